// 2^x for the softmax of the view-cache kernels, two values at a time.
#pragma once

#include "tc_common.cuh"

namespace gsa {
namespace tc {

__device__ __forceinline__ float exp2_mufu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// 2^x on the FMA pipe for x <= 128: x = j + f with j = round(x) (left in the low
// bits of x + 1.5 * 2^23) and f in [-1/2, 1/2]; 2^f by a quartic fitted for the
// least maximum relative error (2.7e-6 evaluated in fp32, below the 2^-9 of the
// bf16 weights and the 1e-5 wanted of fp32 sums of weights); j goes into the
// exponent bits.  x is clamped at -125: the result is then about 2^-125.
__device__ __forceinline__ uint64_t exp2_poly2(uint64_t x2) {
  float x0, x1;
  f2_unpack(x2, x0, x1);
  const uint64_t x = f2_pack(fmaxf(x0, -125.f), fmaxf(x1, -125.f));
  const uint64_t big = f2_pack(12582912.f, 12582912.f);
  const uint64_t t = f2_add(x, big);
  const uint64_t f = f2_sub(x, f2_sub(t, big));
  uint64_t p = f2_fma(f2_pack(0.009570102f, 0.009570102f), f, f2_pack(0.05591786f, 0.05591786f));
  p = f2_fma(p, f, f2_pack(0.24024744f, 0.24024744f));
  p = f2_fma(p, f, f2_pack(0.6931218f, 0.6931218f));
  p = f2_fma(p, f, f2_pack(0.9999993f, 0.9999993f));
  float t0, t1, p0, p1;
  f2_unpack(t, t0, t1);
  f2_unpack(p, p0, p1);
  // the low nine bits of t hold j modulo 512; the rest is shifted out
  return f2_pack(__int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23)),
                 __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23)));
}

// Larger of three; NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

}  // namespace tc
}  // namespace gsa
