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

__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 2^x on the FMA pipe: x = j + f with j = round(x) and f in [-1/2, 1/2];
// 2^f by a quartic fitted for the least maximum relative error (2.7e-6 evaluated in
// fp32, below the 2^-8 of the bf16 weights and the 1e-5 wanted of fp32 sums of
// weights), times 2^j.  x + 1.5 * 2^23 + 127 has j + 127, the exponent of 2^j, in its
// low bits.  x is clamped at -127, where 2^j is 0: what lies below gives 0, -infinity
// included, as the special-function unit does.  The clamp and the product keep a NaN;
// an integer addition of j to the exponent would make a number of it.
// x is at most 128, or with ANY any number: clamped at 128, where 2^j is infinity.
template <bool ANY>
__device__ __forceinline__ uint64_t exp2_poly2(uint64_t x2) {
  float x0, x1;
  f2_unpack(x2, x0, x1);
  if (ANY) {
    x0 = min_nan(x0, 128.f);
    x1 = min_nan(x1, 128.f);
  }
  const uint64_t x = f2_pack(max_nan(x0, -127.f), max_nan(x1, -127.f));
  const uint64_t big = f2_pack(12583039.f, 12583039.f);
  const uint64_t t = f2_add(x, big);
  const uint64_t f = f2_sub(x, f2_sub(t, big));
  uint64_t p = f2_fma(f2_pack(0.009570102f, 0.009570102f), f, f2_pack(0.05591786f, 0.05591786f));
  p = f2_fma(p, f, f2_pack(0.24024744f, 0.24024744f));
  p = f2_fma(p, f, f2_pack(0.6931218f, 0.6931218f));
  p = f2_fma(p, f, f2_pack(0.9999993f, 0.9999993f));
  float t0, t1;
  f2_unpack(t, t0, t1);
  return f2_mul(p, f2_pack(__int_as_float(__float_as_int(t0) << 23), __int_as_float(__float_as_int(t1) << 23)));
}

}  // namespace tc
}  // namespace gsa
