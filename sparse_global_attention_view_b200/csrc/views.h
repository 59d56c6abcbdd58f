// Launchers of the view-cache operators (prefix_attn, key_weights,
// cache_evict), shared between their C-ABI layer and the kernel files.
// Arguments are validated by the caller.
#pragma once

#include <atomic>

#include "internal.h"

namespace gsa {

// One batch of views: sizes, token strides (elements) and device offsets.
struct ViewDims {
  int B, H, Hk, G;           // views, query heads, key heads, query heads per key head
  int n_q, n_own, n_prefix;  // tokens held by the buffers
  int max_q, max_own;        // longest view: queries, own tokens
  int causal;
  long long q_stride, kp_stride, vp_stride, ko_stride, vo_stride, o_stride;
  float scale, c2;           // softmax scale, and times log2(e)
  long long wait_cycles;
  const int* q_off;          // [B + 1] device
  const int* own_off;        // [B + 1] device
};

// How a prefix_attn call is cut up (a function of the sizes alone).
struct ViewPlan {
  // the tensor-core launches: rows packed over views against the prefix
  // alone, rows aligned to views against both, or against their own keys alone
  int packed, aligned, aligned_prefix, aligned_own;
  int rows;        // at most four rows: the prefix by the CUDA-core kernel, instead of `packed`
  int joined;      // by clusters that finish the rows, own keys included
  int small_own;   // the views' own keys by the CUDA-core kernel, which also merges
  int split_packed, split_aligned;  // key splits
  int parts;       // partial results per (query, head); 0: written directly
};
ViewPlan view_plan(const ViewDims& d);

cudaError_t launch_prefix_attn(const ViewDims& d, const ViewPlan& p, const bf16* q, const bf16* kp,
                               const bf16* vp, const bf16* ko, const bf16* vo, bf16* out, float* lse,
                               float* part_o, float* part_lse, unsigned* err, cudaStream_t st);

// How a key_weights call is cut up.
struct WeightsPlan {
  int rows;       // at most eight rows: the kernel for those
  int own_cores;  // views of few rows: their own keys by CUDA cores
  int prefix_units, own_units;    // work items of 512 keys: of the prefix, of one view at most
  int split_prefix, split_own;    // query ranges of an item
};
WeightsPlan weights_plan(const ViewDims& d);
// Work items of the plan: a 32-bit number of them, and the grid's stride more, is what
// the kernel counts to.
inline long long weights_items(const ViewDims& d, const WeightsPlan& p) {
  return ((long long)p.prefix_units * p.split_prefix + (long long)d.B * p.own_units * p.split_own) * d.Hk;
}
constexpr long long kMostItems = 0x7fffffffLL - 1024;

cudaError_t launch_key_weights(const ViewDims& d, const WeightsPlan& p, const bf16* q, const bf16* kp, const bf16* ko,
                               const float* lse, const float* acc, long long acc_stride, float* acc_out,
                               long long acc_out_stride, float decay, float* part_prefix, float* part_own, unsigned* err, cudaStream_t st);

// One cache_evict call.
struct EvictDims {
  int Hk, n, keep, recent_from;
  long long k_stride, v_stride, w_stride;  // elements
};
inline int evict_most_moves(const EvictDims& d) { return d.keep < d.n - d.keep ? d.keep : d.n - d.keep; }
cudaError_t launch_cache_evict(const EvictDims& d, bf16* k, bf16* v, const float* acc, const int* ids, float* acc_out,
                               int* ids_out, int* n_moves, int* src, int* dst, cudaStream_t st);

// Allows a kernel its dynamic shared memory: once for each device (a microsecond a
// call otherwise).  `done` belongs to the kernel: a bit for each device.
template <typename F>
cudaError_t allow_smem(F* kernel, int bytes, std::atomic<unsigned long long>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

// A second kernel of a call: launched while the first one still runs, so that its
// start is not waited for.  The first kernel, launched in the ordinary way, calls
// pdl_launch() at its start; the second one calls pdl_wait() before it reads what the
// first one writes or writes what the first one touches: it goes on when the first one
// has ended and its writes are visible.  What was written before the call (offsets,
// queries, keys) may be read ahead of that, since the first kernel began behind it: so
// a call's only kernel is never launched this way.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_second(void (*kernel)(P...), dim3 grid, unsigned threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// A view's ranges; false (and the device-check bit) when the offsets do not
// describe rows of the buffers or more of them than a view may have.
struct ViewRange {
  int q0, q1, k0, k1;
};
__device__ __forceinline__ bool view_range(const ViewDims& d, int b, ViewRange* r, unsigned* err) {
  r->q0 = d.q_off[b];
  r->q1 = d.q_off[b + 1];
  r->k0 = d.own_off[b];
  r->k1 = d.own_off[b + 1];
  if (r->q0 < 0 || r->q1 < r->q0 || r->q1 > d.n_q || r->q1 - r->q0 > d.max_q || r->k0 < 0 || r->k1 < r->k0 ||
      r->k1 > d.n_own || r->k1 - r->k0 > d.max_own) {
    if (err) atomicOr(err, kErrDeviceCheck);
    return false;
  }
  return true;
}
// Every view's, by `threads` threads.
__device__ __forceinline__ void check_views(const ViewDims& d, int thread, int threads, unsigned* err) {
  ViewRange r;
  for (int b = thread; b < d.B; b += threads) view_range(d, b, &r, err);
}

}  // namespace gsa
