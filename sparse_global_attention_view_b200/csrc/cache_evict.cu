// Shrinking a cache of keys and values to the tokens with the largest account.
//
// For each key head the n_keep tokens with the largest key stay: the account of
// attention received, +infinity for tokens numbered recent_from or later; equal
// keys go to the lower slot.  Slots are not kept in order: the kept tokens below
// n_keep stay where they are, and the r-th kept token at or behind n_keep moves
// into the r-th free slot.  So a token's K and V move only where they must, and
// as sources lie behind n_keep and targets before it, moves need no order and
// the call may be repeated.
//
// select_kernel: one cluster of CTAs a head, each with a slice of the slots, its
// sort keys in shared memory (read again from memory where a slice does not
// fit).  A radix selection finds the n_keep-th key in three passes of 11, 11 and
// 10 bits, with histograms in shared memory that the CTAs read from one another;
// then the counts of equal keys, of free slots and of movers before every warp's
// part of the slots give each its rank.  Integer arithmetic throughout, so the
// result depends on the inputs alone.  Bound by the latency of its passes.
// move_kernel: copies K and V rows, eight lanes a row.  Bound by memory.
#include <cooperative_groups.h>
#include <math_constants.h>

#include "views.h"

namespace gsa {
namespace {

namespace cg = cooperative_groups;

constexpr int CLUSTER = 8;
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int BINS = 2048;
constexpr int kMaxKeys = 40 * 1024;  // sort keys of a slice in shared memory

struct Shared {
  uint32_t hist[BINS];
  uint32_t warp_sum[kWarps];
  uint32_t tot[4];        // this CTA's counts, read by the others
  uint32_t bin, above;    // the bin that holds the wanted key; keys above it
  uint32_t before[kWarps][2];
};

// Larger account, larger key; NaN counts as -infinity and -0 as 0.
__device__ __forceinline__ uint32_t sort_key(float acc, int id, int recent_from) {
  if (id >= recent_from) acc = CUDART_INF_F;
  if (acc != acc) acc = -CUDART_INF_F;
  const uint32_t u = __float_as_uint(acc + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct EvictArgs {
  int Hk, n, keep, recent_from;
  const float* acc;
  const int* ids;
  float* acc_out;
  int* ids_out;
  long long w_stride;
  int most;      // moves a head can need: min(keep, n - keep)
  int* n_moves;  // [Hk]
  int* src;      // [Hk][most]
  int* dst;      // [Hk][most]
};

// Exclusive sum over the warps of the block of a value that lane 0 holds.
__device__ __forceinline__ uint32_t warps_before(uint32_t v, uint32_t* scratch, uint32_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) scratch[warp] = v;
  __syncthreads();
  uint32_t x = scratch[lane], sum = x;  // 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  *total = __shfl_sync(0xffffffffu, sum, 31);
  return __shfl_sync(0xffffffffu, sum - x, warp);
}

template <bool IN_SMEM>
__global__ void __launch_bounds__(kThreads, 1) select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_keys[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), hk = blockIdx.x / CLUSTER;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* acc = a.acc + hk * a.w_stride;
  const int* ids = a.ids + hk * a.w_stride;
  // this CTA's slots [s0, s1), and a warp's part [w0, w1) of them
  const int slice = ((a.n + CLUSTER - 1) / CLUSTER + 31) & ~31;
  const int s0 = min(a.n, rank * slice), s1 = min(a.n, s0 + slice);
  const int part = ((slice + kWarps - 1) / kWarps + 31) & ~31;
  const int w0 = min(s1, s0 + warp * part), w1 = min(s1, w0 + part);
  auto key_of = [&](int slot) -> uint32_t {
    return IN_SMEM ? s_keys[slot - s0] : sort_key(acc[slot], ids[slot], a.recent_from);
  };
  if (IN_SMEM)
    for (int s = s0 + tid; s < s1; s += kThreads) s_keys[s - s0] = sort_key(acc[s], ids[s], a.recent_from);

  // the n_keep-th largest key: its leading bits are settled pass by pass
  uint32_t prefix = 0, mask = 0, want = (uint32_t)a.keep;
  const int shifts[3] = {21, 10, 0};
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = shifts[pass];
    const uint32_t bins = pass == 2 ? 1024u : 2048u;
    for (int b = tid; b < BINS; b += kThreads) sh.hist[b] = 0;
    __syncthreads();
    for (int base = w0; base < w1; base += 32) {
      const int slot = base + lane;
      bool in = slot < w1;
      uint32_t bin = 0;
      if (in) {
        const uint32_t k = key_of(slot);
        in = (k & mask) == prefix;
        bin = (k >> shift) & (bins - 1);
      }
      // many equal keys would queue up at one counter
      const uint32_t live = __ballot_sync(0xffffffffu, in);
      if (live == 0) continue;
      const uint32_t first = __shfl_sync(0xffffffffu, bin, __ffs(live) - 1);
      if (__all_sync(0xffffffffu, !in || bin == first)) {
        if (lane == 0) atomicAdd(&sh.hist[first], (uint32_t)__popc(live));
      } else if (in) {
        atomicAdd(&sh.hist[bin], 1u);
      }
    }
    cluster.sync();
    // every CTA sums all histograms, two bins a thread from the top, and finds
    // the bin in which the count from above reaches `want`
    uint32_t c0 = 0, c1 = 0;
    const int hi = (int)bins - 1 - 2 * tid;
    if (hi > 0)
      for (int r = 0; r < CLUSTER; ++r) {
        const uint32_t* h = cluster.map_shared_rank(sh.hist, r);
        c0 += h[hi];
        c1 += h[hi - 1];
      }
    uint32_t sum = c0 + c1, total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const uint32_t warp_total = __shfl_sync(0xffffffffu, sum, 31);
    const uint32_t above = warps_before(warp_total, sh.warp_sum, &total) + sum - (c0 + c1);
    if (above < want && above + c0 >= want) {
      sh.bin = hi;
      sh.above = above;
    } else if (above + c0 < want && above + c0 + c1 >= want) {
      sh.bin = hi - 1;
      sh.above = above + c0;
    }
    cluster.sync();  // the result is there, and nobody reads a histogram any more
    want -= sh.above;
    prefix |= sh.bin << shift;
    mask |= (bins - 1) << shift;
  }
  const uint32_t limit = prefix;  // `want` of the keys that equal it stay

  // equal keys before every warp's part: first in the CTA, then in the cluster
  uint32_t eq = 0, total;
  for (int base = w0; base < w1; base += 32)
    eq += __popc(__ballot_sync(0xffffffffu, base + lane < w1 && key_of(base + lane) == limit));
  uint32_t eq_before = warps_before(eq, sh.warp_sum, &total);
  if (tid == 0) sh.tot[0] = total;
  cluster.sync();
  for (int r = 0; r < rank; ++r) eq_before += cluster.map_shared_rank(sh.tot, r)[0];

  // free slots below `keep`, and kept tokens at or behind it
  const uint32_t below = (1u << lane) - 1;
  auto kept_ballot = [&](int base, uint32_t* run) -> uint32_t {
    const int slot = base + lane;
    const uint32_t k = slot < w1 ? key_of(slot) : 0u;
    const uint32_t same = __ballot_sync(0xffffffffu, slot < w1 && k == limit);
    const bool kept = slot < w1 && (k > limit || (k == limit && *run + __popc(same & below) < want));
    *run += __popc(same);
    return __ballot_sync(0xffffffffu, kept);
  };
  uint32_t holes = 0, movers = 0, run = eq_before;
  for (int base = w0; base < w1; base += 32) {
    const uint32_t kept = kept_ballot(base, &run);
    const int slot = base + lane;
    const uint32_t low = __ballot_sync(0xffffffffu, slot < a.keep && slot < w1);
    holes += __popc(low & ~kept);
    movers += __popc(kept & ~low);
  }
  uint32_t holes_before = warps_before(holes, sh.warp_sum, &total);
  if (tid == 0) sh.tot[1] = total;
  uint32_t movers_before = warps_before(movers, sh.warp_sum, &total);
  if (tid == 0) sh.tot[2] = total;
  cluster.sync();
  uint32_t all = 0;
  for (int r = 0; r < CLUSTER; ++r) {
    const uint32_t* t = cluster.map_shared_rank(sh.tot, r);
    if (r < rank) {
      holes_before += t[1];
      movers_before += t[2];
    }
    all += t[2];
  }
  if (rank == 0 && tid == 0) a.n_moves[hk] = (int)all;
  run = eq_before;
  for (int base = w0; base < w1; base += 32) {
    const uint32_t kept = kept_ballot(base, &run);
    const int slot = base + lane;
    const bool in = slot < w1, mine = kept >> lane & 1;
    const uint32_t low = __ballot_sync(0xffffffffu, slot < a.keep && in);
    const uint32_t free_here = low & ~kept, move_here = kept & ~low;
    if (in && slot < a.keep) {
      if (mine) {
        a.acc_out[hk * a.w_stride + slot] = acc[slot];
        a.ids_out[hk * a.w_stride + slot] = ids[slot];
      } else {
        a.dst[(long long)hk * a.most + holes_before + __popc(free_here & below)] = slot;
      }
    } else if (mine) {
      a.src[(long long)hk * a.most + movers_before + __popc(move_here & below)] = slot;
    }
    holes_before += __popc(free_here);
    movers_before += __popc(move_here);
  }
  cluster.sync();  // no CTA leaves while another may read its shared memory
}

constexpr int MOVE_THREADS = 256, MOVE_UNROLL = 4;
constexpr int MOVE_BLOCK = MOVE_THREADS / 8 * MOVE_UNROLL;  // moves of a block

__global__ void __launch_bounds__(MOVE_THREADS)
    move_kernel(const EvictArgs a, bf16* __restrict__ k, bf16* __restrict__ v, long long k_stride, long long v_stride) {
  const int hk = blockIdx.y, e = (threadIdx.x & 7) * 8, grp = threadIdx.x >> 3;
  const int n = a.n_moves[hk];
  const int m0 = blockIdx.x * MOVE_BLOCK;
  if (m0 >= n) return;
  uint4 kk[MOVE_UNROLL], vv[MOVE_UNROLL];
  int to[MOVE_UNROLL];
#pragma unroll
  for (int u = 0; u < MOVE_UNROLL; ++u) {
    const int m = m0 + u * (MOVE_THREADS / 8) + grp;
    to[u] = -1;
    if (m < n) {
      const int from = a.src[(long long)hk * a.most + m];
      to[u] = a.dst[(long long)hk * a.most + m];
      kk[u] = *reinterpret_cast<const uint4*>(k + from * k_stride + hk * 64 + e);
      vv[u] = *reinterpret_cast<const uint4*>(v + from * v_stride + hk * 64 + e);
      if (e == 0) a.acc_out[hk * a.w_stride + to[u]] = a.acc[hk * a.w_stride + from];
      if (e == 8) a.ids_out[hk * a.w_stride + to[u]] = a.ids[hk * a.w_stride + from];
    }
  }
#pragma unroll
  for (int u = 0; u < MOVE_UNROLL; ++u)
    if (to[u] >= 0) {
      *reinterpret_cast<uint4*>(k + to[u] * k_stride + hk * 64 + e) = kk[u];
      *reinterpret_cast<uint4*>(v + to[u] * v_stride + hk * 64 + e) = vv[u];
    }
}

template <bool IN_SMEM>
cudaError_t launch_select(const EvictArgs& a, size_t smem, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(select_kernel<IN_SMEM>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.Hk * CLUSTER));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CLUSTER;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<IN_SMEM>, a);
}

}  // namespace

cudaError_t launch_cache_evict(const EvictDims& d, bf16* k, bf16* v, const float* acc, const int* ids, float* acc_out,
                               int* ids_out, int* n_moves, int* src, int* dst, cudaStream_t st) {
  if (d.keep <= 0) return cudaSuccess;
  EvictArgs a;
  a.Hk = d.Hk;
  a.n = d.n;
  a.keep = d.keep;
  a.recent_from = d.recent_from;
  a.acc = acc;
  a.ids = ids;
  a.acc_out = acc_out;
  a.ids_out = ids_out;
  a.w_stride = d.w_stride;
  a.most = evict_most_moves(d);
  a.n_moves = n_moves;
  a.src = src;
  a.dst = dst;
  const int slice = ((d.n + CLUSTER - 1) / CLUSTER + 31) & ~31;
  const cudaError_t e =
      slice <= kMaxKeys ? launch_select<true>(a, (size_t)slice * 4, st) : launch_select<false>(a, 0, st);
  if (e != cudaSuccess || a.most == 0) return e;
  move_kernel<<<dim3((unsigned)((a.most + MOVE_BLOCK - 1) / MOVE_BLOCK), (unsigned)d.Hk), MOVE_THREADS, 0, st>>>(
      a, k, v, d.k_stride, d.v_stride);
  return cudaGetLastError();
}

}  // namespace gsa
