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
// select_kernel: a cluster of four or eight CTAs a head (one for few slots), each with a
// slice of the slots and the leading halves of their sort keys in shared memory
// (16 bits tell almost all keys apart; the others, and slices that do not fit, are
// read again).  A radix selection finds the n_keep-th key in three passes of 11,
// 11 and 10 bits: the CTAs add their counts of each digit to one another's shared
// memory, one barrier a pass.  Then the counts of equal keys, of free slots and of
// movers before every thread's part of the slots give each its rank.  Integer
// arithmetic throughout, so the result depends on the inputs alone.  Bound by
// instruction issue and latency, not by its bytes: counting takes the slots thread
// by thread with a run of equal digits held in a register (a cache of equal
// accounts would queue up at one counter), ranking gives every thread an odd
// number of consecutive slots (no votes, one scan of the block).  CTAs behind the
// clusters' copy the accounts and numbers of all slots below n_keep meanwhile;
// the movers' come over those of the free slots afterwards.  The single CTA of few
// slots does all of it, the moves as well: one launch.
// move_kernel: copies K and V rows, eight lanes a row.  Bound by memory.
#include <cooperative_groups.h>
#include <math_constants.h>

#include "views.h"

namespace gsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int BINS = 2048;
constexpr int kFewSlots = 4096;       // one CTA a head: 19 us for 2000 slots of 16 heads against 33 of a cluster and the moves'
constexpr int kSomeSlots = 65536;      // clusters of four: 32 us for 42594 slots of 16 heads against 38 of eight; equal at 80000
constexpr int kMaxKeys = 96 * 1024;   // sort keys of a slice in shared memory, two bytes each
constexpr int kCopyCtas = 64;

struct Shared {
  uint32_t counts[BINS];   // this CTA's
  uint32_t sums[2][BINS];  // the cluster's, one pass in use while the other is cleared
  uint32_t warp_sum[kWarps];
  uint32_t tot[4];         // this CTA's counts, read by the others
  uint32_t bin, above;     // the bin that holds the wanted key; keys above it
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
  bf16* k;
  bf16* v;
  long long k_stride, v_stride;
};

// Exclusive sum over the threads of the block.
__device__ __forceinline__ uint32_t threads_before(uint32_t v, uint32_t* scratch, uint32_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = sum;
  __syncthreads();
  uint32_t w = scratch[lane];  // 32 warps
  const uint32_t own = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  return __shfl_sync(0xffffffffu, w - own, warp) + sum - v;
}

// Moves m, m + step, ... of a head (MOVE_UNROLL of them); eight lanes a move.
constexpr int MOVE_UNROLL = 2;
__device__ __forceinline__ void move_rows(const EvictArgs& a, int hk, int m, int step, int n) {
  const int e = (threadIdx.x & 7) * 8;
  const long long list = (long long)hk * a.most, row = hk * a.w_stride;
  uint4 kk[MOVE_UNROLL], vv[MOVE_UNROLL];
  int to[MOVE_UNROLL];
#pragma unroll
  for (int u = 0; u < MOVE_UNROLL; ++u, m += step) {
    to[u] = -1;
    if (m < n) {
      const int from = a.src[list + m];
      to[u] = a.dst[list + m];
      kk[u] = *reinterpret_cast<const uint4*>(a.k + from * a.k_stride + hk * 64 + e);
      vv[u] = *reinterpret_cast<const uint4*>(a.v + from * a.v_stride + hk * 64 + e);
      if (e == 0) a.acc_out[row + to[u]] = a.acc[row + from];
      if (e == 8) a.ids_out[row + to[u]] = a.ids[row + from];
    }
  }
#pragma unroll
  for (int u = 0; u < MOVE_UNROLL; ++u)
    if (to[u] >= 0) {
      *reinterpret_cast<uint4*>(a.k + to[u] * a.k_stride + hk * 64 + e) = kk[u];
      *reinterpret_cast<uint4*>(a.v + to[u] * a.v_stride + hk * 64 + e) = vv[u];
    }
}

template <int CLUSTER, bool IN_SMEM>
__global__ void __launch_bounds__(kThreads, CLUSTER < 8 ? 1 : 2) select_kernel(const EvictArgs a) {
  extern __shared__ uint16_t s_top[];
  __shared__ Shared sh;
  const int tid = threadIdx.x;
  pdl_launch();
  if ((int)blockIdx.x >= a.Hk * CLUSTER) {
    // whole clusters of copying CTAs
    const int step = (int)(gridDim.x - a.Hk * CLUSTER) * kThreads, first = (int)(blockIdx.x - a.Hk * CLUSTER) * kThreads + tid;
    for (int h = 0; h < a.Hk; ++h) {
      const long long row = h * a.w_stride;
#pragma unroll 2
      for (int i = first; i < a.keep; i += step) {
        a.acc_out[row + i] = a.acc[row + i];
        a.ids_out[row + i] = a.ids[row + i];
      }
    }
    return;
  }
  cg::cluster_group cluster = cg::this_cluster();
  auto sync_all = [&]() {
    if (CLUSTER > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  auto of_rank = [&](uint32_t* p, int r) -> uint32_t* { return CLUSTER > 1 ? cluster.map_shared_rank(p, r) : p; };
  const int rank = CLUSTER > 1 ? (int)cluster.block_rank() : 0, hk = blockIdx.x / CLUSTER;
  const float* acc = a.acc + hk * a.w_stride;
  const int* ids = a.ids + hk * a.w_stride;
  // this CTA's slots [s0, s1), and the thread's part [t0, t1) of them
  const int slice = ((a.n + CLUSTER - 1) / CLUSTER + 31) & ~31;
  const int s0 = min(a.n, rank * slice), s1 = min(a.n, s0 + slice);
  const int part = ((s1 - s0 + kThreads - 1) / kThreads) | 1;
  const int t0 = min(s1, s0 + tid * part), t1 = min(s1, t0 + part);
  auto key_of = [&](int slot) -> uint32_t { return sort_key(acc[slot], ids[slot], a.recent_from); };
  auto top_of = [&](int slot) -> uint32_t { return IN_SMEM ? s_top[slot - s0] : key_of(slot) >> 16; };
  if (IN_SMEM) {
#pragma unroll 8
    for (int s = s0 + tid; s < s1; s += kThreads) s_top[s - s0] = (uint16_t)(key_of(s) >> 16);
  }
  for (int b = tid; b < BINS; b += kThreads) {
    sh.counts[b] = 0;
    sh.sums[0][b] = 0;
  }
  sync_all();

  // the n_keep-th largest key: its leading bits are settled pass by pass
  uint32_t prefix = 0, mask = 0, want = (uint32_t)a.keep;
  const int shifts[3] = {21, 10, 0};
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = shifts[pass];
    const uint32_t bins = pass == 2 ? 1024u : 2048u;
    uint32_t run_bin = 0, run = 0;  // equal digits seen in a row
    auto flush = [&]() {
      if (run) atomicAdd(&sh.counts[run_bin], run);
    };
#pragma unroll 4
    for (int slot = s0 + tid; slot < s1; slot += kThreads) {
      uint32_t k = top_of(slot) << 16;
      if ((k ^ prefix) & mask & 0xffff0000u) continue;
      if (pass > 0) {
        k = key_of(slot);
        if ((k ^ prefix) & mask) continue;
      }
      const uint32_t bin = (k >> shift) & (bins - 1);
      if (bin != run_bin) {
        flush();
        run = 0;
        run_bin = bin;
      }
      ++run;
    }
    flush();
    __syncthreads();
    // to every CTA's sums; the counts and the other sums are cleared for the next pass
    uint32_t* sums = sh.sums[pass & 1];
    for (int b = tid; b < BINS; b += kThreads) {
      const uint32_t c = sh.counts[b];
      sh.counts[b] = 0;
      sh.sums[(pass & 1) ^ 1][b] = 0;
      if (c) {
#pragma unroll
        for (int r = 0; r < CLUSTER; ++r) atomicAdd(of_rank(sums, r) + b, c);
      }
    }
    sync_all();
    // two bins a thread from the top: the one in which the count reaches `want`
    const int hi = (int)bins - 1 - 2 * tid;
    const uint32_t c0 = hi > 0 ? sums[hi] : 0, c1 = hi > 0 ? sums[hi - 1] : 0;
    uint32_t total;
    const uint32_t above = threads_before(c0 + c1, sh.warp_sum, &total);
    if (above < want && above + c0 >= want) {
      sh.bin = hi;
      sh.above = above;
    } else if (above + c0 < want && above + c0 + c1 >= want) {
      sh.bin = hi - 1;
      sh.above = above + c0;
    }
    __syncthreads();
    want -= sh.above;
    prefix |= sh.bin << shift;
    mask |= (bins - 1) << shift;
  }
  const uint32_t limit = prefix;  // `want` of the keys that equal it stay

  const uint32_t limit_top = limit >> 16;
  // above the limit (2), equal to it (1) or below
  auto rank_of = [&](int slot) -> int {
    const uint32_t t = top_of(slot);
    if (t != limit_top) return t > limit_top ? 2 : 0;
    const uint32_t k = key_of(slot);
    return k > limit ? 2 : (k == limit ? 1 : 0);
  };
  // kept for certain, and equal to the limit, before and behind `keep`
  uint32_t more_low = 0, more_high = 0, eq_low = 0, eq_high = 0, total;
  for (int slot = t0; slot < t1; ++slot) {
    const int x = rank_of(slot);
    const bool low = slot < a.keep;
    more_low += low && x == 2;
    more_high += !low && x == 2;
    eq_low += low && x == 1;
    eq_high += !low && x == 1;
  }
  // equal keys before the thread's part: in the CTA, then in the cluster
  uint32_t eq_before = threads_before(eq_low + eq_high, sh.warp_sum, &total);
  if (tid == 0) sh.tot[0] = total;
  sync_all();
  for (int r = 0; r < rank; ++r) eq_before += of_rank(sh.tot, r)[0];
  // free slots below `keep`, and kept tokens at or behind it
  const uint32_t left = want > eq_before ? want - eq_before : 0;
  const uint32_t stay_low = min(left, eq_low), stay_high = min(left - stay_low, eq_high);
  const uint32_t holes = (uint32_t)max(0, min(t1, a.keep) - t0) - more_low - stay_low, movers = more_high + stay_high;
  uint32_t holes_before = threads_before(holes, sh.warp_sum, &total);
  if (tid == 0) sh.tot[1] = total;
  uint32_t movers_before = threads_before(movers, sh.warp_sum, &total);
  if (tid == 0) sh.tot[2] = total;
  sync_all();
  uint32_t all = 0;
#pragma unroll
  for (int r = 0; r < CLUSTER; ++r) {
    const uint32_t* t = of_rank(sh.tot, r);
    if (r < rank) {
      holes_before += t[1];
      movers_before += t[2];
    }
    all += t[2];
  }
  if (rank == 0 && tid == 0) a.n_moves[hk] = (int)all;
  const long long list = (long long)hk * a.most;
  uint32_t run = eq_before;
  for (int slot = t0; slot < t1; ++slot) {
    const int x = rank_of(slot);
    const bool stays = x == 2 || (x == 1 && run < want);
    run += x == 1;
    if (IN_SMEM) {
      s_top[slot - s0] = stays;  // the thread's own slots, looked at for the last time
    } else {
      if (slot < a.keep && !stays) a.dst[list + holes_before++] = slot;
      if (slot >= a.keep && stays) a.src[list + movers_before++] = slot;
    }
  }
  if (IN_SMEM) {
    // the lists in whole lines: the warp goes over its threads' parts, 32 slots at a time
    __syncwarp();
    const int lane = tid & 31;
    uint32_t hb = __shfl_sync(0xffffffffu, holes_before, 0), mb = __shfl_sync(0xffffffffu, movers_before, 0);
    const int first = __shfl_sync(0xffffffffu, t0, 0), last = __shfl_sync(0xffffffffu, t1, 31);
    const uint32_t below = (1u << lane) - 1;
    for (int base = first; base < last; base += 32) {
      const int slot = base + lane;
      const bool in = slot < last, stays = in && s_top[slot - s0];
      const uint32_t h = __ballot_sync(0xffffffffu, in && !stays && slot < a.keep);
      const uint32_t m = __ballot_sync(0xffffffffu, stays && slot >= a.keep);
      if (h >> lane & 1) a.dst[list + hb + __popc(h & below)] = slot;
      if (m >> lane & 1) a.src[list + mb + __popc(m & below)] = slot;
      hb += __popc(h);
      mb += __popc(m);
    }
  }
  if (CLUSTER == 1) {
    __syncthreads();
    const long long row = hk * a.w_stride;
    for (int slot = tid; slot < a.keep; slot += kThreads)
      if (s_top[slot]) {
        a.acc_out[row + slot] = acc[slot];
        a.ids_out[row + slot] = ids[slot];
      }
    for (int m = tid >> 3; m < (int)all; m += kThreads / 8 * MOVE_UNROLL) move_rows(a, hk, m, kThreads / 8, (int)all);
  }
  sync_all();  // no CTA leaves while another may read its shared memory
}

constexpr int MOVE_THREADS = 256;
constexpr int MOVE_BLOCK = MOVE_THREADS / 8 * MOVE_UNROLL;  // moves of a block

__global__ void __launch_bounds__(MOVE_THREADS) move_kernel(const EvictArgs a) {
  // heads vary fastest: equal ranks of all heads lie near one another in memory
  const int hk = blockIdx.x % a.Hk, m0 = blockIdx.x / a.Hk * MOVE_BLOCK;
  pdl_wait();
  const int n = a.n_moves[hk];
  if (m0 < n) move_rows(a, hk, m0 + (threadIdx.x >> 3), MOVE_THREADS / 8, n);
}

int slice_of(int n, int cluster) { return ((n + cluster - 1) / cluster + 31) & ~31; }

template <int CLUSTER, bool IN_SMEM>
cudaError_t launch_select(const EvictArgs& a, cudaStream_t st) {
  const size_t smem = IN_SMEM ? (size_t)slice_of(a.n, CLUSTER) * 2 : 0;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(select_kernel<CLUSTER, IN_SMEM>, kMaxKeys * 2, &done);
  if (e != cudaSuccess) return e;
  if (CLUSTER == 1) {
    select_kernel<CLUSTER, IN_SMEM><<<(unsigned)a.Hk, kThreads, smem, st>>>(a);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.Hk * CLUSTER + kCopyCtas));
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
  return cudaLaunchKernelEx(&cfg, select_kernel<CLUSTER, IN_SMEM>, a);
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
  a.k = k;
  a.v = v;
  a.k_stride = d.k_stride;
  a.v_stride = d.v_stride;
  if (d.n <= kFewSlots) return launch_select<1, true>(a, st);
  const cudaError_t e = d.n <= kSomeSlots             ? launch_select<4, true>(a, st)
                        : slice_of(d.n, 8) <= kMaxKeys ? launch_select<8, true>(a, st)
                                                       : launch_select<8, false>(a, st);
  if (e != cudaSuccess || a.most == 0) return e;
  const long long blocks = (long long)((a.most + MOVE_BLOCK - 1) / MOVE_BLOCK) * d.Hk;
  return launch_second(move_kernel, dim3((unsigned)blocks), MOVE_THREADS, st, a);
}

}  // namespace gsa
