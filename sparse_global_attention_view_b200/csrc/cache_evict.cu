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
// read again).  A radix selection finds the n_keep-th key in four passes of 11, 5, 8
// and 8 bits, the first two on the halves in shared memory: every CTA adds up all
// CTAs' counts of a digit, one barrier a pass.  Then every warp counts the kept and
// the equal keys of its consecutive slots by votes, one scan gives what lies before
// them, and a second round of votes the ranks.  Integer arithmetic throughout, so
// the result depends on the inputs alone.  Bound by instruction issue and latency,
// not by its bytes: the first digits are counted as the keys arrive, with a run of
// equal ones held in a register (a cache of equal accounts would queue up at one
// counter), and the second ones at a counter a lane.  CTAs behind the
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
constexpr int kFewSlots = 4096;       // one CTA a head: 14 us for 2500 slots of 16 heads against 18 of a cluster and the moves'
constexpr int kSomeSlots = 65536;      // clusters of four: 22 us for 20000 slots of 16 heads against 31 of eight; equal at 80000
// Halves of sort keys in a slice's shared memory, so that two CTAs fit on an SM: 162 us
// for 274800 slots of 16 heads against 185 without; with 400000 slots and one CTA on an
// SM, 303 against 254 without.
constexpr int kMaxKeys = 44 * 1024;
constexpr int kCopyCtas = 64;

// Passes of the radix selection: a digit's place, its bins and their place among the counts.
constexpr int kPasses = 4;
struct Pass {
  int shift, bins, at;
};
__device__ constexpr Pass kPass[kPasses] = {{21, 2048, 0}, {16, 32, 2048}, {8, 256, 2080}, {0, 256, 2336}};
constexpr int kCounts = 2592;
constexpr int kClose = 1024;  // slots whose half equals the limit's that a CTA remembers

struct Shared {
  alignas(16) uint32_t counts[kCounts];  // this CTA's, read by the others
  uint32_t lanes[32 * 32];  // of the second pass, for each lane of a warp
  int close_slot[kClose];
  uint16_t close_low[kClose];  // the lower halves of their keys
  uint32_t n_close;
  uint32_t warp_sum[kWarps];
  uint32_t warp_tot[4][kWarps];
  alignas(16) uint32_t tot[4];  // this CTA's counts, read by the others
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

// Moves m, m + step, ... of a head (N of them); eight lanes a move.
template <int N>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int hk, int m, int step, int n) {
  const int e = (threadIdx.x & 7) * 8;
  const long long list = (long long)hk * a.most, row = hk * a.w_stride;
  uint4 kk[N], vv[N];
  int to[N];
#pragma unroll
  for (int u = 0; u < N; ++u, m += step) {
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
  for (int u = 0; u < N; ++u)
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
  // this CTA's slots [s0, s1), and the warp's part [first, last) of them
  const int lane = tid & 31, warp = tid >> 5;
  const int slice = ((a.n + CLUSTER - 1) / CLUSTER + 31) & ~31;
  const int s0 = min(a.n, rank * slice), s1 = min(a.n, s0 + slice);
  const int part = ((s1 - s0 + kThreads - 1) / kThreads) * 32;
  const int first = min(s1, s0 + warp * part), last = min(s1, first + part);
  auto key_of = [&](int slot) -> uint32_t { return sort_key(acc[slot], ids[slot], a.recent_from); };
  auto top_of = [&](int slot) -> uint32_t { return IN_SMEM ? s_top[slot - s0] : key_of(slot) >> 16; };
  for (int b = tid; b < kCounts; b += kThreads) sh.counts[b] = 0;
  sh.lanes[tid] = 0;
  if (tid == 0) sh.n_close = 0;
  __syncthreads();

  // the n_keep-th largest key: its leading bits are settled pass by pass
  uint32_t prefix = 0, want = (uint32_t)a.keep;
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    uint32_t* counts = sh.counts + kPass[pass].at;
    const int shift = kPass[pass].shift;
    const uint32_t bins = kPass[pass].bins;
    if (pass == 0) {
      uint32_t run_bin = 0, run = 0;  // equal digits seen in a row
      auto flush = [&]() {
        if (run) atomicAdd(&counts[run_bin], run);
      };
      for (int slot = first + lane; slot < last; slot += 128) {
        uint32_t k[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) k[u] = slot + 32 * u < last ? key_of(slot + 32 * u) : 0u;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (slot + 32 * u >= last) break;
          if (IN_SMEM) s_top[slot + 32 * u - s0] = (uint16_t)(k[u] >> 16);
          const uint32_t bin = k[u] >> shift;
          if (bin != run_bin) {
            flush();
            run = 0;
            run_bin = bin;
          }
          ++run;
        }
      }
      flush();
    } else if (pass == 1) {
#pragma unroll 4
      for (int slot = first + lane; slot < last; slot += 32) {
        const uint32_t t = top_of(slot);
        if (t >> 5 == prefix >> 21) atomicAdd(&sh.lanes[(t & 31) * 32 + lane], 1u);
      }
      __syncthreads();
      const uint32_t c = __reduce_add_sync(0xffffffffu, sh.lanes[tid]);
      if (lane == 0) counts[warp] = c;
    } else if (pass == 3 && sh.n_close <= kClose) {
      if (tid < sh.n_close && sh.close_low[tid] >> 8 == (prefix >> 8 & 0xff)) atomicAdd(&counts[sh.close_low[tid] & 0xff], 1u);
    } else {
#pragma unroll 4
      for (int slot = first + lane; slot < last; slot += 32) {
        if (top_of(slot) != prefix >> 16) continue;
        const uint32_t k = key_of(slot);
        if (pass == 2) {
          const uint32_t at = atomicAdd(&sh.n_close, 1u);
          if (at < kClose) {
            sh.close_slot[at] = slot;
            sh.close_low[at] = (uint16_t)k;
          }
        } else if (k >> 8 != prefix >> 8) {
          continue;
        }
        atomicAdd(&counts[(k >> shift) & (bins - 1)], 1u);
      }
    }
    sync_all();
    // two bins a thread from the top: the one in which the count reaches `want`
    const int hi = (int)bins - 1 - 2 * tid;
    uint32_t c0 = 0, c1 = 0, total;
    if (hi > 0) {
#pragma unroll
      for (int r = 0; r < CLUSTER; ++r) {
        const uint2 c = *reinterpret_cast<const uint2*>(of_rank(counts, r) + hi - 1);
        c0 += c.y;
        c1 += c.x;
      }
    }
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
  }
  const uint32_t limit = prefix;  // `want` of the keys that equal it stay

  // Halves that equal the limit's are told apart in shared memory, so that they are
  // enough from here on: no key's half is 0 or 0xffff.
  const uint32_t limit_top = limit >> 16;
  if (IN_SMEM) {
    auto tell = [&](int slot, uint32_t low) {
      if (low != (limit & 0xffff)) s_top[slot - s0] = (uint16_t)(low > (limit & 0xffff) ? limit_top + 1 : limit_top - 1);
    };
    if (sh.n_close <= kClose) {
      if (tid < sh.n_close) tell(sh.close_slot[tid], sh.close_low[tid]);
    } else {
#pragma unroll 4
      for (int slot = first + lane; slot < last; slot += 32)
        if (s_top[slot - s0] == limit_top) tell(slot, key_of(slot) & 0xffff);
    }
    __syncthreads();
  }
  auto short_key = [&](int slot) -> uint32_t { return IN_SMEM ? s_top[slot - s0] : key_of(slot); };
  const uint32_t z = IN_SMEM ? limit_top : limit;
  // kept for certain, and equal to the limit, before `keep` and from there on
  const int low_last = min(last, a.keep), high_first = max(first, a.keep);
  uint32_t tot[4] = {0u, 0u, 0u, 0u};
  auto count = [&](int from, int to, uint32_t* more, uint32_t* equal) {
#pragma unroll 4
    for (int slot = from + lane; slot < to; slot += 32) {
      const uint32_t k = short_key(slot);
      *more += k > z;
      *equal += k == z;
    }
  };
  count(first, low_last, &tot[0], &tot[1]);
  count(high_first, last, &tot[2], &tot[3]);
#pragma unroll
  for (int c = 0; c < 4; ++c) tot[c] = __reduce_add_sync(0xffffffffu, tot[c]);
  // ... before the warp's part: in the CTA, then in the cluster
  if (lane == 0)
#pragma unroll
    for (int c = 0; c < 4; ++c) sh.warp_tot[c][warp] = tot[c];
  __syncthreads();
  uint32_t before[4], all[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t x = sh.warp_tot[c][lane];
    before[c] = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0u);
    const uint32_t sum = __reduce_add_sync(0xffffffffu, x);
    if (tid == 0) sh.tot[c] = sum;
  }
  sync_all();
#pragma unroll
  for (int r = 0; r < CLUSTER; ++r) {
    const uint4 t = *reinterpret_cast<const uint4*>(of_rank(sh.tot, r));
    const uint32_t tc[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (r < rank) before[c] += tc[c];
      all[c] += tc[c];
    }
  }
  // the equal keys that stay are the first ones, so those below `keep` before others
  auto stay_low = [&](const uint32_t (&t)[4]) -> uint32_t { return min(want, t[1]); };
  auto stay_high = [&](const uint32_t (&t)[4]) -> uint32_t { return min(want - stay_low(t), t[3]); };
  const uint32_t n_moves = all[2] + stay_high(all);
  if (rank == 0 && tid == 0) a.n_moves[hk] = (int)n_moves;
  // free slots below `keep`, and kept tokens at or behind it, before the warp's own
  uint32_t holes = (uint32_t)min(first, a.keep) - before[0] - stay_low(before);
  uint32_t movers = before[2] + stay_high(before), run = before[1] + before[3];
  const long long row = hk * a.w_stride;
  int* const dst = a.dst + (long long)hk * a.most;
  int* const src = a.src + (long long)hk * a.most;
  const uint32_t below = (1u << lane) - 1;
  const bool ties = all[1] + all[3] > want;  // not all equal keys stay
  auto stays = [&](int slot, int to) -> bool {
    const uint32_t k = slot < to ? short_key(slot) : 0u;
    bool yes = k >= z;
    if (ties) {
      const uint32_t q = __ballot_sync(0xffffffffu, k == z);
      if (k == z) yes = run + __popc(q & below) < want;
      run += __popc(q);
    }
    return yes;
  };
#pragma unroll 2
  for (int base = first; base < low_last; base += 32) {
    const int slot = base + lane;
    const bool yes = stays(slot, low_last), hole = !yes && slot < low_last;
    const uint32_t h = __ballot_sync(0xffffffffu, hole);
    if (hole) dst[holes + __popc(h & below)] = slot;
    holes += __popc(h);
    if (CLUSTER == 1 && yes) {
      a.acc_out[row + slot] = acc[slot];
      a.ids_out[row + slot] = ids[slot];
    }
  }
#pragma unroll 2
  for (int base = high_first; base < last; base += 32) {
    const int slot = base + lane;
    const bool yes = stays(slot, last);
    const uint32_t m = __ballot_sync(0xffffffffu, yes);
    if (yes) src[movers + __popc(m & below)] = slot;
    movers += __popc(m);
  }
  if (CLUSTER == 1) {
    __syncthreads();
    for (int m = tid >> 3; m < (int)n_moves; m += kThreads / 8 * 2) move_rows<2>(a, hk, m, kThreads / 8, (int)n_moves);
  }
  sync_all();  // no CTA leaves while another may read its shared memory
}

constexpr int MOVE_THREADS = 256;

template <int N>
__global__ void __launch_bounds__(MOVE_THREADS) move_kernel(const EvictArgs a) {
  // heads vary fastest: equal ranks of all heads lie near one another in memory
  const int hk = blockIdx.x % a.Hk, m0 = blockIdx.x / a.Hk * (MOVE_THREADS / 8 * N);
  pdl_wait();
  const int n = a.n_moves[hk];
  if (m0 < n) move_rows<N>(a, hk, m0 + (threadIdx.x >> 3), MOVE_THREADS / 8, n);
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
  // two moves a thread at a time (162 us for 274800 -> 137400 slots of 16 heads; 178 with
  // one, 176 with four), one while that makes two waves of blocks at most (20.6 us for
  // 42594 -> 41220, 22.6 with two; equal at 24000 -> 18000)
  auto blocks = [&](int per) -> long long { return (long long)((a.most + per - 1) / per) * d.Hk; };
  constexpr int kRows = MOVE_THREADS / 8;
  if (blocks(kRows) <= 16 * 148) return launch_second(move_kernel<1>, dim3((unsigned)blocks(kRows)), MOVE_THREADS, st, a);
  return launch_second(move_kernel<2>, dim3((unsigned)blocks(2 * kRows)), MOVE_THREADS, st, a);
}

}  // namespace gsa
