// How much attention every key received: the column sums of a softmax whose row
// sums are known,
//   w[hk][j] = sum over queries i that see j, over the heads h of group hk, of
//              exp(scale q_ih . k_j - lse_ih),
// added to a running account of the cached keys.
//
// key_weights_kernel (tcgen05 / TMEM / TMA): the products are taken transposed,
// S^T = K Q^T with 128 keys as the rows of a tile, so a thread owns a key and its
// sum stays in a register; no atomics, and no reduction over lanes.  A work item
// is 512 keys of one key head (four tiles) against a range of query tiles (128
// (token, head of the group) rows each); one CTA an SM takes items in turn:
//   warp 0       TMA producer: the item's key tiles (two sets of four, so the next
//                item's keys arrive during this one) and a 5-stage ring of query tiles;
//   warp 1       MMA issuer: for each query tile four products, one a key tile;
//   warp 2       the query tile's -lse log2(e) into the ring, and which of its rows count
//                for nothing (and TMEM allocation);
//   warps 4-19   a warpgroup for each key tile: exponentials and sums.
// While one warpgroup waits for its product the three others have the
// exponential units busy: those bound it (half as many tensor flops an
// exponential as in attention, and no maximum, packing or store of weights).
// Few items are cut over query ranges, whose sums are added in order afterwards.
//
// key_weights_own_kernel: the own keys of views of few rows, eight lanes a key.
// key_weights_rows_kernel: at most eight rows in all.  Bound by the read of the
// keys; eight lanes hold a key, and after the dot products lane r takes the
// exponential of row r.
//
// Rows that count for nothing (of no token, of a log sum of -infinity, hidden from a
// key) are told by their place, not by an infinite score or log sum: one that holds
// NaN or infinity, or meets an infinite key, would leave NaN otherwise.
//
// All sums are fp32: a tile's 128 terms in 8 chains, then tile after tile.
#include <math_constants.h>

#include <type_traits>

#include "exp2_poly.cuh"
#include "views.h"

namespace gsa {
namespace {

using namespace tc;

constexpr int kPolyOf8 = 2;  // pairs of exponentials in eight on the FMA pipe
constexpr int SLOTS = 4;     // key tiles of an item
constexpr int ITEM = 128 * SLOTS;
constexpr int ST = 5;        // query ring stages
constexpr int kThreads = 128 + 128 * SLOTS;
constexpr uint32_t kTile = 128 * 128;

constexpr uint32_t OFF_K = 0;
constexpr uint32_t OFF_Q = OFF_K + 2 * SLOTS * kTile;
constexpr uint32_t OFF_L = OFF_Q + ST * kTile;
// a bit for each row of a query tile that counts for nothing, and whether there is one
constexpr uint32_t OFF_NONE = OFF_L + ST * 512, OFF_SOME = OFF_NONE + ST * 16;
constexpr uint32_t OFF_BAR = OFF_SOME + (ST * 4 + 7) / 8 * 8;
constexpr uint32_t OFF_MISC = OFF_BAR + 256;
constexpr uint32_t kSmemBytes = OFF_MISC + 64 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// KF/KE: a set of key tiles filled / free; QF/QE: a query stage; LF: its lse; SF/SE: a score tile
constexpr int B_KF = 0, B_KE = B_KF + 2, B_QF = B_KE + 2, B_QE = B_QF + ST, B_LF = B_QE + ST, B_SF = B_LF + ST,
              B_SE = B_SF + SLOTS, B_DRAIN = B_SE + SLOTS, B_COUNT = B_DRAIN + 1;
static_assert(B_COUNT * 8 <= 256, "barrier area");
constexpr uint32_t kCols = 128 * SLOTS;

struct WeightsArgs {
  ViewDims d;
  int rows_tok;                       // tokens per query tile: 128 / G
  int prefix_units, own_units;        // items of 512 keys: of the prefix, of one view at most
  int prefix_items;                   // items that come before the views' own
  int split_prefix, split_own;        // query ranges of an item
  int n_items;
  uint32_t m_units, m_split, m_tok;   // for quotients by prefix_units, split_prefix and rows_tok (udiv31)
  const float* lse;                   // [n_q][H]
  const float* acc;                   // nullable [Hk][acc_stride]
  float* acc_out;                     // [Hk][acc_out_stride]
  float decay;
  long long acc_stride, acc_out_stride;
  float* part_prefix;                 // [split_prefix][Hk][n_prefix] when split_prefix > 1
  float* part_own;                    // [split_own][Hk][n_own] when split_own > 1
  unsigned* err;
};

// One work item; n_keys = 0: nothing to do.
struct Item {
  int hk, own, split;
  int key0, n_keys;  // rows of the prefix or of the own keys
  int tok0;          // first token of the first query tile
  int tiles;         // query tiles
  int tok_lo, tok_hi;  // tokens that see the keys, apart from causal masks
  int see0;          // causal: key key0 + r is seen by tokens >= see0 + r
};

__device__ __forceinline__ Item get_item(const WeightsArgs& a, int idx, bool report) {
  const ViewDims& d = a.d;
  Item it;
  it.n_keys = 0;
  it.tiles = 0;
  it.see0 = -2147483647;
  int n_split;
  // the prefix's items first: they are the longer ones
  it.own = idx >= a.prefix_items;
  if (!it.own) {
    n_split = a.split_prefix;
    const int r = udiv31(idx, a.prefix_units, a.m_units);
    it.hk = udiv31(r, a.split_prefix, a.m_split);
    it.split = r - it.hk * a.split_prefix;
    it.key0 = (idx - r * a.prefix_units) * ITEM;
    it.n_keys = min(ITEM, d.n_prefix - it.key0);
    it.tok_lo = max(d.q_off[0], 0);
    it.tok_hi = min(d.q_off[d.B], d.n_q);
    it.tok0 = 0;
  } else {
    n_split = a.split_own;
    int r = (idx - a.prefix_items) / a.own_units;
    const int u = idx - a.prefix_items - r * a.own_units;
    it.hk = r / (a.split_own * d.B);
    r -= it.hk * a.split_own * d.B;
    it.split = r / d.B;
    const int b = r - it.split * d.B;
    ViewRange v;
    if (!view_range(d, b, &v, report ? a.err : nullptr)) return it;
    const int nk = v.k1 - v.k0, nq = v.q1 - v.q0;
    if (u * ITEM >= nk) return it;
    it.key0 = v.k0 + u * ITEM;
    it.n_keys = min(ITEM, nk - u * ITEM);
    it.tok_lo = it.tok0 = v.q0;
    it.tok_hi = v.q1;
    if (d.causal) {
      // key j of the view is seen by its queries i >= j + nq - nk
      it.see0 = v.q0 + u * ITEM + nq - nk;
      it.tok0 += max(0, it.see0 - v.q0) / a.rows_tok * a.rows_tok;
    }
  }
  // at most 2^24 tiles and 32 ranges
  const int all = udiv31(max(0, it.tok_hi - it.tok0 + a.rows_tok - 1), a.rows_tok, a.m_tok);
  const int t0 = n_split == 1 ? 0 : all * it.split / n_split;
  it.tiles = n_split == 1 ? all : all * (it.split + 1) / n_split - t0;
  it.tok0 += t0 * a.rows_tok;
  return it;
}

__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tkp,
                       const __grid_constant__ CUtensorMap tko, const WeightsArgs a) {
  extern __shared__ __align__(1024) uint8_t tc_smem_raw[];
  const uint32_t raw = smem_u32(tc_smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* sp = tc_smem_raw + (sb - raw);
  const uint32_t sK = sb + OFF_K, sQ = sb + OFF_Q;
  auto bar = [&](int i) -> uint32_t { return sb + OFF_BAR + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + OFF_MISC + 4);
  float* sL = reinterpret_cast<float*>(sp + OFF_L);
  uint32_t* sNone = reinterpret_cast<uint32_t*>(sp + OFF_NONE);
  uint32_t* sSome = reinterpret_cast<uint32_t*>(sp + OFF_SOME);

  pdl_launch();
  const ViewDims& d = a.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int MT = a.rows_tok, tile_rows = MT * d.G;
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_KF + s), 1);
      mbar_init(bar(B_KE + s), 1);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(bar(B_QF + s), 1);
      mbar_init(bar(B_QE + s), 1 + 4 * SLOTS);  // the products, and every sum warp
      mbar_init(bar(B_LF + s), 1);
    }
    for (int t = 0; t < SLOTS; ++t) {
      mbar_init(bar(B_SF + t), 1);
      mbar_init(bar(B_SE + t), 4);
    }
    mbar_init(bar(B_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // rows of the ring that no copy fills (group sizes that do not divide 128)
  for (int s = 0; s < ST; ++s)
    for (uint32_t o = tile_rows * 128u + tid * 16u; o < kTile; o += kThreads * 16u)
      *reinterpret_cast<uint4*>(sp + OFF_Q + s * kTile + o) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), kCols);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const long long limit = d.wait_cycles;
  auto wait = [&](int b, uint32_t parity) { return mbar_wait(bar(b), parity, abort_flag, a.err, limit); };

  // every role walks the same items; `it_n` counts those with products, `step`
  // the query tiles of all of them
  if (warp == 0) {
    if (lane == 0) {
      int it_n = 0, step = 0;
      bool ok = true;
      for (int idx = blockIdx.x; ok && idx < a.n_items; idx += gridDim.x) {
        const Item it = get_item(a, idx, true);
        if (it.n_keys == 0 || it.tiles == 0) continue;
        const int kb = it_n & 1, slots = (it.n_keys + 127) / 128;
        if (it_n >= 2 && !(ok = wait(B_KE + kb, ((it_n >> 1) - 1) & 1))) break;
        mbar_expect_tx(bar(B_KF + kb), slots * kTile);
        for (int t = 0; t < slots; ++t)
          tma_load_3d(sK + (kb * SLOTS + t) * kTile, it.own ? &tko : &tkp, bar(B_KF + kb), 0, it.hk, it.key0 + t * 128);
        ++it_n;
        for (int i = 0; i < it.tiles; ++i, ++step) {
          const int s = step % ST;
          if (step >= ST && !(ok = wait(B_QE + s, (step / ST - 1) & 1))) break;
          mbar_expect_tx(bar(B_QF + s), tile_rows * 128u);
          tma_load_3d(sQ + s * kTile, &tq, bar(B_QF + s), 0, it.hk * d.G, it.tok0 + i * MT);
        }
      }
      // this CTA's own copies land before its shared memory goes away, whatever
      // becomes of the other warps
      volatile int never = 0;
      for (int k = max(0, it_n - 2); k < it_n; ++k) mbar_wait(bar(B_KF + (k & 1)), (k >> 1) & 1, &never, a.err);
      for (int k = max(0, step - ST); k < step; ++k) mbar_wait(bar(B_QF + k % ST), (k / ST) & 1, &never, a.err);
    }
  } else if (warp == 1) {
    // the whole warp runs the loop and one lane issues
    const bool leader = elect_one();
    const uint32_t id = idesc(128, 128, kFmtBF16, 0, 0);
    const uint64_t k_desc = sdesc_k(sK), q_desc = sdesc_k(sQ);  // count 16-byte units
    auto all_wait = [&](int b, uint32_t parity) { return warp_wait_fast(bar(b), parity, abort_flag, a.err, limit); };
    int it_n = 0, step = 0;
    uint32_t se_seen = 0;  // a bit for each slot: parity of its next free-wait
    uint32_t se_used = 0;  // slots that have been written before
    bool ok = true;
    for (int idx = blockIdx.x; ok && idx < a.n_items; idx += gridDim.x) {
      const Item it = get_item(a, idx, false);
      if (it.n_keys == 0 || it.tiles == 0) continue;
      const int kb = it_n & 1, slots = (it.n_keys + 127) / 128;
      if (!(ok = all_wait(B_KF + kb, (it_n >> 1) & 1))) break;
      for (int i = 0; ok && i < it.tiles; ++i, ++step) {
        const int s = step % ST;
        if (!(ok = all_wait(B_QF + s, (step / ST) & 1))) break;
        const uint64_t qd = q_desc + (uint64_t)(s * (kTile >> 4));
#pragma unroll
        for (int t = 0; t < SLOTS; ++t) {
          if (t >= slots) break;
          if (se_used >> t & 1) {
            if (!(ok = all_wait(B_SE + t, se_seen >> t & 1))) break;
            se_seen ^= 1u << t;
          }
          se_used |= 1u << t;
          fence_after_sync();
          const uint64_t kd = k_desc + (uint64_t)((kb * SLOTS + t) * (kTile >> 4));
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_bf16_ss(tbase + t * 128, kd + kk * 2, qd + kk * 2, id, kk > 0);
            mma_commit(bar(B_SF + t));
          }
        }
        if (ok && leader) mma_commit(bar(B_QE + s));
      }
      if (ok && leader) mma_commit(bar(B_KE + kb));
      ++it_n;
    }
    if (!ok) {
      // wait for the products already issued before TMEM is released
      volatile int never = 0;
      if (leader) mma_commit(bar(B_DRAIN));
      __syncwarp();
      mbar_wait(bar(B_DRAIN), 0, &never, a.err);
    }
  } else if (warp == 2) {
    int step = 0;
    bool ok = true;
    for (int idx = blockIdx.x; ok && idx < a.n_items; idx += gridDim.x) {
      const Item it = get_item(a, idx, false);
      if (it.n_keys == 0) continue;
      for (int i = 0; ok && i < it.tiles; ++i, ++step) {
        const int s = step % ST;
        const int tok0 = it.tok0 + i * MT;
        float v[4];
        uint32_t none[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = u * 32 + lane, tl = row / d.G, tok = tok0 + tl;
          // rows of no token weigh nothing, as do queries that saw no key
          float z = -CUDART_INF_F;
          if (tl < MT && tok >= it.tok_lo && tok < it.tok_hi) z = a.lse[(long long)tok * d.H + it.hk * d.G + row - tl * d.G];
          v[u] = -z * 1.4426950408889634f;
          none[u] = __ballot_sync(0xffffffffu, z == -CUDART_INF_F);
        }
        if (step >= ST && !(ok = __all_sync(0xffffffffu, wait(B_QE + s, (step / ST - 1) & 1)))) break;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          sL[s * 128 + u * 32 + lane] = v[u];
          if (lane == 0) sNone[s * 4 + u] = none[u];
        }
        if (lane == 0) sSome[s] = none[0] | none[1] | none[2] | none[3];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_LF + s));
      }
    }
  } else if (warp == 3) {
    // no item looks at the views' own keys: their offsets are looked at here
    if (blockIdx.x == 0 && a.own_units == 0) check_views(d, lane, 32, a.err);
  } else {
    const int t = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t s_addr = tbase + ((uint32_t)((warp & 3) * 32) << 16) + t * 128;
    const float c2 = d.c2;
    const uint64_t c2p = f2_pack(c2, c2);
    int step = 0;
    uint32_t sf = 0;  // parity of the slot's next product
    bool ok = true;
    for (int idx = blockIdx.x; ok && idx < a.n_items; idx += gridDim.x) {
      const Item it = get_item(a, idx, false);
      if (it.n_keys == 0) continue;
      const int r = t * 128 + row;  // the thread's key of the item
      const bool slot_live = t * 128 < it.n_keys;
      float total = 0.f, before = 0.f;  // the account so far, on its way during the products
      if (!it.own && a.acc && a.split_prefix == 1 && r < it.n_keys) before = a.acc[it.hk * a.acc_stride + it.key0 + r];
      for (int i = 0; ok && i < it.tiles; ++i, ++step) {
        const int s = step % ST;
        ok = warp_wait_fast(bar(B_LF + s), (step / ST) & 1, abort_flag, a.err, limit);
        if (!ok) break;
        if (slot_live) {
          ok = warp_wait_fast(bar(B_SF + t), sf, abort_flag, a.err, limit);
          if (!ok) break;
          sf ^= 1;
          fence_after_sync();
          // rows before lo do not see this key, and there are none from hi on
          const int tok0 = it.tok0 + i * MT;
          const int lo = (max(it.see0 + r, tok0) - tok0) * d.G;
          const int hi = it.tok_hi - tok0 >= MT ? 128 : (it.tok_hi - tok0) * d.G;
          const bool whole = __all_sync(0xffffffffu, lo == 0 && sSome[s] == 0u);
          const float4* nl = reinterpret_cast<const float4*>(sL + s * 128);
          uint64_t ps[4] = {0ull, 0ull, 0ull, 0ull};
          uint32_t sv[32];
          // SOME: without the columns whose bit is set in `skip`
          auto chunk = [&](int c, auto some, uint32_t skip) {
            constexpr bool SOME = decltype(some)::value;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float4 z = nl[8 * c + u];
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const int k = 4 * u + 2 * w;
                uint64_t x2 = f2_fma(f2_pack(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1])), c2p,
                                     w ? f2_pack(z.z, z.w) : f2_pack(z.x, z.y));
                float x0, x1;
                f2_unpack(x2, x0, x1);
                if (SOME) {
                  if (skip >> k & 1) x0 = -CUDART_INF_F;
                  if (skip >> (k + 1) & 1) x1 = -CUDART_INF_F;
                  x2 = f2_pack(x0, x1);
                }
                const uint64_t p2 = ((2 * u + w) & 7) >= 8 - kPolyOf8 ? exp2_poly2<true>(x2) : f2_pack(exp2_mufu(x0), exp2_mufu(x1));
                ps[(2 * u + w) & 3] = f2_add(ps[(2 * u + w) & 3], p2);
              }
            }
          };
          // as far as there are queries (rolled loops: registers to overlap the
          // exponentials in, and little code; with the next load in flight 1159 us at 5496
          // queries and 46716 keys of 16 heads, where it was 943 without; a loop of its
          // own for tiles whose rows all count: 38 us less)
          auto load = [&](int c, bool last) {
            tmem_ld32(s_addr + 32 * c, sv);
            tmem_wait_ld();
            if (last) {
              fence_before_sync();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(B_SE + t));
            }
          };
          if (whole) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              load(c, c == 3);
              chunk(c, std::false_type{}, 0u);
            }
          } else {
            const int chunks = max(1, (min(hi, 128) + 31) >> 5);
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              load(c, c == chunks - 1);
              const int before = lo - 32 * c;
              const uint32_t skip = sNone[s * 4 + c] | (before >= 32 ? 0xffffffffu : before > 0 ? (1u << before) - 1 : 0u);
              if (__any_sync(0xffffffffu, skip != 0u))
                chunk(c, std::true_type{}, skip);
              else
                chunk(c, std::false_type{}, 0u);
            }
          }
          const uint64_t p01 = f2_add(f2_add(ps[0], ps[1]), f2_add(ps[2], ps[3]));
          float p0, p1;
          f2_unpack(p01, p0, p1);
          total += p0 + p1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_QE + s));
      }
      if (ok && r < it.n_keys) {
        const int key = it.key0 + r;
        const int n_split = it.own ? a.split_own : a.split_prefix;
        if (n_split > 1) {
          if (it.own)
            a.part_own[((long long)it.split * d.Hk + it.hk) * d.n_own + key] = total;
          else
            a.part_prefix[((long long)it.split * d.Hk + it.hk) * d.n_prefix + key] = total;
        } else {
          if (!it.own && a.acc) total += a.decay * before;
          a.acc_out[it.hk * a.acc_out_stride + (it.own ? d.n_prefix + key : key)] = total;
        }
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    fence_after_sync();
    tmem_dealloc(tbase, kCols);
  }
}

// The sums of query ranges, in order; key j of the cache and the own keys.
__global__ void __launch_bounds__(256) add_parts_kernel(const WeightsArgs a) {
  const ViewDims& d = a.d;
  const int j = blockIdx.x * 256 + threadIdx.x, hk = blockIdx.y;
  pdl_wait();
  const long long at = hk * a.acc_out_stride + j;
  if (j < d.n_prefix) {
    if (a.split_prefix < 2) return;
    float t = 0.f;
    for (int s = 0; s < a.split_prefix; ++s) t += a.part_prefix[((long long)s * d.Hk + hk) * d.n_prefix + j];
    if (a.acc) t += a.decay * a.acc[hk * a.acc_stride + j];
    a.acc_out[at] = t;
  } else if (j < d.n_prefix + d.n_own) {
    const int k = j - d.n_prefix;
    if (a.split_own < 2 || k < d.own_off[0] || k >= d.own_off[d.B]) return;
    float t = 0.f;
    for (int s = 0; s < a.split_own; ++s) t += a.part_own[((long long)s * d.Hk + hk) * d.n_own + k];
    a.acc_out[at] = t;
  }
}

// ---------------------------------------------------------------------------
// at most eight rows

constexpr int ROWS = 8;
constexpr int KEYS_BLOCK = 128;  // keys of a block: 32 groups of eight lanes, four keys each

__device__ __forceinline__ float dot8(const uint4& u, const float (&q)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(w[i] << 16), q[2 * i], s);
    s = fmaf(__uint_as_float(w[i] & 0xffff0000u), q[2 * i + 1], s);
  }
  return s;
}

__global__ void __launch_bounds__(256)
    key_weights_rows_kernel(const WeightsArgs a, const bf16* __restrict__ q, const bf16* __restrict__ kp,
                            const bf16* __restrict__ ko, int prefix_blocks) {
  const ViewDims& d = a.d;
  const int hk = blockIdx.y, grp = threadIdx.x >> 3, e = threadIdx.x & 7;
  const bool own = (int)blockIdx.x >= prefix_blocks;
  const int key0 = ((int)blockIdx.x - (own ? prefix_blocks : 0)) * KEYS_BLOCK;
  const int n_keys = own ? d.n_own : d.n_prefix;
  const bf16* k = own ? ko : kp;
  const long long stride = own ? d.ko_stride : d.kp_stride;
  const int rows = d.n_q * d.G;
  if (blockIdx.x == 0 && hk == 0) check_views(d, threadIdx.x, 256, a.err);
  uint4 ku[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int j = key0 + u * 32 + grp;
    ku[u] = j < n_keys ? *reinterpret_cast<const uint4*>(k + j * stride + hk * 64 + e * 8) : make_uint4(0u, 0u, 0u, 0u);
  }
  float qf[ROWS][8];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = min(i, rows - 1), tl = row / d.G, h = hk * d.G + row - tl * d.G;
    const uint4 w = *reinterpret_cast<const uint4*>(q + tl * d.q_stride + h * 64 + e * 8);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      qf[i][2 * c] = __uint_as_float(x[c] << 16);
      qf[i][2 * c + 1] = __uint_as_float(x[c] & 0xffff0000u);
    }
  }
  // lane e looks after row e
  const int my_tok = e / d.G;
  const float z = e < rows ? a.lse[(long long)my_tok * d.H + hk * d.G + e - my_tok * d.G] : -CUDART_INF_F;
  const float nl = -z * 1.4426950408889634f;
  int tok_lo = max(d.q_off[0], 0), tok_hi = min(d.q_off[d.B], d.n_q);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int j = key0 + u * 32 + grp;
    bool write = j < n_keys;
    if (own) {
      // the view of the key: the last one that starts at or before it
      int lo = 0, hi = d.B;  // own_off[lo] <= j < own_off[hi], once it holds at all
      write = write && j >= d.own_off[0] && j < d.own_off[d.B];
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (d.own_off[mid] <= j) lo = mid; else hi = mid;
      }
      tok_lo = max(d.q_off[lo], 0);
      tok_hi = min(d.q_off[lo + 1], d.n_q);
      if (d.causal) tok_lo = max(tok_lo, j - d.own_off[lo + 1] + d.q_off[lo + 1]);
    }
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (i >= rows) break;
      float s = dot8(ku[u], qf[i]);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      if (i == e) mine = s;
    }
    float p = z != -CUDART_INF_F && my_tok >= tok_lo && my_tok < tok_hi ? exp2_mufu(fmaf(mine, d.c2, nl)) : 0.f;
    p += __shfl_xor_sync(0xffffffffu, p, 1);
    p += __shfl_xor_sync(0xffffffffu, p, 2);
    p += __shfl_xor_sync(0xffffffffu, p, 4);
    if (write && e == 0) {
      if (!own && a.acc) p += a.decay * a.acc[hk * a.acc_stride + j];
      a.acc_out[hk * a.acc_out_stride + (own ? d.n_prefix + j : j)] = p;
    }
  }
}

// Own keys of views of few rows: a group of eight lanes takes four keys and goes over
// the queries that see any of them.  Of the four dot products' sums over the lanes each
// pair of lanes keeps one, so that a query costs four shuffles and one exponential:
// bound by those and the latency of the reads.  256 views of a token, 250 to 500 own
// keys and 16 heads, prefix of 1374 included: 67 us at 3.1 TB/s, 130 with a key a group.
constexpr int OWN_THREADS = 128, OWN_KEYS = OWN_THREADS / 2;

__global__ void __launch_bounds__(OWN_THREADS)
    key_weights_own_kernel(const WeightsArgs a, const bf16* __restrict__ q, const bf16* __restrict__ k) {
  const ViewDims& d = a.d;
  const int hk = blockIdx.y, lane = threadIdx.x & 7, e = lane * 8;
  const int j0 = blockIdx.x * OWN_KEYS + (threadIdx.x >> 3) * 4;
  uint4 ku[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    ku[u] = j0 + u < d.n_own ? *reinterpret_cast<const uint4*>(k + (j0 + u) * d.ko_stride + hk * 64 + e)
                             : make_uint4(0u, 0u, 0u, 0u);
  if (blockIdx.x == 0 && hk == 0) check_views(d, threadIdx.x, OWN_THREADS, a.err);
  // the view of the lane's key: the last one that starts at or before it
  const int mine = lane >> 1, j = j0 + mine;
  const bool in = j < d.n_own && j >= d.own_off[0] && j < d.own_off[d.B];
  int lo = 0, hi = 0;  // the rows that see it
  if (in) {
    int v = 0;
    for (int end = d.B; end - v > 1;) {
      const int mid = (v + end) >> 1;
      if (d.own_off[mid] <= j) v = mid; else end = mid;
    }
    // offsets may be anything: a row number is formed of what the buffers hold alone
    long long see = d.q_off[v];
    if (d.causal) see = max(see, (long long)j - d.own_off[v + 1] + d.q_off[v + 1]);
    lo = (int)min(max(see, 0ll), (long long)d.n_q) * d.G;
    hi = max(min(d.q_off[v + 1], d.n_q), 0) * d.G;
  }
  float total = 0.f;
  for (int row = -1;;) {
    // the group's next row: the least that one of its keys has left
    int next = max(row + 1, lo);
    if (next >= hi) next = INT32_MAX;
    next = min(next, __shfl_xor_sync(0xffffffffu, next, 2));
    row = min(next, __shfl_xor_sync(0xffffffffu, next, 4));
    if (__all_sync(0xffffffffu, row == INT32_MAX)) break;
    const bool live = row >= lo && row < hi;
    const int x_row = row == INT32_MAX ? 0 : row, t = x_row / d.G, h = hk * d.G + x_row - t * d.G;
    float qf[8];
    const uint4 w = *reinterpret_cast<const uint4*>(q + t * d.q_stride + h * 64 + e);
    const float z = a.lse[(long long)t * d.H + h];
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      qf[2 * c] = __uint_as_float(x[c] << 16);
      qf[2 * c + 1] = __uint_as_float(x[c] & 0xffff0000u);
    }
    float s[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] = dot8(ku[u], qf);
    const bool up = lane & 4, odd = lane & 2;
    const float s0 = (up ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, up ? s[0] : s[2], 4);
    const float s1 = (up ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, up ? s[1] : s[3], 4);
    float y = (odd ? s1 : s0) + __shfl_xor_sync(0xffffffffu, odd ? s0 : s1, 2);
    y += __shfl_xor_sync(0xffffffffu, y, 1);
    if (live && z != -CUDART_INF_F) total += exp2_mufu(fmaf(y, d.c2, -z * 1.4426950408889634f));
    if (row == INT32_MAX) row = INT32_MAX - 1;  // done: stays so when it is counted up
  }
  if (in && !(lane & 1)) a.acc_out[hk * a.acc_out_stride + d.n_prefix + j] = total;
  pdl_wait();  // whoever waits for this kernel waits for the one before it too
}

__global__ void __launch_bounds__(256) check_kernel(const ViewDims d, unsigned* err) { check_views(d, threadIdx.x, 256, err); }

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

}  // namespace

WeightsPlan weights_plan(const ViewDims& d) {
  WeightsPlan p = {};
  p.split_prefix = p.split_own = 1;
  if ((long long)d.n_q * d.G <= ROWS && d.n_q > 0) {
    p.rows = 1;
    return p;
  }
  const int MT = 128 / d.G;
  p.prefix_units = ceil_div(d.n_prefix, ITEM);
  p.own_cores = (long long)d.max_q * d.G <= 16;
  p.own_units = p.own_cores ? 0 : ceil_div(d.max_own, ITEM);
  // query ranges so that the items fill the SMs evenly: an item costs its query
  // tiles and about two more, and there are as many own items as tokens at most
  const int tiles_p = ceil_div(d.n_q, MT), tiles_o = ceil_div(d.max_q, MT);
  long long own_items = (long long)d.B * p.own_units;
  if (own_items > d.n_own / ITEM + d.B) own_items = d.n_own / ITEM + d.B;
  double best = 0;
  for (int s = 1; s <= 32 && s <= (tiles_p > 1 ? tiles_p : 1); ++s) {
    const int per_p = ceil_div(tiles_p, s), so = per_p > 0 && tiles_o > 0 ? ceil_div(tiles_o, per_p) : 1;
    const double items = ((double)p.prefix_units * s + (double)own_items * so) * d.Hk;
    const double work = ((double)p.prefix_units * s * (per_p + 2.0) + (double)own_items * so * (ceil_div(tiles_o, so) + 2.0)) * d.Hk;
    const double longest = (per_p > ceil_div(tiles_o, so) ? per_p : ceil_div(tiles_o, so)) + 2.0;
    const double cost = work / 148.0 + (items > 148.0 ? 0.5 : 1.0) * longest + (s > 1 ? 6.0 : 0.0);
    if (s == 1 || cost < best) {
      WeightsPlan x = p;
      x.split_prefix = s;
      x.split_own = so;
      if (s > 1 && weights_items(d, x) > kMostItems) break;
      best = cost;
      p = x;
    }
  }
  return p;
}

cudaError_t launch_key_weights(const ViewDims& d, const WeightsPlan& p, const bf16* q, const bf16* kp, const bf16* ko,
                               const float* lse, const float* acc, long long acc_stride, float* acc_out,
                               long long acc_out_stride, float decay, float* part_prefix, float* part_own, unsigned* err, cudaStream_t st) {
  if (d.n_prefix + d.n_own <= 0) return cudaSuccess;
  WeightsArgs a = {};
  a.d = d;
  a.lse = lse;
  a.acc = decay != 0.f ? acc : nullptr;
  a.acc_out = acc_out;
  a.decay = decay;
  a.acc_stride = acc_stride;
  a.acc_out_stride = acc_out_stride;
  a.part_prefix = part_prefix;
  a.part_own = part_own;
  a.err = err;
  if (p.rows) {
    const int pb = ceil_div(d.n_prefix, KEYS_BLOCK), ob = ceil_div(d.n_own, KEYS_BLOCK);
    key_weights_rows_kernel<<<dim3((unsigned)(pb + ob), (unsigned)d.Hk), 256, 0, st>>>(a, q, kp, ko, pb);
    return cudaGetLastError();
  }
  const int MT = 128 / d.G;
  a.rows_tok = MT;
  a.prefix_units = p.prefix_units;
  a.own_units = p.own_units;
  a.split_prefix = p.split_prefix;
  a.split_own = p.split_own;
  a.prefix_items = p.prefix_units * p.split_prefix * d.Hk;
  a.m_units = 0xffffffffu / (uint32_t)(p.prefix_units > 0 ? p.prefix_units : 1);
  a.m_split = 0xffffffffu / (uint32_t)p.split_prefix;
  a.m_tok = 0xffffffffu / (uint32_t)MT;
  a.n_items = (int)weights_items(d, p);
  if (a.n_items > 0) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(key_weights_kernel, (int)kSmemBytes, &done);
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mkp, mko;
    auto map = [&](CUtensorMap* m, const bf16* base, int heads, int rows, long long stride, int b1, int b2) {
      return make_tmap_3d(m, false, base, 64, (unsigned long long)heads, (unsigned long long)rows, 128,
                          (unsigned long long)stride * 2, 64, (unsigned)b1, (unsigned)b2);
    };
    bool ok = true;
    if (d.n_prefix > 0) ok = ok && map(&mkp, kp, d.Hk, d.n_prefix, d.kp_stride, 1, 128);
    if (d.n_own > 0) ok = ok && map(&mko, ko, d.Hk, d.n_own, d.ko_stride, 1, 128);
    // a map that no item uses still has to be one
    if (d.n_prefix <= 0) mkp = mko;
    if (d.n_own <= 0) mko = mkp;
    if (d.n_q > 0)
      ok = ok && map(&mq, q, d.H, d.n_q, d.q_stride, d.G, MT);
    else
      mq = mkp;
    if (!ok) return cudaErrorInvalidValue;
    const int grid = a.n_items < 148 ? a.n_items : 148;
    key_weights_kernel<<<(unsigned)grid, kThreads, kSmemBytes, st>>>(mq, mkp, mko, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.n_items == 0 && !(p.own_cores && d.n_own > 0)) {
    // no key to weigh: offsets that say otherwise are reported
    check_kernel<<<1, 256, 0, st>>>(d, err);
    return cudaGetLastError();
  }
  if (p.own_cores && d.n_own > 0) {
    const dim3 grid((unsigned)ceil_div(d.n_own, OWN_KEYS), (unsigned)d.Hk);
    if (a.n_items > 0 && p.split_prefix == 1)
      return launch_second(key_weights_own_kernel, grid, OWN_THREADS, st, a, q, ko);
    key_weights_own_kernel<<<grid, OWN_THREADS, 0, st>>>(a, q, ko);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (p.split_prefix > 1 || p.split_own > 1) {
    return launch_second(add_parts_kernel, dim3((unsigned)ceil_div((long long)d.n_prefix + d.n_own, 256), (unsigned)d.Hk),
                         256, st, a);
  }
  return cudaSuccess;
}

}  // namespace gsa
