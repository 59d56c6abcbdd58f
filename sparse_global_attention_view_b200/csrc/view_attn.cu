// Attention of a batch of views that share one prefix (a cache of the views
// seen so far): softmax over the prefix and the view's own keys.
//
// For query i of view b (rows packed one behind the other, views ragged):
//   s_ij = scale q_i . k_j over the prefix keys and the view's own keys,
//   out_i = sum_j exp(s_ij - lse_i) v_j,  lse_i = log sum_j exp s_ij.
// The softmax is associative over key ranges, so ranges are taken by different
// CTAs where there are few rows, and (out, lse) pairs are merged afterwards.
//
// view_attn_kernel (tcgen05 / TMEM / TMA): one CTA = up to two 128-row query
// tiles of one key head.  A row is a (token, query head of the group) pair, so
// the G query heads that share a key head share its K/V tiles.  20 warps:
//   warp 0      TMA producer: the Q tiles once, then a 6-stage ring of 128-key K/V
//               tiles; zeroes the value rows behind a view's last key;
//   warps 1, 3  MMA issuers of two streams each;
//   warp 2      TMEM allocation;
//   warps 4-19  softmax, one warpgroup a stream, one thread a row.
// A stream is one query tile against one 64-key half of every key tile: it has a
// softmax state, 64 TMEM columns of scores (P is written over them) and 64 of
// output of its own.  Two streams serve a query tile; with one tile of rows all
// four do, each with half of every other key tile.  Streams never wait for one
// another; their results are joined in shared memory at the end.  Four streams
// give every scheduler four softmax warps: a step of one of them (load, maximum,
// exponentials, store, two products) is a chain of latencies that only other
// warps can fill, and with two tiles of 128 x 128 scores and two warps a
// scheduler the exponential units idled half the time.
// view_rows_kernel: at most four rows in all against the prefix.  Bound by the read
// of the cache; CUDA cores, eight lanes a key, four keys' loads in flight a lane.
// Over a short prefix latency is what counts: the blocks of a head are a cluster
// then, whose first one takes the own keys too and joins all of it: one launch.
// view_own_kernel: views of few rows.  Their own keys are read by CUDA cores
// (eight lanes a key, plain 16-byte loads: nothing is read that no query sees),
// and the partial results against the prefix are merged in the same pass.
// merge_kernel: partial results only.
//
// Every sum, maximum and partial result is fp32; P is rounded to bf16 for the
// product with V (a relative 2^-8 each at most, independent between keys), and the
// denominator sums the unrounded weights.
#include <cooperative_groups.h>
#include <math.h>
#include <math_constants.h>

#include "exp2_poly.cuh"
#include "views.h"

namespace gsa {
namespace {

using namespace tc;

constexpr int kPolyOf8 = 1;  // pairs of exponentials in eight on the FMA pipe
constexpr int TK = 128;      // keys per key tile
constexpr int HK = 64;       // keys of a stream's half
constexpr int NS = 4;        // streams
constexpr int ST = 6;        // K/V ring stages
constexpr int kThreads = 128 + 128 * NS;
constexpr uint32_t kTile = 128 * 128;  // bytes of one [128][64] bf16 tile

constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_K = OFF_Q + 2 * kTile;
constexpr uint32_t OFF_V = OFF_K + ST * kTile;
constexpr uint32_t OFF_BAR = OFF_V + ST * kTile;
constexpr uint32_t OFF_MISC = OFF_BAR + 384;
constexpr uint32_t kSmemBytes = OFF_MISC + 64 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
// results on their way to another stream: 64 values, maximum and sum a row, over the ring
constexpr int JOIN = 68;  // floats a row: 16-byte accesses of a thread a row meet no bank conflicts
static_assert((NS - 1) * 128 * JOIN * 4 <= 2 * ST * kTile, "join area");

constexpr int B_Q = 0, B_KF = 1, B_KVE = B_KF + ST, B_SF = B_KVE + ST, B_PF = B_SF + NS,
              B_OF = B_PF + NS, B_VZ = B_OF + NS, B_END = B_VZ + 1, B_JOIN = B_END + 1, B_DRAIN = B_JOIN + 1,
              B_COUNT = B_DRAIN + 2;
static_assert(B_COUNT * 8 <= 384, "barrier area");

constexpr uint32_t kCols = 512, COL_O = 256;  // TMEM: stream x has S, then P, at 64 x, and O at 256 + 64 x

struct ViewAttnArgs {
  ViewDims d;
  int rows_tok;   // tokens per row tile: 128 / G
  int aligned, do_prefix, do_own, check_views;
  int n_split, units_per_view;
  bf16* out;      // written directly when part_o is null
  float* lse;     // nullable
  float* part_o;  // [parts][n_q][H][64], normalised
  float* part_lse;  // [parts][n_q][H], log2 units
  int part0;
  unsigned* err;
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* err,
                                          long long limit) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err, limit));
}

__global__ void __launch_bounds__(kThreads, 1)
    view_attn_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tkp,
                     const __grid_constant__ CUtensorMap tvp, const __grid_constant__ CUtensorMap tko,
                     const __grid_constant__ CUtensorMap tvo, const ViewAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t tc_smem_raw[];
  const uint32_t raw = smem_u32(tc_smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* sp = tc_smem_raw + (sb - raw);
  const uint32_t sQ = sb + OFF_Q, sK = sb + OFF_K, sV = sb + OFF_V;
  auto bar = [&](int i) -> uint32_t { return sb + OFF_BAR + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + OFF_MISC + 4);

  pdl_launch();
  const ViewDims& d = a.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.y;
  const int unit = (int)(blockIdx.x / (unsigned)a.n_split), split = blockIdx.x - unit * a.n_split;
  const int MT = a.rows_tok, unit_tok = 2 * MT;

  // this CTA's rows [tok0, tok_end) and keys; uniform over the CTA
  long long tok0;
  int tok_lo, tok_end, q0 = 0, nq = 0, k0 = 0, nk = 0;
  if (a.aligned) {
    const int b = unit / a.units_per_view, c = unit - b * a.units_per_view;
    ViewRange r;
    if (!view_range(d, b, &r, a.err)) return;
    tok0 = (long long)r.q0 + (long long)c * unit_tok;
    if (tok0 >= r.q1) return;
    tok_lo = q0 = r.q0;
    tok_end = r.q1;
    nq = r.q1 - r.q0;
    k0 = r.k0;
    nk = a.do_own ? r.k1 - r.k0 : 0;
  } else {
    tok0 = (long long)unit * unit_tok;
    tok_lo = max(d.q_off[0], 0);
    tok_end = min(d.q_off[d.B], d.n_q);
    if (tok0 >= tok_end || tok0 + unit_tok <= tok_lo) {
      // a launch that reads no own keys still reports offsets that promise some: a block
      // behind the rows (checks elsewhere in the kernel cost its softmax registers: 1325
      // us at 5496 x 42594 x 16 heads against 1306)
      if (a.check_views && blockIdx.x == gridDim.x - 1 && blockIdx.y == 0) check_views(d, tid, kThreads, a.err);
      return;
    }
  }
  const int last_row = (int)min(tok0 + unit_tok, (long long)tok_end) - 1;
  // own keys seen by at least one of the rows
  int nk_seen = nk;
  if (d.causal) nk_seen = max(0, min(nk, last_row - q0 + nk - nq + 1));
  const int np = a.do_prefix ? (d.n_prefix + TK - 1) / TK : 0;
  const int nt_all = np + (nk_seen + TK - 1) / TK;
  // at most 2^24 tiles and 64 splits
  const int j0 = (int)((unsigned)(nt_all * split) / (unsigned)a.n_split);
  const int nt = (int)((unsigned)(nt_all * (split + 1)) / (unsigned)a.n_split) - j0;
  // one tile of rows: issuer w and its streams take every other key tile, else
  // all key tiles of query tile w.  The i-th step is key tile j0 + at(w, i)
  const bool one = tok0 + MT >= tok_end;
  auto at = [&](int w, int i) -> int { return one ? 2 * i + w : i; };
  auto steps = [&](int w) -> int { return one ? (nt + 1 - w) / 2 : nt; };
  // the value rows behind the view's last seen key hold other tokens: zeroed
  const bool zero_tail = nt > 0 && j0 + nt == nt_all && nt_all > np && (nk_seen % TK) != 0;

  if (tid == 0) {
    mbar_init(bar(B_Q), 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(bar(B_KF + s), 1);
      mbar_init(bar(B_KVE + s), one ? 1 : 2);
    }
    for (int x = 0; x < NS; ++x) {
      mbar_init(bar(B_SF + x), 1);
      mbar_init(bar(B_PF + x), 4);
      mbar_init(bar(B_OF + x), 1);
    }
    mbar_init(bar(B_VZ), 1);
    mbar_init(bar(B_END), 4 * NS);
    mbar_init(bar(B_JOIN), 4 * NS);
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_DRAIN + 1), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), kCols);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const long long limit = d.wait_cycles;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0 && nt > 0) {
      const int q_tiles = one ? 1 : 2;
      mbar_expect_tx(bar(B_Q), (uint32_t)(q_tiles * MT * d.G) * 128u);
      for (int t = 0; t < q_tiles; ++t) tma_load_3d(sQ + t * kTile, &tq, bar(B_Q), 0, hk * d.G, (int)(tok0 + t * MT));
      int issued = 0;
      for (int i = 0; i < nt; ++i) {
        const int s = i % ST;
        if (i >= ST && !mbar_wait(bar(B_KVE + s), ((i / ST) - 1) & 1, abort_flag, a.err, limit)) break;
        const int j = j0 + i;
        const bool pre = j < np;
        const int row = pre ? j * TK : k0 + (j - np) * TK;
        mbar_expect_tx(bar(B_KF + s), 2 * kTile);
        tma_load_3d(sK + s * kTile, pre ? &tkp : &tko, bar(B_KF + s), 0, hk, row);
        tma_load_3d(sV + s * kTile, pre ? &tvp : &tvo, bar(B_KF + s), 0, hk, row);
        issued = i + 1;
      }
      // this CTA's own copies land before its shared memory goes away, whatever
      // becomes of the other warps
      volatile int never = 0;
      mbar_wait(bar(B_Q), 0, &never, a.err);
      for (int i = issued - 1; i >= 0 && i >= issued - ST; --i) {
        mbar_wait(bar(B_KF + i % ST), (i / ST) & 1, &never, a.err);
      }
    }
    __syncwarp();
    if (zero_tail && !*abort_flag) {
      // value rows of other tokens: their weights are 0, but 0 x infinity or NaN
      // is not.  The last copy has been issued, so its phase is the one waited for
      const int i = nt - 1, s = i % ST;
      if (warp_wait(bar(B_KF + s), (i / ST) & 1, abort_flag, a.err, limit)) {
        uint8_t* v = sp + OFF_V + s * kTile;
        for (uint32_t o = (uint32_t)(nk_seen % TK) * 128u + lane * 16u; o < kTile; o += 512u)
          *reinterpret_cast<uint4*>(v + o) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_VZ));
      }
    }
  } else if (warp == 1 || warp == 3) {
    // ---------------- MMA issuer of streams 2 w and 2 w + 1 ----------------
    // the whole warp runs the loop, one lane issues
    const int w = __shfl_sync(0xffffffffu, warp >> 1, 0), n = steps(w);
    if (n > 0) {
      const bool leader = elect_one();
      const uint32_t id_qk = idesc(128, HK, kFmtBF16, 0, 0);
      const uint32_t id_pv = idesc(128, 64, kFmtBF16, 0, 1);
      const uint64_t q_desc = sdesc_k(sQ + (one ? 0 : w) * kTile);
      const uint64_t k_desc = sdesc_k(sK), v_desc = sdesc_mn(sV);
      auto wait = [&](int b, uint32_t parity) { return warp_wait_fast(bar(b), parity, abort_flag, a.err, limit); };
      // descriptors count 16-byte units
      auto issue_s = [&](int s, int half) {
        const uint32_t x = 2 * w + half;
        const uint64_t kd = k_desc + (uint64_t)(s * (kTile >> 4) + half * (HK * 128 >> 4));
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_bf16_ss(tbase + x * 64, q_desc + kk * 2, kd + kk * 2, id_qk, kk > 0);
          mma_commit(bar(B_SF + x));
        }
      };
      // ring stage and phase of the present and the next step
      const int step = one ? 2 : 1;
      int s = one ? w : 0, s1 = s;
      uint32_t ph = 0, ph1 = 0;
      bool ok = wait(B_Q, 0) && wait(B_KF + s, 0);
      if (ok) {
        fence_after_sync();
        issue_s(s, 0);
        issue_s(s, 1);
      }
      for (int i = 0; ok && i < n; ++i) {
        s1 = s + step;
        ph1 = ph;
        if (s1 >= ST) {
          s1 -= ST;
          ph1 ^= 1;
        }
        if (zero_tail && at(w, i) == nt - 1) ok = wait(B_VZ, 0);
        if (ok && i + 1 < n) ok = wait(B_KF + s1, ph1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t x = 2 * w + half;
          if (ok) ok = wait(B_PF + x, i & 1);
          if (!ok) break;
          fence_after_sync();
          const uint64_t vd = v_desc + (uint64_t)(s * (kTile >> 4) + half * (HK * 128 >> 4));
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ts(tbase + COL_O + x * 64, tbase + x * 64 + kk * 8, vd + kk * (2048 >> 4), id_pv,
                          (i > 0 || kk > 0) ? 1u : 0u);
          }
          if (i + 1 < n) {
            // the scores come over the P just read: products complete in order
            issue_s(s1, half);
          } else if (leader) {
            mma_commit(bar(B_OF + x));
          }
        }
        if (ok && leader) mma_commit(bar(B_KVE + s));
        s = s1;
        ph = ph1;
      }
      if (!ok) {
        // wait for the products already issued before TMEM is released
        volatile int never = 0;
        if (leader) mma_commit(bar(B_DRAIN + w));
        __syncwarp();
        mbar_wait(bar(B_DRAIN + w), 0, &never, a.err);
      }
    }
  } else if (warp >= 4) {
    // ---------------- softmax of stream x, one thread a row ----------------
    const int x = (warp - 4) >> 2, w = x >> 1, half = x & 1;
    const int row = (warp & 3) * 32 + lane;
    const int tl = row / d.G, g = row - tl * d.G;
    const long long tok = tok0 + (one ? 0 : w * MT) + tl;
    const bool valid = tl < MT && tok >= tok_lo && tok < tok_end;
    // own keys [0, own_end) of the view are seen by this row
    int own_end = nk;
    if (d.causal && valid) own_end = max(0, min(nk, (int)(tok - q0) + nk - nq + 1));
    const bool work = __any_sync(0xffffffffu, valid);
    const uint32_t s_addr = tbase + ((uint32_t)((warp & 3) * 32) << 16) + x * 64;
    const uint32_t o_addr = s_addr + COL_O;
    const float c2 = d.c2;
    const int n = steps(w);
    float m_used = -CUDART_INF_F, l = 0.f;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      // S of this step, and with it the product of the step before, is complete
      ok = warp_wait(bar(B_SF + x), i & 1, abort_flag, a.err, limit);
      if (!ok) break;
      fence_after_sync();
      if (work) {
        uint32_t sv[2][32];
        tmem_ld32(s_addr, sv[0]);
        tmem_ld32(s_addr + 32, sv[1]);
        tmem_wait_ld();
        const int j = j0 + at(w, i);
        const int end = (j < np ? d.n_prefix - j * TK : own_end - (j - np) * TK) - half * HK;
        if (end < HK) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int u = 0; u < 32; ++u)
              if (32 * c + u >= end) sv[c][u] = __float_as_uint(-CUDART_INF_F);
        }
        // eight independent chains: a thread owns a whole row
        auto sval = [&](int k) -> float { return __uint_as_float(sv[k >> 5][k & 31]); };
        float mq[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) mq[u] = max_nan(sval(u), sval(u + 8));
#pragma unroll
        for (int k = 16; k < HK; k += 16)
#pragma unroll
          for (int u = 0; u < 8; ++u) mq[u] = max3_nan(mq[u], sval(k + u), sval(k + 8 + u));
        const float mx = max3_nan(max3_nan(mq[0], mq[1], mq[2]), max3_nan(mq[3], mq[4], mq[5]), max_nan(mq[6], mq[7]));
        float mxs = mx * c2;
        if (mxs == CUDART_INF_F) mxs = CUDART_NAN_F;  // infinity - infinity
        // the maximum in use is raised only when a score exceeds it by 2^8; a NaN
        // score makes it NaN, and with it the row
        const bool need = !(mxs <= m_used + 8.f);
        if (__any_sync(0xffffffffu, need)) {
          const float corr = need ? exp2f(m_used - mxs) : 1.f;
          if (i > 0) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t ov[16];
              tmem_ld16(o_addr + 16 * c, ov);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 16; ++u) ov[u] = __float_as_uint(__uint_as_float(ov[u]) * corr);
              tmem_st16(o_addr + 16 * c, ov);
            }
          }
          if (need) {
            l *= corr;
            m_used = mxs;
          }
        }
        // a row that has seen no key yet keeps finite arithmetic: weights 2^-inf = 0
        const float shift = m_used == -CUDART_INF_F ? 0.f : -m_used;
        const uint64_t c2p = f2_pack(c2, c2), nmp = f2_pack(shift, shift);
        uint64_t ps2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const uint64_t x2 =
                f2_fma(f2_pack(__uint_as_float(sv[c][2 * u]), __uint_as_float(sv[c][2 * u + 1])), c2p, nmp);
            uint64_t p2;
            if ((u & 7) >= 8 - kPolyOf8) {
              p2 = exp2_poly2<false>(x2);
            } else {
              float x0, x1;
              f2_unpack(x2, x0, x1);
              p2 = f2_pack(exp2_mufu(x0), exp2_mufu(x1));
            }
            ps2[u & 3] = f2_add(ps2[u & 3], p2);
            float p0, p1;
            f2_unpack(p2, p0, p1);
            pk[u] = pack_bf16x2(p0, p1);
          }
          tmem_st16(s_addr + 16 * c, pk);
        }
        tmem_wait_st();
        const uint64_t s01 = f2_add(f2_add(ps2[0], ps2[1]), f2_add(ps2[2], ps2[3]));
        float lo, hi;
        f2_unpack(s01, lo, hi);
        l += lo + hi;
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PF + x));
    }
    if (ok && n > 0) ok = warp_wait(bar(B_OF + x), 0, abort_flag, a.err, limit);
    // all streams are through with the ring: their results meet there
    if (ok) {
      fence_after_sync();
      if (lane == 0) mbar_arrive(bar(B_END));
      ok = warp_wait(bar(B_END), 0, abort_flag, a.err, limit);
    }
    // slot of the join area; the first stream of a tile collects
    const int slot = one ? x - 1 : (half ? w : -1);
    float* join = reinterpret_cast<float*>(sp + OFF_K) + row * JOIN;
    if (ok && slot >= 0) {
      float* mine = join + slot * 128 * JOIN;
      mine[64] = m_used;
      mine[65] = l;
      if (n > 0 && work) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t ov[16];
          tmem_ld16(o_addr + 16 * c, ov);
          tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 16; u += 4)
            *reinterpret_cast<uint4*>(mine + 16 * c + u) = make_uint4(ov[u], ov[u + 1], ov[u + 2], ov[u + 3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_JOIN));
    } else if (ok) {
      if (lane == 0) mbar_arrive(bar(B_JOIN));
      ok = warp_wait(bar(B_JOIN), 0, abort_flag, a.err, limit);
    }
    if (ok && slot < 0 && work) {
      // (maximum, sum, values) of the streams that share the rows
      const int first = one ? 0 : w, others = one ? NS - 1 : 1;
      float m = m_used;
      for (int k = 0; k < others; ++k) m = fmaxf(m, join[(first + k) * 128 * JOIN + 64]);
      // 2^(m_k - m): 0 for a stream that saw no key, NaN for one that saw a NaN
      auto factor = [&](float mk) -> float { return mk == -CUDART_INF_F ? 0.f : exp2f(mk - m); };
      const float f0 = factor(m_used);
      float lt = m_used == -CUDART_INF_F ? l * 0.f : l * f0;
      for (int k = 0; k < others; ++k) {
        const float* o = join + (first + k) * 128 * JOIN;
        lt += o[64] == -CUDART_INF_F ? o[65] * 0.f : o[65] * factor(o[64]);
      }
      // no key seen: zeros and a log sum of -infinity
      const bool empty = lt == 0.f;
      const float inv = empty ? 0.f : 1.f / lt;
      const float lse2 = empty ? -CUDART_INF_F : m + log2f(lt);
      const int h = hk * d.G + g;
      const long long rh = tok * d.H + h;
      const long long part = a.part0 + split;
      // the row is put together where the first of the others left its values, and goes
      // out from there as one copy of whole lines (stores of a thread a row, each of 32
      // rows' 16 bytes, took 7600 cycles of a CTA's 17500 beside its steps)
      float* row_out = join + first * 128 * JOIN;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float o[16];
        uint32_t ov[16];
        if (n > 0) {
          tmem_ld16(o_addr + 16 * c, ov);
          tmem_wait_ld();
        }
#pragma unroll
        for (int u = 0; u < 16; ++u) o[u] = f0 == 0.f ? 0.f : __uint_as_float(ov[u]) * f0;
        for (int k = 0; k < others; ++k) {
          const float* src = join + (first + k) * 128 * JOIN;
          const float f = factor(src[64]);
          if (f == 0.f) continue;  // nothing was stored where no key was seen
#pragma unroll
          for (int u = 0; u < 16; u += 4) {
            const float4 y = *reinterpret_cast<const float4*>(src + 16 * c + u);
            o[u] = fmaf(y.x, f, o[u]);
            o[u + 1] = fmaf(y.y, f, o[u + 1]);
            o[u + 2] = fmaf(y.z, f, o[u + 2]);
            o[u + 3] = fmaf(y.w, f, o[u + 3]);
          }
        }
#pragma unroll
        for (int u = 0; u < 16; ++u) o[u] *= inv;
        if (a.part_o) {
#pragma unroll
          for (int u = 0; u < 16; u += 4)
            *reinterpret_cast<float4*>(row_out + 16 * c + u) = make_float4(o[u], o[u + 1], o[u + 2], o[u + 3]);
        } else {
          // behind what is still to be read of the fp32 values: in the first half of them
          uint32_t pw[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) pw[u] = pack_bf16x2(o[2 * u], o[2 * u + 1]);
          uint4* dst = reinterpret_cast<uint4*>(row_out + 8 * c);
          dst[0] = make_uint4(pw[0], pw[1], pw[2], pw[3]);
          dst[1] = make_uint4(pw[4], pw[5], pw[6], pw[7]);
        }
      }
      fence_proxy_async_smem();
      if (valid && !(a.part_o && empty)) {  // the merge skips an empty part by its log sum
        if (a.part_o)
          bulk_store(a.part_o + (part * d.n_q * d.H + rh) * 64, smem_u32(row_out), 256);
        else
          bulk_store(a.out + tok * d.o_stride + h * 64, smem_u32(row_out), 128);
      }
      if (valid) {
        if (a.part_o)
          a.part_lse[part * d.n_q * d.H + rh] = lse2;
        else if (a.lse)
          a.lse[rh] = lse2 * 0.6931471805599453f;
      }
      bulk_store_wait();  // shared memory has been read before it goes away
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    fence_after_sync();
    tmem_dealloc(tbase, kCols);
  }
}

// ---------------------------------------------------------------------------
// merging partial results

// The kernels below start before the one whose results they read has ended
// (pdl_wait): those pointers carry no __restrict__, which would allow their loads to
// be moved ahead of the wait.
// Merges (o, lse2) pairs; o normalised.  A pair of lse2 = -infinity holds no key.
struct Merge {
  float m;  // largest lse2 so far, NaN ones aside
  float l;  // sum of 2^(lse2 - m)
  __device__ __forceinline__ Merge() : m(-INFINITY), l(0.f) {}
  // factor of the sums so far, and weight of the new pair
  __device__ __forceinline__ bool add(float lse2, float* keep, float* w) {
    if (lse2 == -CUDART_INF_F) return false;
    const float mn = fmaxf(m, lse2);
    *keep = m == -CUDART_INF_F ? 0.f : exp2f(m - mn);
    *w = exp2f(lse2 - mn);
    l = l * *keep + *w;
    m = mn;
    return true;
  }
  __device__ __forceinline__ float lse() const {
    return l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
  }
  __device__ __forceinline__ float inv() const { return l == 0.f ? 0.f : 1.f / l; }
};

// Eight lanes a (token, head); every lane eight of the 64 values.
__global__ void __launch_bounds__(256) merge_kernel(const ViewDims d, int parts, const float* part_o, const float* part_lse,
                                                    bf16* out, float* lse, unsigned* err) {
  if (blockIdx.x == 0) check_views(d, threadIdx.x, 256, err);
  const long long rh = ((long long)blockIdx.x * 256 + threadIdx.x) >> 3;
  const int e = (threadIdx.x & 7) * 8;
  const long long n = (long long)d.n_q * d.H;
  if (rh >= n) return;
  pdl_wait();
  const int tok = (int)(rh / d.H), h = (int)(rh - (long long)tok * d.H);
  if (tok < d.q_off[0] || tok >= d.q_off[d.B]) return;
  Merge mg;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < parts; ++p) {
    float keep, w;
    if (!mg.add(part_lse[p * n + rh], &keep, &w)) continue;
    const float4* src = reinterpret_cast<const float4*>(part_o + (p * n + rh) * 64 + e);
    const float4 x = src[0], y = src[1];
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int u = 0; u < 8; ++u) acc[u] = acc[u] * keep + v[u] * w;
  }
  const float inv = mg.inv();
  uint32_t w[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) w[u] = pack_bf16x2(acc[2 * u] * inv, acc[2 * u + 1] * inv);
  *reinterpret_cast<uint4*>(out + tok * d.o_stride + h * 64 + e) = make_uint4(w[0], w[1], w[2], w[3]);
  if (lse && e == 0) lse[rh] = mg.lse();
}

// ---------------------------------------------------------------------------
// CUDA-core kernels: eight lanes hold a key's 64 values

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// Sum over the eight lanes.
__device__ __forceinline__ float sum8(float s) {
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  return s + __shfl_xor_sync(0xffffffffu, s, 4);
}

// A softmax on its way: maximum, sum, and the lane's eight of 64 values.
struct Row {
  float m, l, o[8];
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = 0.f;
  }
  // takes a key of score s
  __device__ __forceinline__ void add(float s, const float (&v)[8]) {
    // exp2f(-infinity - -infinity) would be NaN for scores of -infinity
    const float mn = fmaxf(m, s);
    const float corr = m == mn ? 1.f : exp2f(m - mn);
    const float p = s == -INFINITY ? 0.f : exp2f(s - mn);
    l = l * corr + p;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = fmaf(p, v[c], o[c] * corr);
    m = mn;
  }
  // raises the maximum to scores that come; take() then turns one into its weight
  template <int N>
  __device__ __forceinline__ void raise(float (&s)[N]) {
    float mn = m;
#pragma unroll
    for (int u = 0; u < N; ++u) mn = fmaxf(mn, s[u]);
    const float corr = m == mn ? 1.f : exp2f(m - mn);
    m = mn;
    l *= corr;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] *= corr;
  }
  __device__ __forceinline__ void take(float s, const float (&v)[8]) {
    const float p = s == -INFINITY ? 0.f : exp2f(s - m);
    l += p;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = fmaf(p, v[c], o[c]);
  }
  // joins another state: its maximum, sum and the lane's values
  __device__ __forceinline__ void join(float mo, float lo, const float* vo) {
    const float mn = fmaxf(m, mo);
    // equal maxima, two infinite ones among them, need no factor
    const float ca = m == mn ? 1.f : exp2f(m - mn), cb = mo == mn ? 1.f : exp2f(mo - mn);
    l = l * ca + lo * cb;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = o[c] * ca + vo[c] * cb;
    m = mn;
  }
  // joins the states of the lanes that differ in bits 3 and 4
  __device__ __forceinline__ void join_groups() {
#pragma unroll
    for (int x = 8; x <= 16; x <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m, x), lo = __shfl_xor_sync(0xffffffffu, l, x);
      const float mn = fmaxf(m, mo);
      // equal maxima, two infinite ones among them, need no factor
      const float ca = m == mn ? 1.f : exp2f(m - mn), cb = mo == mn ? 1.f : exp2f(mo - mn);
      l = l * ca + lo * cb;
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = o[c] * ca + __shfl_xor_sync(0xffffffffu, o[c], x) * cb;
      m = mn;
    }
  }
};

constexpr int ROWS_THREADS = 512, ROWS_UNROLL = 4;

constexpr int ROWS_CLUSTER = 8;

struct RowsArgs {
  const bf16 *q, *kp, *vp, *ko, *vo;
  float *part_o, *part_lse;  // JOINED false: partial results
  bf16* out;                 // JOINED: results
  float* lse;
  unsigned* err;
};

// Block (split, key head): rows [0, R) against the split's part of the prefix.  With
// JOINED the splits of a head are a cluster, and its first block finishes the rows.
template <int R, bool JOINED>
__global__ void __launch_bounds__(ROWS_THREADS, R == 1 && !JOINED ? 2 : 1) view_rows_kernel(const ViewDims d, const RowsArgs a) {
  namespace cg = cooperative_groups;
  if (JOINED)
    cg::this_cluster().barrier_arrive();  // this block has started
  else
    pdl_launch();
  const bf16* __restrict__ q = a.q;
  const bf16* __restrict__ k = a.kp;
  const bf16* __restrict__ v = a.vp;
  constexpr int WARPS = ROWS_THREADS / 32, GROUPS = ROWS_THREADS / 8;
  __shared__ float s_m[WARPS][R], s_l[WARPS][R], s_o[WARPS][R][64], s_row[ROWS_CLUSTER][R][66];
  const int hk = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, e = (lane & 7) * 8;
  const int rows = d.n_q * d.G;
  const int j0 = (int)((long long)d.n_prefix * blockIdx.x / gridDim.x);
  const int j1 = (int)((long long)d.n_prefix * (blockIdx.x + 1) / gridDim.x);
  const bf16* kb = k + hk * 64 + e;
  const bf16* vb = v + hk * 64 + e;
  uint4 ku[ROWS_UNROLL], vu[ROWS_UNROLL];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < ROWS_UNROLL; ++u) {
      const int j = base + u * GROUPS;
      ku[u] = vu[u] = make_uint4(0u, 0u, 0u, 0u);
      if (j < j1) {
        ku[u] = *reinterpret_cast<const uint4*>(kb + j * d.kp_stride);
        vu[u] = *reinterpret_cast<const uint4*>(vb + j * d.vp_stride);
      }
    }
  };
  if (JOINED) load(j0 + (tid >> 3));  // on their way together with the queries
  float qf[R][8];
  Row st[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = min(i, rows - 1), tl = row / d.G, h = hk * d.G + row - tl * d.G;
    unpack8(*reinterpret_cast<const uint4*>(q + tl * d.q_stride + h * 64 + e), qf[i]);
#pragma unroll
    for (int c = 0; c < 8; ++c) qf[i][c] *= d.c2;
    st[i].clear();
  }
  const bool first = JOINED && blockIdx.x == 0;
  int q_lo = 0, q_hi = 0;
  if (first) {
    // looked at behind the prefix: on their way during it
    q_lo = d.q_off[0];
    q_hi = d.q_off[d.B];
    asm volatile("prefetch.global.L1 [%0];\n" ::"l"(d.own_off));
  }
  for (int base = j0 + (tid >> 3); base < j1 + (tid >> 3); base += GROUPS * ROWS_UNROLL) {
    if (!JOINED || base >= j0 + GROUPS) load(base);
    float s[R][ROWS_UNROLL];
#pragma unroll
    for (int u = 0; u < ROWS_UNROLL; ++u) {
      float kf[8];
      unpack8(ku[u], kf);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float x = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) x = fmaf(qf[i][c], kf[c], x);
        x = sum8(x);
        s[i][u] = base + u * GROUPS < j1 ? x : -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) st[i].raise(s[i]);
#pragma unroll
    for (int u = 0; u < ROWS_UNROLL; ++u) {
      float vf[8];
      unpack8(vu[u], vf);
#pragma unroll
      for (int i = 0; i < R; ++i) st[i].take(s[i][u], vf);
    }
  }
  // the first block: which own keys the rows see, and whether they belong to a view
  int own_lo[R], own_hi[R];
  bool mine[R];
  if (first) {
    if (hk == 0) check_views(d, tid, ROWS_THREADS, a.err);
    q_lo = max(q_lo, 0);
    q_hi = min(q_hi, d.n_q);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int tl = min(i, rows - 1) / d.G;
      mine[i] = i < rows && tl >= q_lo && tl < q_hi;
      own_lo[i] = own_hi[i] = 0;
      if (!mine[i]) continue;
      // the view of the token: the last one that starts at or before it
      int lo = 0, hi = d.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (d.q_off[mid] <= tl) lo = mid; else hi = mid;
      }
      ViewRange r;
      mine[i] = view_range(d, lo, &r, nullptr);
      if (!mine[i]) continue;
      const int nk = r.k1 - r.k0;
      own_lo[i] = r.k0;
      own_hi[i] = r.k0 + (d.causal ? max(0, min(nk, tl - r.q0 + nk - (r.q1 - r.q0) + 1)) : nk);
    }
  }
  if (first) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      for (int base = own_lo[i]; base < own_hi[i]; base += GROUPS) {
        const int j = base + (tid >> 3);
        const bool live = j < own_hi[i];
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        float kf[8], vf[8];
        unpack8(live ? *reinterpret_cast<const uint4*>(a.ko + j * d.ko_stride + hk * 64 + e) : zero, kf);
        unpack8(live ? *reinterpret_cast<const uint4*>(a.vo + j * d.vo_stride + hk * 64 + e) : zero, vf);
        float x = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) x = fmaf(qf[i][c], kf[c], x);
        x = sum8(x);
        if (live) st[i].add(x, vf);
      }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    st[i].join_groups();
    if (lane < 8) {
#pragma unroll
      for (int c = 0; c < 8; ++c) s_o[warp][i][e + c] = st[i].o[c];
      if (lane == 0) {
        s_m[warp][i] = st[i].m;
        s_l[warp][i] = st[i].l;
      }
    }
  }
  __syncthreads();
  // thread (row, value): joins the warps
  const int i = tid >> 6, c = tid & 63;
  if (i < min(R, rows)) {
    float m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = fmaxf(m, s_m[w][i]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = s_m[w][i] == m ? 1.f : exp2f(s_m[w][i] - m);
      l += s_l[w][i] * f;
      o += s_o[w][i][c] * f;
    }
    const int tl = i / d.G, h = hk * d.G + i - tl * d.G;
    if (!JOINED) {
      const long long at = ((long long)blockIdx.x * d.n_q + tl) * d.H + h;
      a.part_o[at * 64 + c] = l == 0.f ? 0.f : o / l;
      if (c == 0) a.part_lse[at] = l == 0.f ? -INFINITY : m + log2f(l);
    } else {
      // into the first block's memory
      cg::this_cluster().barrier_wait();
      float* to = cg::this_cluster().map_shared_rank(&s_row[blockIdx.x][i][0], 0);
      to[c] = o;
      if (c == 0) {
        to[64] = m;
        to[65] = l;
      }
    }
  } else if (JOINED) {
    cg::this_cluster().barrier_wait();
  }
  if (JOINED) {
    cg::this_cluster().barrier_arrive();
    if (!first) return;
    cg::this_cluster().barrier_wait();
    if (first && i < min(R, rows)) {
      float m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
      for (int r = 0; r < ROWS_CLUSTER; ++r) m = fmaxf(m, s_row[r][i][64]);
#pragma unroll
      for (int r = 0; r < ROWS_CLUSTER; ++r) {
        const float mr = s_row[r][i][64], f = mr == m ? 1.f : exp2f(mr - m);
        l += s_row[r][i][65] * f;
        o += s_row[r][i][c] * f;
      }
      bool writes = false;
#pragma unroll
      for (int u = 0; u < R; ++u) writes = writes || (u == i && mine[u]);
      if (writes) {
        const int tl = i / d.G, h = hk * d.G + i - tl * d.G;
        a.out[tl * d.o_stride + h * 64 + c] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
        if (a.lse && c == 0) a.lse[(long long)tl * d.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// own keys of views with few rows, merged with the prefix's partial results


// One block = one view, key head and R of the view's rows.  Eight lanes hold a key's
// 64 values; the block's groups of eight take the keys in turn, each with a softmax of
// its own, merged at the end.  Bound by the latency of the key reads: a group has four
// keys under way at a time, or two for two rows, in 64 registers so that an SM holds 32
// warps.  256 views of a token, 250 to 500 own keys and 16 heads, prefix of 1374
// included: 89 us at 4.5 TB/s; 126 with one key at a time, 101 with two, 110 without the
// limit on registers.
template <int R, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 32 / WARPS)
    view_own_kernel(const ViewDims d, const bf16* __restrict__ q, const bf16* __restrict__ k,
                    const bf16* __restrict__ v, int parts, const float* part_o, const float* part_lse, bf16* out,
                    float* lse, unsigned* err) {
  constexpr int GROUPS = 4 * WARPS, OWN_UNROLL = R == 1 ? 4 : 2;
  const int b = blockIdx.x, hk = blockIdx.y;
  ViewRange r;
  if (!view_range(d, b, &r, err)) {
    pdl_wait();  // whoever waits for this kernel waits for the one before it too
    return;
  }
  __shared__ float s_m[WARPS][R], s_l[WARPS][R], s_o[WARPS][R][64];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, e = (lane & 7) * 8, grp = tid >> 3;
  const int nq = r.q1 - r.q0, nk = r.k1 - r.k0, rows = nq * d.G;
  const long long n = (long long)d.n_q * d.H;
  const int r0 = blockIdx.z * R;
  if (r0 >= rows) {
    pdl_wait();
    return;
  }
  const bf16* kb = k + (long long)r.k0 * d.ko_stride + hk * 64 + e;
  const bf16* vb = v + (long long)r.k0 * d.vo_stride + hk * 64 + e;
  float qf[R][8];
  Row st[R];
  int end[R];
  int end_max = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = min(r0 + i, rows - 1), tl = row / d.G, h = hk * d.G + row - tl * d.G;
    unpack8(*reinterpret_cast<const uint4*>(q + (r.q0 + tl) * d.q_stride + h * 64 + e), qf[i]);
#pragma unroll
    for (int c = 0; c < 8; ++c) qf[i][c] *= d.c2;
    st[i].clear();
    end[i] = d.causal ? max(0, min(nk, tl + nk - nq + 1)) : nk;
    end_max = max(end_max, end[i]);
  }
  for (int base = 0; base < end_max; base += GROUPS * OWN_UNROLL) {
    uint4 ku[OWN_UNROLL], vu[OWN_UNROLL];
#pragma unroll
    for (int u = 0; u < OWN_UNROLL; ++u) {
      const int j = base + u * GROUPS + grp;
      ku[u] = vu[u] = make_uint4(0u, 0u, 0u, 0u);
      if (j < end_max) {
        ku[u] = *reinterpret_cast<const uint4*>(kb + j * d.ko_stride);
        vu[u] = *reinterpret_cast<const uint4*>(vb + j * d.vo_stride);
      }
    }
    float s[R][OWN_UNROLL];
#pragma unroll
    for (int u = 0; u < OWN_UNROLL; ++u) {
      float kf[8];
      unpack8(ku[u], kf);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float x = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) x = fmaf(qf[i][c], kf[c], x);
        x = sum8(x);
        s[i][u] = base + u * GROUPS + grp < end[i] ? x : -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) st[i].raise(s[i]);
#pragma unroll
    for (int u = 0; u < OWN_UNROLL; ++u) {
      float vf[8];
      unpack8(vu[u], vf);
#pragma unroll
      for (int i = 0; i < R; ++i) st[i].take(s[i][u], vf);
    }
  }
  // the four groups of a warp, then the warps
#pragma unroll
  for (int i = 0; i < R; ++i) {
    st[i].join_groups();
    if (lane < 8) {
#pragma unroll
      for (int c = 0; c < 8; ++c) s_o[warp][i][e + c] = st[i].o[c];
      if (lane == 0) {
        s_m[warp][i] = st[i].m;
        s_l[warp][i] = st[i].l;
      }
    }
  }
  __syncthreads();
  if (parts > 0) pdl_wait();
  // warp i: row i.  Its four groups take the warps' own results in turn, and then the
  // prefix's
  if (warp >= R || r0 + warp >= rows) return;
  Row x;
  x.clear();
  const int row = r0 + warp, tl = row / d.G, h = hk * d.G + row - tl * d.G, tok = r.q0 + tl;
  const long long rh = (long long)tok * d.H + h;
#pragma unroll
  for (int w = lane >> 3; w < WARPS; w += 4) x.join(s_m[w][warp], s_l[w][warp], &s_o[w][warp][e]);
#pragma unroll 2
  for (int p = lane >> 3; p < parts; p += 4) {
    const float z = part_lse[p * n + rh];
    const float4* src = reinterpret_cast<const float4*>(part_o + (p * n + rh) * 64 + e);
    const float4 y0 = src[0], y1 = src[1];
    if (z == -INFINITY) continue;  // nothing was written
    const float pv[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
    x.join(z, 1.f, pv);
  }
  x.join_groups();
  if (lane < 8) {
    const float inv = x.l == 0.f ? 0.f : 1.f / x.l;
    uint32_t w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      w[c] = x.l == 0.f ? 0u : pack_bf16x2(x.o[2 * c] * inv, x.o[2 * c + 1] * inv);
    *reinterpret_cast<uint4*>(out + tok * d.o_stride + h * 64 + e) = make_uint4(w[0], w[1], w[2], w[3]);
    if (lse && e == 0) lse[rh] = x.l == 0.f ? -INFINITY : (x.m + log2f(x.l)) * 0.6931471805599453f;
  }
}

__global__ void __launch_bounds__(256) check_kernel(const ViewDims d, unsigned* err) { check_views(d, threadIdx.x, 256, err); }

// ---------------------------------------------------------------------------
// host

cudaError_t prepare_kernel() {
  static std::atomic<unsigned long long> done{0};
  return allow_smem(view_attn_kernel, (int)kSmemBytes, &done);
}

template <int R>
cudaError_t launch_joined(const ViewDims& d, const RowsArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ROWS_CLUSTER, (unsigned)d.Hk);
  cfg.blockDim = dim3(ROWS_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ROWS_CLUSTER;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, view_rows_kernel<R, true>, d, a);
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Key splits for `units` CTAs (one with a single tile of rows counts half) of `tiles`
// key tiles each on 148 SMs.  Costs are counted in key tiles: a CTA's start and end
// take about as long as ten of them (measured over splits of 96 to 1152 CTAs), and a
// merged result costs `merge` more for each split.
int choose_split(double units, int tiles, int most, double merge) {
  int best = 1;
  double best_cost = 0;
  for (int s = 1; s <= most && s <= tiles; ++s) {
    const double waves = ceil(units * s / 148.0);
    const double cost = waves * (ceil_div(tiles, s) + 10.0) + (s > 1 ? merge * s : 0.0);
    if (s == 1 || cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return best;
}

}  // namespace

ViewPlan view_plan(const ViewDims& d) {
  ViewPlan p = {};
  p.split_packed = p.split_aligned = 1;
  const int MT = 128 / d.G;
  const int np = ceil_div(d.n_prefix, TK), no = ceil_div(d.max_own, TK);
  const bool has_own = d.n_own > 0 && d.max_own > 0;
  const bool short_views = (long long)d.max_q * d.G <= 16 && d.max_own <= 4096;
  if (!has_own || short_views || (d.n_prefix > 0 && d.B > 1 && d.n_q < 2LL * MT * d.B)) {
    p.packed = d.n_prefix > 0;
    p.small_own = has_own && short_views;
    p.aligned = p.aligned_own = has_own && !short_views;
  } else {
    p.aligned = p.aligned_own = 1;
    p.aligned_prefix = d.n_prefix > 0;
  }
  // partial results of one launch of a kind: their bytes against a key tile's time
  const double merge = 1.0 + (double)d.n_q * d.H * 64 * 8 / 3.0e6;
  p.rows = p.packed && (long long)d.n_q * d.G <= 4 && (p.small_own || !has_own);
  if (p.rows) {
    // one launch while its eight blocks a head keep up with the memory; two blocks an
    // SM beyond (95 us for a token at 137400 keys of 16 heads, 117 with one)
    p.joined = d.n_prefix <= 16384;
    if (p.joined) {
      p.small_own = 0;
      return p;
    }
    int s = 296 / d.Hk;
    p.split_packed = s > 1 ? s : 1;
    p.parts = p.split_packed;
    return p;
  }
  if (p.packed) {
    const double units = d.n_q <= 2 * MT ? 1.0 : (double)d.n_q / (2 * MT) + 0.25;
    p.split_packed = choose_split(units * d.Hk, np, 64, merge);
    p.parts += p.split_packed;
  }
  if (p.aligned) {
    // rows there are, and a quarter of a CTA for the ragged end of a view
    double units = (double)d.n_q / (2 * MT) + 0.25 * d.B;
    const double most = (double)d.B * ceil_div(d.max_q, 2 * MT);
    if (units > most) units = most;
    p.split_aligned = choose_split(units * d.Hk, (p.aligned_prefix ? np : 0) + no, 64, merge);
    p.parts += p.split_aligned;
  }
  // one part that nothing else joins is the result
  if (p.parts == 1 && !p.small_own) p.parts = 0;
  return p;
}

cudaError_t launch_prefix_attn(const ViewDims& d, const ViewPlan& p, const bf16* q, const bf16* kp, const bf16* vp,
                               const bf16* ko, const bf16* vo, bf16* out, float* lse, float* part_o, float* part_lse,
                               unsigned* err, cudaStream_t st) {
  if (d.n_q <= 0) return cudaSuccess;
  if (d.max_q <= 0) {
    // no view has a query: offsets that say otherwise are reported
    check_kernel<<<1, 256, 0, st>>>(d, err);
    return cudaGetLastError();
  }
  const int MT = 128 / d.G;
  if (p.rows) {
    const int rows = d.n_q * d.G;
    const RowsArgs a = {q, kp, vp, ko, vo, part_o, part_lse, out, lse, err};
    if (p.joined)
      return rows == 1 ? launch_joined<1>(d, a, st) : rows == 2 ? launch_joined<2>(d, a, st) : launch_joined<4>(d, a, st);
    const dim3 grid((unsigned)p.split_packed, (unsigned)d.Hk);
    if (rows == 1)
      view_rows_kernel<1, false><<<grid, ROWS_THREADS, 0, st>>>(d, a);
    else if (rows == 2)
      view_rows_kernel<2, false><<<grid, ROWS_THREADS, 0, st>>>(d, a);
    else
      view_rows_kernel<4, false><<<grid, ROWS_THREADS, 0, st>>>(d, a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  } else if (p.packed || p.aligned) {
    cudaError_t e = prepare_kernel();
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mkp, mvp, mko, mvo;
    auto map = [&](CUtensorMap* m, const bf16* base, int heads, int rows, long long stride, int b1, int b2) {
      return make_tmap_3d(m, false, base, 64, (unsigned long long)heads, (unsigned long long)rows, 128,
                          (unsigned long long)stride * 2, 64, (unsigned)b1, (unsigned)b2);
    };
    bool ok = map(&mq, q, d.H, d.n_q, d.q_stride, d.G, MT);
    if (d.n_prefix > 0)
      ok = ok && map(&mkp, kp, d.Hk, d.n_prefix, d.kp_stride, 1, TK) && map(&mvp, vp, d.Hk, d.n_prefix, d.vp_stride, 1, TK);
    if (d.n_own > 0)
      ok = ok && map(&mko, ko, d.Hk, d.n_own, d.ko_stride, 1, TK) && map(&mvo, vo, d.Hk, d.n_own, d.vo_stride, 1, TK);
    if (!ok) return cudaErrorInvalidValue;
    // a map that no tile uses still has to be one
    if (d.n_prefix <= 0) mkp = mvp = mq;
    if (d.n_own <= 0) mko = mvo = mq;
    ViewAttnArgs a = {};
    a.d = d;
    a.rows_tok = MT;
    a.out = out;
    a.lse = lse;
    a.part_o = p.parts ? part_o : nullptr;
    a.part_lse = part_lse;
    a.err = err;
    if (p.packed) {
      a.aligned = 0;
      a.do_prefix = 1;
      a.do_own = 0;
      a.check_views = !p.aligned && !p.small_own && !p.parts;  // the merge does it
      a.n_split = p.split_packed;
      a.units_per_view = 0;
      a.part0 = 0;
      const dim3 grid((unsigned)(ceil_div(d.n_q, 2 * MT) * a.n_split + (a.check_views ? 1 : 0)), (unsigned)d.Hk);
      view_attn_kernel<<<grid, kThreads, kSmemBytes, st>>>(mq, mkp, mvp, mko, mvo, a);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      a.part0 = p.split_packed;
    }
    if (p.aligned) {
      a.aligned = 1;
      a.check_views = 0;
      a.do_prefix = p.aligned_prefix;
      a.do_own = p.aligned_own;
      a.n_split = p.split_aligned;
      a.units_per_view = ceil_div(d.max_q, 2 * MT);
      const dim3 grid((unsigned)(d.B * a.units_per_view * a.n_split), (unsigned)d.Hk);
      view_attn_kernel<<<grid, kThreads, kSmemBytes, st>>>(mq, mkp, mvp, mko, mvo, a);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  }
  if (p.small_own) {
    // two rows a block share the reads (64 us for 64 views of four tokens and 250 to 500
    // own keys, 77 with one), or one where views have no more; large blocks where there are
    // few of them and many keys (69 us for 16 tokens with up to 4000 own keys, 226 with
    // small ones and one key at a time)
    const int rows = d.max_q * d.G, r = rows > 1 ? 2 : 1;
    const bool large = d.max_own >= 256 && (long long)d.B * d.Hk * ceil_div(rows, r) < 8 * 148;
    const dim3 grid((unsigned)d.B, (unsigned)d.Hk, (unsigned)ceil_div(rows, r));
    auto kernel = r == 1 ? (large ? view_own_kernel<1, 16> : view_own_kernel<1, 4>)
                         : (large ? view_own_kernel<2, 16> : view_own_kernel<2, 4>);
    const unsigned threads = large ? 512 : 128;
    if (p.parts > 0)
      return launch_second(kernel, grid, threads, st, d, q, ko, vo, p.parts, (const float*)part_o, (const float*)part_lse, out,
                           lse, err);
    kernel<<<grid, threads, 0, st>>>(d, q, ko, vo, 0, part_o, part_lse, out, lse, err);
    return cudaGetLastError();
  }
  if (p.parts > 0 || (!p.packed && !p.aligned)) {
    const long long blocks = ((long long)d.n_q * d.H * 8 + 255) / 256;
    if (p.parts == 0) {
      // no keys at all: the call's only kernel
      merge_kernel<<<(unsigned)blocks, 256, 0, st>>>(d, 0, part_o, part_lse, out, lse, err);
      return cudaGetLastError();
    }
    return launch_second(merge_kernel, dim3((unsigned)blocks), 256, st, d, p.parts, (const float*)part_o,
                         (const float*)part_lse, out, lse, err);
  }
  return cudaSuccess;
}

}  // namespace gsa
