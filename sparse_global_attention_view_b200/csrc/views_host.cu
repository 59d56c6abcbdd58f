// The C ABI of the view-cache operators (include/gsa.h): argument validation,
// workspace layout and the enqueueing of each call.
#include <math.h>
#include <stdint.h>

#include "views.h"

using gsa::bf16;
using gsa::ViewDims;
using gsa::ViewPlan;

namespace {

inline bool dev_ptr(const void* p) { return p != nullptr && ((uintptr_t)p & 15u) == 0; }
inline bool word_ptr(const void* p) { return p != nullptr && ((uintptr_t)p & 3u) == 0; }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline gsa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GSA_OK : GSA_ERR_CUDA; }

// A token stride of `heads` heads: 0 stands for a dense layout.  TMA maps hold
// strides below 2^40 bytes.
bool take_stride(int64_t s, int heads, long long* out) {
  const long long dense = (long long)heads * gsa::kHeadDim;
  if (s == 0) s = dense;
  if (s < dense || s % 8 != 0 || s >= (1LL << 39)) return false;
  *out = s;
  return true;
}

gsa_status make_view_dims(const gsa_view_batch* b, ViewDims* d) {
  if (b == nullptr) return GSA_ERR_INVALID_ARG;
  if (b->n_views < 1 || b->n_heads < 1 || b->n_kv_heads < 1 || b->head_dim < 1 || b->n_q < 0 || b->n_own < 0 ||
      b->n_prefix < 0)
    return GSA_ERR_INVALID_ARG;
  if (b->n_heads % b->n_kv_heads != 0) return GSA_ERR_INVALID_ARG;
  if (b->max_q < 0 || b->max_q > b->n_q || b->max_own < 0 || b->max_own > b->n_own) return GSA_ERR_INVALID_ARG;
  if (b->causal != 0 && b->causal != 1) return GSA_ERR_INVALID_ARG;
  if (!(b->scale >= 0.f) || isinf(b->scale) || b->wait_limit_ns < 0) return GSA_ERR_INVALID_ARG;
  if (b->head_dim != gsa::kHeadDim || b->n_heads > 128) return GSA_ERR_UNSUPPORTED;
  // slots of the cache after an append, tile starts and grids are int32
  constexpr long long most = INT32_MAX - 1024;
  if ((long long)b->n_prefix + b->n_own > most || b->n_q > most / 128) return GSA_ERR_INVALID_ARG;
  // so is the grid of the views' row tiles, two a block, in at most 64 key ranges
  const long long unit = 2 * (128 / (b->n_heads / b->n_kv_heads)), units = (b->max_q + unit - 1) / unit;
  if (b->n_views * (units > 1 ? units : 1) > INT32_MAX / 64) return GSA_ERR_INVALID_ARG;
  ViewDims t = {};
  t.B = b->n_views;
  t.H = b->n_heads;
  t.Hk = b->n_kv_heads;
  t.G = b->n_heads / b->n_kv_heads;
  t.n_q = b->n_q;
  t.n_own = b->n_own;
  t.n_prefix = b->n_prefix;
  t.max_q = b->max_q;
  t.max_own = b->max_own;
  t.causal = b->causal;
  if (!take_stride(b->q_stride, t.H, &t.q_stride) || !take_stride(b->out_stride, t.H, &t.o_stride) ||
      !take_stride(b->k_prefix_stride, t.Hk, &t.kp_stride) || !take_stride(b->v_prefix_stride, t.Hk, &t.vp_stride) ||
      !take_stride(b->k_own_stride, t.Hk, &t.ko_stride) || !take_stride(b->v_own_stride, t.Hk, &t.vo_stride))
    return GSA_ERR_INVALID_ARG;
  t.scale = b->scale > 0.f ? b->scale : 0.125f;
  t.c2 = t.scale * 1.4426950408889634f;
  // SM clocks stay below 2 GHz: two cycles per nanosecond is at least the time asked
  t.wait_cycles = b->wait_limit_ns > 0 ? 2LL * b->wait_limit_ns : 4000000000LL;
  *d = t;
  return GSA_OK;
}

struct AttnLayout {
  size_t part_o, part_lse, total;
};
AttnLayout attn_layout(const ViewDims& d, const ViewPlan& p) {
  AttnLayout l;
  const size_t rows = (size_t)p.parts * d.n_q * d.H;
  l.part_o = GSA_WS_HEADER_BYTES;
  l.part_lse = l.part_o + up256(rows * gsa::kHeadDim * 4);
  l.total = l.part_lse + up256(rows * 4);
  return l;
}

struct WeightsLayout {
  size_t prefix, own, total;
};
WeightsLayout weights_layout(const ViewDims& d, const gsa::WeightsPlan& p) {
  WeightsLayout l;
  l.prefix = GSA_WS_HEADER_BYTES;
  l.own = l.prefix + (p.split_prefix > 1 ? up256((size_t)p.split_prefix * d.Hk * d.n_prefix * 4) : 0);
  l.total = l.own + (p.split_own > 1 ? up256((size_t)p.split_own * d.Hk * d.n_own * 4) : 0);
  return l;
}

struct CacheLayout {
  size_t moves, src, dst, total;
};
gsa_status make_evict_dims(const gsa_cache* c, gsa::EvictDims* d, CacheLayout* l) {
  if (c == nullptr || c->n_kv_heads < 1 || c->head_dim < 1 || c->n_tokens < 0 || c->n_keep < 0 ||
      c->n_keep > c->n_tokens || c->w_stride < c->n_tokens || c->w_stride >= (1LL << 40))
    return GSA_ERR_INVALID_ARG;
  if (c->head_dim != gsa::kHeadDim || c->n_kv_heads > 128) return GSA_ERR_UNSUPPORTED;
  if (c->n_tokens > INT32_MAX - (1 << 20)) return GSA_ERR_INVALID_ARG;  // slots plus a stride are int32
  d->Hk = c->n_kv_heads;
  d->n = c->n_tokens;
  d->keep = c->n_keep;
  d->recent_from = c->recent_from;
  d->w_stride = c->w_stride;
  if (!take_stride(c->k_stride, d->Hk, &d->k_stride) || !take_stride(c->v_stride, d->Hk, &d->v_stride))
    return GSA_ERR_INVALID_ARG;
  const size_t most = (size_t)gsa::evict_most_moves(*d) * d->Hk * 4;
  l->moves = GSA_WS_HEADER_BYTES;
  l->src = l->moves + up256((size_t)d->Hk * 4);
  l->dst = l->src + up256(most);
  l->total = l->dst + up256(most);
  return GSA_OK;
}

// Bytes that `heads` rows of n 32-bit words reach over, `stride` words apart.
uintptr_t span(int heads, long long n, long long stride) {
  return n > 0 ? (uintptr_t)((heads - 1) * stride + n) * 4 : 0;
}
bool overlap(const void* a, uintptr_t na, const void* b, uintptr_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

}  // namespace

extern "C" {

gsa_status view_workspace_size(const gsa_view_batch* batch, size_t* bytes) {
  ViewDims d;
  if (bytes == nullptr) return GSA_ERR_INVALID_ARG;
  gsa_status st = make_view_dims(batch, &d);
  if (st != GSA_OK) return st;
  const size_t x = attn_layout(d, gsa::view_plan(d)).total, y = weights_layout(d, gsa::weights_plan(d)).total;
  *bytes = x > y ? x : y;
  return GSA_OK;
}

gsa_status prefix_attn(const gsa_view_batch* batch, const gsa_bf16* q, const gsa_bf16* k_prefix,
                       const gsa_bf16* v_prefix, const gsa_bf16* k_own, const gsa_bf16* v_own,
                       const int32_t* q_off, const int32_t* own_off, gsa_bf16* out, float* lse, void* ws,
                       size_t ws_bytes, void* stream) {
  ViewDims d;
  gsa_status st = make_view_dims(batch, &d);
  if (st != GSA_OK) return st;
  if (!word_ptr(q_off) || !word_ptr(own_off) || !dev_ptr(ws) || (lse != nullptr && !word_ptr(lse)))
    return GSA_ERR_INVALID_ARG;
  if (d.n_q > 0 && (!dev_ptr(q) || !dev_ptr(out))) return GSA_ERR_INVALID_ARG;
  if (d.n_prefix > 0 && (!dev_ptr(k_prefix) || !dev_ptr(v_prefix))) return GSA_ERR_INVALID_ARG;
  if (d.n_own > 0 && (!dev_ptr(k_own) || !dev_ptr(v_own))) return GSA_ERR_INVALID_ARG;
  const ViewPlan p = gsa::view_plan(d);
  const AttnLayout l = attn_layout(d, p);
  if (ws_bytes < l.total) return GSA_ERR_WORKSPACE;
  d.q_off = q_off;
  d.own_off = own_off;
  char* base = static_cast<char*>(ws);
  return cuda_status(gsa::launch_prefix_attn(d, p, (const bf16*)q, (const bf16*)k_prefix, (const bf16*)v_prefix,
                                             (const bf16*)k_own, (const bf16*)v_own, (bf16*)out, lse,
                                             (float*)(base + l.part_o), (float*)(base + l.part_lse), (unsigned*)ws,
                                             as_stream(stream)));
}

gsa_status key_weights(const gsa_view_batch* batch, const gsa_bf16* q, const gsa_bf16* k_prefix,
                       const gsa_bf16* k_own, const int32_t* q_off, const int32_t* own_off, const float* lse,
                       const float* acc, int64_t acc_stride, float* acc_out, int64_t acc_out_stride,
                       float decay, void* ws, size_t ws_bytes, void* stream) {
  ViewDims d;
  gsa_status st = make_view_dims(batch, &d);
  if (st != GSA_OK) return st;
  const long long keys = (long long)d.n_prefix + d.n_own;
  if (!word_ptr(q_off) || !word_ptr(own_off) || !dev_ptr(ws)) return GSA_ERR_INVALID_ARG;
  if (d.n_q > 0 && (!dev_ptr(q) || !word_ptr(lse))) return GSA_ERR_INVALID_ARG;
  if (d.n_prefix > 0 && !dev_ptr(k_prefix)) return GSA_ERR_INVALID_ARG;
  if (d.n_own > 0 && !dev_ptr(k_own)) return GSA_ERR_INVALID_ARG;
  if (keys > 0 && !word_ptr(acc_out)) return GSA_ERR_INVALID_ARG;
  if (acc != nullptr && !word_ptr(acc)) return GSA_ERR_INVALID_ARG;
  if (acc_out_stride < keys || acc_out_stride >= (1LL << 40) || !(decay >= 0.f) || isinf(decay))
    return GSA_ERR_INVALID_ARG;
  if (acc != nullptr && (acc_stride < d.n_prefix || acc_stride >= (1LL << 40))) return GSA_ERR_INVALID_ARG;
  // in place, or apart: a shifted account would be read after it was written.  One row
  // has no stride
  if (acc != nullptr && !(acc == acc_out && (acc_stride == acc_out_stride || d.Hk == 1)) &&
      overlap(acc, span(d.Hk, d.n_prefix, acc_stride), acc_out, span(d.Hk, keys, acc_out_stride)))
    return GSA_ERR_INVALID_ARG;
  const gsa::WeightsPlan p = gsa::weights_plan(d);
  if (gsa::weights_items(d, p) > gsa::kMostItems) return GSA_ERR_INVALID_ARG;
  const WeightsLayout l = weights_layout(d, p);
  if (ws_bytes < l.total) return GSA_ERR_WORKSPACE;
  d.q_off = q_off;
  d.own_off = own_off;
  char* base = static_cast<char*>(ws);
  return cuda_status(gsa::launch_key_weights(d, p, (const bf16*)q, (const bf16*)k_prefix, (const bf16*)k_own, lse, acc,
                                             acc_stride, acc_out, acc_out_stride, decay, (float*)(base + l.prefix),
                                             (float*)(base + l.own), (unsigned*)ws, as_stream(stream)));
}

gsa_status cache_workspace_size(const gsa_cache* cache, size_t* bytes) {
  gsa::EvictDims d;
  CacheLayout l;
  if (bytes == nullptr) return GSA_ERR_INVALID_ARG;
  const gsa_status st = make_evict_dims(cache, &d, &l);
  if (st != GSA_OK) return st;
  *bytes = l.total;
  return GSA_OK;
}

gsa_status cache_evict(const gsa_cache* cache, gsa_bf16* k, gsa_bf16* v, const float* acc, const int32_t* ids,
                       float* acc_out, int32_t* ids_out, void* ws, size_t ws_bytes, void* stream) {
  gsa::EvictDims d;
  CacheLayout l;
  const gsa_status st = make_evict_dims(cache, &d, &l);
  if (st != GSA_OK) return st;
  if (!dev_ptr(ws)) return GSA_ERR_INVALID_ARG;
  if (d.n > 0 && (!dev_ptr(k) || !dev_ptr(v) || !word_ptr(acc) || !word_ptr(ids) || !word_ptr(acc_out) || !word_ptr(ids_out)))
    return GSA_ERR_INVALID_ARG;
  const uintptr_t w = span(d.Hk, d.n, d.w_stride);
  if (overlap(acc, w, acc_out, w) || overlap(ids, w, ids_out, w) || overlap(acc, w, ids_out, w) ||
      overlap(ids, w, acc_out, w) || overlap(acc_out, w, ids_out, w))
    return GSA_ERR_INVALID_ARG;
  if (ws_bytes < l.total) return GSA_ERR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  return cuda_status(gsa::launch_cache_evict(d, (bf16*)k, (bf16*)v, acc, ids, acc_out, ids_out, (int*)(base + l.moves),
                                             (int*)(base + l.src), (int*)(base + l.dst), as_stream(stream)));
}

}  // extern "C"
