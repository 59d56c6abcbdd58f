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
  if ((long long)b->n_views * ((b->max_q + 127LL) / 128 + 1) * 64 * 128 > INT32_MAX) return GSA_ERR_INVALID_ARG;
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

}  // namespace

extern "C" {

gsa_status view_workspace_size(const gsa_view_batch* batch, size_t* bytes) {
  ViewDims d;
  if (bytes == nullptr) return GSA_ERR_INVALID_ARG;
  gsa_status st = make_view_dims(batch, &d);
  if (st != GSA_OK) return st;
  *bytes = attn_layout(d, gsa::view_plan(d)).total;
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

}  // extern "C"
