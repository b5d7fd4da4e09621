// gdn_attn_checks.cuh -- host-side argument checks that the full-attention entry
// points share (gdn_attn_api.cu, gdn_kv8_api.cu).
#pragma once

#include <math.h>
#include <string.h>

#include "gdn_attn.cuh"

#define GDN_EXPORT extern "C" __attribute__((visibility("default")))

namespace gdn {
namespace attn {

constexpr size_t kAlign = 256;
constexpr int64_t kMostTokens = 0x7fff0000;   // the kernels' block ends stay below 2^31
// Waits give up after 4 s (a block of keys takes microseconds); the test flag shortens
// that to 2 ms and has some hand-overs withheld.
inline uint64_t wait_ns_of(const gdn_attn_dims* d) {
  return d->flags & GDN_TEST_WAIT_TIMEOUT ? 2000000ull : 4000000000ull;
}

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int elem(const gdn_attn_dims* d) { return d->io == GDN_FP32 ? 4 : 2; }

inline int check_dims(const gdn_attn_dims* d, bool fp32) {
  if (!d) return GDN_EINVAL;
  if (d->h_q <= 0 || d->h_kv <= 0 || d->h_q % d->h_kv != 0) return GDN_EINVAL;
  if (d->flags & ~GDN_TEST_WAIT_TIMEOUT) return GDN_EINVAL;
  if (!(d->norm_eps >= 0.f) || d->norm_eps > 1e30f) return GDN_EINVAL;   // also rejects NaN
  if (!(d->scale >= 0.f) || d->scale > 1e30f) return GDN_EINVAL;
  if (d->rope != GDN_ROPE_HALF && d->rope != GDN_ROPE_INTERLEAVED) return GDN_EINVAL;
  if (d->d != 64 && d->d != 128 && d->d != 256) return GDN_EUNSUPPORTED;
  if (d->io != GDN_BF16 && d->io != GDN_FP16 && !(fp32 && d->io == GDN_FP32))
    return GDN_EUNSUPPORTED;
  if (d->rot_dim < 0 || d->rot_dim > d->d || d->rot_dim % 16 != 0) return GDN_EUNSUPPORTED;
  if (d->h_q > 65535) return GDN_EUNSUPPORTED;
  return GDN_OK;
}

inline bool page_ok(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128; }
inline int page_shift(int32_t p) { return p == 16 ? 4 : p == 32 ? 5 : p == 64 ? 6 : 7; }

// A view [tokens][heads][d] with data: its address and strides keep every row
// 16-byte aligned, no two rows of it are the same (a tensor map has no stride of
// zero), and its rows lie within what a tensor map and 64-bit offsets can address.
inline int check_view(const gdn_attn_dims* d, const gdn_view* v, int64_t tokens, int64_t heads) {
  if (!aligned16(v->data)) return GDN_EALIGN;
  if (v->token_stride < 0 || v->head_stride < 0) return GDN_EINVAL;
  if (v->token_stride * elem(d) % 16 != 0 || v->head_stride * elem(d) % 16 != 0) return GDN_EALIGN;
  if ((tokens > 1 && v->token_stride == 0) || (heads > 1 && v->head_stride == 0))
    return GDN_EUNSUPPORTED;
  if (v->token_stride >= (1LL << 36) || v->head_stride >= (1LL << 36)) return GDN_EUNSUPPORTED;
  return GDN_OK;
}

inline gdn_view view_or_none(const gdn_view* v) {
  gdn_view none = {nullptr, 0, 0};
  return v ? *v : none;
}

template <typename Cache>   // gdn_kv_cache, gdn_kv8_cache
inline int check_cache(const gdn_attn_dims* d, const Cache* c) {
  if (!c || !c->k || !c->v || !c->block_table) return GDN_EINVAL;
  if (c->num_pages <= 0 || c->num_seqs < 0 || c->pages_per_seq <= 0) return GDN_EINVAL;
  if (!page_ok(d->page_size)) return GDN_EUNSUPPORTED;
  // rows of the pool are 32-bit coordinates of a tensor map
  if (c->num_pages > 0x7fffffffLL / ((int64_t)d->h_kv * d->page_size)) return GDN_EUNSUPPORTED;
  if ((int64_t)c->pages_per_seq * d->page_size > kMostTokens) return GDN_EUNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v)) return GDN_EALIGN;
  return GDN_OK;
}

inline int cuda_rc(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ECUDA; }

inline int check_axes(const gdn_attn_dims* d, const gdn_rope_axes* axes) {
  if (!axes || axes->count < 1 || axes->count > GDN_ROPE_MAX_AXES) return GDN_EINVAL;
  for (int i = 0; i < d->rot_dim / 2; ++i)
    if (axes->pair[i] >= axes->count) return GDN_EINVAL;
  return GDN_OK;
}

// The norm's and rotation's arguments of a call that has passed check_dims and, with
// axes, check_axes (everything but a cache's).
inline int rope_args(const gdn_attn_dims* d, const gdn_rope_params* pr, const gdn_rope_axes* axes,
                     const gdn_view& q, const gdn_view& k, const gdn_view& v,
                     const int32_t* positions, int64_t n, void* q_out, void* k_out,
                     int32_t* d_status, GdnRopeArgs& a) {
  if (!positions || (d->rot_dim > 0 && !pr->inv_freq)) return GDN_EINVAL;
  if (!isfinite(pr->rope_scale)) return GDN_EINVAL;
  if ((q.data && !q_out) || (k.data && !v.data && !k_out)) return GDN_EINVAL;
  if (n > 0x7fffffffLL) return GDN_EUNSUPPORTED;
  if (!aligned16(q_out) || !aligned16(k_out) || !aligned16(pr->q_norm) || !aligned16(pr->k_norm))
    return GDN_EALIGN;
  for (const gdn_view* w : {&q, &k, &v})
    if (w->data) {
      const int rc = check_view(d, w, n, w == &q ? d->h_q : d->h_kv);
      if (rc != GDN_OK) return rc;
    }
  memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.v = v;
  a.q_out = q_out; a.k_out = k_out;
  a.q_norm = pr->q_norm; a.k_norm = pr->k_norm; a.inv_freq = pr->inv_freq;
  a.rope_scale = pr->rope_scale;
  a.positions = positions; a.n = n;
  if (axes) a.axes = *axes;
  a.d_status = d_status;
  a.h_q = d->h_q; a.h_kv = d->h_kv; a.d = d->d; a.rot_dim = d->rot_dim;
  a.interleaved = d->rope == GDN_ROPE_INTERLEAVED;
  a.eps = d->norm_eps;
  a.wait_ns = wait_ns_of(d);
  a.withhold = d->flags & GDN_TEST_WAIT_TIMEOUT ? 1 : 0;
  return GDN_OK;
}

inline float scale_log2_of(const gdn_attn_dims* d) {
  const double s = d->scale > 0.f ? (double)d->scale : 1.0 / sqrt((double)d->d);
  return (float)(s * 1.4426950408889634074);
}

}  // namespace attn
}  // namespace gdn
