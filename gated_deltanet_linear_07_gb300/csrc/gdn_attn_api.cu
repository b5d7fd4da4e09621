// gdn_attn_api.cu -- the full-attention entry points declared in
// include/gdn.h: host-side argument checks, workspace carve-up and dispatch.
// Nothing here allocates, synchronises or keeps state between calls.
#include <math.h>
#include <string.h>

#include "gdn_attn_checks.cuh"

using namespace gdn::attn;

namespace {

int rope_impl(const gdn_attn_dims* d, const gdn_rope_params* pr, const gdn_rope_axes* axes,
              const gdn_view& q, const gdn_view& k, const gdn_view& v, const int32_t* positions,
              const int32_t* row_seq, int64_t n, const gdn_kv_cache* cache, void* q_out,
              void* k_out, int32_t* d_status, gdn_stream_t stream) {
  GdnRopeArgs a;
  const int rc = rope_args(d, pr, axes, q, k, v, positions, n, q_out, k_out, d_status, a);
  if (rc != GDN_OK) return rc;
  a.row_seq = row_seq;
  if (cache) {
    a.cache = *cache;
    a.page_shift = page_shift(d->page_size);
  }
  return cuda_rc(gdn_launch_rope(a, d->io, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

GDN_EXPORT int gdn_qk_norm_rope(const gdn_attn_dims* dims, const gdn_rope_params* params,
                                const gdn_view* q, const gdn_view* k, const int32_t* positions,
                                int64_t n, void* q_out, void* k_out, gdn_stream_t stream) {
  const int rc = check_dims(dims, true);
  if (rc != GDN_OK) return rc;
  if (!params || n < 0) return GDN_EINVAL;
  const gdn_view qv = view_or_none(q), kv = view_or_none(k), none = {nullptr, 0, 0};
  if (n == 0) return GDN_OK;
  if (!qv.data && !kv.data) return GDN_EINVAL;
  return rope_impl(dims, params, nullptr, qv, kv, none, positions, nullptr, n, nullptr, q_out, k_out,
                   params->d_status, stream);
}

GDN_EXPORT int gdn_qk_norm_rope_axes(const gdn_attn_dims* dims, const gdn_rope_params* params,
                                     const gdn_rope_axes* axes, const gdn_view* q,
                                     const gdn_view* k, const int32_t* positions, int64_t n,
                                     void* q_out, void* k_out, gdn_stream_t stream) {
  int rc = check_dims(dims, true);
  if (rc != GDN_OK) return rc;
  if (!params || n < 0) return GDN_EINVAL;
  if ((rc = check_axes(dims, axes)) != GDN_OK) return rc;
  const gdn_view qv = view_or_none(q), kv = view_or_none(k), none = {nullptr, 0, 0};
  if (n == 0) return GDN_OK;
  if (!qv.data && !kv.data) return GDN_EINVAL;
  return rope_impl(dims, params, axes, qv, kv, none, positions, nullptr, n, nullptr, q_out, k_out,
                   params->d_status, stream);
}

GDN_EXPORT int gdn_kv_append(const gdn_attn_dims* dims, const gdn_rope_params* params,
                             const gdn_view* q, const gdn_view* k, const gdn_view* v,
                             const int32_t* positions, const int32_t* row_seq, int64_t n,
                             const gdn_kv_cache* cache, void* q_out, void* k_out,
                             int32_t* d_status, gdn_stream_t stream) {
  int rc = check_dims(dims, true);
  if (rc != GDN_OK) return rc;
  if (!params || n < 0) return GDN_EINVAL;
  if ((rc = check_cache(dims, cache)) != GDN_OK) return rc;
  if (!row_seq && n > cache->num_seqs) return GDN_EINVAL;
  if (n == 0) return GDN_OK;
  const gdn_view qv = view_or_none(q), kv = view_or_none(k), vv = view_or_none(v);
  if (!kv.data || !vv.data) return GDN_EINVAL;
  return rope_impl(dims, params, nullptr, qv, kv, vv, positions, row_seq, n, cache, q_out, k_out,
                   d_status, stream);
}

GDN_EXPORT int gdn_attn_prefill(const gdn_attn_dims* dims, const gdn_view* q, const gdn_view* k,
                                const gdn_view* v, const int32_t* cu_seqlens_q,
                                const int32_t* cu_seqlens_kv, int32_t num_seqs, int64_t total_q,
                                int64_t total_kv, const gdn_view* gate, void* o,
                                int32_t* d_status, gdn_stream_t stream) {
  int rc = check_dims(dims, false);
  if (rc != GDN_OK) return rc;
  if (num_seqs < 0 || total_q < 0 || total_kv < 0) return GDN_EINVAL;
  if (num_seqs == 0 && (total_q > 0 || total_kv > 0)) return GDN_EINVAL;
  if (!cu_seqlens_kv && total_kv != total_q) return GDN_EINVAL;
  if (total_q == 0) return GDN_OK;
  const gdn_view gv = view_or_none(gate);
  if (!q || !k || !v || !q->data || !o || !cu_seqlens_q) return GDN_EINVAL;
  if (total_kv > 0 && (!k->data || !v->data)) return GDN_EINVAL;
  if (o == q->data || o == k->data || o == v->data || o == gv.data) return GDN_EINVAL;
  if (total_q > kMostTokens || total_kv > kMostTokens) return GDN_EUNSUPPORTED;
  if (!aligned16(o)) return GDN_EALIGN;
  if ((rc = check_view(dims, q, total_q, dims->h_q)) != GDN_OK) return rc;
  if (total_kv > 0 && ((rc = check_view(dims, k, total_kv, dims->h_kv)) != GDN_OK ||
                       (rc = check_view(dims, v, total_kv, dims->h_kv)) != GDN_OK))
    return rc;
  if (gv.data && (rc = check_view(dims, &gv, total_q, dims->h_q)) != GDN_OK) return rc;
  GdnAttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = *q; a.k = *k; a.v = *v; a.gate = gv;
  if (total_kv == 0) a.k = a.v = *q;   // no key is read; a tensor map wants an address
  a.o = o;
  a.cu_q = cu_seqlens_q;
  a.cu_kv = cu_seqlens_kv ? cu_seqlens_kv : cu_seqlens_q;
  a.num_seqs = num_seqs;
  a.total_q = total_q; a.total_kv = total_kv;
  a.d_status = d_status;
  a.wait_ns = wait_ns_of(dims);
  a.withhold = dims->flags & GDN_TEST_WAIT_TIMEOUT ? 1 : 0;
  a.scale_log2 = scale_log2_of(dims);
  a.h_q = dims->h_q; a.h_kv = dims->h_kv; a.d = dims->d;
  return cuda_rc(gdn_launch_attn_prefill(a, dims->io, reinterpret_cast<cudaStream_t>(stream)));
}

GDN_EXPORT size_t gdn_attn_decode_workspace_size(const gdn_attn_dims* dims, int32_t n,
                                                 int64_t shared_len) {
  if (check_dims(dims, false) != GDN_OK || n < 0 || shared_len < 0) return 0;
  if (!page_ok(dims->page_size) || shared_len % dims->page_size != 0) return 0;
  const int64_t slots = gdn_attn_decode_slots(dims->h_q, dims->h_kv, dims->d, n, shared_len);
  return align_up((size_t)slots * dims->d * 4) + align_up((size_t)slots * sizeof(float2));
}

GDN_EXPORT int gdn_attn_decode(const gdn_attn_dims* dims, const gdn_view* q,
                               const gdn_kv_cache* cache, const int32_t* seq_lens, int32_t n,
                               int64_t shared_len, const gdn_view* gate, void* o, void* workspace,
                               size_t workspace_bytes, int32_t* d_status, gdn_stream_t stream) {
  int rc = check_dims(dims, false);
  if (rc != GDN_OK) return rc;
  if (n < 0 || shared_len < 0) return GDN_EINVAL;
  if ((rc = check_cache(dims, cache)) != GDN_OK) return rc;
  if (n > cache->num_seqs || shared_len % dims->page_size != 0 ||
      shared_len > (int64_t)cache->pages_per_seq * dims->page_size)
    return GDN_EINVAL;
  if (n == 0) return GDN_OK;
  const gdn_view gv = view_or_none(gate);
  if (!q || !q->data || !seq_lens || !o) return GDN_EINVAL;
  if (o == q->data || o == gv.data) return GDN_EINVAL;
  if ((int64_t)n * dims->h_q > 0x7fffffffLL) return GDN_EUNSUPPORTED;
  if (!workspace || workspace_bytes < gdn_attn_decode_workspace_size(dims, n, shared_len))
    return GDN_EWORKSPACE;
  if (!aligned16(o) || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
    return GDN_EALIGN;
  if ((rc = check_view(dims, q, n, dims->h_q)) != GDN_OK) return rc;
  if (gv.data && (rc = check_view(dims, &gv, n, dims->h_q)) != GDN_OK) return rc;
  GdnAttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = *q; a.gate = gv;
  a.cache = *cache;
  a.page_shift = page_shift(dims->page_size);
  a.seq_lens = seq_lens;
  a.o = o;
  a.total_q = n;
  a.shared_len = shared_len;
  a.splits = gdn_attn_prefix_splits(dims->h_q, dims->h_kv, dims->d, n, shared_len);
  const int64_t slots = gdn_attn_decode_slots(dims->h_q, dims->h_kv, dims->d, n, shared_len);
  a.part_o = reinterpret_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(reinterpret_cast<char*>(workspace) +
                                        align_up((size_t)slots * dims->d * 4));
  a.d_status = d_status;
  a.wait_ns = wait_ns_of(dims);
  a.withhold = dims->flags & GDN_TEST_WAIT_TIMEOUT ? 1 : 0;
  a.scale_log2 = scale_log2_of(dims);
  a.h_q = dims->h_q; a.h_kv = dims->h_kv; a.d = dims->d;
  return cuda_rc(gdn_launch_attn_decode(a, dims->io, reinterpret_cast<cudaStream_t>(stream)));
}
