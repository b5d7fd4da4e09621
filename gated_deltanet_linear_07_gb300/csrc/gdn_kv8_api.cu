// gdn_kv8_api.cu -- the entry points of the 8-bit cache declared in include/gdn.h:
// host-side argument checks, workspace carve-up and dispatch.  Nothing here
// allocates, synchronises or keeps state between calls.
#include "gdn_attn_checks.cuh"
#include "gdn_kv8.cuh"

using namespace gdn::attn;

namespace {

int check_kv8(const gdn_attn_dims* d, const gdn_kv8_cache* c) {
  const int rc = check_cache(d, c);
  if (rc != GDN_OK) return rc;
  if (!c->k_scale || !c->v_scale) return GDN_EINVAL;
  if ((reinterpret_cast<uintptr_t>(c->k_scale) & 3u) || (reinterpret_cast<uintptr_t>(c->v_scale) & 3u))
    return GDN_EALIGN;
  return GDN_OK;
}

int64_t capacity_of(const gdn_attn_dims* d, const gdn_kv8_cache* c) {
  return (int64_t)c->pages_per_seq * d->page_size;
}

// The rows' scores are counted in 64 bits, with room for what follows them.
bool scores_ok(const gdn_attn_dims* d, int64_t n, int64_t capacity) {
  return n * d->h_q <= 0x7fffffffLL && n * d->h_q * capacity <= (1LL << 48);
}

// Where the parts of the decode's workspace begin; the last entry is its size.
struct DecodeWorkspace {
  size_t part_ml, row_ml, scores, size;
  DecodeWorkspace(const gdn_attn_dims* d, int64_t n, int64_t capacity) {
    const size_t slots = (size_t)gdn_kv8_decode_slots(d->h_q, d->h_kv);
    part_ml = align_up(slots * d->d * 4);
    row_ml = part_ml + align_up(slots * sizeof(float2));
    scores = row_ml + (capacity > 0 ? align_up((size_t)n * d->h_q * sizeof(float2)) : 0);
    size = scores + align_up((size_t)n * d->h_q * capacity * 4);
  }
};

}  // namespace

GDN_EXPORT int gdn_kv8_append(const gdn_attn_dims* dims, const gdn_rope_params* params,
                              const gdn_rope_axes* axes, const gdn_view* q, const gdn_view* k,
                              const gdn_view* v, const int32_t* positions,
                              const int32_t* cu_seqlens, const int32_t* starts, int32_t num_seqs,
                              int64_t n, const gdn_kv8_cache* cache, void* q_out, void* k_out,
                              int32_t* d_status, gdn_stream_t stream) {
  int rc = check_dims(dims, false);
  if (rc != GDN_OK) return rc;
  if (!params || n < 0 || num_seqs < 0) return GDN_EINVAL;
  if (axes && (rc = check_axes(dims, axes)) != GDN_OK) return rc;
  if ((rc = check_kv8(dims, cache)) != GDN_OK) return rc;
  if (num_seqs > cache->num_seqs || (!cu_seqlens && num_seqs != n)) return GDN_EINVAL;
  if (n == 0) return GDN_OK;
  if (num_seqs == 0 || !starts) return GDN_EINVAL;
  const gdn_view qv = view_or_none(q), kv = view_or_none(k), vv = view_or_none(v);
  if (!kv.data || !vv.data) return GDN_EINVAL;
  GdnKv8AppendArgs a;
  memset(&a, 0, sizeof(a));
  if ((rc = rope_args(dims, params, axes, qv, kv, vv, positions, n, q_out, k_out, d_status, a.r)) !=
      GDN_OK)
    return rc;
  a.r.page_shift = page_shift(dims->page_size);
  a.cache = *cache;
  a.cu = cu_seqlens;
  a.starts = starts;
  a.num_seqs = num_seqs;
  return cuda_rc(gdn_launch_kv8_append(a, dims->io, reinterpret_cast<cudaStream_t>(stream)));
}

GDN_EXPORT int gdn_kv8_gather(const gdn_attn_dims* dims, const gdn_kv8_cache* cache,
                              const int32_t* cu_seqlens, int32_t num_seqs, int64_t total,
                              void* k_out, void* v_out, int32_t* d_status, gdn_stream_t stream) {
  int rc = check_dims(dims, false);
  if (rc != GDN_OK) return rc;
  if (total < 0 || num_seqs < 0) return GDN_EINVAL;
  if ((rc = check_kv8(dims, cache)) != GDN_OK) return rc;
  if (num_seqs > cache->num_seqs) return GDN_EINVAL;
  if (total == 0) return GDN_OK;
  if (num_seqs == 0 || !cu_seqlens || (!k_out && !v_out) || k_out == v_out) return GDN_EINVAL;
  if (total > kMostTokens) return GDN_EUNSUPPORTED;
  if (!aligned16(k_out) || !aligned16(v_out)) return GDN_EALIGN;
  GdnKv8GatherArgs a;
  memset(&a, 0, sizeof(a));
  a.cache = *cache;
  a.cu = cu_seqlens;
  a.k_out = k_out;
  a.v_out = v_out;
  a.d_status = d_status;
  a.total = total;
  a.num_seqs = num_seqs;
  a.h_kv = dims->h_kv;
  a.d = dims->d;
  a.page_shift = page_shift(dims->page_size);
  return cuda_rc(gdn_launch_kv8_gather(a, dims->io, reinterpret_cast<cudaStream_t>(stream)));
}

GDN_EXPORT size_t gdn_attn_decode_kv8_workspace_size(const gdn_attn_dims* dims, int32_t n,
                                                     int64_t capacity) {
  if (check_dims(dims, false) != GDN_OK || n < 0 || capacity < 0 || capacity > kMostTokens) return 0;
  if (!page_ok(dims->page_size) || capacity % dims->page_size != 0) return 0;
  if (!scores_ok(dims, n, capacity)) return 0;
  return DecodeWorkspace(dims, n, capacity).size;
}

GDN_EXPORT int gdn_attn_decode_kv8(const gdn_attn_dims* dims, const gdn_view* q,
                                   const gdn_kv8_cache* cache, const int32_t* seq_lens, int32_t n,
                                   const gdn_view* gate, float* weights, void* o, void* workspace,
                                   size_t workspace_bytes, int32_t* d_status,
                                   gdn_stream_t stream) {
  int rc = check_dims(dims, false);
  if (rc != GDN_OK) return rc;
  if (n < 0) return GDN_EINVAL;
  if ((rc = check_kv8(dims, cache)) != GDN_OK) return rc;
  if (n > cache->num_seqs) return GDN_EINVAL;
  if (n == 0) return GDN_OK;
  const gdn_view gv = view_or_none(gate);
  if (!q || !q->data || !seq_lens || !o) return GDN_EINVAL;
  if (o == q->data || o == gv.data) return GDN_EINVAL;
  // (the weights' sums take up to 64 CTAs for a head of a row)
  const int64_t capacity = capacity_of(dims, cache);
  if (!scores_ok(dims, n, weights ? capacity : 0) ||
      (weights && (int64_t)n * dims->h_kv > 0x1ffffff))
    return GDN_EUNSUPPORTED;
  const DecodeWorkspace ws(dims, n, weights ? capacity : 0);
  if (!workspace || workspace_bytes < ws.size) return GDN_EWORKSPACE;
  if (!aligned16(o) || !aligned16(weights) ||
      (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
    return GDN_EALIGN;
  if ((rc = check_view(dims, q, n, dims->h_q)) != GDN_OK) return rc;
  if (gv.data && (rc = check_view(dims, &gv, n, dims->h_q)) != GDN_OK) return rc;
  GdnKv8DecodeArgs a;
  memset(&a, 0, sizeof(a));
  a.q = *q; a.gate = gv;
  a.cache = *cache;
  a.seq_lens = seq_lens;
  a.weights = weights;
  a.o = o;
  a.d_status = d_status;
  char* w = reinterpret_cast<char*>(workspace);
  a.part_o = reinterpret_cast<float*>(w);
  a.part_ml = reinterpret_cast<float2*>(w + ws.part_ml);
  a.row_ml = reinterpret_cast<float2*>(w + ws.row_ml);
  a.scores = reinterpret_cast<float*>(w + ws.scores);
  a.capacity = capacity;
  a.wait_ns = wait_ns_of(dims);
  a.withhold = dims->flags & GDN_TEST_WAIT_TIMEOUT ? 1 : 0;
  a.scale_log2 = scale_log2_of(dims);
  a.n = n; a.h_q = dims->h_q; a.h_kv = dims->h_kv; a.d = dims->d;
  a.page_shift = page_shift(dims->page_size);
  return cuda_rc(gdn_launch_kv8_decode(a, dims->io, reinterpret_cast<cudaStream_t>(stream)));
}

GDN_EXPORT int gdn_kv8_evict(const gdn_attn_dims* dims, const gdn_kv8_cache* from,
                             const float* weights, const int32_t* seq_lens, int32_t n, int32_t keep,
                             int32_t first, int32_t last, const gdn_kv8_cache* to,
                             float* weights_out, int32_t* new_lens, int32_t* kept,
                             int32_t* d_status, gdn_stream_t stream) {
  int rc = check_dims(dims, false);
  if (rc != GDN_OK) return rc;
  if (n < 0 || keep <= 0 || first < 0 || last < 0 || (int64_t)first + last > keep) return GDN_EINVAL;
  if ((rc = check_kv8(dims, from)) != GDN_OK || (rc = check_kv8(dims, to)) != GDN_OK) return rc;
  if (n > from->num_seqs || n > to->num_seqs || capacity_of(dims, to) < keep) return GDN_EINVAL;
  if (n == 0) return GDN_OK;
  if (!weights || !seq_lens || !new_lens || !kept) return GDN_EINVAL;
  if (weights_out == weights || new_lens == seq_lens) return GDN_EINVAL;
  if (!aligned16(weights)) return GDN_EALIGN;
  // the selection takes a CTA per sequence and head, the copy several: all of both, or nothing is launched
  const int64_t items = (int64_t)n * dims->h_kv;
  if (items > 0x7fffffffLL || GdnKv8MoveGrid(items, keep).ctas > 0x7fffffffLL) return GDN_EUNSUPPORTED;
  GdnKv8EvictArgs a;
  memset(&a, 0, sizeof(a));
  a.from = *from;
  a.to = *to;
  a.weights = weights;
  a.weights_out = weights_out;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.kept = kept;
  a.d_status = d_status;
  a.n = n; a.keep = keep; a.first = first; a.last = last;
  a.h_kv = dims->h_kv; a.d = dims->d;
  a.page_shift = page_shift(dims->page_size);
  return cuda_rc(gdn_launch_kv8_evict(a, reinterpret_cast<cudaStream_t>(stream)));
}
