// gdn_rope.cu -- per-head RMS norm of queries and keys, the rotation by
// position, and the append of keys and values to a paged cache, in one pass.
//
// For a head row x of token t at position p:
//   y = x / sqrt(mean_i x_i^2 + eps) * w,
//   (y_a, y_b) <- s (y_a cos - y_b sin, y_a sin + y_b cos),  angle = p f_i,
// over the pairs (a, b) = (i, i + rot/2) or (2i, 2i + 1) of the first rot
// channels.  Rows are read and written once, so the bytes of q, k and v bound
// it.  An angle belongs to a (token, pair), not to a head: the CTA computes
// its tokens' cosines and sines once into shared memory and all heads of those
// tokens read them (per row they would cost more instructions than the row's
// bytes leave time for).
#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_BATCH = 4;   // rows in flight per lane group

// D / 8 lanes hold one row, eight channels each; TOK tokens per CTA.
template <typename IO, int D, int TOK>
__global__ void __launch_bounds__(ROPE_THREADS)
    norm_rope_kernel(const __grid_constant__ GdnRopeArgs a) {
  constexpr int LPR = D / 8;
  constexpr int GROUPS = ROPE_THREADS / LPR;
  __shared__ __align__(16) float2 cs[TOK * (D / 2)];
  const int tid = threadIdx.x;
  const int part = tid % LPR;            // this lane's channels: 8 part .. 8 part + 7
  const int group = tid / LPR;
  const int64_t t0 = (int64_t)blockIdx.x * TOK;
  const int toks = (int)(a.n - t0 < TOK ? a.n - t0 : TOK);
  const int half = a.rot_dim >> 1;
  const int nq = a.q.data ? a.h_q : 0, nk = a.k.data ? a.h_kv : 0, nv = a.v.data ? a.h_kv : 0;
  const int per = nq + nk + nv;          // rows of one token: q heads, k heads, v heads
  const int rows = toks * per;

  // The angle in turns, reduced in fp64 (positions may be far), then fp32.
  for (int i = tid; i < toks * half; i += ROPE_THREADS) {
    const int tt = i / half;
    const double turns = (double)a.positions[t0 + tt] *
                         (a.inv_freq[i - tt * half] * 0.15915494309189533577);
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    cs[i] = make_float2(c * a.rope_scale, s * a.rope_scale);
  }
  __syncthreads();

  for (int r0 = group; r0 < rows + group; r0 += GROUPS * ROPE_BATCH) {
    Vec8<IO> x[ROPE_BATCH];
#pragma unroll
    for (int u = 0; u < ROPE_BATCH; ++u) {
      const int r = r0 + u * GROUPS;
      if (r >= rows) continue;
      const int tt = r / per, h = r - tt * per;
      const gdn_view& w = h < nq ? a.q : h < nq + nk ? a.k : a.v;
      const int hh = h < nq ? h : h < nq + nk ? h - nq : h - nq - nk;
      x[u].load(reinterpret_cast<const IO*>(w.data) + (t0 + tt) * w.token_stride +
                hh * w.head_stride + 8 * part);
    }
#pragma unroll
    for (int u = 0; u < ROPE_BATCH; ++u) {
      const int r = r0 + u * GROUPS;
      // the lanes of a group take this branch together, other groups of the
      // warp may not: every shuffle below is masked to the group
      if (r >= rows) continue;
      const uint32_t mask = LPR == 32 ? 0xffffffffu
                                      : ((1u << (LPR & 31)) - 1u) << ((tid & 31) / LPR * LPR);
      const int tt = r / per, h = r - tt * per;
      const int64_t t = t0 + tt;
      const bool is_q = h < nq, is_v = h >= nq + nk;
      const int hh = is_q ? h : is_v ? h - nq - nk : h - nq;
      const int32_t pos = a.positions[t];
      float f[8];
      if (!is_v) {
        x[u].get(f);
        const float* wp = is_q ? a.q_norm : a.k_norm;
        if (wp) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
          for (int m = LPR / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(mask, ss, m, LPR);
          const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
          const float4 w0 = __ldg(reinterpret_cast<const float4*>(wp + 8 * part));
          const float4 w1 = __ldg(reinterpret_cast<const float4*>(wp + 8 * part + 4));
          const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * w[i];
        }
        const float2* c2 = cs + tt * half;
        if (a.interleaved) {
          if (8 * part < a.rot_dim) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 c = c2[4 * part + i];
              const float ya = f[2 * i], yb = f[2 * i + 1];
              f[2 * i] = ya * c.x - yb * c.y;
              f[2 * i + 1] = ya * c.y + yb * c.x;
            }
          }
        } else if (half > 0) {
          // the other channel of each pair sits half / 8 lanes away
          const bool lo = 8 * part < half, in = 8 * part < a.rot_dim;
          const int other = !in ? part : lo ? part + (half >> 3) : part - (half >> 3);
          const int i0 = !in ? 0 : lo ? 8 * part : 8 * part - half;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float y = __shfl_sync(mask, f[i], other, LPR);
            if (in) {
              const float2 c = c2[i0 + i];
              f[i] = lo ? f[i] * c.x - y * c.y : y * c.y + f[i] * c.x;
            }
          }
        }
        x[u].set(f);
      }
      if (is_q) {
        if (pos < 0 && a.v.data) {   // padding row of an append
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = 0.f;
          x[u].set(f);
        }
        x[u].store(reinterpret_cast<IO*>(a.q_out) + (t * a.h_q + hh) * D + 8 * part);
      } else if (!a.v.data) {
        x[u].store(reinterpret_cast<IO*>(a.k_out) + (t * a.h_kv + hh) * D + 8 * part);
      } else if (pos >= 0) {
        // the row's place in the cache; a row without one is reported and left out
        const int64_t b = a.row_seq ? (int64_t)a.row_seq[t] : t;
        const int32_t pg = pos >> a.page_shift;
        if (b < 0 || b >= a.cache.num_seqs || pg >= a.cache.pages_per_seq) {
          if (part == 0) set_status(a.d_status, GDN_DEV_BAD_LENGTH);
          continue;
        }
        const int32_t page = __ldg(a.cache.block_table + b * a.cache.pages_per_seq + pg);
        if (page < 0 || page >= a.cache.num_pages) {
          if (part == 0) set_status(a.d_status, GDN_DEV_BAD_PAGE);
          continue;
        }
        const int64_t row = (((int64_t)page * a.h_kv + hh) << a.page_shift) +
                            (pos & ((1 << a.page_shift) - 1));
        x[u].store(reinterpret_cast<IO*>(is_v ? a.cache.v : a.cache.k) + row * D + 8 * part);
      }
    }
  }
}

template <typename IO, int D>
static cudaError_t launch_rope_d(const GdnRopeArgs& a, cudaStream_t s) {
  // Four tokens to a CTA once there are enough of them to fill the SMs that
  // way; below that one, so that few tokens still spread over the SMs.
  if (a.n >= 2048) {
    norm_rope_kernel<IO, D, 4><<<(unsigned)((a.n + 3) / 4), ROPE_THREADS, 0, s>>>(a);
  } else {
    norm_rope_kernel<IO, D, 1><<<(unsigned)a.n, ROPE_THREADS, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename IO>
static cudaError_t launch_rope_io(const GdnRopeArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_rope_d<IO, 64>(a, s)
                   : a.d == 128 ? launch_rope_d<IO, 128>(a, s) : launch_rope_d<IO, 256>(a, s);
}

}  // namespace attn
}  // namespace gdn

cudaError_t gdn_launch_rope(const GdnRopeArgs& a, int io, cudaStream_t s) {
  using namespace gdn::attn;
  return io == GDN_FP32 ? launch_rope_io<float>(a, s)
                        : io == GDN_BF16 ? launch_rope_io<__nv_bfloat16>(a, s)
                                         : launch_rope_io<__half>(a, s);
}
