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

// Which of a token's rows a lane group works on: a q head, a k head or a v head.
enum RowKind { ROW_Q, ROW_K, ROW_V };

// D / 8 lanes hold one row, eight channels each.  A lane group stays with one
// head for the CTA's TOK tokens, whose rows are all in flight at once: the
// head's weights and addresses are formed once, and the next head's rows are
// fetched while this one's are worked on.
template <typename IO, int D, int TOK>
__global__ void __launch_bounds__(ROPE_THREADS)
    norm_rope_kernel(const __grid_constant__ GdnRopeArgs a) {
  constexpr int LPR = D / 8;
  constexpr int GROUPS = ROPE_THREADS / LPR;
  __shared__ __align__(16) float cs[TOK][2][D / 2];   // cosines, sines
  const int tid = threadIdx.x;
  const int part = tid % LPR;            // this lane's channels: 8 part .. 8 part + 7
  const int64_t t0 = (int64_t)blockIdx.x * TOK;
  const int toks = (int)(a.n - t0 < TOK ? a.n - t0 : TOK);
  const int half = a.rot_dim >> 1;
  const int nq = a.q.data ? a.h_q : 0, nk = a.k.data ? a.h_kv : 0, nv = a.v.data ? a.h_kv : 0;
  const int per = nq + nk + nv;          // rows of one token: q heads, k heads, v heads
  // every shuffle is among the lanes of one row
  const uint32_t mask = LPR == 32 ? 0xffffffffu
                                  : ((1u << (LPR & 31)) - 1u) << ((tid & 31) / LPR * LPR);
  // half layout: the other channel of each pair sits half / 8 lanes away
  const bool rotated = 8 * part < a.rot_dim;
  const bool low = 8 * part < half;
  const int other = !rotated || a.interleaved ? part : low ? part + (half >> 3) : part - (half >> 3);

  auto kind_of = [&](int h) { return h < nq ? ROW_Q : h < nq + nk ? ROW_K : ROW_V; };
  auto fetch = [&](int h, Vec8<IO> (&x)[TOK]) {
    const RowKind kind = kind_of(h);
    const gdn_view& w = kind == ROW_Q ? a.q : kind == ROW_K ? a.k : a.v;
    const int hh = kind == ROW_Q ? h : kind == ROW_K ? h - nq : h - nq - nk;
    const IO* p = reinterpret_cast<const IO*>(w.data) + t0 * w.token_stride + hh * w.head_stride +
                  8 * part;
#pragma unroll
    for (int u = 0; u < TOK; ++u)
      if (u < toks) x[u].load(p + u * w.token_stride);
  };
  const int step = GROUPS * gridDim.y;
  int h = blockIdx.y * GROUPS + tid / LPR;
  Vec8<IO> x[TOK];
  if (h < per) fetch(h, x);

  // The angle in turns, reduced in fp64 (positions may be far), then fp32.
  for (int i = tid; i < toks * half; i += ROPE_THREADS) {
    const int tt = i / half, f = i - tt * half;
    const double turns = (double)a.positions[t0 + tt] * (a.inv_freq[f] * 0.15915494309189533577);
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    cs[tt][0][f] = c * a.rope_scale;
    cs[tt][1][f] = s * a.rope_scale;
  }
  __syncthreads();

  for (; h < per; h += step) {
    const RowKind kind = kind_of(h);
    const int hh = kind == ROW_Q ? h : kind == ROW_K ? h - nq : h - nq - nk;
    Vec8<IO> next[TOK];
    if (h + step < per) fetch(h + step, next);
    if (kind != ROW_V) {
      const float* wp = kind == ROW_Q ? a.q_norm : a.k_norm;
      float w[8], wo[8];   // this lane's weights and those of the pairs' other channels
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = wo[i] = 1.f;
      if (wp) {
        reinterpret_cast<float4*>(w)[0] = __ldg(reinterpret_cast<const float4*>(wp + 8 * part));
        reinterpret_cast<float4*>(w)[1] = __ldg(reinterpret_cast<const float4*>(wp + 8 * part + 4));
        reinterpret_cast<float4*>(wo)[0] = __ldg(reinterpret_cast<const float4*>(wp + 8 * other));
        reinterpret_cast<float4*>(wo)[1] =
            __ldg(reinterpret_cast<const float4*>(wp + 8 * other + 4));
      }
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        if (u >= toks) break;
        float f[8];
        x[u].get(f);
        float inv = 1.f;
        if (wp) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
          for (int m = LPR / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(mask, ss, m, LPR);
          inv = rsqrtf(ss * (1.0f / D) + a.eps);
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = f[i] * inv * w[i];
        if (a.interleaved) {
          if (rotated) {
            float c[4], s[4];
            *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(&cs[u][0][4 * part]);
            *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(&cs[u][1][4 * part]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float ya = y[2 * i], yb = y[2 * i + 1];
              y[2 * i] = ya * c[i] - yb * s[i];
              y[2 * i + 1] = ya * s[i] + yb * c[i];
            }
          }
        } else if (half > 0) {
          Vec8<IO> xo = x[u];
          xo.exchange(mask, other, LPR);   // the raw channels: half the words of the normed ones
          if (rotated) {
            float o[8], c[8], s[8];
            xo.get(o);
            const int i0 = low ? 8 * part : 8 * part - half;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              reinterpret_cast<float4*>(c)[q] =
                  *reinterpret_cast<const float4*>(&cs[u][0][i0 + 4 * q]);
              reinterpret_cast<float4*>(s)[q] =
                  *reinterpret_cast<const float4*>(&cs[u][1][i0 + 4 * q]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float yo = o[i] * inv * wo[i];
              y[i] = y[i] * c[i] + (low ? -yo : yo) * s[i];
            }
          }
        }
        x[u].set(y);
      }
    }
    // ---- to q_out, k_out or the cache ----
    if (kind == ROW_Q || !a.v.data) {
      const int heads = kind == ROW_Q ? a.h_q : a.h_kv;
      IO* dst = reinterpret_cast<IO*>(kind == ROW_Q ? a.q_out : a.k_out) + (t0 * heads + hh) * D +
                8 * part;
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        if (u >= toks) break;
        if (a.v.data && a.positions[t0 + u] < 0) {   // padding row of an append
          const float zero[8] = {};
          x[u].set(zero);
        }
        x[u].store(dst + (int64_t)u * heads * D);
      }
    } else {
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        if (u >= toks) break;
        const int64_t t = t0 + u;
        const int32_t pos = a.positions[t];
        if (pos < 0) continue;
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
        x[u].store(reinterpret_cast<IO*>(kind == ROW_V ? a.cache.v : a.cache.k) + row * D +
                   8 * part);
      }
    }
#pragma unroll
    for (int u = 0; u < TOK; ++u) x[u] = next[u];
  }
}

template <typename IO, int D>
static cudaError_t launch_rope_d(const GdnRopeArgs& a, cudaStream_t s) {
  constexpr int GROUPS = ROPE_THREADS / (D / 8);
  // Four tokens to a CTA once there are enough of them to fill the SMs that
  // way.  Below that one, and with few tokens their heads over several CTAs
  // too, so that no lane group has more than one row.
  if (a.n >= 2048) {
    norm_rope_kernel<IO, D, 4><<<(unsigned)((a.n + 3) / 4), ROPE_THREADS, 0, s>>>(a);
  } else {
    const int per = (a.q.data ? a.h_q : 0) + (a.k.data ? a.h_kv : 0) + (a.v.data ? a.h_kv : 0);
    const unsigned split = a.n <= 128 ? (unsigned)((per + GROUPS - 1) / GROUPS) : 1u;
    norm_rope_kernel<IO, D, 1><<<dim3((unsigned)a.n, split), ROPE_THREADS, 0, s>>>(a);
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
