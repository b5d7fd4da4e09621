// gdn_rope.cu -- per-head RMS norm of queries and keys, the rotation by
// position, and the append of keys and values to a paged cache, in one pass.
//
// For a head row x of token t at position p:
//   y = x / sqrt(mean_i x_i^2 + eps) * w,
//   (y_a, y_b) <- s (y_a cos - y_b sin, y_a sin + y_b cos),  angle = p f_i,
// over the pairs (a, b) = (i, i + rot/2) or (2i, 2i + 1) of the first rot
// channels.  Rows are read and written once, so the bytes of q, k and v bound
// it.  An angle belongs to a (token, pair), not to a head: a token's cosines
// and sines are formed once in shared memory and all of its heads read them
// (per row they would cost more instructions than the row's bytes leave time
// for).
//
// The angle: only the fraction of a turn matters.  f / 2 pi modulo 1 is kept as
// a 64-bit fixed-point fraction, and p times it, modulo 2^64, is the fraction
// of the turn exactly as the product of integers: no far position loses bits,
// and no fp64 arithmetic runs per angle (this GPU has little of it).
//
// Two kernels of the same arithmetic: few tokens are spread as thinly as they
// go (one lane group per row where they are very few: 2.3 us for one token);
// many go through a ring of shared-memory stages that one warp per CTA keeps
// filled by TMA, four tokens to a stage, so that eight warps have four
// independent rows each to work on.  Measured, inputs beyond L2: 30011 tokens of
// 16 + 4 heads of 256 in 103 us, 6.0 TB/s; of 32 + 8 heads of 128, wholly
// rotated, 110 us, 5.6 TB/s (88 and 82 % of the copy rate); one token to a stage:
// 137 and 128 us; loads straight into registers: 187 and 160 us.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_attn.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace attn {

using gdn::tc::fence_mbar_init;
using gdn::tc::mbar_arrive;
using gdn::tc::mbar_expect_tx;
using gdn::tc::mbar_init;
using gdn::tc::mbar_wait;
using gdn::tc::smem_u32;

// f radians per position as a fraction of a turn, in 2^-64 of it.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const double t = f * 0.15915494309189533577;
  return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}
// Cosine and sine of position p, from the top 32 bits of the turn's fraction
// as a signed one in half turns.  For 16-bit rows they come from the
// special-function unit, within 2^-20.5 on this range (the rows are rounded by
// 2^-12 or more): the warp that forms the angles would otherwise be what bounds
// wholly rotated heads (30011 tokens of 40 heads of 128: 119 us with sincospif).
template <typename IO>
__device__ __forceinline__ void angle(int32_t p, uint64_t fraction, float scale, float& c, float& s) {
  const uint64_t turn = (uint64_t)(int64_t)p * fraction;
  const float x = (float)(int32_t)(turn >> 32);
  if (sizeof(IO) == 2) {
    const float r = x * (0x1p-31f * 3.14159265358979f);
    asm("cos.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(r));
    asm("sin.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(r));
  } else {
    sincospif(x * 0x1p-31f, &s, &c);
  }
  c *= scale;
  s *= scale;
}

__device__ __forceinline__ float fast_rsqrt(float x) {   // special-function unit, 2 ulp
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The rows of one token, in this order: q heads, k heads, v heads.
enum RowKind { ROW_Q, ROW_K, ROW_V };
struct Row {
  RowKind kind;
  int head;
};
struct RowSet {
  int nq, nk, nv;
  __device__ __forceinline__ explicit RowSet(const GdnRopeArgs& a)
      : nq(a.q.data ? a.h_q : 0), nk(a.k.data ? a.h_kv : 0), nv(a.v.data ? a.h_kv : 0) {}
  __device__ __forceinline__ int per_token() const { return nq + nk + nv; }
  __device__ __forceinline__ Row operator[](int r) const {
    return r < nq ? Row{ROW_Q, r} : r < nq + nk ? Row{ROW_K, r - nq} : Row{ROW_V, r - nq - nk};
  }
};
template <typename IO>
__device__ __forceinline__ const IO* row_ptr(const GdnRopeArgs& a, Row w, int64_t t) {
  const gdn_view& v = w.kind == ROW_Q ? a.q : w.kind == ROW_K ? a.k : a.v;
  return reinterpret_cast<const IO*>(v.data) + t * v.token_stride + w.head * v.head_stride;
}

// A lane's place in a row of D channels (eight per lane) and, in the half
// layout, the lane that holds the other channels of its pairs.
template <int D>
struct LanePlace {
  static constexpr int LPR = D / 8;
  int part, other, i0;
  uint32_t mask;
  bool rotated, low;
  __device__ __forceinline__ explicit LanePlace(const GdnRopeArgs& a) {
    const int half = a.rot_dim >> 1, lane = threadIdx.x & 31;
    part = lane % LPR;
    mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << (lane / LPR * LPR);
    rotated = 8 * part < a.rot_dim;
    low = 8 * part < half;
    other = !rotated || a.interleaved ? part : low ? part + (half >> 3) : part - (half >> 3);
    i0 = !rotated ? 0 : a.interleaved ? 4 * part : low ? 8 * part : 8 * part - half;
  }
};

// A token's cosines, sines and negated sines, D / 2 floats each: the low half of
// a pair takes the negated sine, so that no lane has a sign to apply.
template <typename IO, int D>
__device__ __forceinline__ void put_angle(float* cs, int i, int32_t pos, uint64_t fraction,
                                          float scale) {
  float c, s;
  angle<IO>(pos, fraction, scale, c, s);
  cs[i] = c;
  cs[D / 2 + i] = s;
  cs[D + i] = -s;
}

// Norm (w: this lane's weights; norm false: neither root nor weights) and
// rotation (cs: the tokens', as above, 3 D / 2 floats each) of one head's rows of
// the first `toks` of N tokens, step by step side by side: one row alone is a
// chain of thirteen shuffles.  By the lanes of the row together.
template <typename IO, int D, int N>
__device__ __forceinline__ void norm_rotate(const LanePlace<D>& at, int toks, bool norm,
                                            bool interleaved, bool rotate, float eps,
                                            const float4 (&w)[2], const float* cs,
                                            Vec8<IO> (&x)[N]) {
  uint64_t y[N][4];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    float f[8];
    x[u].get(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[u][i] = pk(f[2 * i], f[2 * i + 1]);
  }
  if (norm) {
    float ss[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      uint64_t sq = mul2(y[u][0], y[u][0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) sq = fma2(y[u][i], y[u][i], sq);
      float s0, s1;
      unpk(sq, s0, s1);
      ss[u] = s0 + s1;
    }
#pragma unroll
    for (int m = at.LPR / 2; m > 0; m >>= 1)
#pragma unroll
      for (int u = 0; u < N; ++u) ss[u] += __shfl_xor_sync(at.mask, ss[u], m, at.LPR);
    const uint64_t w2[4] = {pk(w[0].x, w[0].y), pk(w[0].z, w[0].w), pk(w[1].x, w[1].y),
                            pk(w[1].z, w[1].w)};
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const float inv = fast_rsqrt(ss[u] * (1.0f / D) + eps);
      const uint64_t inv2 = pk(inv, inv);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[u][i] = mul2(mul2(y[u][i], inv2), w2[i]);
    }
  }
  if (rotate && interleaved) {
    if (at.rotated) {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        if (N > 1 && u >= toks) break;
        const float4 c = *reinterpret_cast<const float4*>(cs + u * (D / 2 * 3) + at.i0);
        const float4 s = *reinterpret_cast<const float4*>(cs + u * (D / 2 * 3) + D / 2 + at.i0);
        const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float ya, yb;
          unpk(y[u][i], ya, yb);
          y[u][i] = fma2(y[u][i], pk(cc[i], cc[i]), mul2(pk(yb, ya), pk(-sn[i], sn[i])));
        }
      }
    }
  } else if (rotate) {
    const float* cp = cs + at.i0;
    const float* sp = cp + (at.low ? D : D / 2);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      uint64_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float ya, yb;
        unpk(y[u][i], ya, yb);
        o[i] = pk(__shfl_sync(at.mask, ya, at.other, at.LPR),
                  __shfl_sync(at.mask, yb, at.other, at.LPR));
      }
      if (at.rotated && (N == 1 || u < toks)) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 c = *reinterpret_cast<const float4*>(cp + u * (D / 2 * 3) + 4 * q);
          const float4 s = *reinterpret_cast<const float4*>(sp + u * (D / 2 * 3) + 4 * q);
          y[u][2 * q] = fma2(y[u][2 * q], pk(c.x, c.y), mul2(o[2 * q], pk(s.x, s.y)));
          y[u][2 * q + 1] = fma2(y[u][2 * q + 1], pk(c.z, c.w), mul2(o[2 * q + 1], pk(s.z, s.w)));
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpk(y[u][i], f[2 * i], f[2 * i + 1]);
    x[u].set(f);
  }
}

// Row of the cache pool (before the head) that token t's keys and values go
// to; < 0: none, and reported where that is an error.
__device__ __forceinline__ int64_t cache_row(const GdnRopeArgs& a, int64_t t, int32_t pos) {
  if (pos < 0) return -1;
  const int64_t b = a.row_seq ? (int64_t)a.row_seq[t] : t;
  const int32_t pg = pos >> a.page_shift;
  if (b < 0 || b >= a.cache.num_seqs || pg >= a.cache.pages_per_seq) {
    set_status(a.d_status, GDN_DEV_BAD_LENGTH);
    return -1;
  }
  const int32_t page = __ldg(a.cache.block_table + b * a.cache.pages_per_seq + pg);
  if (page < 0 || page >= a.cache.num_pages) {
    set_status(a.d_status, GDN_DEV_BAD_PAGE);
    return -1;
  }
  return (((int64_t)page * a.h_kv) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// The finished row to q_out, k_out or the cache (dst: cache_row); a padding row of
// an append is zeros.
template <typename IO, int D>
__device__ __forceinline__ void put_row(const GdnRopeArgs& a, Row w, int64_t t, int32_t pos,
                                        int64_t dst, int part, Vec8<IO>& x) {
  const bool append = a.v.data != nullptr;
  if (append && pos < 0) {
    const float zero[8] = {};
    x.set(zero);
  }
  if (append && w.kind != ROW_Q && dst >= 0) {
    const int64_t row = dst + ((int64_t)w.head << a.page_shift);
    x.store(reinterpret_cast<IO*>(w.kind == ROW_V ? a.cache.v : a.cache.k) + row * D + 8 * part);
  }
  IO* out = reinterpret_cast<IO*>(w.kind == ROW_Q ? a.q_out : w.kind == ROW_K ? a.k_out : nullptr);
  if (out) x.store(out + (t * (w.kind == ROW_Q ? a.h_q : a.h_kv) + w.head) * D + 8 * part);
}

// ---- few tokens: one CTA per token, or several with a share of its rows -----

constexpr int FEW_THREADS = 256;

template <typename IO, int D>
__global__ void __launch_bounds__(FEW_THREADS)
    norm_rope_kernel(const __grid_constant__ GdnRopeArgs a) {
  constexpr int GROUPS = FEW_THREADS / (D / 8);
  __shared__ __align__(16) float cs[D / 2 * 3];
  const LanePlace<D> at(a);
  const RowSet set(a);
  const int64_t t = blockIdx.x;
  const int per = set.per_token(), step = GROUPS * gridDim.y;
  int r = blockIdx.y * GROUPS + threadIdx.x / (D / 8);
  Vec8<IO> x[1];
  if (r < per) x[0].load(row_ptr<IO>(a, set[r], t) + 8 * at.part);
  const int32_t pos = a.positions[t];
  const int64_t dst = a.v.data ? cache_row(a, t, pos) : -1;
  for (int i = threadIdx.x; i < a.rot_dim / 2; i += FEW_THREADS)
    put_angle<IO, D>(cs, i, pos, turn_fraction(a.inv_freq[i]), a.rope_scale);
  __syncthreads();
  for (; r < per; r += step) {
    const Row w = set[r];
    Vec8<IO> next;
    if (r + step < per) next.load(row_ptr<IO>(a, set[r + step], t) + 8 * at.part);
    if (w.kind != ROW_V) {
      const float* wp = w.kind == ROW_Q ? a.q_norm : a.k_norm;
      float4 wt[2] = {};
      if (wp) {
        wt[0] = __ldg(reinterpret_cast<const float4*>(wp + 8 * at.part));
        wt[1] = __ldg(reinterpret_cast<const float4*>(wp + 8 * at.part + 4));
      }
      norm_rotate<IO, D, 1>(at, 1, wp != nullptr, a.interleaved, a.rot_dim > 0, a.eps, wt, cs, x);
    }
    put_row<IO, D>(a, w, t, pos, dst, at.part, x[0]);
    x[0] = next;
  }
}

// ---- many tokens: a ring of stages ---------------------------------------------

constexpr int MANY_WARPS = 8;                          // consumers; one more warp loads
constexpr int MANY_THREADS = 32 * (MANY_WARPS + 1);
constexpr int MANY_TOKENS = 4;                         // tokens of a stage
constexpr int MANY_STAGES = 2;
constexpr int MANY_PER_SM = 2;
constexpr int MANY_CTAS = MANY_PER_SM * SMS;
constexpr uint32_t STAGE_ROWS_BYTES = 49152;           // rows of one stage, at most

struct ManyShared {
  uint64_t full[MANY_STAGES], empty[MANY_STAGES];
  int64_t dst[MANY_STAGES][MANY_TOKENS];
  int32_t pos[MANY_STAGES][MANY_TOKENS];
};

// How a unit is cut: `parts` of a token's heads, hq q heads and hkv k and v heads
// each, so that a stage's rows fit.
struct ManyCut {
  int32_t parts, hq, hkv;
  uint32_t stage_bytes;
};

// A unit is MANY_TOKENS tokens, or a part of their heads.  The loading warp looks
// up positions and cache rows for eight units at a time (chains of dependent loads,
// side by side), brings a unit's rows in by one TMA box each for q, k and v, and
// forms the unit's cosines and sines in its stage; a lane group takes one head's
// rows of the unit's tokens at a time.
template <typename IO, int D>
__global__ void __launch_bounds__(MANY_THREADS, MANY_PER_SM)
    norm_rope_ring_kernel(const __grid_constant__ GdnRopeArgs a, const __grid_constant__ ManyCut cut,
                          const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap) {
  constexpr int N = MANY_TOKENS;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(16) ManyShared sh;
  __shared__ __align__(16) float wts[2][D];
  __shared__ uint64_t fraction[D / 2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int parts = cut.parts;
  const int nq = a.q.data ? cut.hq : 0, nk = a.k.data ? cut.hkv : 0, nv = a.v.data ? cut.hkv : 0;
  const int64_t units = (a.n + N - 1) / N * parts;
  // each stage: per token cosines, sines, negated sines [3][D / 2] fp32; then the
  // rows: q [token][head][D], k, v alike
  constexpr int CS = D / 2 * 3;
  constexpr uint32_t CS_BYTES = N * CS * 4;
  constexpr uint32_t ROW_BYTES = D * sizeof(IO);
  bool ok = true;
  int s = 0;               // stage, and the parity of its phase
  uint32_t phase = 0;
  auto advance = [&]() {
    if (++s == MANY_STAGES) {
      s = 0;
      phase ^= 1;
    }
  };
  auto box = [&](uint32_t dst, const CUtensorMap* map, int head, int token) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(token),
        "r"(smem_u32(&sh.full[s]))
        : "memory");
  };
  // the copies of unit u into stage s, by one thread; heads and tokens past the
  // end arrive as zeros
  auto load = [&](int64_t u) {
    const int64_t g = parts == 1 ? u : u / parts;
    const int part = parts == 1 ? 0 : (int)(u - g * parts);
    uint32_t dst = smem_u32(smem) + (uint32_t)s * cut.stage_bytes + CS_BYTES;
    mbar_expect_tx(&sh.full[s], (uint32_t)((nq + nk + nv) * N) * ROW_BYTES);
    if (nq) box(dst, &qmap, part * nq, (int)(g * N));
    dst += (uint32_t)(nq * N) * ROW_BYTES;
    if (nk) box(dst, &kmap, part * nk, (int)(g * N));
    dst += (uint32_t)(nk * N) * ROW_BYTES;
    if (nv) box(dst, &vmap, part * nv, (int)(g * N));
  };
  if (warp == MANY_WARPS && lane == 0) {
    for (int i = 0; i < MANY_STAGES; ++i) {
      mbar_init(&sh.full[i], 2);   // the copies' bytes expected, the angles written
      mbar_init(&sh.empty[i], MANY_WARPS);
    }
    fence_mbar_init();
    // the first units are on their way before anything else
    for (int i = 0; i < MANY_STAGES; ++i, advance())
      if (blockIdx.x + (int64_t)i * gridDim.x < units &&
          !(a.withhold && blockIdx.x == 0 && i == 0))   // (the test's)
        load(blockIdx.x + (int64_t)i * gridDim.x);
  }
  s = 0;
  phase = 0;
  for (int i = tid; i < D; i += MANY_THREADS) {
    wts[0][i] = a.q_norm ? a.q_norm[i] : 1.f;
    wts[1][i] = a.k_norm ? a.k_norm[i] : 1.f;
    if (i < a.rot_dim / 2) fraction[i] = turn_fraction(a.inv_freq[i]);
  }
  __syncthreads();
  if (warp == MANY_WARPS) {
    const int half = a.rot_dim / 2;
    const float scale = a.rope_scale;
    bool first = true;
    int64_t done = 0;        // this CTA's units so far
    for (int64_t base = blockIdx.x; base < units && ok; base += (32LL / N) * gridDim.x) {
      int32_t pos = 0;     // of token lane % N of unit lane / N
      int64_t dst = -1;
      const int64_t unit = base + (int64_t)(lane / N) * gridDim.x;
      const int64_t mine = (parts == 1 ? unit : unit / parts) * N + lane % N;
      if (unit < units && mine < a.n) {
        pos = a.positions[mine];
        if (a.v.data) dst = cache_row(a, mine, pos);
      }
      for (int k = 0; k < 32 / N && base + (int64_t)k * gridDim.x < units; ++k) {
        if (!(first && k < MANY_STAGES)) {   // those are there already
          ok = mbar_wait(&sh.empty[s], phase ^ 1, a.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) load(base + (int64_t)k * gridDim.x);
        }
        // the angles while the copies are on their way
        float* cs = reinterpret_cast<float*>(smem + (size_t)s * cut.stage_bytes);
        int32_t p[N];
#pragma unroll
        for (int tt = 0; tt < N; ++tt) {
          p[tt] = __shfl_sync(0xffffffffu, pos, k * N + tt);
          const int64_t d = __shfl_sync(0xffffffffu, dst, k * N + tt);
          if (lane == 0) {
            sh.pos[s][tt] = p[tt];
            sh.dst[s][tt] = d;
          }
        }
        for (int i = lane; i < half; i += 32) {
          const uint64_t f = fraction[i];
#pragma unroll
          for (int tt = 0; tt < N; ++tt) put_angle<IO, D>(cs + tt * CS, i, p[tt], f, scale);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.full[s]);
        advance();
        ++done;
      }
      first = false;
    }
    // What is in flight lands before this CTA's memory is another's: the consumers wait for
    // it too, unless a wait of theirs has run out.
    for (int64_t x = max(done - MANY_STAGES, (int64_t)0); x < done; ++x)
      mbar_wait(&sh.full[x % MANY_STAGES], (uint32_t)(x / MANY_STAGES) & 1, GRACE_NS);
  } else {
    const LanePlace<D> at(a);
    constexpr int GROUPS = MANY_WARPS * 32 / (D / 8);
    const int group = tid / (D / 8);
    const bool q_normed = a.q_norm != nullptr, k_normed = a.k_norm != nullptr;
    const bool interleaved = a.interleaved, rotate = a.rot_dim > 0, append = a.v.data != nullptr;
    const float eps = a.eps;
    const int64_t n = a.n;
    const int h_q = a.h_q, h_kv = a.h_kv, page_shift = a.page_shift;
    IO* const q_out = reinterpret_cast<IO*>(a.q_out) + 8 * at.part;
    IO* const k_out = a.k_out ? reinterpret_cast<IO*>(a.k_out) + 8 * at.part : nullptr;
    IO* const k_cache = reinterpret_cast<IO*>(a.cache.k) + 8 * at.part;
    IO* const v_cache = reinterpret_cast<IO*>(a.cache.v) + 8 * at.part;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x, advance()) {
      const int64_t g = parts == 1 ? u : u / parts;
      const int part = parts == 1 ? 0 : (int)(u - g * parts);
      const int toks = (int)min((int64_t)N, n - g * N);
      ok = mbar_wait(&sh.full[s], phase, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);   // the rows' lanes leave together
      if (!ok) break;
      const unsigned char* stage = smem + (size_t)s * cut.stage_bytes;
      const float* cs = reinterpret_cast<const float*>(stage);
      const IO* in = reinterpret_cast<const IO*>(stage + CS_BYTES) + 8 * at.part;
      for (int r = group; r < nq + nk + nv; r += GROUPS) {
        const bool is_q = r < nq, is_v = r >= nq + nk;
        const int rr = is_q ? r : is_v ? r - nq - nk : r - nq;
        const int across = is_q ? nq : is_v ? nv : nk;      // rows between tokens in the stage
        const int head = part * across + rr;
        if (head >= (is_q ? h_q : h_kv)) continue;           // a ragged last part
        const IO* src = in + ((is_q ? 0 : is_v ? (nq + nk) * N : nq * N) + rr) * D;
        Vec8<IO> x[N];
#pragma unroll
        for (int tt = 0; tt < N; ++tt) x[tt].load(src + tt * across * D);
        if (!is_v) {
          const float* wp = wts[is_q ? 0 : 1];
          const float4 wt[2] = {*reinterpret_cast<const float4*>(wp + 8 * at.part),
                                *reinterpret_cast<const float4*>(wp + 8 * at.part + 4)};
          norm_rotate<IO, D, N>(at, toks, is_q ? q_normed : k_normed, interleaved, rotate, eps, wt,
                                cs, x);
        }
        if (append) {
#pragma unroll
          for (int tt = 0; tt < N; ++tt)
            if (sh.pos[s][tt] < 0) {   // padding row
              const float zero[8] = {};
              x[tt].set(zero);
            }
        }
        if (append && !is_q) {
          IO* out = (is_v ? v_cache : k_cache) + ((int64_t)head << page_shift) * D;
#pragma unroll
          for (int tt = 0; tt < N; ++tt) {
            const int64_t dst = sh.dst[s][tt];
            if (tt < toks && dst >= 0) x[tt].store(out + dst * D);
          }
        }
        if (is_q || (!is_v && k_out)) {
          const int heads = is_q ? h_q : h_kv;
          IO* out = (is_q ? q_out : k_out) + (g * N * heads + head) * D;
#pragma unroll
          for (int tt = 0; tt < N; ++tt)
            if (tt < toks) x[tt].store(out + (int64_t)tt * heads * D);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[s]);
    }
  }
  if (!ok) set_status(a.d_status, GDN_DEV_WAIT_TIMEOUT);
}

// Rows of a view as (channel, head, token); a box is `heads` heads of MANY_TOKENS.
template <typename IO, int D>
static bool rope_map(CUtensorMap* map, const gdn_view& v, int h, int64_t n, int heads) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(gdn_tensor_map_encoder());
  if (!enc) return false;
  constexpr CUtensorMapDataType type = sizeof(IO) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t dims[3] = {D, (cuuint64_t)h, (cuuint64_t)n};
  // the stride of an axis of extent one is never used: any legal value does
  const cuuint64_t strides[2] = {h > 1 ? (cuuint64_t)v.head_stride * sizeof(IO) : 16,
                                 n > 1 ? (cuuint64_t)v.token_stride * sizeof(IO) : 16};
  const cuuint32_t box[3] = {D, (cuuint32_t)heads, MANY_TOKENS};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, type, 3, const_cast<void*>(v.data), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename IO, int D>
static cudaError_t launch_rope_d(const GdnRopeArgs& a, cudaStream_t s) {
  constexpr int GROUPS = FEW_THREADS / (D / 8);
  const int hq = a.q.data ? a.h_q : 0, hkv = a.k.data ? a.h_kv : 0;
  const int kvs = (a.k.data ? 1 : 0) + (a.v.data ? 1 : 0);
  const int per = hq + kvs * hkv;
  // The two kernels cross near 600 tokens (16 + 4 heads of 256, us, this one and
  // the ring: 512 tokens 5.0 and 5.4, 768 tokens 7.6 and 7.0; of 128 with 32 + 8:
  // 4.6 and 4.7, 6.9 and 5.7).
  if (a.n < 640) {
    // very few tokens: their rows over several CTAs, one row per lane group
    const unsigned split = a.n <= 128 ? (unsigned)((per + GROUPS - 1) / GROUPS) : 1u;
    norm_rope_kernel<IO, D><<<dim3((unsigned)a.n, split), FEW_THREADS, 0, s>>>(a);
    return cudaGetLastError();
  }
  constexpr int MOST = (int)(STAGE_ROWS_BYTES / (MANY_TOKENS * D * sizeof(IO)));
  ManyCut cut;
  cut.parts = (per + MOST - 1) / MOST;
  for (;; ++cut.parts) {   // the parts' shares are rounded up: one more if they do not fit
    cut.hq = (hq + cut.parts - 1) / cut.parts;
    cut.hkv = (hkv + cut.parts - 1) / cut.parts;
    if (cut.hq + kvs * cut.hkv <= MOST && cut.hq <= 256 && cut.hkv <= 256) break;
  }
  const uint32_t angles = MANY_TOKENS * D / 2 * 3 * 4;
  cut.stage_bytes = angles + (uint32_t)((cut.hq + kvs * cut.hkv) * MANY_TOKENS * D) * sizeof(IO);
  CUtensorMap qmap = {}, kmap = {}, vmap = {};
  if ((a.q.data && !rope_map<IO, D>(&qmap, a.q, a.h_q, a.n, cut.hq)) ||
      (a.k.data && !rope_map<IO, D>(&kmap, a.k, a.h_kv, a.n, cut.hkv)) ||
      (a.v.data && !rope_map<IO, D>(&vmap, a.v, a.h_kv, a.n, cut.hkv)))
    return cudaErrorInvalidValue;
  auto kernel = norm_rope_ring_kernel<IO, D>;
  cudaError_t e = cudaSuccess;
  static int opted_in[64] = {};
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !opted_in[dev]) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)(MANY_STAGES * (STAGE_ROWS_BYTES + angles)))) != cudaSuccess)
      return e;
    if (dev >= 0 && dev < 64) opted_in[dev] = 1;
  }
  const int64_t units = (a.n + MANY_TOKENS - 1) / MANY_TOKENS * cut.parts;
  const unsigned grid = (unsigned)(units < MANY_CTAS ? units : MANY_CTAS);
  kernel<<<grid, MANY_THREADS, MANY_STAGES * cut.stage_bytes, s>>>(a, cut, qmap, kmap, vmap);
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
