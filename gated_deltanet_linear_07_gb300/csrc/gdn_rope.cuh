// gdn_rope.cuh -- the arithmetic of the per-head norm and rotation, shared by
// the kernels that norm and rotate rows (gdn_rope.cu) and the one that stores
// them in 8 bits (gdn_kv8.cu).
#pragma once

#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

// f radians per position as a fraction of a turn, in 2^-64 of it.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const double t = f * 0.15915494309189533577;
  return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}
// Cosine and sine of position p, from the top 32 bits of the turn's fraction
// as a signed one in half turns.  For 16-bit rows they come from the
// special-function unit, within 2^-20.5 on this range (the rows are rounded by
// 2^-12 or more): the warp that forms the angles would otherwise be what bounds
// wholly rotated heads (30011 tokens of 40 heads of 128: 119 us with sincospif).  Keys that are
// stored in 8 bits take the same, so that the packed ones beside them are the rotation's bits;
// more of them than with fp32's own functions round to the other side of a border (16,384 tokens of
// 4 heads of 256, a quarter rotated: 2.3 of a million numbers, 0.7 with those).
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
    i0 = !rotated ? 0 : a.interleaved || low ? 4 * part : 4 * part - (half >> 1);
  }
};

// A token's cosines, sines and negated sines, D / 2 floats each: the low half of
// a pair takes the negated sine, so that no lane has a sign to apply.  In the half layout a
// lane reads eight pairs, four at a time: the first fours of all lanes lie side by side, and
// the second ones, so that eight lanes read 128 bytes in a row (with a lane's eight side by
// side two of them meet in every bank: 16,411 tokens of 40 heads of 128, all rotated, 76 us
// where this takes 64).
template <int D>
__device__ __forceinline__ int angle_place(bool interleaved, int i) {
  return interleaved ? i : (i & 4) * (D / 16) + (i >> 3) * 4 + (i & 3);
}
template <typename IO, int D>
__device__ __forceinline__ void put_angle(float* cs, int place, int32_t pos, uint64_t fraction,
                                          float scale) {
  float c, s;
  angle<IO>(pos, fraction, scale, c, s);
  cs[place] = c;
  cs[D / 2 + place] = s;
  cs[D + place] = -s;
}

// Norm (w: this lane's weights; norm false: neither root nor weights) and
// rotation (cs: the tokens', as above, 3 D / 2 floats each) of one head's rows of
// the first `toks` of N tokens, step by step side by side: one row alone is a
// chain of thirteen shuffles.  By the lanes of the row together; y: pairs of channels in fp32.
template <typename IO, int D, int N>
__device__ __forceinline__ void norm_rotate_fp32(const LanePlace<D>& at, int toks, bool norm,
                                                 bool interleaved, bool rotate, float eps,
                                                 const float4 (&w)[2], const float* cs,
                                                 const Vec8<IO> (&x)[N], uint64_t (&y)[N][4]) {
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
          const float4 c = *reinterpret_cast<const float4*>(cp + u * (D / 2 * 3) + D / 4 * q);
          const float4 s = *reinterpret_cast<const float4*>(sp + u * (D / 2 * 3) + D / 4 * q);
          y[u][2 * q] = fma2(y[u][2 * q], pk(c.x, c.y), mul2(o[2 * q], pk(s.x, s.y)));
          y[u][2 * q + 1] = fma2(y[u][2 * q + 1], pk(c.z, c.w), mul2(o[2 * q + 1], pk(s.z, s.w)));
        }
      }
    }
  }
}
// The same, rounded to the rows' type in their place.
template <typename IO, int D, int N>
__device__ __forceinline__ void norm_rotate(const LanePlace<D>& at, int toks, bool norm,
                                            bool interleaved, bool rotate, float eps,
                                            const float4 (&w)[2], const float* cs,
                                            Vec8<IO> (&x)[N]) {
  uint64_t y[N][4];
  norm_rotate_fp32<IO, D, N>(at, toks, norm, interleaved, rotate, eps, w, cs, x, y);
#pragma unroll
  for (int u = 0; u < N; ++u) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpk(y[u][i], f[2 * i], f[2 * i + 1]);
    x[u].set(f);
  }
}

}  // namespace attn
}  // namespace gdn
