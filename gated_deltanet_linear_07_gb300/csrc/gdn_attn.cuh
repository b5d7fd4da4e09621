// gdn_attn.cuh -- what the full-attention kernels share: 16-bit and 32-bit
// element vectors and the launch descriptors between the API translation unit
// and the kernels.
#pragma once

#include <cuda_fp16.h>

#include "gdn_common.cuh"

namespace gdn {
namespace attn {

constexpr int SMS = 152;                 // of the one GPU this is built for
constexpr int PREFIX_SMS = 96;           // of them, the shared prefix's pass of a decode: about
                                         // two thirds, a number that 2, 3, 4, 6 and 8 divide

// For copies and products in flight when a wait has run out (they take microseconds).
constexpr uint64_t GRACE_NS = 1000000;

// Eight consecutive channels of a row: one 16-byte access (16-bit types) or
// two (fp32).
template <typename IO>
struct Vec8;

template <>
struct Vec8<float> {
  float4 lo, hi;
  __device__ __forceinline__ void load(const float* p) {
    lo = *reinterpret_cast<const float4*>(p);
    hi = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = lo;
    *reinterpret_cast<float4*>(p + 4) = hi;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = lo.x; f[1] = lo.y; f[2] = lo.z; f[3] = lo.w;
    f[4] = hi.x; f[5] = hi.y; f[6] = hi.z; f[7] = hi.w;
  }
  // The same channels of lane `src` of a group of `width` lanes.
  __device__ __forceinline__ void exchange(uint32_t mask, int src, int width) {
    lo = make_float4(__shfl_sync(mask, lo.x, src, width), __shfl_sync(mask, lo.y, src, width),
                     __shfl_sync(mask, lo.z, src, width), __shfl_sync(mask, lo.w, src, width));
    hi = make_float4(__shfl_sync(mask, hi.x, src, width), __shfl_sync(mask, hi.y, src, width),
                     __shfl_sync(mask, hi.z, src, width), __shfl_sync(mask, hi.w, src, width));
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    lo = make_float4(f[0], f[1], f[2], f[3]);
    hi = make_float4(f[4], f[5], f[6], f[7]);
  }
};

template <typename IO>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename IO>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <typename IO>
struct Vec8 {
  uint4 w;
  __device__ __forceinline__ void load(const IO* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(IO* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2<IO>(u[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  __device__ __forceinline__ void exchange(uint32_t mask, int src, int width) {
    w = make_uint4(__shfl_sync(mask, w.x, src, width), __shfl_sync(mask, w.y, src, width),
                   __shfl_sync(mask, w.z, src, width), __shfl_sync(mask, w.w, src, width));
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    w = make_uint4(pack2<IO>(f[0], f[1]), pack2<IO>(f[2], f[3]), pack2<IO>(f[4], f[5]),
                   pack2<IO>(f[6], f[7]));
  }
};

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pk(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpk(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The softmax weights on their way to the product with v, 2^(c (s - m)) with a
// reference m that may lag behind the row's true maximum by up to LAG_LOG2, are
// formed SCALE_LOG2 larger (the row's sum too: the quotient is the same).  bf16 has
// the range of fp32 and needs no scale.  fp16 has 30 powers of two in its normal
// range: with 2^12 and a lag of 2^3.9 the largest weight is 61147 of 65504 (the
// rounding of the exponent stays far below the rest of it) and those down to
// 2^-26 of the reference keep their relative accuracy (unscaled, weights below 2^-25
// were zeros, which 2048 keys of 2^-26 together are not).  A lag of 2^3 rescales
// so much more often that 24,001 fp16 tokens of 16 sequences took 3.5 % longer.
template <typename IO>
struct WeightRange {
  static constexpr float LAG_LOG2 = 8.0f, SCALE_LOG2 = 0.0f;
};
template <>
struct WeightRange<__half> {
  static constexpr float LAG_LOG2 = 3.9f, SCALE_LOG2 = 12.0f;
};
// What is added to c s for the weight's exponent (m: -inf before the first key).
template <typename IO>
__device__ __forceinline__ float weight_offset(float m, float c) {
  constexpr float up = WeightRange<IO>::SCALE_LOG2;
  return m == -INFINITY ? 0.f : up == 0.f ? -m * c : fmaf(-m, c, up);
}

// sigmoid(x) with the exponential and the quotient on the special-function
// unit: a few ulp, 0 and 1 at the ends.
__device__ __forceinline__ float gate_sigmoid(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * x));
  return __fdividef(1.0f, 1.0f + e);
}

}  // namespace attn
}  // namespace gdn

// One call of gdn_qk_norm_rope, gdn_qk_norm_rope_axes or gdn_kv_append.
struct GdnRopeArgs {
  gdn_view q, k, v;            // null data: left out (v: no append)
  void* q_out;
  void* k_out;                 // may be null with an append: k goes to the cache
  const float* q_norm;
  const float* k_norm;
  const double* inv_freq;
  const int32_t* positions;
  const int32_t* row_seq;
  gdn_kv_cache cache;
  int32_t* d_status;
  int64_t n;
  uint64_t wait_ns;
  int32_t withhold;            // GDN_TEST_WAIT_TIMEOUT: one unit's copies never come
  int32_t h_q, h_kv, d, rot_dim, interleaved, page_shift;
  float eps, rope_scale;
  gdn_rope_axes axes;          // count 0: one axis; else positions [count][n]
};

// One attention call; the prefix pass of gdn_attn_decode uses the same kernel
// as gdn_attn_prefill, with the batch's rows as its tokens.
struct GdnAttnArgs {
  gdn_view q, k, v;            // k, v: packed keys and values (prefill)
  gdn_view gate;               // null data: none
  void* o;
  const int32_t* cu_q;
  const int32_t* cu_kv;
  gdn_kv_cache cache;          // decode
  const int32_t* seq_lens;     // decode
  int32_t* d_status;
  float* part_o;               // decode workspace: partial outputs, [slot][d] fp32,
  float2* part_ml;             // and their (reference maximum in log2 units, sum)
  int64_t total_q, total_kv, shared_len;
  uint64_t wait_ns;
  int32_t withhold;            // GDN_TEST_WAIT_TIMEOUT: some hand-overs never come
  float scale_log2;            // scale * log2(e)
  int32_t h_q, h_kv, d, num_seqs, page_shift;
  int32_t splits;              // prefix pass: how many CTA groups share the prefix
};

cudaError_t gdn_launch_rope(const GdnRopeArgs& a, int io, cudaStream_t s);
cudaError_t gdn_launch_attn_prefill(const GdnAttnArgs& a, int io, cudaStream_t s);
// Decode: slots of partial results that n rows behind shared_len shared tokens
// need, and the launches (prefix pass, per-sequence pass, merge).
int64_t gdn_attn_decode_slots(int h_q, int h_kv, int d, int n, int64_t shared_len);
cudaError_t gdn_launch_attn_decode(const GdnAttnArgs& a, int io, cudaStream_t s);
// How many CTA groups share the keys of the prefix pass (0: no pass).
int gdn_attn_prefix_splits(int h_q, int h_kv, int d, int n, int64_t shared_len);
// SMs that the prefix pass takes.
int gdn_attn_prefix_ctas(int h_q, int h_kv, int d, int n, int64_t shared_len);
cudaError_t gdn_launch_attn_prefix(const GdnAttnArgs& a, int io, cudaStream_t s);
