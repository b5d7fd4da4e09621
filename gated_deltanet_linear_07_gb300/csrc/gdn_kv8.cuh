// gdn_kv8.cuh -- what the kernels of the 8-bit cache share: e4m3 conversions, the
// block's scale, and the launch descriptors between the API translation unit
// and the kernels.
#pragma once

#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

constexpr int KV8_BLOCK = GDN_KV8_BLOCK;
constexpr int KV8_MIN_EXP = -40, KV8_MAX_EXP = 40;

// Four numbers as e4m3 (nearest, ties to even; above 448 as 448, NaN as NaN).
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Four e4m3 numbers as two pairs of fp16 (every one is an fp16 number).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float4 from_e4m3x4(uint32_t w) {
  uint32_t lo, hi;
  e4m3x4_to_f16(w, lo, hi);
  const float2 a = unpack2<__half>(lo), b = unpack2<__half>(hi);
  return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The smallest 2^e, e in [KV8_MIN_EXP, KV8_MAX_EXP], with top <= 448 * 2^e: 448 is
// 1.75 * 2^8, so the exponent of top decides, and whether its mantissa is above 1.75.
__device__ __forceinline__ int kv8_exponent(float top) {
  const uint32_t bits = __float_as_uint(top);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, KV8_MIN_EXP), KV8_MAX_EXP);
}
// A block's scale as the calls take it (0: all that it holds stands for 0).
__device__ __forceinline__ bool kv8_scale_ok(float s) {
  return s == 0.f || (s >= 0x1p-40f && s <= 0x1p40f);
}

}  // namespace attn
}  // namespace gdn

struct GdnKv8AppendArgs {
  GdnRopeArgs r;               // its cache and row_seq are not used
  gdn_kv8_cache cache;
  const int32_t* cu;           // null: row t is sequence t
  const int32_t* starts;
  int32_t num_seqs;
};

struct GdnKv8GatherArgs {
  gdn_kv8_cache cache;
  const int32_t* cu;
  void* k_out;
  void* v_out;
  int32_t* d_status;
  int64_t total;
  int32_t num_seqs, h_kv, d, page_shift;
};

struct GdnKv8EvictArgs {
  gdn_kv8_cache from, to;
  const float* weights;
  float* weights_out;
  const int32_t* seq_lens;
  int32_t* new_lens;
  int32_t* kept;
  int32_t* d_status;
  int32_t n, keep, first, last, h_kv, d, page_shift;
};

// The eviction's copy: each CTA has `blocks` blocks of the new pages of one sequence and head,
// `across` CTAs each of these; ctas in all.
struct GdnKv8MoveGrid {
  static constexpr int WARPS = 8, BLOCKS = 16;   // of a CTA, at most
  int blocks;
  int64_t across, ctas;
  GdnKv8MoveGrid(int64_t items, int32_t keep) : blocks(BLOCKS) {
    const int64_t all = ((int64_t)keep + GDN_KV8_BLOCK - 1) / GDN_KV8_BLOCK;
    // fewer where that leaves SMs idle, down to a unit (a block's keys or values) per warp
    while (blocks > WARPS / 2 && items * ((all + blocks - 1) / blocks) < 4 * gdn::attn::SMS) blocks /= 2;
    across = (all + blocks - 1) / blocks;
    ctas = items * across;
  }
};

struct GdnKv8DecodeArgs {
  gdn_view q, gate;
  gdn_kv8_cache cache;
  const int32_t* seq_lens;
  float* weights;              // null: none are collected
  void* o;
  int32_t* d_status;
  float* part_o;               // workspace: partial outputs [slot][d],
  float2* part_ml;             // their (reference maximum in log2 units, sum);
  float2* row_ml;              // with weights: the rows' [n][h_q] alike,
  float* scores;               // and [n][h_q][capacity] scores in log2 units
  int64_t capacity;            // tokens of a block table row
  uint64_t wait_ns;
  int32_t withhold;            // GDN_TEST_WAIT_TIMEOUT: some hand-overs never come
  float scale_log2;            // scale * log2(e)
  int32_t n, h_q, h_kv, d, page_shift;
};

cudaError_t gdn_launch_kv8_append(const GdnKv8AppendArgs& a, int io, cudaStream_t s);
cudaError_t gdn_launch_kv8_gather(const GdnKv8GatherArgs& a, int io, cudaStream_t s);
cudaError_t gdn_launch_kv8_evict(const GdnKv8EvictArgs& a, cudaStream_t s);
// Slots of partial results that a decode of these heads needs.
int64_t gdn_kv8_decode_slots(int h_q, int h_kv);
cudaError_t gdn_launch_kv8_decode(const GdnKv8DecodeArgs& a, int io, cudaStream_t s);
