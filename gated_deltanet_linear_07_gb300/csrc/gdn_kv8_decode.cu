// gdn_kv8_decode.cu -- one query token per sequence against the cache held in 8
// bits.  With k8, v8 the stored numbers and a, b their blocks' scales,
//
//   s_p = c a_p (q . k8_p),   o = sum_p 2^(s_p - M) b_p v8_p / sum_p 2^(s_p - M).
//
// Every cached byte is used for one token's few query heads only, so the reads of the
// cache bound it, and at half the bytes per key, what a key costs to compute has half the
// time.  The products therefore have the keys, and the channels of the values, on the
// 16-row side of mma.sync m16n8k16 and the query heads on its 8-row side: S^T = K Q^T
// and O^T = V^T P^T, half the instructions and half the exponentials of the
// other way round for up to 8 heads.  An e4m3 number is an fp16 number: one conversion
// for two of them, no scale applied to any.  (mma.sync of e4m3 itself is put together
// from conversions and fp16 products here: 29 cycles of a scheduler where an m16n8k16
// takes 8.5, and with the operands in two or three terms each the step of 64
// sequences took 165 us instead of 123.)  K's fragments come straight from ldmatrix of
// bytes, with the channels of a 16-byte chunk in an order that Q's share (a sum does
// not mind); V's from its transposing form, two keys' bytes put side by side by one
// permutation.  P^T passes from the accumulators' layout to the operand's by a transpose
// between lanes.
//
// Two references per head: M for the sum of the weights, and M' for the largest
// contribution s_p + log2 b_p, by which the weights are scaled for the product with v
// in fp16: blocks of large and small values may follow each other in any order
// without either leaving fp16's range unless it is negligible beside the other.  Both may
// lag behind the true maxima by 2^3.9, so that they move at the first keys only and no
// lane asks the others for a maximum in between.
//
// The work is cut by bytes: all units of 32 KB (64 keys of 256, 128 of 128, 256 of 64) of
// all (sequence, key/value head) items form one line, with a little added for the beginning
// and end of each item, which the resident CTAs share in equal runs.  A run that covers an
// item writes its output; an item cut by a run's border leaves partial results that the
// merge kernel joins (the borders follow from seq_lens alone).  Few keys in all: a cluster of
// CTAs per item, joined through distributed shared memory, no second launch.  Within a CTA
// one warp keeps TMA loads of keys in flight and brings each item's queries into the
// products' form, another loads values; four more (eight at head dim 64) take 32 keys of a
// unit each.  Two such CTAs per SM: one's products fill the time that the other takes to join
// its warps between items.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_attn_device.cuh"
#include "gdn_kv8.cuh"

namespace gdn {
namespace attn {

using namespace gdn::tc;

constexpr int K8_TILE = 32;              // keys of a warp's tile: two blocks
constexpr int K8_MAX_WARPS = 8;          // that consume; two more warps load
constexpr int K8_MAX_BARS = 8;
// Keys of a CTA of a cluster, at most (replayed, 16 + 4 heads of 256: 16 sequences of 2048 21 us in
// clusters, 25 as runs with a merge; one of 4096 13.9 and 14.1, where the two meet).  The block
// table's width decides, not the lengths, which the host does not know: a short sequence under a
// wide table is cut in runs (one of 700 keys under a table of 704 or 4096 places 9.9 us, of 8192 or
// 131,072 12.1; of 3000 keys 12.8 and 13.9; of 64 keys 9.4 both; 32 + 8 heads of 128, 700 keys 7.9 and 9.6).
constexpr int K8_FEW_KEYS = 512;
constexpr int K8_SCALES = 16;            // units whose scales are kept: the stages' and two batches
// What a unit and the ends of an item cost, as far as the cut goes: the ends as much as four units
// (200 rows of 8 heads of 128: 124 us with nothing for the ends, 116 with 3, 106 with 16, 111 with 36; of 4
// heads of 256: 137, 127, 114, 114).
constexpr int K8_UNIT_COST = 4, K8_ITEM_COST = 16;

// NT: query heads of an item in eights.
template <int D, int NT>
struct K8Cfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int KEYS = 16384 / D;                   // of a unit
  static constexpr int BLOCKS = KEYS / KV8_BLOCK;
  static constexpr int BATCH = 32 / BLOCKS;                // units that a loading warp looks up at a time
  static constexpr uint32_t TILE = KEYS * D;               // bytes of one of K, V
  static constexpr uint32_t STAGE = 2 * TILE;
  // O^T takes 4 NT registers per 16 channels.  Where a warp does not have them, the groups of
  // warps take every unit and a half of the channels each (the scores twice).
  static constexpr bool HALVES = NT * D > 256;
  static constexpr int GROUP = KEYS / K8_TILE;             // warps that share a unit
  static constexpr int WARPS = GROUP < 4 ? 4 : GROUP;
  static constexpr int GROUPS = HALVES ? 1 : WARPS / GROUP;   // that take the units in turn
  static constexpr int THREADS = 32 * (WARPS + 2);
  static constexpr int JOIN = HALVES ? GROUP : WARPS;      // warps that add up their O
  // Q's fragments of two items; joining the warps' O takes those of the item that is done and
  // as much again.
  static constexpr uint32_t QBUF = D / 16 * NT * 32 * 8;
  static_assert(2 * QBUF == ROWS * D * 4, "half of O's rows in Q's place");
  static constexpr uint32_t BOOK = 2048 + 12 * K8_SCALES * BLOCKS;   // K8Shared and the scales
  static constexpr uint32_t HEAD = (BOOK + 3 * QBUF + 1023) / 1024 * 1024;
  static constexpr int PER_SM = 2;
  static constexpr int CTAS = SMS * PER_SM;
  static constexpr int STAGES = (int)((233472u / PER_SM - 1024u - HEAD) / STAGE);
  // A wait by parity tells a phase from the next one only: each barrier is one group's.
  static constexpr int BARS = STAGES % GROUPS == 0 ? STAGES : STAGES * GROUPS;
  static constexpr uint32_t SMEM = HEAD + STAGES * STAGE;
  static_assert(STAGES >= 2 && BARS <= K8_MAX_BARS, "a unit in flight beside the one in use");
};

struct __align__(16) K8Shared {
  uint64_t full[K8_MAX_BARS], empty[K8_MAX_BARS];
  uint64_t q_full[2], q_empty[2];        // of every other item
  float q_scale[2][16];                  // of the item's heads
  float m[K8_MAX_WARPS][16], l[K8_MAX_WARPS][16];
  float2 ml[16];         // of the whole CTA, for its cluster
  int64_t sum[K8_MAX_WARPS + 2], found_first;
  int64_t walk[K8_MAX_WARPS + 2][5];     // each warp's K8Walk
  int32_t found;
};

struct K8Args {
  GdnKv8DecodeArgs a;
  int32_t rows;          // query heads per item, <= 8 NT
  int32_t subs;          // items per (sequence, key/value head)
  int32_t box_rows;      // rows per TMA box
  int32_t unit_shift;    // keys of a unit, log2
  int32_t ctas;          // CTAs that share the units
  int32_t cluster;       // CTAs per item (the form for few keys; 0: runs of units)
  int32_t merge_rows;    // rows of an item that a CTA of the merge joins
};

// Keys of a sequence by its entry of seq_lens (a block table row holds fewer than 2^31).
__device__ __forceinline__ int k8_clip(const K8Args& p, int len) {
  if (len > p.a.capacity) {
    set_status(p.a.d_status, GDN_DEV_BAD_LENGTH);
    len = (int)p.a.capacity;
  }
  return max(len, 0);
}
__device__ __forceinline__ int k8_len(const K8Args& p, int b) {
  return k8_clip(p, p.a.seq_lens[b]);
}
__device__ __forceinline__ int units_of(const K8Args& p, int keys) {
  return (int)(((int64_t)keys + (1 << p.unit_shift) - 1) >> p.unit_shift);
}

// An item's place on the line: nt units and its ends.
__device__ __forceinline__ int64_t span_of(int nt) {
  return nt > 0 ? (int64_t)nt * K8_UNIT_COST + K8_ITEM_COST : 0;
}
// Run c of the line is [start(c), start(c + 1)); a unit is in the run that its first point is
// in.  (No run is shorter than a unit.)
struct K8Line {
  int64_t length;
  int ctas;
  __device__ __forceinline__ K8Line(int64_t n, int most)
      : length(n), ctas(n < (int64_t)most * K8_UNIT_COST ? max((int)(n / K8_UNIT_COST), 1) : most) {}
  __device__ __forceinline__ int64_t start(int c) const { return length * c / ctas; }
  // The CTA whose run holds point u: the last whose run starts at or before it.
  __device__ __forceinline__ int owner(int64_t u) const {
    return (int)(((u + 1) * ctas - 1) / length);
  }
};

// First query head and number of query heads of item hs of a sequence.
template <int NT>
__device__ __forceinline__ int k8_head(const K8Args& p, int hs) {
  return hs / p.subs * (p.a.h_q / p.a.h_kv) + hs % p.subs * (8 * NT);
}
template <int NT>
__device__ __forceinline__ int k8_rows(const K8Args& p, int hs) {
  return min(p.rows, p.a.h_q / p.a.h_kv - hs % p.subs * (8 * NT));
}

// The gate of four channels of an output, and four channels of a finished one: y / l, gated
// (zeros where no key was seen).
template <typename IO>
__device__ __forceinline__ uint2 k8_gate(const GdnKv8DecodeArgs& a, int b, int h, int col) {
  if (!a.gate.data) return make_uint2(0, 0);
  return *reinterpret_cast<const uint2*>(reinterpret_cast<const IO*>(a.gate.data) +
                                         (int64_t)b * a.gate.token_stride +
                                         (int64_t)h * a.gate.head_stride + col);
}
template <typename IO, int D>
__device__ __forceinline__ void k8_put_four(const GdnKv8DecodeArgs& a, int b, int h, int col, float l,
                                            float (&y)[4], uint2 g) {
  const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] *= inv;
  if (a.gate.data && l != 0.f) {
    const float2 g0 = unpack2<IO>(g.x), g1 = unpack2<IO>(g.y);
    y[0] *= gate_sigmoid(g0.x);
    y[1] *= gate_sigmoid(g0.y);
    y[2] *= gate_sigmoid(g1.x);
    y[3] *= gate_sigmoid(g1.y);
  }
  *reinterpret_cast<uint2*>(reinterpret_cast<IO*>(a.o) + ((int64_t)b * a.h_q + h) * D + col) =
      make_uint2(pack2<IO>(y[0], y[1]), pack2<IO>(y[2], y[3]));
}

// The run [w, end) of the line, item by item.  (In shared memory, one for each warp: only
// looked at between items, when the accumulators leave no registers for it.)
struct K8Segment {
  int b, hs;             // sequence, and key/value head * subs + sub
  int keys;              // of the sequence
  int t0, t1;            // units of the item in this run
  int whole;             // all of the item is in this run
};
struct K8Walk {
  int64_t w, end, item_first;
  int nt, keys, b, hs;   // of the item to come
  // ahead: the entry of seq_lens of sequence b + 1, on its way while the items of b are worked on.
  __device__ bool next(const K8Args& p, int heads, K8Segment& s, int& ahead) {
    for (;;) {
      if (b >= p.a.n || item_first >= end) return false;
      const int64_t from = max(w - item_first, (int64_t)0);
      const int64_t to = (end - item_first + K8_UNIT_COST - 1) / K8_UNIT_COST;
      s.t0 = (int)min((from + K8_UNIT_COST - 1) / K8_UNIT_COST, (int64_t)nt);
      s.t1 = (int)min(to, (int64_t)nt);
      s.whole = s.t0 == 0 && s.t1 == nt;
      s.b = b;
      s.hs = hs;
      s.keys = keys;
      item_first += span_of(nt);
      if (++hs == heads) {
        hs = 0;
        ++b;
        keys = k8_clip(p, ahead);
        nt = units_of(p, keys);
        while (b < p.a.n && nt == 0) {
          if (++b < p.a.n) keys = k8_len(p, b);
          nt = units_of(p, keys);
        }
        if (b + 1 < p.a.n) ahead = p.a.seq_lens[b + 1];
      }
      if (s.t0 < s.t1) return true;
    }
  }
};

// Byte offset of a 16-byte chunk of a key's row in a tile: column blocks of up to 128
// bytes, each [key][bytes], swizzled as TMA leaves them (row: key % 8).
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int key, int row, int chunk) {
  if (D == 64) return (uint32_t)(key * 64 + ((chunk ^ (row >> 1)) << 4));
  return (uint32_t)((chunk >> 3) * (16384 / D) * 128 + key * 128 + (((chunk & 7) ^ row) << 4));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Bytes of asynchronous copies to come on `bar` (no arrival).
__device__ __forceinline__ void mbar_add_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}
template <int WARPS>
__device__ __forceinline__ void k8_consumers_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
}

template <typename IO, int D, int NT, bool FEW>
__global__ void __launch_bounds__(K8Cfg<D, NT>::THREADS, K8Cfg<D, NT>::PER_SM)
    kv8_decode_kernel(const __grid_constant__ K8Args p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  using C = K8Cfg<D, NT>;
  constexpr int CHUNKS = D / 16;
  constexpr float UP = WeightRange<__half>::SCALE_LOG2, LAG = WeightRange<__half>::LAG_LOG2;
  constexpr int W = C::WARPS, OWN = C::HALVES ? CHUNKS / 2 : CHUNKS;   // chunks of a warp's O
  extern __shared__ __align__(1024) unsigned char smem[];
  K8Shared* sh = reinterpret_cast<K8Shared*>(smem);
  // of the units' blocks: keys' scales, values' scales and their logarithms
  static_assert(sizeof(K8Shared) <= 2048, "shared bookkeeping");
  float* const sh_scale = reinterpret_cast<float*>(smem + 2048);
  constexpr int KIND = K8_SCALES * C::BLOCKS;
  // Q's fragments [chunk][nt][lane] of every other item; the third part: O's second half of rows
  const auto q_at = [&](int par) { return reinterpret_cast<uint2*>(smem + C::BOOK + par * C::QBUF); };
  const auto o_offset = [](int par, int row) {
    return (row < C::ROWS / 2 ? par * C::QBUF + row * D * 4
                              : 2 * C::QBUF + (row - C::ROWS / 2) * D * 4) + C::BOOK;
  };
  const GdnKv8DecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem) + C::HEAD;
  const int heads = a.h_kv * p.subs;
  const int n = a.n;

  if (tid == 0) {
    for (int s = 0; s < C::BARS; ++s) {
      mbar_init(&sh->full[s], 2);     // keys, values
      mbar_init(&sh->empty[s], C::HALVES ? W : C::GROUP);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->q_full[i], 1);
      mbar_init(&sh->q_empty[i], W);
    }
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch();   // (the merge reads seq_lens before it waits: what wrote them is done with here)
  K8Walk walk;
  int64_t w0, w1;
  if (FEW) {
    // ---- this CTA's share of its cluster's item ----
    const int item = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
    walk.b = item / heads;
    walk.hs = item % heads;
    walk.keys = k8_len(p, walk.b);
    walk.nt = units_of(p, walk.keys);
    walk.item_first = 0;
    w0 = (int64_t)walk.nt * rank / p.cluster * K8_UNIT_COST;
    w1 = (int64_t)walk.nt * (rank + 1) / p.cluster * K8_UNIT_COST;
    if (tid < 16) sh->ml[tid] = make_float2(-INFINITY, 0.f);
    __syncthreads();
  } else {
    // ---- this CTA's run of the line ----
    int64_t total = 0, span = 0, before = 0;
    for (int base = 0; base < n; base += C::THREADS) {
      const int b = base + tid;
      span = b < n ? span_of(units_of(p, k8_len(p, b))) * heads : 0;
      total += block_scan(span, sh->sum, W + 2, before);
    }
    const K8Line line(total, p.ctas);
    const int c = (int)blockIdx.x;
    w0 = total > 0 && c < line.ctas ? line.start(c) : 0;
    w1 = total > 0 && c < line.ctas ? line.start(c + 1) : 0;
    int64_t seen = 0;
    for (int base = 0; base < n && w0 < w1; base += C::THREADS) {
      const int b = base + tid;
      int64_t all = total;
      if (n > C::THREADS) {   // else the scan above has it all
        span = b < n ? span_of(units_of(p, k8_len(p, b))) * heads : 0;
        all = block_scan(span, sh->sum, W + 2, before);
      }
      if (w0 >= seen + before && w0 < seen + before + span) {
        sh->found = b;
        sh->found_first = seen + before;
      }
      seen += all;
    }
    __syncthreads();
  }

  if (w0 < w1) {
    walk.w = w0;
    walk.end = w1;
    if (!FEW) {
      walk.b = sh->found;
      walk.keys = k8_len(p, walk.b);
      walk.nt = units_of(p, walk.keys);
      walk.hs = (int)((w0 - sh->found_first) / span_of(walk.nt));
      walk.item_first = sh->found_first + walk.hs * span_of(walk.nt);
    }
    static_assert(sizeof(K8Walk) <= sizeof(sh->walk[0]), "room for a walk");
    K8Walk& at = *reinterpret_cast<K8Walk*>(sh->walk[warp]);
    if (lane == 0) at = walk;
    __syncwarp();
    // one lane walks, all of them read what it found
    int ahead = 0;
    if (lane == 0 && walk.b + 1 < n) ahead = a.seq_lens[walk.b + 1];
    auto next = [&](K8Segment& g) {
      int found = 0;
      if (lane == 0) found = at.next(p, heads, g, ahead);
      found = __shfl_sync(0xffffffffu, found, 0);
      g.b = __shfl_sync(0xffffffffu, g.b, 0);
      g.hs = __shfl_sync(0xffffffffu, g.hs, 0);
      g.keys = __shfl_sync(0xffffffffu, g.keys, 0);
      g.t0 = __shfl_sync(0xffffffffu, g.t0, 0);
      g.t1 = __shfl_sync(0xffffffffu, g.t1, 0);
      g.whole = __shfl_sync(0xffffffffu, g.whole, 0);
      return found != 0;
    };
    K8Segment g = {};
    bool ok = true;
    int j = 0, items = 0;            // units and items so far: the rings' positions
    if (warp >= W) {
      // ---- loads: one warp of K, with the items' queries, and one of V ----
      constexpr int COLS = D == 256 ? 2 : 1;
      const bool is_v = warp > W;
      const CUtensorMap* const map = is_v ? &vmap : &kmap;
      const int cb = lane % COLS, r = lane / COLS * p.box_rows;   // of this lane's box of a unit
      // Pages and scales are looked up for BATCH units at a time, a lane for each block: pages two
      // batches ahead, scales, by them, one; and the first ones of the item to come.  What a
      // lane can work out for its block is done there too: from unit to unit this warp is a chain
      // of dependent instructions, and with the rows' coordinates among them it was what
      // bounded the smaller heads (1150 cycles for four boxes).
      const int bu = lane / C::BLOCKS, brow = lane % C::BLOCKS * KV8_BLOCK;
      const float* const scales = is_v ? a.cache.v_scale : a.cache.k_scale;
      float* const scale_to = sh_scale + (is_v ? KIND : 0);
      auto page_at = [&](const K8Segment& g, int t) {
        t += bu;
        const int64_t pos = (int64_t)t * C::KEYS + brow;
        return t < g.t1 && pos < g.keys
                   ? __ldg(a.cache.block_table + (int64_t)g.b * a.cache.pages_per_seq +
                           (pos >> a.page_shift))
                   : 0;
      };
      // Row of the pool that a lane's block starts at (of page 0 where there is no such page).
      auto row_at = [&](const K8Segment& g, int t, int32_t page) {
        const int64_t pos = (int64_t)(t + bu) * C::KEYS + brow;
        if (page < 0 || page >= a.cache.num_pages) {
          set_status(a.d_status, GDN_DEV_BAD_PAGE);
          page = 0;
        }
        return (int)((((int64_t)page * a.h_kv + g.hs / p.subs) << a.page_shift) +
                     (pos & ((1 << a.page_shift) - 1)));
      };
      auto scale_at = [&](const K8Segment& g, int t, int row) {
        t += bu;
        return t < g.t1 && (int64_t)t * C::KEYS + brow < g.keys ? __ldg(scales + row / KV8_BLOCK) : 0.f;
      };
      // An item's queries: head lane / 4 of each eight, four channels of each chunk.
      uint2 q[NT][CHUNKS];
      auto load_q = [&](const K8Segment& g) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int head = nt * 8 + (lane >> 2);
          const IO* src = reinterpret_cast<const IO*>(a.q.data) + (int64_t)g.b * a.q.token_stride +
                          (int64_t)(k8_head<NT>(p, g.hs) + head) * a.q.head_stride + (lane & 3) * 4;
#pragma unroll
          for (int ch = 0; ch < CHUNKS; ++ch)
            q[nt][ch] = head < k8_rows<NT>(p, g.hs) ? __ldg(reinterpret_cast<const uint2*>(src + ch * 16))
                                                    : make_uint2(0, 0);
        }
      };
      auto put_q = [&](int par) {   // each row times a power of two that brings its largest element to [1, 2)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float top = 0.f;
#pragma unroll
          for (int ch = 0; ch < CHUNKS; ++ch) {
            const float2 x = unpack2<IO>(q[nt][ch].x), y = unpack2<IO>(q[nt][ch].y);
            top = max3(max3(top, fabsf(x.x), fabsf(x.y)), fabsf(y.x), fabsf(y.y));
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // (an Inf, and a row of zeros or of subnormals, as it is)
          const int ex = (int)(__float_as_uint(top) >> 23);
          const int up = ex == 0 || ex == 255 ? 0 : max(-126, min(126, 127 - ex));
          const float f = pow2(up);
#pragma unroll
          for (int ch = 0; ch < CHUNKS; ++ch) {
            const float2 x = unpack2<IO>(q[nt][ch].x), y = unpack2<IO>(q[nt][ch].y);
            q_at(par)[(ch * NT + nt) * 32 + lane] =
                make_uint2(pack2<__half>(x.x * f, x.y * f), pack2<__half>(y.x * f, y.y * f));
          }
          if ((lane & 3) == 0) sh->q_scale[par][nt * 8 + (lane >> 2)] = a.scale_log2 * pow2(-up);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->q_full[par]);
      };
      // Unit u of a batch, whose blocks start at the lanes' rows, into stage j % STAGES; the
      // arrival, which says that its scales are there, apart.
      auto load_unit = [&](const K8Segment& g, int t, int u, int row) {
        uint64_t* full = &sh->full[j % C::BARS];
        const int left = min(g.keys - t * C::KEYS, C::KEYS);
        const uint32_t dst = ring + (uint32_t)(j % C::STAGES) * C::STAGE + (is_v ? C::TILE : 0u);
        // (the test's: of the first CTA, or of the last one of the first cluster)
        const bool withheld = a.withhold && j == 0 && !is_v && blockIdx.x == (FEW ? p.cluster - 1 : 0);
        const int there = (left + p.box_rows - 1) / p.box_rows * p.box_rows;
        const int from = __shfl_sync(0xffffffffu, row, (u * C::BLOCKS + r / KV8_BLOCK) & 31);
        if (lane == 0 && !withheld) mbar_add_tx(full, (uint32_t)there * D);
        __syncwarp();
        if (r < there && !withheld)
          tma_box(dst + (uint32_t)(cb * C::KEYS + r) * (D < 128 ? 64u : 128u), map, from, cb, full);
        __syncwarp();
        return !withheld;
      };
      auto put_scales = [&](int at_unit, float scale) {
        const int place = (at_unit + bu) % K8_SCALES * C::BLOCKS + lane % C::BLOCKS;
        scale_to[place] = scale;
        if (is_v) scale_to[KIND + place] = __log2f(scale);
        __syncwarp();
      };
      K8Segment h = {};
      bool more = next(h);
      int32_t page_h = more ? page_at(h, h.t0) : 0;
      if (more && !is_v) load_q(h);
      int row_h = more ? row_at(h, h.t0, page_h) : 0;
      float scale_h = more ? scale_at(h, h.t0, row_h) : 0.f;
      for (; ok && more; ++items) {
        g = h;
        int row = row_h;
        int32_t page1 = page_at(g, g.t0 + C::BATCH);
        float scale = scale_h;
        // The first item's first units are on their way before its scales and queries are there.
        int early = 0;
        if (items == 0) {
          bool all = true;
          for (; early < min(C::STAGES, C::BATCH) && g.t0 + early < g.t1; ++early, ++j)
            all &= load_unit(g, g.t0 + early, early, row);
          j = 0;
          put_scales(0, scale);
          if (lane == 0)
            for (int u = all ? 0 : 1; u < early; ++u) mbar_arrive(&sh->full[u]);
          __syncwarp();
        }
        more = next(h);
        if (more) page_h = page_at(h, h.t0);
        if (!is_v) {
          // the queries, once the item before the last is done with their place
          const int par = items & 1;
          if (items > 1) ok = mbar_wait(&sh->q_empty[par], (items / 2 - 1) & 1, a.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          put_q(par);
          if (more) load_q(h);
        }
        if (more) {
          row_h = row_at(h, h.t0, page_h);
          scale_h = scale_at(h, h.t0, row_h);
        }
        for (int tb = g.t0; tb < g.t1 && ok; tb += C::BATCH) {
          const int row1 = row_at(g, tb + C::BATCH, page1);
          const float scale1 = scale_at(g, tb + C::BATCH, row1);
          page1 = page_at(g, tb + 2 * C::BATCH);
          // (their places were those of the batch before the last: no stage holds one of its units)
          if (early == 0) put_scales(j, scale);
          j += early;
          for (int u = early; u < C::BATCH && tb + u < g.t1; ++u, ++j) {
            if (j >= C::STAGES) {
              const int was = j - C::STAGES;
              ok = mbar_wait(&sh->empty[was % C::BARS], (was / C::BARS) & 1, a.wait_ns);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            load_unit(g, tb + u, u, row);
            if (lane == 0) mbar_arrive(&sh->full[j % C::BARS]);
            __syncwarp();
          }
          early = 0;
          row = row1;
          scale = scale1;
        }
      }
      // (the consumers wait for these too, unless they have given up)
      for (int x = max(0, j - C::STAGES); x < j; ++x)
        mbar_wait(&sh->full[x % C::BARS], (x / C::BARS) & 1, GRACE_NS);
    } else {
      // ---- 32 keys of every unit of this warp's group, with its own reference, sum and O ----
      const int group = warp / C::GROUP, part = warp % C::GROUP;
      const int ch0 = C::HALVES ? group * OWN : 0;
      const int row8 = lane >> 2, col = (lane & 3) * 2;   // key or channel pair; heads col, col + 1
      const int mi = lane >> 3, mr = lane & 7;            // this lane's row of an ldmatrix
      const int k_key = part * K8_TILE + (mi & 1) * 8 + mr, v_key = part * K8_TILE + mi * 8 + mr;
      while (next(g)) {
        const int h0 = k8_head<NT>(p, g.hs), rows = k8_rows<NT>(p, g.hs);
        const int par = items & 1;
        if (ok) ok = mbar_wait(&sh->q_full[par], (items / 2) & 1, a.wait_ns);
        __syncwarp();
        ++items;
        const uint2* const q = q_at(par) + lane;
        float cs[NT][2];                                  // scale of heads col, col + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) cs[nt][e] = sh->q_scale[par][nt * 8 + col + e];
        float o[OWN][NT][4];
#pragma unroll
        for (int ch = 0; ch < OWN; ++ch)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            o[ch][nt][0] = o[ch][nt][1] = o[ch][nt][2] = o[ch][nt][3] = 0.f;
        // of heads col, col + 1: references of the sum and of the contributions, sum, and what
        // a weight is scaled by for the product, 2^(M - M' + UP)
        float m[NT][2], mv[NT][2], l[NT][2], pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            m[nt][e] = mv[nt][e] = -INFINITY;
            l[nt][e] = pf[nt][e] = 0.f;
          }

        for (int t = g.t0; t < g.t1; ++t, ++j) {
          if (C::GROUPS > 1 && j % C::GROUPS != group) continue;
          const int s = j % C::STAGES;
          if (ok) ok = mbar_wait(&sh->full[j % C::BARS], (j / C::BARS) & 1, a.wait_ns);
          __syncwarp();
          const int left = min(C::KEYS, g.keys - t * C::KEYS) - part * K8_TILE;
          const uint32_t kt = ring + (uint32_t)s * C::STAGE, vt = kt + C::TILE;
          if (left > 0) {
            float x[2][NT][4];   // [block][eight][key row8: 2 heads, row8 + 8: 2 heads]
            {
              float sc[2][2][NT][4] = {};   // [block][sums of even and odd chunks]
#pragma unroll
              for (int ch = 0; ch < CHUNKS; ch += 2) {
                uint32_t w[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  ldsm4(kt + chunk_at<D>(k_key + i * KV8_BLOCK, mr, ch + (mi >> 1)), w[i]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint2 qf[NT];
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) qf[nt] = q[((ch + h) * NT + nt) * 32];
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    uint32_t ka[4];
                    e4m3x4_to_f16(w[i][2 * h], ka[0], ka[2]);
                    e4m3x4_to_f16(w[i][2 * h + 1], ka[1], ka[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                      mma16816<__half>(sc[i][h][nt], ka, qf[nt].x, qf[nt].y);
                  }
                }
              }
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 4; ++e) x[i][nt][e] = sc[i][0][nt][e] + sc[i][1][nt][e];
            }
            if (left < K8_TILE) {
              // Values past the end may be anything, and 0 x NaN is not 0: cleared.
              constexpr int ROW = D / 16;
              for (int i = lane; i < (K8_TILE - left) * ROW; i += 32) {
                const int key = part * K8_TILE + left + i / ROW;
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 vt + chunk_at<D>(key, key & 7, i % ROW)),
                             "r"(0)
                             : "memory");
              }
              __syncwarp();
            }
            // Scores in log2 units.
            const float* const sc_at = sh_scale + j % K8_SCALES * C::BLOCKS + 2 * part;
            const float2 ks = *reinterpret_cast<const float2*>(sc_at);
            const float2 vs = *reinterpret_cast<const float2*>(sc_at + KIND);
            const float2 lv = *reinterpret_cast<const float2*>(sc_at + 2 * KIND);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                x[0][nt][e] *= cs[nt][e & 1] * ks.x;
                x[1][nt][e] *= cs[nt][e & 1] * ks.y;
              }
            if (left < K8_TILE) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (i * KV8_BLOCK + row8 + (e >> 1) * 8 >= left) x[i][nt][e] = -INFINITY;
            }
            bool far = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float y0 = fmaxf(x[0][nt][e], x[0][nt][2 + e]);
                const float y1 = fmaxf(x[1][nt][e], x[1][nt][2 + e]);
                far |= fmaxf(y0, y1) > m[nt][e] + LAG;
                far |= fmaxf(y0 + lv.x, y1 + lv.y) > mv[nt][e] + LAG;
              }
            // A head's references follow from the head alone.
            if (__any_sync(0xffffffffu, far)) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float y0 = fmaxf(x[0][nt][e], x[0][nt][2 + e]);
                  const float y1 = fmaxf(x[1][nt][e], x[1][nt][2 + e]);
                  float top = fmaxf(y0, y1), topv = fmaxf(y0 + lv.x, y1 + lv.y);
#pragma unroll
                  for (int o = 4; o < 32; o <<= 1) {
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, o));
                  }
                  f[e] = 1.f;
                  if (top > m[nt][e] + LAG) {
                    l[nt][e] *= ex2(m[nt][e] - top);
                    m[nt][e] = top;
                  }
                  if (topv > mv[nt][e] + LAG) {
                    f[e] = ex2(mv[nt][e] - topv);
                    mv[nt][e] = topv;
                  }
                  // (a weight of 0 until there is a contribution.  M - M' is 44 at most where the
                  // largest weights' scales are not 0; else 80 of it are kept, and what is less
                  // than 2^-76 of the largest weight comes out smaller or as 0.)
                  pf[nt][e] = mv[nt][e] == -INFINITY ? 0.f : ex2(fminf(m[nt][e] - mv[nt][e], 80.f) + UP);
                }
#pragma unroll
                for (int ch = 0; ch < OWN; ++ch) {
                  o[ch][nt][0] *= f[0];
                  o[ch][nt][1] *= f[1];
                  o[ch][nt][2] *= f[0];
                  o[ch][nt][3] *= f[1];
                }
              }
            }
            if (a.weights) {   // the scores, for the weights' sums
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const int head = nt * 8 + col + (e & 1);
                    const int key = i * KV8_BLOCK + row8 + (e >> 1) * 8;
                    if (head < rows && key < left)
                      a.scores[((int64_t)g.b * a.h_q + h0 + head) * a.capacity + t * C::KEYS +
                               part * K8_TILE + key] = x[i][nt][e];
                  }
            }
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float f = pf[nt][e] * (i ? vs.y : vs.x);
#pragma unroll
                  for (int r = 0; r < 2; ++r) {
                    // (no fma with the scale: the reference is such a rounded product)
                    const float w = ex2(x[i][nt][2 * r + e] - m[nt][e]);
                    l[nt][e] += w;
                    y[2 * r + e] = w * f;
                  }
                }
                pb[i][nt][0] = transpose_8x8(pack2<__half>(y[0], y[1]));
                pb[i][nt][1] = transpose_8x8(pack2<__half>(y[2], y[3]));
              }
#pragma unroll
            for (int ch = 0; ch < OWN; ++ch) {
              uint32_t w[4];
              ldsm4t(vt + chunk_at<D>(v_key, mr, ch0 + ch), w);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t va[4];   // channels 2 row8 (even rows) and 2 row8 + 1 of the chunk
                e4m3x4_to_f16(__byte_perm(w[2 * i], 0, 0x3120), va[0], va[1]);
                e4m3x4_to_f16(__byte_perm(w[2 * i + 1], 0, 0x3120), va[2], va[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16816<__half>(o[ch][nt], va, pb[i][nt][0], pb[i][nt][1]);
              }
            }
            // the cleared rows are written by a copy next
            if (left < K8_TILE) fence_async_smem();
          }
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&sh->empty[j % C::BARS]);
        }

        // the gate of this thread's part of the output, on its way while the warps join
        constexpr int OUT = (C::ROWS * (D / 4) + 32 * W - 1) / (32 * W);
        uint2 gate[OUT] = {};
        const bool direct = !FEW && g.whole;
        if (direct)
#pragma unroll
          for (int k = 0; k < OUT; ++k) {
            const int i = tid + k * 32 * W, row = i / (D / 4);
            if (row < rows)
              gate[k] = k8_gate<IO>(a, g.b, h0 + row, i % (D / 4) * 4);
          }
        // ---- join the warps ----
        const bool all_ok = __all_sync(0xffffffffu, ok);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
            if (!all_ok) l[nt][e] = NAN;
            if (row8 == 0) {
              sh->m[warp][nt * 8 + col + e] = m[nt][e];
              sh->l[warp][nt * 8 + col + e] = l[nt][e];
            }
          }
        k8_consumers_bar<W>();
        float f[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < C::JOIN; ++w) mm = fmaxf(mm, sh->m[w][nt * 8 + col + e]);
            f[nt][e] = mv[nt][e] == -INFINITY ? 0.f : ex2(mv[nt][e] - UP - mm);
          }
        // The warps add up in one slab, a share of the channels at a time, each at another
        // one: every sum has a fixed order.
#pragma unroll
        for (int st = 0; st < C::JOIN; ++st) {
          const int share = (warp + st) % C::JOIN;
#pragma unroll
          for (int ch = 0; ch < OWN; ++ch) {
            if (ch % C::JOIN != share) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + col + e;
                if (row >= rows) continue;
                float2* dst = reinterpret_cast<float2*>(smem + o_offset(par, row)) + (ch0 + ch) * 8 + row8;
                float2 v = make_float2(o[ch][nt][e] * f[nt][e], o[ch][nt][2 + e] * f[nt][e]);
                if (st > 0) {
                  const float2 w = *dst;
                  v.x += w.x;
                  v.y += w.y;
                }
                *dst = v;
              }
          }
          k8_consumers_bar<W>();
        }
        // ---- out: the output itself, or a partial result ----
        const int64_t slot = (2 * (int64_t)blockIdx.x + (g.t0 > 0 ? 0 : 1)) * p.rows;
#pragma unroll
        for (int k = 0; k < OUT; ++k) {
          const int i = tid + k * 32 * W, row = i / (D / 4), c4 = i % (D / 4) * 4;
          if (row >= rows) break;
          float mm = -INFINITY, ll = 0.f;
#pragma unroll
          for (int w = 0; w < C::JOIN; ++w) mm = fmaxf(mm, sh->m[w][row]);
#pragma unroll
          for (int w = 0; w < C::JOIN; ++w)
            ll += mm == -INFINITY ? sh->l[w][row]
                                  : sh->l[w][row] * ex2(sh->m[w][row] - mm);
          const float4 v = reinterpret_cast<const float4*>(smem + o_offset(par, row))[c4 / 4];
          if (FEW) {
            if (c4 == 0) sh->ml[row] = make_float2(mm, ll);
          } else if (direct) {
            float y[4] = {v.x, v.y, v.z, v.w};
            k8_put_four<IO, D>(a, g.b, h0 + row, c4, ll, y, gate[k]);
            if (a.weights && c4 == 0) a.row_ml[(int64_t)g.b * a.h_q + h0 + row] = make_float2(mm, ll);
          } else {
            *reinterpret_cast<float4*>(a.part_o + (slot + row) * D + c4) = v;
            if (c4 == 0) a.part_ml[slot + row] = make_float2(mm, ll);
          }
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&sh->q_empty[par]);   // (O had Q's place)
        k8_consumers_bar<W>();   // m, l and the rest of O's place are free again
      }
    }
    if (!ok) set_status(a.d_status, GDN_DEV_WAIT_TIMEOUT);
  }
  if (FEW) {
    // ---- the cluster's partials joined, a share of the channels by each CTA ----
    __syncwarp();
    cluster_barrier();
    const int rank = blockIdx.x % p.cluster;
    const int rows = k8_rows<NT>(p, walk.hs), h0 = k8_head<NT>(p, walk.hs);
    const uint32_t ml_at = smem_u32(sh->ml), o_at = smem_u32(smem);   // (an item at most: the first)
    for (int x = rank * C::THREADS + tid; x < rows * (D / 4); x += p.cluster * C::THREADS) {
      const int row = x / (D / 4), c4 = x % (D / 4) * 4;
      float mm = -INFINITY, ll = 0.f;
      for (int r = 0; r < p.cluster; ++r)
        mm = fmaxf(mm, ld_peer_8(peer_addr(ml_at + 8u * row, r)).x);
      float y[4] = {};
      for (int r = 0; r < p.cluster; ++r) {
        const float2 v = ld_peer_8(peer_addr(ml_at + 8u * row, r));
        if (v.y == 0.f) continue;   // saw no key
        const float f = ex2(v.x - mm);
        const float4 o = ld_peer_16(peer_addr(o_at + o_offset(0, row) + (uint32_t)c4 * 4u, r));
        ll += f * v.y;
        y[0] = fmaf(f, o.x, y[0]);
        y[1] = fmaf(f, o.y, y[1]);
        y[2] = fmaf(f, o.z, y[2]);
        y[3] = fmaf(f, o.w, y[3]);
      }
      k8_put_four<IO, D>(a, walk.b, h0 + row, c4, ll, y, k8_gate<IO>(a, walk.b, h0 + row, c4));
      if (a.weights && c4 == 0)
        a.row_ml[(int64_t)walk.b * a.h_q + h0 + row] = make_float2(mm, ll);
    }
    cluster_barrier();   // the others may still read this CTA's
  }
}

// ---- merge ------------------------------------------------------------------------

// Joins the partial results of one item:
//   M = max m_i,  o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// Few items: a CTA per item and a few of its rows.  Many: a CTA per border of two runs, at work
// where it is the first inside an item (most items are whole then, and a CTA for each of 3200
// cost 10 us more).  All that does not need the partials is done before they are waited for.
constexpr int K8_MERGE_THREADS = 256, K8_MERGE_WARPS = K8_MERGE_THREADS / 32;
constexpr int K8_MERGE_SMEM = 64 * 1024;   // one head of 16 rows, all runs in one item: 40 KB

// Partials of one item, at most: with equal runs every head of a sequence has as
// many units, so an item is at most 1 / heads of the line, and its ends cut two runs.
static __host__ __device__ __forceinline__ int k8_most_parts(const K8Args& p) {
  return p.ctas / (p.a.h_kv * p.subs) + 2;
}

// By item, a few rows of it per CTA.
template <typename IO, int D, int NT>
__global__ void __launch_bounds__(K8_MERGE_THREADS)
    kv8_merge_kernel(const __grid_constant__ K8Args p) {
  extern __shared__ __align__(16) unsigned char merge_smem[];
  __shared__ int64_t sums[K8_MERGE_THREADS / 32], s_mine;
  __shared__ float sum_l[16];
  __shared__ float4 shares[K8_MERGE_THREADS];
  const GdnKv8DecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int heads = a.h_kv * p.subs;
  const int n = a.n;
  float2* ml = reinterpret_cast<float2*>(merge_smem);   // [part][row]: statistics, then (factor, sum)
  int32_t* first_row = reinterpret_cast<int32_t*>(ml + (size_t)k8_most_parts(p) * p.merge_rows);
  const int slices = (p.rows + p.merge_rows - 1) / p.merge_rows;
  const int item = blockIdx.x / slices, r0 = blockIdx.x % slices * p.merge_rows;
  const int b = item / heads, hs = item % heads;
  const int h0 = k8_head<NT>(p, hs) + r0;
  const int rows = min(p.merge_rows, k8_rows<NT>(p, hs) - r0);
  int64_t total = 0;
  for (int base = 0; base < n; base += K8_MERGE_THREADS) {
    const int i = base + tid;
    int64_t before;
    const int64_t u = i < n ? span_of(units_of(p, k8_len(p, i))) * heads : 0;
    const int64_t all = block_scan(u, sums, K8_MERGE_THREADS / 32, before);
    if (i == b) s_mine = total + before;
    total += all;
  }
  __syncthreads();
  const int nt = units_of(p, k8_len(p, b));
  const int64_t u0 = s_mine + hs * span_of(nt);
  const K8Line line(total, p.ctas);
  int c0 = 0, c1 = -1;
  if (nt > 0) {   // the CTAs whose runs hold its first and last unit
    c0 = line.owner(u0);
    c1 = line.owner(u0 + (int64_t)(nt - 1) * K8_UNIT_COST);
  }
  const int parts = c1 - c0 + 1;
  // partial i's first row: a run that starts inside the item left its first partial, else its last
  for (int i = tid; i < parts; i += K8_MERGE_THREADS)
    first_row[i] = (2 * (c0 + i) + (line.start(c0 + i) > u0 ? 0 : 1)) * p.rows + r0;
  pdl_wait();
  if (nt > 0 && c0 == c1) return;   // written already
  if (rows <= 0) return;            // the last heads' item may be shorter
  __syncthreads();
  for (int i = tid; i < parts * rows; i += K8_MERGE_THREADS)
    ml[i] = a.part_ml[first_row[i / rows] + i % rows];
  __syncthreads();
  for (int row = warp; row < rows; row += K8_MERGE_THREADS / 32) {
    float mm = -INFINITY, ll = 0.f;
    for (int i = lane; i < parts; i += 32) mm = fmaxf(mm, ml[i * rows + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    for (int i = lane; i < parts; i += 32) {
      const float2 v = ml[i * rows + row];
      const float f = v.y == 0.f ? 0.f : ex2(v.x - mm);
      ll += v.y == 0.f ? 0.f : f * v.y;
      ml[i * rows + row].x = f;
    }
    ll = warp_sum(ll);
    if (lane == 0) {
      sum_l[row] = ll;
      if (a.weights) a.row_ml[(int64_t)b * a.h_q + h0 + row] = make_float2(mm, ll);
    }
  }
  __syncthreads();
  // The threads that the rows leave over share the partials: group g takes every
  // groups-th one, and the groups' sums are added in their order.
  const int units = rows * (D / 4), groups = max(1, K8_MERGE_THREADS / units);
  for (int x0 = 0; x0 < units; x0 += K8_MERGE_THREADS) {
    const int g = groups > 1 ? tid / units : 0, x = groups > 1 ? tid - g * units : x0 + tid;
    const int row = x / (D / 4), col = x % (D / 4) * 4;
    float y[4] = {};
    const bool mine = x < units && g < groups;
    if (mine) {
#pragma unroll 8
      for (int i = g; i < parts; i += groups) {
        const float2 w = ml[i * rows + row];
        const float4 v =
            *reinterpret_cast<const float4*>(a.part_o + (int64_t)(first_row[i] + row) * D + col);
        if (w.y != 0.f) {
          y[0] = fmaf(w.x, v.x, y[0]);
          y[1] = fmaf(w.x, v.y, y[1]);
          y[2] = fmaf(w.x, v.z, y[2]);
          y[3] = fmaf(w.x, v.w, y[3]);
        }
      }
    }
    if (groups > 1) {
      if (mine) shares[tid] = make_float4(y[0], y[1], y[2], y[3]);
      __syncthreads();
      for (int i = 1; i < groups && g == 0; ++i) {
        const float4 v = shares[i * units + x];
        y[0] += v.x;
        y[1] += v.y;
        y[2] += v.z;
        y[3] += v.w;
      }
    }
    if (mine && g == 0)
      k8_put_four<IO, D>(a, b, h0 + row, col, sum_l[row], y, k8_gate<IO>(a, b, h0 + row, col));
  }
}

// By border: CTA c has the border of runs c and c + 1.
template <typename IO, int D, int NT>
__global__ void __launch_bounds__(K8_MERGE_THREADS)
    kv8_merge_border_kernel(const __grid_constant__ K8Args p) {
  extern __shared__ __align__(16) unsigned char merge_smem[];
  __shared__ int64_t sums[K8_MERGE_WARPS], s_first;
  __shared__ int s_b;
  __shared__ float sum_l[16];
  __shared__ float4 shares[K8_MERGE_THREADS];
  const GdnKv8DecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int heads = a.h_kv * p.subs;
  const int n = a.n;
  float2* ml = reinterpret_cast<float2*>(merge_smem);   // [part][row]: statistics, then (factor, sum)
  int32_t* first_row = reinterpret_cast<int32_t*>(ml + (size_t)k8_most_parts(p) * p.rows);
  int64_t total = 0;
  for (int base = 0; base < n; base += K8_MERGE_THREADS) {
    const int i = base + tid;
    const int64_t u = i < n ? span_of(units_of(p, k8_len(p, i))) * heads : 0;
    int64_t before;
    const int64_t all = block_scan(u, sums, K8_MERGE_WARPS, before);
    total += all;
  }
  const K8Line line(total, p.ctas);
  int b, hs, nt = 0, c0 = 0, c1 = -1;
  int64_t u0 = 0;
  bool mine = true;
  const int c = blockIdx.x + 1;
  mine = total > 0 && c < line.ctas;
  const int64_t w = mine ? line.start(c) : -1;
  int64_t seen = 0;
  for (int base = 0; base < n && mine; base += K8_MERGE_THREADS) {
    const int i = base + tid;
    const int64_t u = i < n ? span_of(units_of(p, k8_len(p, i))) * heads : 0;
    int64_t before;
    const int64_t all = block_scan(u, sums, K8_MERGE_WARPS, before);
    if (w >= seen + before && w < seen + before + u) {
      s_b = i;
      s_first = seen + before;
    }
    seen += all;
  }
  __syncthreads();
  b = hs = 0;
  if (mine) {
    b = s_b;
    nt = units_of(p, k8_len(p, b));
    hs = (int)((w - s_first) / span_of(nt));
    u0 = s_first + hs * span_of(nt);
    c0 = line.owner(u0);
    c1 = line.owner(u0 + (int64_t)(nt - 1) * K8_UNIT_COST);
    mine = c0 == c - 1 && c1 > c0;
  }
  // rows that see no key
  for (int i = blockIdx.x; i < n; i += gridDim.x)
    if (k8_len(p, i) == 0)
      for (int x = tid; x < a.h_q * D / 8; x += K8_MERGE_THREADS)
        reinterpret_cast<uint4*>(a.o)[(int64_t)i * (a.h_q * D / 8) + x] = make_uint4(0, 0, 0, 0);
  const int h0 = k8_head<NT>(p, hs), rows = k8_rows<NT>(p, hs);
  const int parts = c1 - c0 + 1;
  // The threads that the rows leave over share the partials: group g takes every groups-th one, and
  // the groups' sums are added in their order.
  const int units = rows * (D / 4), groups = max(1, K8_MERGE_THREADS / units);
  const int g = groups > 1 ? tid / units : 0;
  uint2 gate = {};
  if (mine) {
    // partial i's first row: a run that starts inside the item left its first partial, else its last
    for (int i = tid; i < parts; i += K8_MERGE_THREADS)
      first_row[i] = (2 * (c0 + i) + (line.start(c0 + i) > u0 ? 0 : 1)) * p.rows;
    if (tid < units) gate = k8_gate<IO>(a, b, h0 + tid / (D / 4), tid % (D / 4) * 4);
    __syncthreads();
  }
  pdl_wait();
  if (!mine) return;
  for (int i = tid; i < parts * rows; i += K8_MERGE_THREADS)
    ml[i] = a.part_ml[first_row[i / rows] + i % rows];
  for (int x0 = 0; x0 < units; x0 += K8_MERGE_THREADS) {
    const int x = groups > 1 ? tid - g * units : x0 + tid;
    const int row = x / (D / 4), col = x % (D / 4) * 4;
    const bool here = x < units && g < groups;
    auto partial = [&](int i) {
      return *reinterpret_cast<const float4*>(a.part_o + (int64_t)(first_row[i] + row) * D + col);
    };
    if (x0 == 0) {
      __syncthreads();
      for (int r = warp; r < rows; r += K8_MERGE_WARPS) {
        float mm = -INFINITY, ll = 0.f;
        for (int i = lane; i < parts; i += 32) mm = fmaxf(mm, ml[i * rows + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        for (int i = lane; i < parts; i += 32) {
          const float2 v = ml[i * rows + r];
          const float f = v.y == 0.f ? 0.f : ex2(v.x - mm);
          ll += v.y == 0.f ? 0.f : f * v.y;
          ml[i * rows + r].x = f;
        }
        ll = warp_sum(ll);
        if (lane == 0) {
          sum_l[r] = ll;
          if (a.weights) a.row_ml[(int64_t)b * a.h_q + h0 + r] = make_float2(mm, ll);
        }
      }
      __syncthreads();
    }
    float y[4] = {};
    if (here) {
      // (a partial that saw no key is zeros, its factor too)
#pragma unroll 16
      for (int i = g; i < parts; i += groups) {
        const float4 v = partial(i);
        const float f = ml[i * rows + row].x;
        y[0] = fmaf(f, v.x, y[0]);
        y[1] = fmaf(f, v.y, y[1]);
        y[2] = fmaf(f, v.z, y[2]);
        y[3] = fmaf(f, v.w, y[3]);
      }
    }
    if (groups > 1) {
      if (here) shares[tid] = make_float4(y[0], y[1], y[2], y[3]);
      __syncthreads();
      for (int i = 1; i < groups && g == 0; ++i) {
        const float4 v = shares[i * units + x];
        y[0] += v.x;
        y[1] += v.y;
        y[2] += v.z;
        y[3] += v.w;
      }
    }
    if (here && g == 0)
      k8_put_four<IO, D>(a, b, h0 + row, col, sum_l[row], y,
                         x0 == 0 ? gate : k8_gate<IO>(a, b, h0 + row, col));
  }
}

// ---- what the cached tokens received -----------------------------------------------

// weights[b][j][p] += sum over head j's query heads of 2^(s_p - M) / l.
constexpr int RECEIVED_THREADS = 256, RECEIVED_KEYS = 4 * RECEIVED_THREADS;

__global__ void __launch_bounds__(RECEIVED_THREADS)
    kv8_received_kernel(const __grid_constant__ GdnKv8DecodeArgs a, int across) {
  pdl_wait();
  const int group = a.h_q / a.h_kv;
  const int item = blockIdx.x / across, b = item / a.h_kv, j = item % a.h_kv;
  int64_t len = a.seq_lens[b];
  len = min(len, a.capacity);
  const float2* ml = a.row_ml + (int64_t)b * a.h_q + j * group;
  const float* s = a.scores + ((int64_t)b * a.h_q + j * group) * a.capacity;
  float* w = a.weights + ((int64_t)b * a.h_kv + j) * a.capacity;
  for (int64_t p0 = (int64_t)(blockIdx.x % across) * RECEIVED_KEYS; p0 < len;
       p0 += (int64_t)across * RECEIVED_KEYS) {
    const int64_t p = p0 + threadIdx.x * 4;      // capacity is a multiple of 16
    if (p >= len) continue;
    float y[4] = {};
    for (int h = 0; h < group; ++h) {
      const float2 v = __ldg(ml + h);
      const float4 x = *reinterpret_cast<const float4*>(s + h * a.capacity + p);
      const float inv = 1.0f / v.y;
      y[0] = fmaf(ex2(x.x - v.x), inv, y[0]);
      y[1] = fmaf(ex2(x.y - v.x), inv, y[1]);
      y[2] = fmaf(ex2(x.z - v.x), inv, y[2]);
      y[3] = fmaf(ex2(x.w - v.x), inv, y[3]);
    }
    if (p + 4 <= len) {
      float4* at = reinterpret_cast<float4*>(w + p);
      const float4 old = *at;
      *at = make_float4(old.x + y[0], old.y + y[1], old.z + y[2], old.w + y[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (p + e < len) w[p + e] += y[e];
    }
  }
}

// ---- host ------------------------------------------------------------------------

template <typename IO, int D, int NT>
static cudaError_t launch_decode(const GdnKv8DecodeArgs& a, cudaStream_t s) {
  using C = K8Cfg<D, NT>;
  cudaError_t e = cudaSuccess;
  K8Args p;
  p.a = a;
  const int group = a.h_q / a.h_kv;
  p.rows = group < C::ROWS ? group : C::ROWS;
  p.subs = (group + C::ROWS - 1) / C::ROWS;
  p.ctas = C::CTAS;
  const int page = 1 << a.page_shift;
  p.box_rows = page < C::KEYS ? page : C::KEYS;
  p.unit_shift = C::KEYS == 64 ? 6 : C::KEYS == 128 ? 7 : 8;
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(gdn_tensor_map_encoder());
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap kmap, vmap;
  constexpr int WIDE = D < 128 ? 64 : 128;
  for (int i = 0; i < 2; ++i) {   // cache rows: (channel, row of the pool, column block)
    const cuuint64_t dims[3] = {WIDE, (cuuint64_t)a.cache.num_pages * a.h_kv << a.page_shift,
                                D / WIDE};
    const cuuint64_t strides[2] = {D, WIDE};
    const cuuint32_t box[3] = {WIDE, (cuuint32_t)p.box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (enc(i ? &vmap : &kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, i ? a.cache.v : a.cache.k, dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            WIDE == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kernel = kv8_decode_kernel<IO, D, NT, false>;
  auto few = kv8_decode_kernel<IO, D, NT, true>;
  auto merge = kv8_merge_kernel<IO, D, NT>;
  auto border = kv8_merge_border_kernel<IO, D, NT>;
  static int opted_in[64] = {};
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !opted_in[dev]) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)C::SMEM)) != cudaSuccess)
      return e;
    if ((e = cudaFuncSetAttribute(few, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)C::SMEM)) != cudaSuccess)
      return e;
    if ((e = cudaFuncSetAttribute(merge, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  K8_MERGE_SMEM)) != cudaSuccess)
      return e;
    if ((e = cudaFuncSetAttribute(border, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  K8_MERGE_SMEM)) != cudaSuccess)
      return e;
    if (dev >= 0 && dev < 64) opted_in[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Few keys: the block table bounds the sequences' lengths, which are not known here.
  p.cluster = 1;
  const int64_t items = (int64_t)a.n * a.h_kv * p.subs;
  const int64_t units = (a.capacity + C::KEYS - 1) / C::KEYS;
  while (p.cluster < 8 && items * p.cluster * 2 <= C::CTAS && p.cluster < units) p.cluster *= 2;
  if (items * p.cluster <= C::CTAS && a.capacity <= (int64_t)K8_FEW_KEYS * p.cluster) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(items * p.cluster));
    cfg.numAttrs = 2;
    if ((e = cudaLaunchKernelEx(&cfg, few, p, kmap, vmap)) != cudaSuccess) return e;
  } else {
    p.cluster = 0;
    cfg.gridDim = dim3((unsigned)p.ctas);
    if ((e = cudaLaunchKernelEx(&cfg, kernel, p, kmap, vmap)) != cudaSuccess) return e;
    p.merge_rows = p.rows;
    int64_t slices = 1;
    const bool by_border = items > 2 * p.ctas;
    if (items <= SMS)
      while (p.merge_rows > 1 && items * slices * 2 <= 4 * SMS) {
        p.merge_rows = (p.merge_rows + 1) / 2;
        slices = (p.rows + p.merge_rows - 1) / p.merge_rows;
      }
    cfg.gridDim = dim3((unsigned)(by_border ? p.ctas - 1 : items * slices));
    cfg.blockDim = dim3(K8_MERGE_THREADS);
    cfg.dynamicSmemBytes = (size_t)k8_most_parts(p) * (8 * p.merge_rows + 4);
    if ((e = cudaLaunchKernelEx(&cfg, by_border ? border : merge, p)) != cudaSuccess) return e;
  }
  if (!a.weights) return cudaSuccess;
  const int64_t most = (a.capacity + RECEIVED_KEYS - 1) / RECEIVED_KEYS;
  const int across = most < 64 ? (int)most : 64;
  return launch_behind(kv8_received_kernel, dim3((unsigned)(a.n * a.h_kv * across)), RECEIVED_THREADS, 0,
                       s, a, across);
}

// Up to eight query heads of a key/value head: one eight of them; more: two (64 sequences of up to
// 8192, 4 key/value heads of 256, replayed: 96 us with 4 query heads each, 102 with 8, 114 with 12, 118
// with 16; 8 of 128: 92 with 8, 99 with 12, 100 with 16; 64 of up to 16,384, 4 of 64: 56 with 8, 85 with 16).
template <typename IO, int D>
static cudaError_t launch_decode_n(const GdnKv8DecodeArgs& a, cudaStream_t s) {
  return a.h_q / a.h_kv <= 8 ? launch_decode<IO, D, 1>(a, s) : launch_decode<IO, D, 2>(a, s);
}
template <typename IO>
static cudaError_t launch_decode_d(const GdnKv8DecodeArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_decode_n<IO, 64>(a, s)
                   : a.d == 128 ? launch_decode_n<IO, 128>(a, s) : launch_decode_n<IO, 256>(a, s);
}

}  // namespace attn
}  // namespace gdn

int64_t gdn_kv8_decode_slots(int h_q, int h_kv) {
  using namespace gdn::attn;
  const int group = h_q / h_kv, most = group <= 8 ? 8 : 16;
  // two cut items per CTA
  return 2 * K8Cfg<256, 1>::CTAS * (int64_t)(group < most ? group : most);
}

cudaError_t gdn_launch_kv8_decode(const GdnKv8DecodeArgs& a, int io, cudaStream_t s) {
  using namespace gdn::attn;
  return io == GDN_BF16 ? launch_decode_d<__nv_bfloat16>(a, s) : launch_decode_d<__half>(a, s);
}
