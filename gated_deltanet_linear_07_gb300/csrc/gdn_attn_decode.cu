// gdn_attn_decode.cu -- one query token per sequence against a paged cache.
//
//   o_b = sum_s 2^(c (q_b . k_s - m)) v_s / sum_s 2^(c (q_b . k_s - m))
//
// Every cached byte is used for one token's few query heads only, so the reads
// of the cache bound it.  The work is cut by bytes, not by sequences: all
// blocks of 64 keys of all (sequence, key/value head) items form one line of
// units, which the resident CTAs share in equal runs, whatever the lengths.  A
// run that covers an item writes its output; an item cut by a run's border
// leaves partial results (O, m, l) that the merge kernel joins.  The borders
// follow from seq_lens alone, so both kernels work them out for themselves and
// nothing has to be handed over but the partials.
//
// Within a CTA one warp keeps TMA loads of K and V blocks in flight through a
// ring that fills shared memory, and four warps take 16 keys of each block
// with their own m, l and O (the 16 x D accumulator of mma.sync m16n8k16, its
// 16 rows being the item's query heads): no barrier between them inside a run.
// Every wait is bounded: a consumer whose wait ran out frees no stage any more and
// makes the sums of its items NaN, the loading warp then runs out too, and what it
// has in flight lands before it leaves.
//
// Few keys in all (at most FEW_BLOCKS blocks per CTA with a cluster of CTAs to an
// item and no more CTAs than fit at once): the same kernel with the items cut over
// the clusters, which join their partials through distributed shared memory.  No
// search for the run, no second launch: 700 keys of 4 heads, 8 us instead of 10.
//
// Behind a shared prefix (gdn_attn_tc.cu computes it once for all rows) the
// items start at shared_len and the merge adds the prefix's partials.  A row that
// ends inside the prefix is not part of that pass, whose products run over all of
// the prefix's values (a weight of zero does not keep an Inf or NaN out): all of
// its keys are its own item here, from key 0, in the prefix's pages.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_attn.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace attn {

using namespace gdn::tc;

constexpr int KEYS = 64;              // keys per block
constexpr int ROWS = 16;              // query heads per item, at most
constexpr int DEC_WARPS = 4;          // consumer warps, 16 keys of a block each
constexpr int DEC_THREADS = 32 * (DEC_WARPS + 1);
constexpr int DEC_MAX_STAGES = 8;
constexpr int FEW_BLOCKS = 4;

template <int D>
struct DecCfg {
  static constexpr uint32_t TILE = KEYS * D * 2;           // one of K, V
  static constexpr uint32_t STAGE = 2 * TILE;
  static constexpr uint32_t OBUF = ROWS * D * 4;           // joining the four warps' O
  static constexpr uint32_t Q_ROW = D * 2 + 16;            // padded: no bank conflicts in ldmatrix
  static constexpr uint32_t HEAD = (1024 + ROWS * Q_ROW + OBUF + 1023) / 1024 * 1024;
  // Smaller heads want more warps to keep up with the loads; at 256 one warp's
  // accumulator takes the registers of two.
  static constexpr int PER_SM = D == 256 ? 1 : D == 128 ? 2 : 3;
  static constexpr int CTAS = SMS * PER_SM;
  static constexpr int FIT = (int)((233472u / PER_SM - 1024u - HEAD) / STAGE);
  static constexpr int STAGES = FIT < DEC_MAX_STAGES ? FIT : DEC_MAX_STAGES;
  static constexpr uint32_t SMEM = HEAD + STAGES * STAGE;
};

struct __align__(16) DecShared {
  uint64_t full[DEC_MAX_STAGES], empty[DEC_MAX_STAGES], q_full, q_empty;
  float m[DEC_WARPS][ROWS], l[DEC_WARPS][ROWS];
  float2 ml[ROWS];       // of the whole CTA, for its cluster
  int64_t sum[DEC_WARPS + 1], found_first;
  int32_t found;
};
static_assert(sizeof(DecShared) <= 1024, "shared bookkeeping");

struct DecArgs {
  GdnAttnArgs a;
  int64_t start;         // first key of this pass: shared_len, or 0 (rows that end before it
                         // have all of theirs here)
  int64_t base_row;      // first row of the partials of this pass
  int32_t rows;          // query heads per item, <= ROWS
  int32_t subs;          // items per (sequence, key/value head)
  int32_t box_rows;      // rows per TMA box
  int32_t ctas;          // CTAs that share the units
  int32_t early, delay;  // of them, those that start beside the prefix pass, and how many units
                         // of time before the others (0: no prefix pass)
  int32_t prefix;        // prefix partials per row (0: none)
  int32_t cluster;       // CTAs per item (the form for few keys; 0: runs of units)
  int32_t merge_rows;    // rows of an item that a CTA of the merge joins
};

// Keys of sequence b that this pass sees, from `first` on.
__device__ __forceinline__ int64_t own_keys(const DecArgs& p, int b, int64_t& first) {
  int64_t len = p.a.seq_lens[b];
  const int64_t cap = (int64_t)p.a.cache.pages_per_seq << p.a.page_shift;
  if (len > cap) {
    set_status(p.a.d_status, GDN_DEV_BAD_LENGTH);
    len = cap;
  }
  first = len < p.start ? 0 : p.start;
  return len > first ? len - first : 0;
}
__device__ __forceinline__ int64_t own_keys(const DecArgs& p, int b) {
  int64_t first;
  return own_keys(p, b, first);
}
__device__ __forceinline__ int64_t blocks_of(int64_t keys) { return (keys + KEYS - 1) / KEYS; }

// Which units each CTA takes: run c is [start(c), start(c + 1)).  Without a prefix
// pass the runs are equal.  Behind one, the first `early` CTAs start on the SMs
// that the prefix pass leaves free and the others when it ends, `delay` units of
// time later: the line is stretched by that much for each of those, and their
// runs leave the stretch out.  (Where the early ones can do all of it before, they
// do.)  Behind a long prefix some runs may be empty.
struct Line {
  int64_t units, stretched;
  int ctas, early, delay;
  __device__ __forceinline__ Line(const DecArgs& p, int64_t n) : units(n), stretched(n), delay(p.delay) {
    const bool alone = p.early > 0 && n < (int64_t)p.delay * p.early;
    if (p.early == 0 || alone) {
      const int most = alone ? p.early : p.ctas;
      ctas = n < most ? (int)n : most;
      early = ctas;
    } else {
      ctas = p.ctas;
      early = p.early;
      stretched += (int64_t)delay * (ctas - early);
    }
  }
  __device__ __forceinline__ int64_t start(int c) const {
    return stretched * c / ctas - (c > early ? (int64_t)delay * (c - early) : 0);
  }
  // The CTA whose run holds unit u: the last whose run starts at or before it.
  __device__ __forceinline__ int owner(int64_t u) const {
    if (early == ctas) return (int)(((u + 1) * ctas - 1) / stretched);
    int lo = 0, hi = ctas;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      const int64_t out = mid > early ? (int64_t)delay * (mid - early) : 0;
      if (stretched * mid < (u + out + 1) * ctas)   // start(mid) <= u
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  }
};

// Sum of v over the CTA's threads (in every thread) and, in `before`, over the
// threads below this one.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums, int warps, int64_t& before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t all = 0, off = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) off += sums[w];
    all += sums[w];
  }
  before = off + incl - v;
  __syncthreads();
  return all;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <typename IO>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                 uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int row, int kb,
                                        uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(kb), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(__cvta_generic_to_global(src))), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
// The next kernel of the stream may start once every CTA has said so; what it
// reads of this one it waits for with pdl_wait.
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void consumers_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * DEC_WARPS) : "memory");
}

// First query head and number of query heads of item hs of a sequence.
__device__ __forceinline__ int item_head(const DecArgs& p, int hs) {
  return hs / p.subs * (p.a.h_q / p.a.h_kv) + hs % p.subs * ROWS;
}
__device__ __forceinline__ int item_rows(const DecArgs& p, int hs) {
  return min(p.rows, p.a.h_q / p.a.h_kv - hs % p.subs * ROWS);
}

// Four channels of a finished output: y / l, gated (zeros where no key was seen).
template <typename IO, int D>
__device__ __forceinline__ void put_four(const GdnAttnArgs& a, int b, int h, int col, float l,
                                         float (&y)[4]) {
  const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] *= inv;
  if (a.gate.data && l != 0.f) {
    const uint2 g = *reinterpret_cast<const uint2*>(reinterpret_cast<const IO*>(a.gate.data) +
                                                    (int64_t)b * a.gate.token_stride +
                                                    h * a.gate.head_stride + col);
    const float2 g0 = unpack2<IO>(g.x), g1 = unpack2<IO>(g.y);
    y[0] *= gate_sigmoid(g0.x);
    y[1] *= gate_sigmoid(g0.y);
    y[2] *= gate_sigmoid(g1.x);
    y[3] *= gate_sigmoid(g1.y);
  }
  *reinterpret_cast<uint2*>(reinterpret_cast<IO*>(a.o) + ((int64_t)b * a.h_q + h) * D + col) =
      make_uint2(pack2<IO>(y[0], y[1]), pack2<IO>(y[2], y[3]));
}

// The run [w, end) of units, item by item.
struct Segment {
  int b, hs;             // sequence, and key/value head * subs + sub
  int64_t keys, first;   // keys of the sequence in this pass, from key `first` on
  int64_t t0, t1;        // blocks of the item in this run
  bool whole;            // all of the item is in this run
};
struct Walk {
  int64_t w, end, item_first, nt, keys, first;
  int b, hs;
  __device__ bool next(const DecArgs& p, int heads, Segment& s) {
    if (w >= end) return false;
    while (w >= item_first + nt) {   // on to the item that holds unit w
      item_first += nt;
      if (++hs == heads) {
        hs = 0;
        do {
          ++b;
          keys = own_keys(p, b, first);
          nt = blocks_of(keys);
        } while (nt == 0);
      }
    }
    s.b = b;
    s.hs = hs;
    s.keys = keys;
    s.first = first;
    s.t0 = w - item_first;
    s.t1 = min(end - item_first, nt);
    s.whole = s.t0 == 0 && s.t1 == nt;
    w = item_first + s.t1;
    return true;
  }
};

__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_peer_16(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_peer_8(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

template <typename IO, int D, bool FEW>
__global__ void __launch_bounds__(DEC_THREADS, DecCfg<D>::PER_SM)
    attn_decode_kernel(const __grid_constant__ DecArgs p, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  using C = DecCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  DecShared* sh = reinterpret_cast<DecShared*>(smem);
  const uint32_t q_smem = smem_u32(smem) + 1024;
  float* obuf = reinterpret_cast<float*>(smem + 1024 + ROWS * C::Q_ROW);
  const GdnAttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem) + C::HEAD;
  const int heads = a.h_kv * p.subs;
  const int n = (int)a.total_q;

  pdl_launch();
  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], DEC_WARPS);
    }
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, DEC_WARPS);
    fence_mbar_init();
  }
  Walk walk;
  int64_t w0, w1;
  if (FEW) {
    // ---- this CTA's share of its cluster's item ----
    const int item = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
    walk.b = item / heads;
    walk.hs = item % heads;
    walk.keys = own_keys(p, walk.b, walk.first);
    walk.nt = blocks_of(walk.keys);
    walk.item_first = 0;
    w0 = walk.nt * rank / p.cluster;
    w1 = walk.nt * (rank + 1) / p.cluster;
    if (tid < ROWS) sh->ml[tid] = make_float2(-INFINITY, 0.f);
    __syncthreads();
  } else {
    // ---- this CTA's run of units ----
    int64_t total = 0, units = 0, before = 0;
    for (int base = 0; base < n; base += DEC_THREADS) {
      const int b = base + tid;
      units = b < n ? blocks_of(own_keys(p, b)) * heads : 0;
      total += block_scan(units, sh->sum, DEC_WARPS + 1, before);
    }
    const Line line(p, total);
    const int c = (int)blockIdx.x;
    w0 = c < line.ctas ? line.start(c) : 0;
    w1 = c < line.ctas ? line.start(c + 1) : 0;
    int64_t seen = 0;
    for (int base = 0; base < n && w0 < w1; base += DEC_THREADS) {
      const int b = base + tid;
      int64_t all = total;
      if (n > DEC_THREADS) {   // else the scan above has it all
        units = b < n ? blocks_of(own_keys(p, b)) * heads : 0;
        all = block_scan(units, sh->sum, DEC_WARPS + 1, before);
      }
      if (w0 >= seen + before && w0 < seen + before + units) {
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
      walk.keys = own_keys(p, walk.b, walk.first);
      walk.nt = blocks_of(walk.keys);
      walk.hs = (int)((w0 - sh->found_first) / walk.nt);
      walk.item_first = sh->found_first + walk.hs * walk.nt;
    }
    Segment g;
    bool ok = true;
    int j = 0, items = 0;            // blocks and items so far: the rings' positions
    if (warp == DEC_WARPS) {
      // ---- loads: each lane one box of the block (K or V, rows, channels) ----
      const int per_kv = (KEYS / p.box_rows) * (D / 64);
      const bool is_v = lane >= per_kv;
      const int box = is_v ? lane - per_kv : lane;
      const int kb = box % (D / 64), r = box / (D / 64) * p.box_rows;
      while (ok && walk.next(p, heads, g)) {
        const int kvh = g.hs / p.subs;
        // the prefix's pages are those of row 0
        const int32_t* table =
            a.cache.block_table + (int64_t)(g.first < p.start ? 0 : g.b) * a.cache.pages_per_seq;
        // the item's queries, once the consumers have the last item's in registers
        if (items > 0) ok = mbar_wait(&sh->q_empty, (items - 1) & 1, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++items;
        const int h0 = item_head(p, g.hs);
        const int rows = item_rows(p, g.hs);
        if (lane == 0) mbar_expect_tx(&sh->q_full, (uint32_t)rows * D * 2);
        __syncwarp();
        if (lane < rows)
          bulk_load(q_smem + (uint32_t)lane * C::Q_ROW,
                    reinterpret_cast<const IO*>(a.q.data) + (int64_t)g.b * a.q.token_stride +
                        (int64_t)(h0 + lane) * a.q.head_stride,
                    D * 2, &sh->q_full);
        auto page_at = [&](int64_t t) {
          const int64_t pos = t * KEYS + r;
          return lane < 2 * per_kv && t < g.t1 && pos < g.keys
                     ? __ldg(table + ((g.first + pos) >> a.page_shift))
                     : 0;
        };
        int32_t page = page_at(g.t0);
        for (int64_t t = g.t0; t < g.t1 && ok; ++t, ++j) {
          const int32_t next = page_at(t + 1);   // on its way while this block waits for room
          const int s = j % C::STAGES;
          if (j >= C::STAGES)
            ok = mbar_wait(&sh->empty[s], ((j / C::STAGES) - 1) & 1, a.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const int64_t left = g.keys - t * KEYS;
          const int there = (int)min((int64_t)KEYS, (left + p.box_rows - 1) / p.box_rows * p.box_rows);
          // (the test's: of the first CTA, or of the last one of the first cluster)
          const bool withheld = a.withhold && j == 0 && blockIdx.x == (FEW ? p.cluster - 1 : 0);
          if (lane == 0 && !withheld) mbar_expect_tx(&sh->full[s], (uint32_t)there * D * 4);
          __syncwarp();
          if (lane < 2 * per_kv && r < there && !withheld) {
            if (page < 0 || page >= a.cache.num_pages) {
              set_status(a.d_status, GDN_DEV_BAD_PAGE);
              page = 0;
            }
            const int64_t pos = g.first + t * KEYS + r;
            const int64_t row = (((int64_t)page * a.h_kv + kvh) << a.page_shift) +
                                (pos & ((1 << a.page_shift) - 1));
            tma_box(ring + (uint32_t)s * C::STAGE + (is_v ? C::TILE : 0u) +
                        (uint32_t)(kb * KEYS + r) * 128u,
                    is_v ? &vmap : &kmap, (int)row, kb, &sh->full[s]);
          }
          page = next;
        }
      }
      // (the consumers wait for these too, unless they have given up)
      for (int x = max(0, j - C::STAGES); x < j; ++x)
        mbar_wait(&sh->full[x % C::STAGES], (x / C::STAGES) & 1, GRACE_NS);
      if (items > 0) mbar_wait(&sh->q_full, (items - 1) & 1, GRACE_NS);
    } else {
      // ---- 16 keys of every block, with this warp's own m, l, O ----
      const int qrow = lane >> 2, qcol = (lane & 3) * 2;
      const float c = a.scale_log2;
      // this lane's row of the four 8 x 8 blocks of an ldmatrix
      const int mi = lane >> 3, mr = lane & 7;
      const int k_tok = warp * 16 + (mi >> 1) * 8 + mr, k_d = (mi & 1) * 8;
      const int v_tok = warp * 16 + (mi & 1) * 8 + mr, v_d = (mi >> 1) * 8;
      while (walk.next(p, heads, g)) {
        const int h0 = item_head(p, g.hs);
        const int rows = item_rows(p, g.hs);
        if (ok) ok = mbar_wait(&sh->q_full, items & 1, a.wait_ns);
        __syncwarp();
        ++items;
        // rows past the item's heads hold anything: they stay in their own rows
        uint32_t qa[D / 16][4];
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          ldsm4(q_smem + (uint32_t)((mi & 1) * 8 + mr) * C::Q_ROW +
                    (uint32_t)(ks * 32 + (mi >> 1) * 16),
                qa[ks]);
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&sh->q_empty);
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int64_t t = g.t0; t < g.t1; ++t, ++j) {
          const int s = j % C::STAGES;
          if (ok) ok = mbar_wait(&sh->full[s], (j / C::STAGES) & 1, a.wait_ns);
          __syncwarp();
          const int left = (int)min((int64_t)KEYS, g.keys - t * KEYS) - warp * 16;   // keys of these 16
          const uint32_t kt = ring + (uint32_t)s * C::STAGE, vt = kt + C::TILE;
          if (left > 0) {
            float sc[2][2][4] = {};
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              uint32_t kf[4];
              const int d = ks * 16 + k_d;
              ldsm4(kt + (uint32_t)((d >> 6) * KEYS * 128 + k_tok * 128) +
                        ((uint32_t)((d & 63) * 2) ^ (uint32_t)(mr << 4)),
                    kf);
              mma16816<IO>(sc[ks & 1][0], qa[ks], kf[0], kf[1]);
              mma16816<IO>(sc[ks & 1][1], qa[ks], kf[2], kf[3]);
            }
            float x[2][4];   // [keys 0-7, 8-15][row: 2, row + 8: 2]
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                x[nt][e] = sc[0][nt][e] + sc[1][nt][e];
                if (nt * 8 + qcol + (e & 1) >= left) x[nt][e] = -INFINITY;
              }
            float mt[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              mt[r] = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
              mt[r] = fmaxf(mt[r], __shfl_xor_sync(0xffffffffu, mt[r], 1));
              mt[r] = fmaxf(mt[r], __shfl_xor_sync(0xffffffffu, mt[r], 2));
            }
            // The reference maximum may lag (WeightRange).  A row's follows from the
            // row alone, and rows without a head ask for nothing.
            bool far[2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
              far[r] = qrow + 8 * r < rows && mt[r] > m[r] &&
                       (m[r] == -INFINITY || (mt[r] - m[r]) * c > WeightRange<IO>::LAG_LOG2);
            if (__any_sync(0xffffffffu, far[0] || far[1])) {
              float f[2];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                f[r] = far[r] ? fast_exp2((m[r] - mt[r]) * c) : 1.f;
                m[r] = far[r] ? mt[r] : m[r];
                l[r] *= f[r];
              }
#pragma unroll
              for (int i = 0; i < D / 8; ++i) {
                o[i][0] *= f[0];
                o[i][1] *= f[0];
                o[i][2] *= f[1];
                o[i][3] *= f[1];
              }
            }
            // The weights go to the product with v in the I/O type, as the prefill's do (a
            // prompt's last token and a decoded one round alike); their sum does not.
            uint32_t pa[4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float nm = weight_offset<IO>(m[r], c);
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                const float e0 = fast_exp2(fmaf(x[nt][2 * r], c, nm));
                const float e1 = fast_exp2(fmaf(x[nt][2 * r + 1], c, nm));
                l[r] += e0 + e1;
                pa[nt * 2 + r] = pack2<IO>(e0, e1);
              }
            }
            // values past the end may be anything: cleared, as 0 x NaN is not 0
            uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
            if (left < 16) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int k = e * 8 + qcol;
                keep[e] = (k < left ? 0x0000ffffu : 0u) | (k + 1 < left ? 0xffff0000u : 0u);
              }
            }
#pragma unroll
            for (int nb = 0; nb < D / 16; ++nb) {
              uint32_t vf[4];
              const int d = nb * 16 + v_d;
              ldsm4t(vt + (uint32_t)((d >> 6) * KEYS * 128 + v_tok * 128) +
                         ((uint32_t)((d & 63) * 2) ^ (uint32_t)(mr << 4)),
                     vf);
              mma16816<IO>(o[2 * nb], pa, vf[0] & keep[0], vf[1] & keep[1]);
              mma16816<IO>(o[2 * nb + 1], pa, vf[2] & keep[0], vf[3] & keep[1]);
            }
          }
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&sh->empty[s]);
        }

        // ---- join the four warps ----
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
          l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
          if (!__all_sync(0xffffffffu, ok)) l[r] = NAN;
        }
        if ((lane & 3) == 0) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            sh->m[warp][qrow + 8 * r] = m[r];
            sh->l[warp][qrow + 8 * r] = l[r];
          }
        }
        consumers_bar();
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mm = -INFINITY;
#pragma unroll
          for (int w = 0; w < DEC_WARPS; ++w) mm = fmaxf(mm, sh->m[w][qrow + 8 * r]);
          f[r] = mm == -INFINITY ? 0.f : fast_exp2((m[r] - mm) * c);
        }
        // Up to four rows: each warp its own slab, summed on the way out.  More
        // do not fit, and the warps add up in one slab, a quarter of the channels
        // at a time, each at another one.  Either way every sum has a fixed order.
        const int slabs = rows <= ROWS / DEC_WARPS ? DEC_WARPS : 1;
#pragma unroll
        for (int st = 0; st < DEC_WARPS; ++st) {
          if (slabs > 1 && st > 0) break;
          const int qt = (warp + st) % DEC_WARPS;
          float* slab = obuf + (slabs > 1 ? warp * rows * D : 0);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            if (slabs == 1 && i / (D / 32) != qt) continue;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int row = qrow + 8 * r;
              if (row >= rows) continue;
              float2* dst = reinterpret_cast<float2*>(slab + row * D + i * 8 + qcol);
              float2 v = make_float2(o[i][2 * r] * f[r], o[i][2 * r + 1] * f[r]);
              if (st > 0) {
                const float2 w = *dst;
                v.x += w.x;
                v.y += w.y;
              }
              *dst = v;
            }
          }
          consumers_bar();
        }
        // ---- out: the output itself, or a partial result ----
        const bool direct = !FEW && g.whole && p.prefix == 0;
        const int64_t slot = g.whole ? 2 * (int64_t)p.ctas + (int64_t)g.b * heads + g.hs
                                     : 2 * (int64_t)blockIdx.x + (g.t0 > 0 ? 0 : 1);
        const int64_t part = p.base_row + slot * p.rows;
        for (int x = tid; x < rows * (D / 8); x += 32 * DEC_WARPS) {
          const int row = x / (D / 8), col = x % (D / 8) * 8;
          float mm = -INFINITY, ll = 0.f;
#pragma unroll
          for (int w = 0; w < DEC_WARPS; ++w) mm = fmaxf(mm, sh->m[w][row]);
#pragma unroll
          for (int w = 0; w < DEC_WARPS; ++w)
            ll += mm == -INFINITY ? sh->l[w][row] : sh->l[w][row] * fast_exp2((sh->m[w][row] - mm) * c);
          float4 v0 = *reinterpret_cast<const float4*>(obuf + row * D + col);
          float4 v1 = *reinterpret_cast<const float4*>(obuf + row * D + col + 4);
          for (int w = 1; w < slabs; ++w) {
            const float4 u0 = *reinterpret_cast<const float4*>(obuf + (w * rows + row) * D + col);
            const float4 u1 = *reinterpret_cast<const float4*>(obuf + (w * rows + row) * D + col + 4);
            v0.x += u0.x; v0.y += u0.y; v0.z += u0.z; v0.w += u0.w;
            v1.x += u1.x; v1.y += u1.y; v1.z += u1.z; v1.w += u1.w;
          }
          if (FEW) {
            float4* dst = reinterpret_cast<float4*>(obuf + row * D + col);
            dst[0] = v0;
            dst[1] = v1;
            if (col == 0) sh->ml[row] = make_float2(mm, ll);
          } else if (direct) {
            const float inv = 1.0f / ll;
            float y[8] = {v0.x * inv, v0.y * inv, v0.z * inv, v0.w * inv,
                          v1.x * inv, v1.y * inv, v1.z * inv, v1.w * inv};
            if (a.gate.data) {
              Vec8<IO> gv;
              gv.load(reinterpret_cast<const IO*>(a.gate.data) + (int64_t)g.b * a.gate.token_stride +
                      (h0 + row) * a.gate.head_stride + col);
              float gf[8];
              gv.get(gf);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] *= gate_sigmoid(gf[e]);
            }
            Vec8<IO> ov;
            ov.set(y);
            ov.store(reinterpret_cast<IO*>(a.o) + ((int64_t)g.b * a.h_q + h0 + row) * D + col);
          } else {
            float4* dst = reinterpret_cast<float4*>(a.part_o + (part + row) * D + col);
            dst[0] = v0;
            dst[1] = v1;
            if (col == 0) a.part_ml[part + row] = make_float2(mm * c, ll);
          }
        }
        consumers_bar();   // obuf and m, l are free again
      }
    }
    if (!ok) set_status(a.d_status, GDN_DEV_WAIT_TIMEOUT);
  }
  if (FEW) {
    // ---- the cluster's partials joined, a share of the channels by each CTA ----
    __syncwarp();
    cluster_barrier();
    const int rank = blockIdx.x % p.cluster;
    const int rows = item_rows(p, walk.hs), h0 = item_head(p, walk.hs);
    const uint32_t ml_at = smem_u32(sh->ml), o_at = smem_u32(obuf);
    for (int x = rank * DEC_THREADS + tid; x < rows * (D / 4); x += p.cluster * DEC_THREADS) {
      const int row = x / (D / 4), col = x % (D / 4) * 4;
      float mm = -INFINITY, ll = 0.f;
      for (int r = 0; r < p.cluster; ++r)
        mm = fmaxf(mm, ld_peer_8(peer_addr(ml_at + 8u * row, r)).x);
      float y[4] = {};
      for (int r = 0; r < p.cluster; ++r) {
        const float2 v = ld_peer_8(peer_addr(ml_at + 8u * row, r));
        if (v.y == 0.f) continue;   // saw no key
        const float f = fast_exp2((v.x - mm) * a.scale_log2);
        const float4 o = ld_peer_16(peer_addr(o_at + (uint32_t)(row * D + col) * 4u, r));
        ll += f * v.y;
        y[0] = fmaf(f, o.x, y[0]);
        y[1] = fmaf(f, o.y, y[1]);
        y[2] = fmaf(f, o.z, y[2]);
        y[3] = fmaf(f, o.w, y[3]);
      }
      put_four<IO, D>(a, walk.b, h0 + row, col, ll, y);
    }
    cluster_barrier();   // the others may still read this CTA's
  }
  // The merge waits for this kernel, and reads the prefix pass's partials too:
  // this kernel may have started before that pass had ended.
  pdl_wait();
}

// Joins the partial results of one item (sequence, key/value head, sub):
//   M = max m_i,  o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// A CTA joins merge_rows rows of it.  The partials' statistics are fetched side by side and
// turned into one factor per partial and row first, so that the sums over the
// partial outputs are independent loads (one after the other they would cost a
// memory latency each).
constexpr int MERGE_THREADS = 256;

// Partials of one item, at most.  With equal runs every head of a sequence has as
// many units, so an item is at most 1 / heads of the line, and its ends cut two
// runs; the short runs behind a prefix pass may all meet one item.
static __host__ __device__ __forceinline__ int most_parts(const DecArgs& p) {
  return p.prefix + (p.early > 0 ? p.ctas : p.ctas / (p.a.h_kv * p.subs) + 2);
}

// One item of 16 rows behind a prefix in PREFIX_SMS parts, runs of 3 SMS CTAs: 75 KB.
constexpr int MERGE_SMEM = 96 * 1024;

template <typename IO, int D, bool SPLIT>
__global__ void __launch_bounds__(MERGE_THREADS)
    attn_merge_kernel(const __grid_constant__ DecArgs p) {
  extern __shared__ __align__(16) unsigned char merge_smem[];
  __shared__ int64_t sums[MERGE_THREADS / 32], s_mine;
  __shared__ float sum_l[ROWS];
  __shared__ float4 shares[SPLIT ? MERGE_THREADS : 1];
  const GdnAttnArgs& a = p.a;
  int64_t* first_row = reinterpret_cast<int64_t*>(merge_smem);          // [part]
  float2* ml = reinterpret_cast<float2*>(first_row + most_parts(p));    // [part][row]: statistics,
                                                                        // then (factor, sum)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int heads = a.h_kv * p.subs;
  const int n = (int)a.total_q;
  const int slices = SPLIT ? (p.rows + p.merge_rows - 1) / p.merge_rows : 1;
  const int item = blockIdx.x / slices, r0 = SPLIT ? blockIdx.x % slices * p.merge_rows : 0;
  const int b = item / heads, hs = item % heads;
  const int h0 = item_head(p, hs) + r0;
  const int rows = SPLIT ? min(p.merge_rows, item_rows(p, hs) - r0) : item_rows(p, hs);
  int64_t total = 0;
  for (int base = 0; base < n; base += MERGE_THREADS) {
    const int i = base + tid;
    int64_t before;
    const int64_t u = i < n ? blocks_of(own_keys(p, i)) * heads : 0;
    const int64_t all = block_scan(u, sums, MERGE_THREADS / 32, before);
    if (i == b) s_mine = total + before;
    total += all;
  }
  __syncthreads();
  const int64_t nt = blocks_of(own_keys(p, b));
  const int64_t u0 = s_mine + hs * nt, u1 = u0 + nt;
  // the CTAs whose runs meet [u0, u1)
  const Line line(p, total);
  int c0 = 0, c1 = -1;
  bool whole = false;
  if (nt > 0) {
    c0 = line.owner(u0);
    c1 = line.owner(u1 - 1);
    whole = c0 == c1;
  }
  const int parts = p.prefix + c1 - c0 + 1;
  for (int i = tid; i < parts; i += MERGE_THREADS) {   // partial i's first row of the workspace
    if (i < p.prefix) {
      first_row[i] = ((int64_t)i * n + b) * a.h_q + h0 - r0;
    } else if (whole) {
      first_row[i] = p.base_row + (2 * (int64_t)p.ctas + (int64_t)b * heads + hs) * p.rows;
    } else {
      const int c = c0 + (i - p.prefix);
      // a run that starts inside the item left its first partial, else its last
      const int64_t at = line.start(c);
      first_row[i] = at == line.start(c + 1) ? -1 : p.base_row + (2 * c + (at > u0 ? 0 : 1)) * p.rows;
    }
  }
  pdl_wait();
  if (nt > 0 && whole && p.prefix == 0) return;   // written already
  if (SPLIT && rows <= 0) return;                 // the last heads' item may be shorter
  __syncthreads();
  for (int i = tid; i < parts * rows; i += MERGE_THREADS)
    ml[i] = first_row[i / rows] < 0 ? make_float2(0.f, 0.f)   // an empty run
                                    : a.part_ml[first_row[i / rows] + r0 + i % rows];
  __syncthreads();
  for (int row = warp; row < rows; row += MERGE_THREADS / 32) {
    float mm = -INFINITY, ll = 0.f;
    for (int i = lane; i < parts; i += 32)
      if (ml[i * rows + row].y != 0.f) mm = fmaxf(mm, ml[i * rows + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    for (int i = lane; i < parts; i += 32) {
      const float2 v = ml[i * rows + row];
      // a partial that saw no key has factor 0, and its O was not written
      const float f = v.y == 0.f ? 0.f : fast_exp2(v.x - mm);
      ll += v.y == 0.f ? 0.f : f * v.y;
      ml[i * rows + row].x = f;
    }
    ll = warp_sum(ll);
    if (lane == 0) sum_l[row] = ll;
  }
  __syncthreads();
  auto add_up = [&](int row, int col, int first, int step, float (&y)[4]) {
#pragma unroll 8
    for (int i = first; i < parts; i += step) {
      const float2 w = ml[i * rows + row];
      // (of an empty run, anything that is there: its factor is 0)
      const float4 v = *reinterpret_cast<const float4*>(
          a.part_o + (max(first_row[i], (int64_t)0) + r0 + row) * D + col);
      if (w.y != 0.f) {
        y[0] = fmaf(w.x, v.x, y[0]);
        y[1] = fmaf(w.x, v.y, y[1]);
        y[2] = fmaf(w.x, v.z, y[2]);
        y[3] = fmaf(w.x, v.w, y[3]);
      }
    }
  };
  const int units = rows * (D / 4);
  const int groups = SPLIT ? MERGE_THREADS / units : 1;
  if (groups > 1) {
    // The threads that the rows leave over share the partials: group g takes every
    // groups-th one, and the groups' sums are added in their order.
    const int g = tid / units, x = tid - g * units;
    const int row = x / (D / 4), col = x % (D / 4) * 4;
    float y[4] = {};
    if (g < groups) {
      add_up(row, col, g, groups, y);
      shares[SPLIT ? tid : 0] = make_float4(y[0], y[1], y[2], y[3]);
    }
    __syncthreads();
    if (g > 0) return;
    for (int i = 1; i < groups; ++i) {
      const float4 v = shares[SPLIT ? i * units + x : 0];
      y[0] += v.x;
      y[1] += v.y;
      y[2] += v.z;
      y[3] += v.w;
    }
    put_four<IO, D>(a, b, h0 + row, col, sum_l[row], y);
    return;
  }
  for (int x = tid; x < units; x += MERGE_THREADS) {
    const int row = x / (D / 4), col = x % (D / 4) * 4;
    float y[4] = {};
    add_up(row, col, 0, 1, y);
    put_four<IO, D>(a, b, h0 + row, col, sum_l[row], y);
  }
}

// ---- host ------------------------------------------------------------------------

static int group_rows(int h_q, int h_kv) {
  const int g = h_q / h_kv;
  return g < ROWS ? g : ROWS;
}

template <typename IO, int D>
static cudaError_t launch_decode(const GdnAttnArgs& a, int io, cudaStream_t s) {
  using C = DecCfg<D>;
  cudaError_t e = cudaSuccess;
  DecArgs p;
  p.a = a;
  const int group = a.h_q / a.h_kv;
  p.rows = group_rows(a.h_q, a.h_kv);
  p.subs = (group + ROWS - 1) / ROWS;
  p.prefix = a.splits;
  p.start = a.splits > 0 ? a.shared_len : 0;
  p.base_row = (int64_t)a.splits * a.total_q * a.h_q;
  p.ctas = C::CTAS;
  p.early = p.delay = 0;
  if (a.splits > 0) {
    // The SMs that the prefix pass leaves free, and its length in units of 64 keys:
    // 128 keys of it take about as long as 0.8 units, or 0.6 below head dim 256
    // where the units are smaller, and it starts and ends in about 5.
    const int left = SMS - gdn_attn_prefix_ctas(a.h_q, a.h_kv, D, (int)a.total_q, a.shared_len);
    if (left > 0) {
      const int64_t blocks = ((a.shared_len + 127) / 128 + a.splits - 1) / a.splits;
      p.early = left * C::PER_SM;
      p.delay = (int)(blocks * (D == 256 ? 8 : 6) / 10 + 5);
    }
  }
  const int page = 1 << a.page_shift;
  p.box_rows = page < KEYS ? page : KEYS;
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(gdn_tensor_map_encoder());
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap kmap, vmap;
  for (int i = 0; i < 2; ++i) {   // cache rows: (64 channels, row of the pool, 64-channel block)
    const cuuint64_t dims[3] = {64, (cuuint64_t)a.cache.num_pages * a.h_kv << a.page_shift, D / 64};
    const cuuint64_t strides[2] = {D * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (enc(i ? &vmap : &kmap,
            io == GDN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            i ? a.cache.v : a.cache.k, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kernel = attn_decode_kernel<IO, D, false>;
  auto few = attn_decode_kernel<IO, D, true>;
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
    if ((e = cudaFuncSetAttribute(attn_merge_kernel<IO, D, false>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  MERGE_SMEM)) != cudaSuccess)
      return e;
    if ((e = cudaFuncSetAttribute(attn_merge_kernel<IO, D, true>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  MERGE_SMEM)) != cudaSuccess)
      return e;
    if (dev >= 0 && dev < 64) opted_in[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(DEC_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  // Few keys: the block table bounds the sequences' lengths, which are not known here.
  p.cluster = 1;
  const int64_t items = a.total_q * a.h_kv * p.subs;
  const int64_t blocks = (((int64_t)a.cache.pages_per_seq << a.page_shift) + KEYS - 1) / KEYS;
  while (p.cluster < 8 && items * p.cluster * 2 <= C::CTAS && p.cluster < blocks) p.cluster *= 2;
  if (a.splits == 0 && items * p.cluster <= C::CTAS && blocks <= (int64_t)FEW_BLOCKS * p.cluster) {
    cudaLaunchAttribute cluster[1];
    cluster[0].id = cudaLaunchAttributeClusterDimension;
    cluster[0].val.clusterDim.x = (unsigned)p.cluster;
    cluster[0].val.clusterDim.y = 1;
    cluster[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(items * p.cluster));
    cfg.attrs = cluster;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, few, p, kmap, vmap);
  }
  p.cluster = 0;
  // This pass needs nothing of the prefix pass and starts on SMs as they become
  // free of it; the merge's search for its partials overlaps this pass's end.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 0 ? 1 : 0;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, p, kmap, vmap)) != cudaSuccess) return e;
  // The merge: a CTA per item, or where that leaves SMs without one, per row or a few of
  // them (one sequence of 100,000 keys of 4 heads: 73.9 and 69.2 us, two of 2112 16.0 and 14.1; eight of 3000
  // with 16 heads of 64, rows alone but their partials shared out: 27.9 and 25.9).
  // More items cut like that lose as much as they gain or more, their searches being the
  // longer part then (64 sequences behind 2048 keys: 19.0 and 20.7).
  p.merge_rows = p.rows;
  int64_t slices = 1;
  if (items <= SMS)
    while (p.merge_rows > 1 && items * slices * 2 <= 4 * SMS) {
      p.merge_rows = (p.merge_rows + 1) / 2;
      slices = (p.rows + p.merge_rows - 1) / p.merge_rows;
    }
  const bool split =
      slices > 1 || (items <= SMS && p.merge_rows * (D / 4) * 2 <= MERGE_THREADS);
  cfg.gridDim = dim3((unsigned)(items * slices));
  cfg.blockDim = dim3(MERGE_THREADS);
  cfg.dynamicSmemBytes = (size_t)most_parts(p) * (8 + 8 * p.merge_rows);
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(
      &cfg, split ? attn_merge_kernel<IO, D, true> : attn_merge_kernel<IO, D, false>, p);
}

template <typename IO>
static cudaError_t launch_decode_d(const GdnAttnArgs& a, int io, cudaStream_t s) {
  return a.d == 64 ? launch_decode<IO, 64>(a, io, s)
                   : a.d == 128 ? launch_decode<IO, 128>(a, io, s) : launch_decode<IO, 256>(a, io, s);
}

}  // namespace attn
}  // namespace gdn

int64_t gdn_attn_decode_slots(int h_q, int h_kv, int d, int n, int64_t shared_len) {
  using namespace gdn::attn;
  const int64_t splits = gdn_attn_prefix_splits(h_q, h_kv, d, n, shared_len);
  const int rows = group_rows(h_q, h_kv);
  const int64_t items = (int64_t)n * h_kv * ((h_q / h_kv + ROWS - 1) / ROWS);
  // prefix partials, two cut items per CTA, and with a prefix one per whole item
  const int ctas = d == 64 ? DecCfg<64>::CTAS : d == 128 ? DecCfg<128>::CTAS : DecCfg<256>::CTAS;
  return splits * n * h_q + (2 * ctas + (splits > 0 ? items : 0)) * rows;
}

cudaError_t gdn_launch_attn_decode(const GdnAttnArgs& a, int io, cudaStream_t s) {
  using namespace gdn::attn;
  if (a.splits > 0) {
    const cudaError_t e = gdn_launch_attn_prefix(a, io, s);
    if (e != cudaSuccess) return e;
  }
  return io == GDN_BF16 ? launch_decode_d<__nv_bfloat16>(a, io, s)
                        : launch_decode_d<__half>(a, io, s);
}
