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
//
// Behind a shared prefix (gdn_attn_tc.cu computes it once for all rows) the
// items start at shared_len and the merge adds the prefix's partials.
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

template <int D>
struct DecCfg {
  static constexpr uint32_t TILE = KEYS * D * 2;           // one of K, V
  static constexpr uint32_t STAGE = 2 * TILE;
  static constexpr uint32_t OBUF = ROWS * D * 4;           // joining the four warps' O
  static constexpr int FIT = (int)((232448u - 4096u - OBUF) / STAGE);
  static constexpr int STAGES = FIT < DEC_MAX_STAGES ? FIT : DEC_MAX_STAGES;
  static constexpr uint32_t SMEM = 4096 + OBUF + STAGES * STAGE;
};

struct __align__(16) DecShared {
  uint64_t full[DEC_MAX_STAGES], empty[DEC_MAX_STAGES];
  float m[DEC_WARPS][ROWS], l[DEC_WARPS][ROWS];
  int64_t sum[DEC_WARPS + 1], found_first;
  int32_t found;
};

struct DecArgs {
  GdnAttnArgs a;
  int64_t start;         // first key of this pass: shared_len, or 0
  int64_t base_row;      // first row of the partials of this pass
  int32_t rows;          // query heads per item, <= ROWS
  int32_t subs;          // items per (sequence, key/value head)
  int32_t box_rows;      // rows per TMA box
  int32_t ctas;          // CTAs that share the units
  int32_t prefix;        // prefix partials per row (0: none)
};

// Keys of sequence b that this pass sees.
__device__ __forceinline__ int64_t own_keys(const DecArgs& p, int b) {
  int64_t len = p.a.seq_lens[b];
  const int64_t cap = (int64_t)p.a.cache.pages_per_seq << p.a.page_shift;
  if (len > cap) {
    set_status(p.a.d_status, GDN_DEV_BAD_LENGTH);
    len = cap;
  }
  return len > p.start ? len - p.start : 0;
}
__device__ __forceinline__ int64_t blocks_of(int64_t keys) { return (keys + KEYS - 1) / KEYS; }

// The units are shared by this many CTAs, in runs [units i / runs, units (i + 1) / runs):
// none of them is empty.
__device__ __forceinline__ int64_t runs_of(const DecArgs& p, int64_t units) {
  return units < p.ctas ? units : (int64_t)p.ctas;
}

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
__device__ __forceinline__ void consumers_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * DEC_WARPS) : "memory");
}

// The run [w, end) of units, item by item.
struct Segment {
  int b, hs;             // sequence, and key/value head * subs + sub
  int64_t keys;          // keys of the sequence in this pass
  int64_t t0, t1;        // blocks of the item in this run
  bool whole;            // all of the item is in this run
};
struct Walk {
  int64_t w, end, item_first, nt, keys;
  int b, hs;
  __device__ bool next(const DecArgs& p, int heads, Segment& s) {
    if (w >= end) return false;
    while (w >= item_first + nt) {   // on to the item that holds unit w
      item_first += nt;
      if (++hs == heads) {
        hs = 0;
        do {
          ++b;
          keys = own_keys(p, b);
          nt = blocks_of(keys);
        } while (nt == 0);
      }
    }
    s.b = b;
    s.hs = hs;
    s.keys = keys;
    s.t0 = w - item_first;
    s.t1 = min(end - item_first, nt);
    s.whole = s.t0 == 0 && s.t1 == nt;
    w = item_first + s.t1;
    return true;
  }
};

template <typename IO, int D>
__global__ void __launch_bounds__(DEC_THREADS, 1)
    attn_decode_kernel(const __grid_constant__ DecArgs p, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  using C = DecCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  DecShared* sh = reinterpret_cast<DecShared*>(smem);
  float* obuf = reinterpret_cast<float*>(smem + 4096);
  const GdnAttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem) + 4096 + C::OBUF;
  const int heads = a.h_kv * p.subs;
  const int n = (int)a.total_q;

  // ---- this CTA's run of units ----
  int64_t total = 0;
  for (int base = 0; base < n; base += DEC_THREADS) {
    const int b = base + tid;
    int64_t before;
    total += block_scan(b < n ? blocks_of(own_keys(p, b)) * heads : 0, sh->sum, DEC_WARPS + 1,
                        before);
  }
  const int64_t runs = runs_of(p, total), c = blockIdx.x;
  const int64_t w0 = c < runs ? total * c / runs : 0, w1 = c < runs ? total * (c + 1) / runs : 0;
  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], DEC_WARPS);
    }
    fence_mbar_init();
  }
  int64_t seen = 0;
  for (int base = 0; base < n && w0 < w1; base += DEC_THREADS) {
    const int b = base + tid;
    const int64_t u = b < n ? blocks_of(own_keys(p, b)) * heads : 0;
    int64_t before;
    const int64_t all = block_scan(u, sh->sum, DEC_WARPS + 1, before);
    if (w0 >= seen + before && w0 < seen + before + u) {
      sh->found = b;
      sh->found_first = seen + before;
    }
    seen += all;
  }
  __syncthreads();

  if (w0 < w1) {
    Walk walk;
    walk.w = w0;
    walk.end = w1;
    walk.b = sh->found;
    walk.keys = own_keys(p, walk.b);
    walk.nt = blocks_of(walk.keys);
    walk.hs = (int)((w0 - sh->found_first) / walk.nt);
    walk.item_first = sh->found_first + walk.hs * walk.nt;
    Segment g;
    bool ok = true;
    int j = 0;                       // blocks so far: the ring's position
    if (warp == DEC_WARPS) {
      // ---- loads: each lane one box of the block (K or V, rows, channels) ----
      const int per_kv = (KEYS / p.box_rows) * (D / 64);
      const bool is_v = lane >= per_kv;
      const int box = is_v ? lane - per_kv : lane;
      const int kb = box % (D / 64), r = box / (D / 64) * p.box_rows;
      while (ok && walk.next(p, heads, g)) {
        const int kvh = g.hs / p.subs;
        const int32_t* table = a.cache.block_table + (int64_t)g.b * a.cache.pages_per_seq;
        auto page_at = [&](int64_t t) {
          const int64_t pos = t * KEYS + r;
          return lane < 2 * per_kv && t < g.t1 && pos < g.keys
                     ? __ldg(table + ((p.start + pos) >> a.page_shift))
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
          const int rows = (int)min((int64_t)KEYS, (left + p.box_rows - 1) / p.box_rows * p.box_rows);
          if (lane == 0) mbar_expect_tx(&sh->full[s], (uint32_t)rows * D * 4);
          __syncwarp();
          if (lane < 2 * per_kv && r < rows) {
            if (page < 0 || page >= a.cache.num_pages) {
              set_status(a.d_status, GDN_DEV_BAD_PAGE);
              page = 0;
            }
            const int64_t pos = p.start + t * KEYS + r;
            const int64_t row = (((int64_t)page * a.h_kv + kvh) << a.page_shift) +
                                (pos & ((1 << a.page_shift) - 1));
            tma_box(ring + (uint32_t)s * C::STAGE + (is_v ? C::TILE : 0u) +
                        (uint32_t)(kb * KEYS + r) * 128u,
                    is_v ? &vmap : &kmap, (int)row, kb, &sh->full[s]);
          }
          page = next;
        }
      }
    } else {
      // ---- 16 keys of every block, with this warp's own m, l, O ----
      const int qrow = lane >> 2, qcol = (lane & 3) * 2;
      const float c = a.scale_log2;
      // this lane's row of the four 8 x 8 blocks of an ldmatrix
      const int mi = lane >> 3, mr = lane & 7;
      const int k_tok = warp * 16 + (mi >> 1) * 8 + mr, k_d = (mi & 1) * 8;
      const int v_tok = warp * 16 + (mi & 1) * 8 + mr, v_d = (mi >> 1) * 8;
      while (walk.next(p, heads, g)) {
        const int kvh = g.hs / p.subs, sub = g.hs % p.subs;
        const int group = a.h_q / a.h_kv;
        const int h0 = kvh * group + sub * ROWS;
        const int rows = min(p.rows, group - sub * ROWS);
        const IO* q = reinterpret_cast<const IO*>(a.q.data) + (int64_t)g.b * a.q.token_stride +
                      h0 * a.q.head_stride;
        uint32_t qa[D / 16][4];
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = qrow + (e & 1) * 8, i = ks * 16 + qcol + (e >> 1) * 8;
            qa[ks][e] = r < rows
                            ? *reinterpret_cast<const uint32_t*>(q + r * a.q.head_stride + i)
                            : 0u;
          }
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
            // the reference maximum may lag by 2^8: see gdn_attn_tc.cu
            bool far = false;
#pragma unroll
            for (int r = 0; r < 2; ++r)
              far |= mt[r] > m[r] && (m[r] == -INFINITY || (mt[r] - m[r]) * c > 8.0f);
            if (__any_sync(0xffffffffu, far)) {
              float f[2];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float mn = fmaxf(m[r], mt[r]);
                f[r] = fast_exp2((m[r] - (mn == -INFINITY ? 0.f : mn)) * c);
                m[r] = mn;
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
            uint32_t pa[4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float nm = m[r] == -INFINITY ? 0.f : -m[r] * c;
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
          if (lane == 0) mbar_arrive(&sh->empty[s]);
        }

        // ---- join the four warps ----
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
          l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
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
        // one quarter of the channels at a time, each warp at another one: every
        // sum has a fixed order
#pragma unroll
        for (int st = 0; st < DEC_WARPS; ++st) {
          const int qt = (warp + st) % DEC_WARPS;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            if (i / (D / 32) != qt) continue;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int row = qrow + 8 * r;
              if (row >= rows) continue;
              float2* dst = reinterpret_cast<float2*>(obuf + row * D + i * 8 + qcol);
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
        const bool direct = g.whole && p.prefix == 0;
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
          const float4 v0 = *reinterpret_cast<const float4*>(obuf + row * D + col);
          const float4 v1 = *reinterpret_cast<const float4*>(obuf + row * D + col + 4);
          if (direct) {
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
}

// Joins the partial results of one item (sequence, key/value head, sub):
//   M = max m_i,  o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
constexpr int MERGE_THREADS = 256;

template <typename IO, int D>
__global__ void __launch_bounds__(MERGE_THREADS)
    attn_merge_kernel(const __grid_constant__ DecArgs p) {
  __shared__ int64_t sums[MERGE_THREADS / 32];
  const GdnAttnArgs& a = p.a;
  const int tid = threadIdx.x;
  const int heads = a.h_kv * p.subs;
  const int n = (int)a.total_q;
  const int b = blockIdx.x / heads, hs = blockIdx.x % heads;
  const int group = a.h_q / a.h_kv, kvh = hs / p.subs, sub = hs % p.subs;
  const int h0 = kvh * group + sub * ROWS;
  const int rows = min(p.rows, group - sub * ROWS);
  int64_t total = 0, mine = 0;
  for (int base = 0; base < n; base += MERGE_THREADS) {
    const int i = base + tid;
    const int64_t u = i < n ? blocks_of(own_keys(p, i)) * heads : 0;
    int64_t before;
    total += block_scan(u, sums, MERGE_THREADS / 32, before);
    mine += block_scan(i < b ? u : 0, sums, MERGE_THREADS / 32, before);
  }
  const int64_t nt = blocks_of(own_keys(p, b));
  const int64_t u0 = mine + hs * nt, u1 = u0 + nt;
  // the CTAs whose runs meet [u0, u1)
  const int64_t runs = runs_of(p, total);
  int64_t c0 = 0, c1 = -1;
  bool whole = false;
  if (nt > 0) {
    c0 = ((u0 + 1) * runs - 1) / total;
    c1 = (u1 * runs - 1) / total;
    whole = c0 == c1;
    if (whole && p.prefix == 0) return;   // written already
  }
  const int own = nt > 0 ? (int)(c1 - c0 + 1) : 0;
  auto row_of = [&](int i, int row) -> int64_t {   // partial i's row of the workspace
    if (i < p.prefix) return ((int64_t)i * n + b) * a.h_q + h0 + row;
    if (whole) return p.base_row + (2 * (int64_t)p.ctas + (int64_t)b * heads + hs) * p.rows + row;
    const int64_t c = c0 + (i - p.prefix);
    // a run that starts inside the item left its first partial, else its last
    const int64_t slot = 2 * c + (total * c / runs > u0 ? 0 : 1);
    return p.base_row + slot * p.rows + row;
  };
  const int parts = p.prefix + own;
  for (int x = tid; x < rows * (D / 8); x += MERGE_THREADS) {
    const int row = x / (D / 8), col = x % (D / 8) * 8;
    float mm = -INFINITY;
    for (int i = 0; i < parts; ++i) {
      const float2 ml = a.part_ml[row_of(i, row)];
      if (ml.y != 0.f) mm = fmaxf(mm, ml.x);
    }
    float ll = 0.f, y[8] = {};
    for (int i = 0; i < parts; ++i) {
      const int64_t r = row_of(i, row);
      const float2 ml = a.part_ml[r];
      if (ml.y == 0.f) continue;   // saw no key; its O was not written
      const float f = fast_exp2(ml.x - mm);
      ll += f * ml.y;
      const float4 v0 = *reinterpret_cast<const float4*>(a.part_o + r * D + col);
      const float4 v1 = *reinterpret_cast<const float4*>(a.part_o + r * D + col + 4);
      y[0] = fmaf(f, v0.x, y[0]);
      y[1] = fmaf(f, v0.y, y[1]);
      y[2] = fmaf(f, v0.z, y[2]);
      y[3] = fmaf(f, v0.w, y[3]);
      y[4] = fmaf(f, v1.x, y[4]);
      y[5] = fmaf(f, v1.y, y[5]);
      y[6] = fmaf(f, v1.z, y[6]);
      y[7] = fmaf(f, v1.w, y[7]);
    }
    const float inv = ll == 0.f ? 0.f : 1.0f / ll;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= inv;
    if (a.gate.data && ll != 0.f) {
      Vec8<IO> gv;
      gv.load(reinterpret_cast<const IO*>(a.gate.data) + (int64_t)b * a.gate.token_stride +
              (h0 + row) * a.gate.head_stride + col);
      float gf[8];
      gv.get(gf);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= gate_sigmoid(gf[e]);
    }
    Vec8<IO> ov;
    ov.set(y);
    ov.store(reinterpret_cast<IO*>(a.o) + ((int64_t)b * a.h_q + h0 + row) * D + col);
  }
}

// ---- host ------------------------------------------------------------------------

static int group_rows(int h_q, int h_kv) {
  const int g = h_q / h_kv;
  return g < ROWS ? g : ROWS;
}

constexpr int DEC_CTAS = 152;   // one per SM: the ring takes an SM's shared memory

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
  p.ctas = DEC_CTAS;
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
  auto kernel = attn_decode_kernel<IO, D>;
  static int opted_in[64] = {};
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !opted_in[dev]) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)C::SMEM)) != cudaSuccess)
      return e;
    if (dev >= 0 && dev < 64) opted_in[dev] = 1;
  }
  kernel<<<p.ctas, DEC_THREADS, C::SMEM, s>>>(p, kmap, vmap);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  attn_merge_kernel<IO, D>
      <<<(unsigned)(a.total_q * a.h_kv * p.subs), MERGE_THREADS, 0, s>>>(p);
  return cudaGetLastError();
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
  return splits * n * h_q + (2 * DEC_CTAS + (splits > 0 ? items : 0)) * rows;
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
