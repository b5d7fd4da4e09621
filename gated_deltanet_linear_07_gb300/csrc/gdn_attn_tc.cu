// gdn_attn_tc.cu -- attention of many query rows over the same keys on the
// tensor cores: causal attention over packed prompts (gdn_attn_prefill), and
// the pass of gdn_attn_decode over a prefix that the whole batch shares.
//
// For a block of 128 query rows per CTA and blocks of 128 keys, one pass:
//   S = Q K^T,  m' = max(m, rowmax S),  P = 2^(c (S - m')),  c = scale log2 e
//   l = l 2^(c (m - m')) + rowsum P,    O = O 2^(c (m - m')) + P V,
// and o = O / l at the end.  S and O live in tensor memory (fp32); P goes
// back there in the I/O type as the A operand of the second product.  The
// reference maximum m may lag behind the true one by up to 2^LAG_LOG2 (WeightRange):
// P is then larger than one but the quotient is the same, and O is rescaled
// only when a row really passes that, which is rare after the first blocks.
//
// Rows: a key/value head's query heads are packed with the tokens, so that
// one block of 128 rows covers 128 / gp tokens x gp heads (gp the largest
// power of two that divides the group) and every key block that is loaded
// serves gp heads at once.
//
// CTA pairs (CG = 2): the two CTAs of a cluster take 256 rows of the same
// key/value head and each loads one half of every K and V block; one
// tcgen05.mma.cta_group::2 works on both CTAs' tensor memories.  That halves
// both the bytes fetched from L2 per product and the operand bytes read from
// shared memory, which at head dim 256 would otherwise be the bound (128 keys
// x 256 channels x 2 operands = 128 KB per 2048 cycles of products).
//
// Warps: 0-7 softmax (warps w and w + 4 share 32 rows, 64 of a block's 128
// columns each), 8 the TMA loads, 9 the MMAs, 10 the order of work, 11-14 the output
// of packed prompts below head dim 256 (else the softmax warps').  K and V
// blocks run through one ring in the order in which the MMA warp consumes them:
// S is formed one or two blocks ahead of the product with V, so that the softmax
// of one block and the products of the others overlap.
//
// Work items (a row block of one head group) are the clusters of the grid; a
// running pair takes over items that have not been launched yet
// (clusterlaunchcontrol), so that the loads and first scores of its next item run
// under the last blocks and the output of this one.  Launched one by one, an item
// cost 12 us beside its blocks.  The heaviest items come first.
//
// Every wait is bounded.  A warp whose wait ran out hands nothing on any more and
// writes no output, so that the warps that depend on it run out too; what two warps
// or two CTAs do together (the row's maxima, the barriers of the end) they still do,
// and the pair leaves when its copies and products in flight have had time to end.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_attn.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace attn {

using namespace gdn::tc;

constexpr int BM = 128;            // query rows per CTA (tensor-memory lanes)
constexpr int BN = 128;            // keys per block
constexpr int WARP_LOAD = 8, WARP_MMA = 9, WARP_ORDER = 10, WARP_OUT = 11;
constexpr uint64_t BLOCK_NS = 8192;   // a key block takes a fifth of it: for waits that span items
constexpr uint32_t MISC_BYTES = 3072;
constexpr int MAX_RING = 8;

// The ring takes what shared memory is left, except that packed keys of head dim 256
// do better with four stages than with five (they come from L2, and a load that runs
// further ahead holds the next item's queries back: 4096 tokens 94 and 99 us); a
// prefix comes from HBM and wants them all.
template <int D, int CG, bool PREFIX>
struct TcCfg {
  // Output by warps of its own, while the next item's softmax begins: packed prompts of
  // 16 sequences with 32 + 8 heads of 128 372 -> 339 us, 40 of 125 tokens 50 -> 45.  At
  // head dim 256 four more warps of registers are all there is, and their output takes
  // longer than the softmax of a first block: 4096 gated tokens 90 us by the softmax
  // warps, 97 by these.
  static constexpr bool OUT_WARPS = !PREFIX && D < 256;
  static constexpr int THREADS = OUT_WARPS ? 480 : 352;
  static constexpr int ITEMS = OUT_WARPS ? 3 : 2;     // under way at a time
  static constexpr uint32_t SUMS = OUT_WARPS ? ITEMS * 2 * BM * 4 : 0;   // their row sums
  static constexpr uint32_t Q_BYTES = BM * D * 2;
  static constexpr uint32_t STAGE = BN * D * 2 / CG;
  static constexpr int FIT = (int)((232448u - MISC_BYTES - SUMS - Q_BYTES) / STAGE);
  static constexpr int MOST = D == 256 && !PREFIX ? 4 : MAX_RING;
  static constexpr int RING = FIT < MOST ? FIT : MOST;
  static constexpr uint32_t SMEM = MISC_BYTES + SUMS + Q_BYTES + RING * STAGE;
  static constexpr int NS = D == 256 ? 2 : 3;        // S buffers: 512 columns less O's
  static constexpr uint32_t TMEM_O = NS * BN;
};

// One work item, as the order warp hands it to the others.
struct TcItem {
  int32_t q0, len_q, k0, len_k;   // the sequence's queries and keys (totals stay 2^16
                                  // below 2^31, so that block ends fit too)
  int32_t tile;                   // row block of the pair within the sequence
  int32_t kvh, h0;                // key/value head, first packed query head
  int32_t split, first_block;     // prefix pass: which share of the keys
  int32_t blocks;                 // key blocks; < 0: no more items
};

struct __align__(16) TcShared {
  uint4 taken[2];        // answers of the launch control
  uint64_t full[MAX_RING], empty[MAX_RING];
  uint64_t q_full, q_empty, s_full[3], p_ready[3], o_done[3], o_free, v_tail[3], l_full[3];
  uint64_t item_full[3], item_empty[3], taken_full[2], taken_free;
  TcItem item[3];
  uint32_t tmem;
  uint32_t gave_up;      // a wait of the pair has run out
  int32_t tail_stage[3]; // ring stage of an item's last V block, where it passes the end
  uint32_t going[2][2][4];   // [turn][column half][quarter]: the warp goes on to the next item
  float red[2][2][BM];   // row maxima of the two column halves, two turns
};
static_assert(sizeof(TcShared) <= MISC_BYTES, "shared bookkeeping");

// ---- PTX: clusters and the pair forms of the tensor-core operations --------

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Arrive on another CTA's mbarrier.  What the two CTAs hand over lies in tensor
// memory, ordered by the tcgen05 fences, so a release at cluster scope (a memory
// barrier: it was the softmax warps' longest stall, 2.2 of 7.5 cycles per issue)
// is left to the one block whose V rows were cleared in shared memory.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
__device__ __forceinline__ void arrive_remote_release(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait; once one has run out (ok false) the later ones return at once.
__device__ __forceinline__ void wait_on(bool& ok, uint64_t* bar, uint32_t parity,
                                        uint64_t budget_ns) {
  if (ok) ok = mbar_wait(bar, parity, budget_ns);
}
// The same without suspending the warp: for the MMA warp, whose next products
// wait for nothing else.  All lanes together.
__device__ __forceinline__ void spin_on(bool& ok, uint64_t* bar, uint32_t parity,
                                        uint64_t budget_ns) {
  if (ok) ok = mbar_spin(bar, parity, budget_ns);
  ok = __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(e)
      :
      : "memory");
  return e != 0;
}
// The same for arrivals with a release at cluster scope.  All lanes together.
__device__ __forceinline__ void wait_on_cluster(bool& ok, uint64_t* bar, uint32_t parity,
                                                uint64_t budget_ns) {
  if (ok) {
    const uint64_t t0 = globaltimer_ns();
    while (!try_wait_cluster(smem_u32(bar), parity))
      if (globaltimer_ns() - t0 > budget_ns) {
        ok = false;
        break;
      }
  }
  ok = __all_sync(0xffffffffu, ok);
}
template <int CG>
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                           int c2, int c3, uint32_t cluster_bar) {
  if (CG == 2) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
        "r"(cluster_bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
        "r"(cluster_bar)
        : "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t* dst, uint32_t ncols) {
  if (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(dst)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, ncols);
    tmem_relinquish();
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t taddr, uint32_t ncols) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
  else
    tmem_dealloc(taddr, ncols);
}
template <int CG>
__device__ __forceinline__ void mma_ss_cg(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_ss(d, a, b, idesc, acc);
}
template <int CG>
__device__ __forceinline__ void mma_ts_cg(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_ts(d, a, b, idesc, acc);
}
// Arrive on `bar` of every CTA of the pair when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void commit_cg(uint64_t* bar) {
  if (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    mma_commit(bar);
}
// 32 consecutive columns of this thread's lane, without the wait.
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
}
// A whole 32-byte sector by one thread: rows are a thread each, so narrower
// stores would reach L2 as parts of sectors.
__device__ __forceinline__ void st_global_32b(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                              uint32_t e, uint32_t f, uint32_t g, uint32_t h) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                   __cvta_generic_to_global(p)),
               "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
               : "memory");
}
__device__ __forceinline__ void ld_global_32b(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                 "=r"(b.w)
               : "l"(__cvta_generic_to_global(p)));
}
// Without a branch, in the loop over the blocks (8192 tokens of 16 heads of 64: 167.9 us
// where the arrival knew of no condition, 168.0 so, 170.0 with a branch).
__device__ __forceinline__ void mbar_arrive_if(uint64_t* bar, bool yes) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"((uint32_t)yes)
      : "memory");
}
// Sets the word at this address of CTA c of the pair.
template <int CG>
__device__ __forceinline__ void tell_gave_up(uint32_t addr, uint32_t c) {
  if (CG == 2)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_cta(addr, c)), "r"(1u) : "memory");
  else
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(1u) : "memory");
}
__device__ __forceinline__ void pair_bar(int id) {   // the two warps that share 32 rows
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}

template <typename IO>
__host__ __device__ constexpr uint32_t idesc_io(int M, int N, bool b_mn);
template <>
__host__ __device__ constexpr uint32_t idesc_io<__nv_bfloat16>(int M, int N, bool b_mn) {
  return idesc_bf16(M, N, false, b_mn);
}
template <>
__host__ __device__ constexpr uint32_t idesc_io<__half>(int M, int N, bool b_mn) {
  return idesc_f16(M, N, false, b_mn);
}

// 32 columns of O of this thread's row on their way out: divided by l, gated.
template <typename IO>
__device__ __forceinline__ void put_32(IO* out, bool wide, const uint32_t (&o)[32], float l,
                                       float inv, bool gated, const Vec8<IO>* g8) {
#pragma unroll
  for (int k = 0; k < 32; k += 16) {
    Vec8<IO> ov[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = l == 0.f ? 0.f : __uint_as_float(o[k + 8 * v + e]) * inv;
      if (gated) {
        float g[8];
        g8[k / 8 + v].get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= gate_sigmoid(g[e]);
      }
      ov[v].set(f);
    }
    if (wide) {
      st_global_32b(out + k, ov[0].w.x, ov[0].w.y, ov[0].w.z, ov[0].w.w, ov[1].w.x, ov[1].w.y,
                    ov[1].w.z, ov[1].w.w);
    } else {
      ov[0].store(out + k);
      ov[1].store(out + k + 8);
    }
  }
}
// The same columns of the gate.  Rows are a thread each, so an access of a warp touches
// 32 lines whatever its width, and the load/store unit takes one a cycle: 32 bytes at a
// time where they are aligned.
template <typename IO>
__device__ __forceinline__ void get_32(const IO* gate, bool sectors, Vec8<IO>* g8) {
#pragma unroll
  for (int v = 0; v < 4; v += 2) {
    if (sectors) {
      ld_global_32b(gate + 8 * v, g8[v].w, g8[v + 1].w);
    } else {
      g8[v].load(gate + 8 * v);
      g8[v + 1].load(gate + 8 * v + 8);
    }
  }
}

// ---- the kernel ---------------------------------------------------------------

struct TcLaunch {
  GdnAttnArgs a;
  int32_t gp_shift;       // log2 of the query heads packed into a row block
  int32_t subs;           // groups of 2^gp_shift query heads per key/value head
  int32_t k_rows, v_rows; // rows of one K / V box
};

// Which sequence and which of its row blocks is row block j of the grid, counting
// from the last block of the last sequence: within a sequence the longest rows
// come first.  By one warp, which keeps its place between calls.
struct TileSearch {
  int base = -1;           // 32 sequences from here (counted from the last one), one to a lane
  int before = 0;          // row blocks of the sequences before them
  int q0, len_q, k0, len_k;   // this lane's sequence
  int nt, incl;               // its row blocks, and with those before it

  static __device__ __forceinline__ bool fits(const GdnAttnArgs& a, int b, int lo, int hi, int klo,
                                              int khi) {
    return hi >= lo && lo >= 0 && hi <= a.total_q && khi >= klo && klo >= 0 && khi <= a.total_kv &&
           (b > 0 || (lo == 0 && klo == 0)) &&
           (b < a.num_seqs - 1 || (hi == a.total_q && khi == a.total_kv));
  }
  // False in a lane whose sequence is not within the totals, in its order.
  __device__ bool load(const GdnAttnArgs& a, int tokens, int first) {
    const int lane = threadIdx.x & 31, b = a.num_seqs - 1 - first - lane;
    base = first;
    q0 = len_q = k0 = len_k = nt = 0;
    bool fine = true;
    if (b >= 0) {
      const int q1 = a.cu_q[b + 1], k1 = a.cu_kv[b + 1];
      q0 = a.cu_q[b];
      k0 = a.cu_kv[b];
      fine = fits(a, b, q0, q1, k0, k1);
      if (fine) {
        len_q = q1 - q0;
        len_k = k1 - k0;
        nt = (len_q + tokens - 1) / tokens;
      }
    }
    incl = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    return fine;
  }
  // Whether all sequences are; leaves the search at the first ones.
  __device__ bool check(const GdnAttnArgs& a, int tokens) {
    bool fine = load(a, tokens, 0);
#pragma unroll 8
    for (int b = a.num_seqs - 33 - (int)(threadIdx.x & 31); b >= 0; b -= 32)
      fine = fits(a, b, a.cu_q[b], a.cu_q[b + 1], a.cu_kv[b], a.cu_kv[b + 1]) && fine;
    return __all_sync(0xffffffffu, fine);
  }
  // False: there is no such block.
  __device__ bool find(const GdnAttnArgs& a, int tokens, int j, TcItem& it) {
    if (j < before) {
      before = 0;
      load(a, tokens, 0);
    }
    for (;;) {
      const int all = __shfl_sync(0xffffffffu, incl, 31);
      if (j < before + all) break;
      if (base + 32 >= a.num_seqs) return false;
      before += all;
      load(a, tokens, base + 32);
    }
    const int at = j - before;
    const int src = __ffs(__ballot_sync(0xffffffffu, at < incl)) - 1;
    const int n = __shfl_sync(0xffffffffu, nt, src), end = __shfl_sync(0xffffffffu, incl, src);
    it.tile = n - 1 - (at - (end - n));
    it.q0 = __shfl_sync(0xffffffffu, q0, src);
    it.len_q = __shfl_sync(0xffffffffu, len_q, src);
    it.k0 = __shfl_sync(0xffffffffu, k0, src);
    it.len_k = __shfl_sync(0xffffffffu, len_k, src);
    return true;
  }
};

// Asks for a cluster that has not been launched yet; the answer goes to the same
// place in both CTAs of a pair and reports to their barriers.
template <int CG>
__device__ __forceinline__ void take_cluster(uint32_t answer, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(answer),
        "r"(bar)
        : "memory");
  else
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
        "[%0], [%1];" ::"r"(answer),
        "r"(bar)
        : "memory");
}
// The taken cluster's first CTA, or -1.
__device__ __forceinline__ int taken_cluster(uint32_t answer) {
  uint32_t x, got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\tld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %1, 1, 0, p;\n\tmov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}\n"
      : "=r"(x), "=r"(got)
      : "r"(answer)
      : "memory");
  return got ? (int)x : -1;
}

template <typename IO, int D, int CG, bool PREFIX>
__global__ void __launch_bounds__(TcCfg<D, CG, PREFIX>::THREADS, 1)
    attn_tc_kernel(const __grid_constant__ TcLaunch p, const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
  using C = TcCfg<D, CG, PREFIX>;
  extern __shared__ __align__(1024) unsigned char smem[];
  TcShared* sh = reinterpret_cast<TcShared*>(smem);
  const GdnAttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // known to be the same in all lanes
  const uint32_t rank = CG == 2 ? cta_rank() : 0u;
  // [item in turn][column half][row]
  float(*sums)[2][BM] = reinterpret_cast<float(*)[2][BM]>(smem + MISC_BYTES);
  const uint32_t q_smem = smem_u32(smem) + MISC_BYTES + C::SUMS;
  const uint32_t ring = q_smem + C::Q_BYTES;
  // the per-sequence pass of a decode needs nothing of this one but its SMs
  if (PREFIX) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int gp = 1 << p.gp_shift;
  const int cta_tokens = BM >> p.gp_shift;
  const int heads = a.h_kv * p.subs;             // row groups that share a tile of tokens
  if (tid == 0) {
    for (int s = 0; s < C::RING; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&sh->s_full[s], 1);
      // its own eight warps, and in a pair's first CTA the other one's together
      mbar_init(&sh->p_ready[s], CG == 2 && rank == 0 ? 9 : 8);
      mbar_init(&sh->o_done[s], 1);
    }
    mbar_init(&sh->o_free, (C::OUT_WARPS ? 4 : 8) * CG);
    for (int s = 0; s < C::ITEMS; ++s) {
      mbar_init(&sh->v_tail[s], 1);
      mbar_init(&sh->item_full[s], 1);
      mbar_init(&sh->item_empty[s], C::OUT_WARPS ? 14 : 10);   // softmax, loads, MMAs, output
      mbar_init(&sh->l_full[s], 8);
    }
    mbar_init(&sh->taken_full[0], 1);
    mbar_init(&sh->taken_full[1], 1);
    mbar_init(&sh->taken_free, CG);
    sh->gave_up = 0;
    fence_mbar_init();
  }
  if (warp == WARP_MMA) tmem_alloc_cg<CG>(&sh->tmem, 512);
  // the sequences' places are looked up while the pair sets itself up (512 tokens of
  // 16 + 4 heads of 256: 13.3 us, looked up after it 14.8)
  TileSearch search;
  bool sequences_fit = true;
  if (!PREFIX && warp == WARP_ORDER) sequences_fit = search.check(a, cta_tokens * CG);
  if (warp == WARP_LOAD && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(
                     reinterpret_cast<uint64_t>(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap))
                 : "memory");
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  bool ok = (smem_u32(smem) & 1023u) == 0;
  constexpr int NS = C::NS, AHEAD = NS - 1;   // S blocks formed ahead of the products with V
  const uint64_t wait_ns = a.wait_ns;

  // Items as the other warps see them, one after the other.
  int at_item = 0;                  // buffer of the item, and the parity of its phase
  uint32_t item_turn = 0;
  auto step_item = [&]() {
    if (++at_item == C::ITEMS) {
      at_item = 0;
      item_turn ^= 1;
    }
  };
  auto next_item = [&](TcItem& it) {
    wait_on(ok, &sh->item_full[at_item], item_turn, wait_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    it = sh->item[at_item];
    return it.blocks >= 0;
  };
  auto item_over = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->item_empty[at_item]);
    step_item();
  };
  auto has_tail = [&](const TcItem& it) {        // the last block passes the keys' end
    return (it.first_block + it.blocks) * BN > it.len_k;
  };

  if (warp == WARP_ORDER) {
    // ---- the order of work: this cluster's own item, then taken ones ----
    int item = blockIdx.x / CG;
    // (alike in every CTA, and before any of them has been given an item)
    if (!sequences_fit) {
      if (lane == 0) set_status(a.d_status, GDN_DEV_BAD_CU_SEQLENS);
      item = -1;
    }
    int asked = 0;
    uint64_t items_ns = wait_ns;         // the longest items under way, and some more
    for (int k = 0; ok;) {
      bool there = item >= 0;
      TcItem it = {};
      if (there) {
        const int rest = item / heads, head = item - rest * heads;
        it.kvh = head / p.subs;
        it.h0 = it.kvh * (a.h_q / a.h_kv) + (head % p.subs) * gp;
        if (PREFIX) {
          it.tile = rest / a.splits;
          it.split = rest - it.tile * a.splits;
          it.len_q = (int32_t)a.total_q;
          it.len_k = (int32_t)a.shared_len;
          const int64_t all = (a.shared_len + BN - 1) / BN;
          it.first_block = (int)(all * it.split / a.splits);
          it.blocks = (int)(all * (it.split + 1) / a.splits) - it.first_block;
        } else {
          there = search.find(a, cta_tokens * CG, rest, it);
          if (there) {
            // the keys that the last token of the pair's rows sees
            const int last = min(it.len_q, (it.tile + 1) * CG * cta_tokens) - 1;
            const int seen = last + it.len_k - it.len_q + 1;
            it.blocks = seen > 0 ? (seen + BN - 1) / BN : 0;
          }
        }
      } else {
        it.blocks = -1;
      }
      if (there || item < 0) {
        // the first wait of each buffer is for nothing
        if (k >= C::ITEMS) wait_on(ok, &sh->item_empty[at_item], item_turn ^ 1, items_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          sh->item[at_item] = it;
          mbar_arrive(&sh->item_full[at_item]);
        }
        ++k;
        step_item();
        if (it.blocks > 0)
          items_ns = max(items_ns, wait_ns + (uint64_t)it.blocks * (C::ITEMS * BLOCK_NS));
        if (item < 0) break;
      }
      // The next one, once this item's buffer after next is free again: a pair
      // holds no more than the item it works on and one more.
      if (there && k >= C::ITEMS)
        wait_on(ok, &sh->item_empty[at_item], item_turn ^ 1, items_ns);
      const int s = asked & 1;
      if (rank == 0) {
        if (asked > 0) wait_on(ok, &sh->taken_free, (asked - 1) & 1, wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_expect_tx(&sh->taken_full[s], 16);
        if (rank == 0) take_cluster<CG>(smem_u32(&sh->taken[s]), smem_u32(&sh->taken_full[s]));
      }
      __syncwarp();
      wait_on(ok, &sh->taken_full[s], (asked >> 1) & 1, wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int first = taken_cluster(smem_u32(&sh->taken[s]));
      fence_async_smem();                       // read before the next answer lands there
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          arrive_remote_release(map_cta(smem_u32(&sh->taken_free), 0));
        else
          mbar_arrive(&sh->taken_free);
      }
      ++asked;
      item = first < 0 ? -1 : first / CG;
    }
  } else if (warp == WARP_LOAD) {
    // ---- TMA loads; in a pair every copy reports to the first CTA's barrier ----
    auto lead = [&](uint64_t* bar) {
      return CG == 2 ? map_cta(smem_u32(bar), 0) : smem_u32(bar);
    };
    int s = 0;                      // ring stage and the parity of its phase
    uint32_t phase = 0;
    int used = 0;                   // items with keys so far
    int tail_at = 0;                // where the next tail reports
    TcItem it;
    // In the cache a block's rows lie in pages: each lane brings one box of the block
    // (rows of one page, 64 channels) and looks its page up a block ahead.  (One
    // lane after the other with a lookup each held a pair to 45 GB/s per SM.)
    const int k_box = lane % (D / 64), k_row = lane / (D / 64) * p.k_rows;
    const int v_box = lane % (D / 64 / CG), v_row = lane / (D / 64 / CG) * p.v_rows;
    while (next_item(it)) {
      if (it.blocks > 0) {
        const int kvh = it.kvh, h0 = it.h0;
        const int tok0 = (it.tile * CG + (int)rank) * cta_tokens;
        const bool tail = has_tail(it);
        const int keys = PREFIX ? it.len_k : 0;
        auto page_at = [&](int pos) {
          int32_t page = PREFIX && pos < keys ? __ldg(a.cache.block_table + (pos >> a.page_shift)) : 0;
          if (PREFIX && (page < 0 || page >= a.cache.num_pages)) {
            set_status(a.d_status, GDN_DEV_BAD_PAGE);
            page = 0;
          }
          return page;
        };
        auto row_at = [&](int32_t page, int pos) {
          return (int)((((int64_t)page * a.h_kv + kvh) << a.page_shift) +
                       (pos & ((1 << a.page_shift) - 1)));
        };
        // rows of [t, t + n) that exist, in whole boxes
        auto rows_of = [&](int t, int n, int box_mask) {
          return !PREFIX || t + n <= keys ? n : max(0, keys - t + box_mask) & ~box_mask;
        };
        const int k_pos = it.first_block * BN + (int)rank * (BN / CG) + k_row;
        const int v_pos = it.first_block * BN + v_row;
        int32_t k_page = 0, v_page = 0;
        if (PREFIX && k_row < BN / CG) k_page = page_at(k_pos);
        if (PREFIX && v_row < BN) v_page = page_at(v_pos);
        auto room = [&]() {         // the stage's last user is through with it
          wait_on(ok, &sh->empty[s], phase ^ 1, wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          return ok;
        };
        auto next_stage = [&]() {
          if (++s == C::RING) {
            s = 0;
            phase ^= 1;
          }
        };
        for (int i = 0; i < it.blocks + AHEAD && ok; ++i) {
          if (i < it.blocks) {   // K block i: this CTA's share of its rows
            if (!room()) break;
            const int t = (it.first_block + i) * BN;
            constexpr int n = BN / CG;
            const uint32_t dst = ring + (uint32_t)s * C::STAGE;
            const uint32_t bar = lead(&sh->full[s]);
            if (rank == 0 && lane == 0) {
              int rows = 0;
              for (int c = 0; c < CG; ++c) rows += rows_of(t + c * n, n, p.k_rows - 1);
              mbar_expect_tx(&sh->full[s], (uint32_t)rows * D * 2);
            }
            __syncwarp();
            if (!PREFIX) {
              if (lane == 0)
                tma_load_4d<CG>(dst, &kmap, 0, it.k0 + t + (int)rank * n, 0, kvh, bar);
            } else if (k_row < n) {
              const int pos = k_pos + i * BN;
              if (pos < keys)
                tma_load_4d<CG>(dst + (uint32_t)(k_box * n + k_row) * 128u, &kmap, 0,
                                row_at(k_page, pos), k_box, 0, bar);
              k_page = page_at(i + 1 < it.blocks ? pos + BN : keys);
            }
            next_stage();
          }
          if (i == 0) {          // Q, once the last item's scores are all formed
            if (used > 0) wait_on(ok, &sh->q_empty, (used - 1) & 1, wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
              if (rank == 0) mbar_expect_tx(&sh->q_full, C::Q_BYTES * CG);
              tma_load_4d<CG>(q_smem, &qmap, 0, h0, it.q0 + tok0, 0, lead(&sh->q_full));
            }
          }
          if (i >= AHEAD) {      // V block i - AHEAD: this CTA's share of its channels
            if (!room()) break;
            if (a.withhold && blockIdx.x < CG && used == 0 && i == AHEAD) {   // (the test's)
              next_stage();
              continue;
            }
            const int t = (it.first_block + i - AHEAD) * BN;
            const uint32_t bytes = (uint32_t)rows_of(t, BN, p.v_rows - 1) * (D / CG) * 2;
            // a tail reports here: this CTA clears its rows past the end
            const bool own = tail && i == it.blocks + AHEAD - 1;
            uint64_t* const own_bar = &sh->v_tail[tail_at];
            const uint32_t dst = ring + (uint32_t)s * C::STAGE;
            const uint32_t bar = !own ? lead(&sh->full[s])
                                      : CG == 2 ? map_cta(smem_u32(own_bar), rank) : smem_u32(own_bar);
            if (lane == 0) {
              if (own) {
                sh->tail_stage[tail_at] = s;
                mbar_expect_tx(own_bar, bytes);
              }
              if (rank == 0) {
                if (own)
                  mbar_arrive(&sh->full[s]);   // nobody waits for it; the phase has to pass
                else
                  mbar_expect_tx(&sh->full[s], bytes * CG);
              }
            }
            __syncwarp();
            constexpr int kbs = D / 64 / CG;
            if (!PREFIX) {
              if (lane == 0)
                tma_load_4d<CG>(dst, &vmap, 0, it.k0 + t, (int)rank * kbs, kvh, bar);
            } else if (v_row < BN) {
              const int pos = v_pos + (i - AHEAD) * BN;
              if (pos < keys)
                tma_load_4d<CG>(dst + (uint32_t)(v_box * BN + v_row) * 128u, &vmap, 0,
                                row_at(v_page, pos), (int)rank * kbs + v_box, 0, bar);
              v_page = page_at(i - AHEAD + 1 < it.blocks ? pos + BN : keys);
            }
            next_stage();
          }
        }
        ++used;
        if (tail && ++tail_at == C::ITEMS) tail_at = 0;
      }
      if (!ok) break;
      item_over();
    }
  } else if (warp == WARP_MMA) {
    // ---- MMAs, for both CTAs of a pair ----
    // The whole warp walks through the loop and one elected lane issues: the
    // descriptors are then uniform values.  From a branch of one lane each MMA
    // took 60 to 100 cycles to issue, as long as it runs.
    constexpr uint32_t id_s = idesc_io<IO>(BM * CG, BN, false);
    constexpr uint32_t id_o = idesc_io<IO>(BM * CG, D, true);
    const uint64_t q_desc = sdesc_kmaj(q_smem, BM, 0);
    const uint64_t k_desc = sdesc_kmaj(ring, BN / CG, 0), v_desc = sdesc_mnmaj(ring, BN, 0);
    int s = 0;                      // ring stage and the parity of its phase
    uint32_t phase = 0;
    auto next_stage = [&]() {
      if (++s == C::RING) {
        s = 0;
        phase ^= 1;
      }
    };
    int sb = 0;                     // S buffer of the next scores
    auto scores = [&](bool last) {
      spin_on(ok, &sh->full[s], phase, wait_ns);
      if (!ok) return;
      tc_fence_after();
      const uint64_t kd = sdesc_add(k_desc, (uint32_t)s * C::STAGE);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ss_cg<CG>(tmem + (uint32_t)sb * BN,
                        sdesc_add(q_desc, (uint32_t)((ks >> 2) * BM * 128 + (ks & 3) * 32)),
                        sdesc_add(kd, (uint32_t)((ks >> 2) * (BN / CG) * 128 + (ks & 3) * 32)), id_s,
                        ks > 0 ? 1u : 0u);
        commit_cg<CG>(&sh->empty[s]);
        commit_cg<CG>(&sh->s_full[sb]);
        if (last) commit_cg<CG>(&sh->q_empty);
      }
      __syncwarp();
      next_stage();
      sb = sb == NS - 1 ? 0 : sb + 1;
    };
    int pb = 0;                     // buffer of the next weights, and its phase
    uint32_t turn = 0;
    int used = 0;
    TcItem it;
    while (next_item(it)) {
      if (it.blocks > 0 && rank == 0) {
        const bool tail = has_tail(it);
        spin_on(ok, &sh->q_full, used & 1, wait_ns);
        for (int i = 0; i < AHEAD && i < it.blocks && ok; ++i) scores(i == it.blocks - 1);
        for (int i = 0; i < it.blocks && ok; ++i) {
          if (i + AHEAD < it.blocks) scores(i + AHEAD == it.blocks - 1);
          const bool last = tail && i == it.blocks - 1;   // V's arrival is part of the weights' then
          if (!last) spin_on(ok, &sh->full[s], phase, wait_ns);
          // the last item's output has been read
          if (i == 0 && used > 0) spin_on(ok, &sh->o_free, (used - 1) & 1, wait_ns);
          if (last)
            wait_on_cluster(ok, &sh->p_ready[pb], turn, wait_ns);
          else
            spin_on(ok, &sh->p_ready[pb], turn, wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = sdesc_add(v_desc, (uint32_t)s * C::STAGE);
          const uint32_t pt = tmem + (uint32_t)pb * BN;
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < BN / 16; ++ks)
              mma_ts_cg<CG>(tmem + C::TMEM_O, pt + (uint32_t)((ks >> 2) * 64 + (ks & 3) * 8),
                            sdesc_add(vd, (uint32_t)(ks * 16 * 128)), id_o,
                            (i > 0 || ks > 0) ? 1u : 0u);
            commit_cg<CG>(&sh->empty[s]);
            commit_cg<CG>(&sh->o_done[pb]);
          }
          __syncwarp();
          next_stage();
          if (++pb == NS) {
            pb = 0;
            turn ^= 1;
          }
        }
        ++used;
      }
      if (CG == 2 && rank == 1) {
        // The second CTA's weights are reported by this warp, which has nothing else to
        // do: an arrival at the other CTA took each softmax warp 140 cycles.
        const uint32_t ready = map_cta(smem_u32(&sh->p_ready[0]), 0);
        const bool tail = has_tail(it);
        for (int i = 0; i < it.blocks && ok; ++i) {
          spin_on(ok, &sh->p_ready[pb], turn, wait_ns);
          if (!ok) break;
          if (lane == 0) {
            if (tail && i == it.blocks - 1)
              arrive_remote_release(ready + 8u * pb);
            else
              arrive_remote(ready + 8u * pb);
          }
          __syncwarp();
          if (++pb == NS) {
            pb = 0;
            turn ^= 1;
          }
        }
      }
      if (!ok) break;
      item_over();
    }
  } else if (C::OUT_WARPS && warp >= WARP_OUT) {
    // ---- output: o = O / l, gated; a warp has 32 rows, a thread one of them ----
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t o_at = tmem + ((uint32_t)(quarter * 32) << 16) + C::TMEM_O;
    const uint32_t freed = CG == 2 ? map_cta(smem_u32(&sh->o_free), 0) : 0u;
    const bool wide = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
    int nb = 0;               // S buffer of the item's first block, and the parity of its phase
    uint32_t turn = 0;
    TcItem it;
    while (next_item(it)) {
      const int h = it.h0 + (row & (gp - 1));
      const int tok = (it.tile * CG + (int)rank) * cta_tokens + (row >> p.gp_shift);
      const bool live = tok < it.len_q;
      const int64_t t = (int64_t)it.q0 + tok;
      const bool gated = a.gate.data && live;
      Vec8<IO> gv[C::OUT_WARPS ? D / 8 : 1];     // the gate's row comes in under the products
      if (gated) {
        const IO* gate = reinterpret_cast<const IO*>(a.gate.data) + t * a.gate.token_stride +
                         h * a.gate.head_stride;
        const bool sectors = (reinterpret_cast<uintptr_t>(gate) & 31u) == 0;
#pragma unroll
        for (int n = 0; n < (C::OUT_WARPS ? D : 0); n += 32) get_32(gate + n, sectors, gv + n / 8);
      }
      wait_on(ok, &sh->l_full[at_item], item_turn, wait_ns + (uint64_t)it.blocks * BLOCK_NS);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const float l = sums[at_item][0][row] + sums[at_item][1][row];
      if (it.blocks > 0) {
        // The last scores were formed after the product NS before them, so of the
        // products that report to one of the NS barriers only the last can be under way.
        const int last = nb + it.blocks - 1;
        wait_on(ok, &sh->o_done[last % NS], turn ^ ((last / NS) & 1), wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        turn ^= ((last + 1) / NS) & 1;
        nb = (last + 1) % NS;
        tc_fence_after();
      }
      const float inv = l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l;   // no key: zeros; NaN stays
      IO* out = reinterpret_cast<IO*>(a.o) + (t * a.h_q + h) * D;
#pragma unroll
      for (int n = 0; n < (C::OUT_WARPS ? D : 0); n += 32) {
        uint32_t o[32];
        if (it.blocks > 0) {
          tmem_ld32_nowait(o_at + n, o);
          tmem_wait_ld(o);
          if (n + 32 == D) {            // all of O is in registers: the next item may write it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (CG == 1 || rank == 0)   // the first CTA's own arrivals stay in it
                mbar_arrive(&sh->o_free);
              else
                arrive_remote(freed);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (live) put_32(out + n, wide, o, l, inv, gated, gv + n / 8);
      }
      item_over();
    }
  } else {
    // ---- softmax: warps w and w + 4 share rows 32 (w % 4) .. + 31 ----
    const int quarter = warp & 3, half = warp >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const float c = a.scale_log2;
    const uint32_t freed = CG == 2 ? map_cta(smem_u32(&sh->o_free), 0) : 0u;
    // the first CTA's own arrivals stay in it
    const bool local = CG == 1 || rank == 0;
    int b = -1;               // this block's S buffer, and the parity of its phase
    uint32_t turn = 1;
    int flip = 0;
    int tail_at = 0;          // where the next tail reports, and the parity of its phase
    uint32_t tail_turn = 0;
    const bool stumbles = a.withhold && blockIdx.x / CG == 1 && warp == 5;   // (the test's)
    uint32_t meet = 0;
    // The two warps of a row meet at a barrier in every block: they go on to an item
    // together or leave together, whichever's wait has run out.
    auto both_next = [&](TcItem& it) {
      wait_on(ok, &sh->item_full[at_item], item_turn, wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      meet ^= 1;
      if (lane == 0) sh->going[meet][half][quarter] = ok;
      pair_bar(1 + quarter);
      ok = ok && sh->going[meet][half ^ 1][quarter];
      if (!ok) return false;
      it = sh->item[at_item];
      return it.blocks >= 0;
    };
    TcItem it;
    while (both_next(it)) {
      const int blocks = it.blocks;
      const bool tail = has_tail(it) && blocks > 0;
      const int h = it.h0 + (row & (gp - 1));
      const int tok = (it.tile * CG + (int)rank) * cta_tokens + (row >> p.gp_shift);
      const bool live = tok < it.len_q;
      // how many keys this row sees; rows past the end follow the last one, so
      // that they ask for no mask of their own
      const int vt = live ? tok : it.len_q - 1;
      int lim;
      if (PREFIX) {   // all of the prefix, or none: a shorter row is not part of this pass
        lim = a.seq_lens[vt] < it.len_k ? 0 : it.len_k;
      } else {
        lim = vt + it.len_k - it.len_q + 1;   // causal: the queries are the last of the keys
        lim = lim < 0 ? 0 : lim;
      }
      int low = lim;   // the least of the warp's rows
      if (PREFIX) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
      } else {
        low = __shfl_sync(0xffffffffu, lim, 0);
      }
      if (stumbles) ok = false;
      float m = -INFINITY;      // reference maximum of the raw scores
      float l = 0.f;            // this thread's half of the row sum

      for (int i = 0; i < blocks; ++i) {
        const int last_b = b;
        const uint32_t last_turn = turn;
        b = b == NS - 1 ? 0 : b + 1;
        turn ^= b == 0;
        wait_on(ok, &sh->s_full[b], turn, wait_ns);
        if (!__all_sync(0xffffffffu, ok)) ok = false;
        tc_fence_after();
        const uint32_t st = tmem + lanes + (uint32_t)b * BN + (uint32_t)half * 64;
        uint32_t r0[32], r1[32];
        tmem_ld32_nowait(st, r0);
        tmem_ld32_nowait(st + 32, r1);
        tmem_wait_ld(r0);
        tmem_wait_ld(r1);
        const int key = (it.first_block + i) * BN + half * 64;
        if (low < key + 64) {
          const int seen = lim - key;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (k >= seen) r0[k] = 0xff800000u;
            if (k + 32 >= seen) r1[k] = 0xff800000u;
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          mx[0] = max3(mx[0], __uint_as_float(r0[k]), __uint_as_float(r0[k + 1]));
          mx[1] = max3(mx[1], __uint_as_float(r0[k + 2]), __uint_as_float(r0[k + 3]));
          mx[2] = max3(mx[2], __uint_as_float(r1[k]), __uint_as_float(r1[k + 1]));
          mx[3] = max3(mx[3], __uint_as_float(r1[k + 2]), __uint_as_float(r1[k + 3]));
        }
        float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        flip ^= 1;
        sh->red[flip][half][row] = mt;
        pair_bar(1 + quarter);      // (a warp that has given up still comes here)
        mt = fmaxf(mt, sh->red[flip][half ^ 1][row]);
        // both warps of a row see the same maxima and so decide alike
        const bool far = live && mt > m && (m == -INFINITY || (mt - m) * c > WeightRange<IO>::LAG_LOG2);
        if (__any_sync(0xffffffffu, far)) {
          // a row's reference follows from the row alone: the others of the warp keep
          // theirs (factor 1), and rows that are not there ask for nothing
          const float f = far ? fast_exp2((m - mt) * c) : 1.f;    // 0 for a first maximum
          m = far ? mt : m;
          if (i > 0) {
            // S(i) was formed after product i - NS, so of the products that report
            // to one of the NS barriers at most one is under way
            wait_on(ok, &sh->o_done[last_b], last_turn, wait_ns);
            if (!__all_sync(0xffffffffu, ok)) ok = false;
            tc_fence_after();
            const int cols = ok ? D / 2 : 0;   // else O may still be the last item's
#pragma unroll 1
            for (int n = 0; n < cols; n += 32) {
              uint32_t o[32];
              const uint32_t at = tmem + lanes + C::TMEM_O + (uint32_t)(half * (D / 2) + n);
              tmem_ld32_nowait(at, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st32(at, o);
            }
          }
          l *= f;
        }
        const float nm = weight_offset<IO>(m, c);
        const uint64_t c2 = pk(c, c), nm2 = pk(nm, nm);
        uint32_t w[32];
        uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          float e0, e1, e2, e3;
          unpk(fma2(pk(__uint_as_float(r0[k]), __uint_as_float(r0[k + 1])), c2, nm2), e0, e1);
          unpk(fma2(pk(__uint_as_float(r1[k]), __uint_as_float(r1[k + 1])), c2, nm2), e2, e3);
          e0 = fast_exp2(e0);
          e1 = fast_exp2(e1);
          e2 = fast_exp2(e2);
          e3 = fast_exp2(e3);
          sum[k / 2 % 2] = add2(sum[k / 2 % 2], pk(e0, e1));
          sum[2 + k / 2 % 2] = add2(sum[2 + k / 2 % 2], pk(e2, e3));
          w[k / 2] = pack2<IO>(e0, e1);
          w[16 + k / 2] = pack2<IO>(e2, e3);
        }
        float la, lb;
        unpk(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), la, lb);
        l += la + lb;
        // over this half's own scores, which are in registers by now
        tmem_st32(st, w);
        tmem_wait_st();
        const bool last = tail && i == blocks - 1;
        if (last) {
          // the rows of V past the end are someone else's, or nothing: clear them
          // (a barrier per item under way: the loads may be that far ahead)
          wait_on(ok, &sh->v_tail[tail_at], tail_turn, wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          const int from = ok ? it.len_k - (it.first_block + i) * BN : BN;
          // (ok: else tail_stage has not been written)
          const uint32_t vt2 = ring + (uint32_t)(ok ? sh->tail_stage[tail_at] : 0) * C::STAGE;
          constexpr int ATOMS = D / 64 / CG;
          for (int x = from * 8 + tid; x < BN * 8; x += 256)
#pragma unroll
            for (int at = 0; at < ATOMS; ++at)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                               vt2 + (uint32_t)(at * BN * 128 + x * 16)),
                           "r"(0)
                           : "memory");
          fence_async_smem();
        }
        tc_fence_before();
        const bool arrives = ok;
        __syncwarp();
        if (lane == 0) mbar_arrive_if(&sh->p_ready[b], arrives);
      }
      if (tail && ++tail_at == C::ITEMS) {
        tail_at = 0;
        tail_turn ^= 1;
      }

      if (C::OUT_WARPS) {       // the output warps do the rest
        if (ok) {
          sums[at_item][half][row] = l;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->l_full[at_item]);
        }
      } else {
        // ---- the end: o = O / l ----
        // the gate's row comes in under the last product
        const int64_t t = (int64_t)it.q0 + tok;
        constexpr int COLS = C::OUT_WARPS ? 0 : D / 2;
        Vec8<IO> gv[PREFIX || C::OUT_WARPS ? 1 : D / 16];
        const bool gated = !PREFIX && a.gate.data && live;
        if (gated) {
          const IO* gate = reinterpret_cast<const IO*>(a.gate.data) + t * a.gate.token_stride +
                           h * a.gate.head_stride + half * (D / 2);
          const bool sectors = (reinterpret_cast<uintptr_t>(gate) & 31u) == 0;
#pragma unroll
          for (int n = 0; n < (PREFIX ? 0 : COLS); n += 32) get_32(gate + n, sectors, gv + n / 8);
        }
        flip ^= 1;
        sh->red[flip][half][row] = l;
        pair_bar(1 + quarter);
        l += sh->red[flip][half ^ 1][row];
        if (blocks > 0) {
          wait_on(ok, &sh->o_done[b], turn, wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
        }
        if (!ok) continue;
        const float inv = l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l;   // no key: zeros; NaN stays
        IO* out = reinterpret_cast<IO*>(a.o) + (t * a.h_q + h) * D + half * (D / 2);
        const bool wide = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
        const int64_t slot =
            PREFIX ? ((int64_t)it.split * a.total_q + (live ? tok : 0)) * a.h_q + h : 0;
        if (PREFIX && live && half == 0) a.part_ml[slot] = make_float2(m * c, l);
#pragma unroll
        for (int n = 0; n < COLS; n += 32) {
          uint32_t o[32];
          const int col = half * (D / 2) + n;
          if (blocks > 0) {
            tmem_ld32_nowait(tmem + lanes + C::TMEM_O + (uint32_t)col, o);
            tmem_wait_ld(o);
            if (n + 32 == D / 2) {      // all of O is in registers: the next item may write it
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if (local)
                  mbar_arrive(&sh->o_free);
                else
                  arrive_remote(freed);
              }
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (PREFIX) {
            if (live && l != 0.f) {
              float* dst = a.part_o + slot * D + col;
#pragma unroll
              for (int k = 0; k < 32; k += 8)
                st_global_32b(dst + k, o[k], o[k + 1], o[k + 2], o[k + 3], o[k + 4], o[k + 5],
                              o[k + 6], o[k + 7]);
            }
          } else if (live) {
            put_32(out + n, wide, o, l, inv, gated, gv + (PREFIX ? 0 : n / 8));
          }
        }
      }
      if (ok) item_over();
    }
  }
  if (!ok) {
    set_status(a.d_status, GDN_DEV_WAIT_TIMEOUT);
    for (uint32_t c = 0; c < CG; ++c) tell_gave_up<CG>(smem_u32(&sh->gave_up), c);
  }
  __syncwarp();
  // nothing of the pair is still to arrive at the other's barriers
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  if (sh->gave_up) {
    // Copies, products and answers of the launch control may be in flight that nobody
    // waited for (a CTA's report to the other's barriers, in phases that will not end):
    // nothing new is asked for by now, and they end in microseconds.
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < GRACE_NS) __nanosleep(20000);
  }
  tc_fence_after();
  if (warp == WARP_MMA) tmem_dealloc_cg<CG>(tmem, 512);
}

// ---- host -------------------------------------------------------------------------

static cudaError_t encode(CUtensorMap* map, int io, const void* ptr, const cuuint64_t (&dims)[4],
                          const cuuint64_t (&strides)[3], const cuuint32_t (&box)[4]) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(gdn_tensor_map_encoder());
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r =
      enc(map, io == GDN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
          4, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Strides of axes of extent one are never used: any legal value does.
static cuuint64_t stride_bytes(int64_t elements, int64_t extent) {
  return extent > 1 ? (cuuint64_t)elements * 2 : 16;
}

template <typename IO, int D, int CG, bool PREFIX>
static cudaError_t launch_tc(const GdnAttnArgs& a, int io, cudaStream_t s) {
  using C = TcCfg<D, CG, PREFIX>;
  cudaError_t e = cudaSuccess;
  TcLaunch p;
  p.a = a;
  const int group = a.h_q / a.h_kv;
  p.gp_shift = 0;
  while ((group >> p.gp_shift) % 2 == 0 && p.gp_shift < 7) ++p.gp_shift;
  const int gp = 1 << p.gp_shift;
  p.subs = group / gp;
  const int cta_tokens = BM / gp;
  CUtensorMap qmap, kmap, vmap;
  {   // Q: (64 channels, head, token, 64-channel block): rows token-major, then heads
    const cuuint64_t dims[4] = {64, (cuuint64_t)a.h_q, (cuuint64_t)a.total_q, D / 64};
    const cuuint64_t str[3] = {stride_bytes(a.q.head_stride, a.h_q),
                               stride_bytes(a.q.token_stride, a.total_q), 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)gp, (cuuint32_t)cta_tokens, D / 64};
    if ((e = encode(&qmap, io, a.q.data, dims, str, box)) != cudaSuccess) return e;
  }
  if (PREFIX) {   // cache rows: (64 channels, row of the pool, 64-channel block, -)
    const cuuint64_t rows = (cuuint64_t)a.cache.num_pages * a.h_kv << a.page_shift;
    const cuuint64_t dims[4] = {64, rows, D / 64, 1};
    const cuuint64_t str[3] = {D * 2, 128, 16};
    const int page = 1 << a.page_shift;
    p.k_rows = page < BN / CG ? page : BN / CG;
    p.v_rows = page < BN ? page : BN;
    const cuuint32_t kbox[4] = {64, (cuuint32_t)p.k_rows, 1, 1};
    const cuuint32_t vbox[4] = {64, (cuuint32_t)p.v_rows, 1, 1};
    if ((e = encode(&kmap, io, a.cache.k, dims, str, kbox)) != cudaSuccess) return e;
    if ((e = encode(&vmap, io, a.cache.v, dims, str, vbox)) != cudaSuccess) return e;
  } else {        // packed: (64 channels, token, 64-channel block, head)
    const cuuint64_t rows = a.total_kv > 0 ? (cuuint64_t)a.total_kv : 1;   // none: never loaded
    const cuuint64_t dims[4] = {64, rows, D / 64, (cuuint64_t)a.h_kv};
    const cuuint64_t kstr[3] = {stride_bytes(a.k.token_stride, a.total_kv), 128,
                                stride_bytes(a.k.head_stride, a.h_kv)};
    const cuuint64_t vstr[3] = {stride_bytes(a.v.token_stride, a.total_kv), 128,
                                stride_bytes(a.v.head_stride, a.h_kv)};
    const cuuint32_t kbox[4] = {64, BN / CG, D / 64, 1};
    const cuuint32_t vbox[4] = {64, BN, D / 64 / CG, 1};
    p.k_rows = BN / CG;
    p.v_rows = BN;
    if ((e = encode(&kmap, io, a.k.data, dims, kstr, kbox)) != cudaSuccess) return e;
    if ((e = encode(&vmap, io, a.v.data, dims, vstr, vbox)) != cudaSuccess) return e;
  }
  auto kernel = attn_tc_kernel<IO, D, CG, PREFIX>;
  static int opted_in[64] = {};
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !opted_in[dev]) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)C::SMEM)) != cudaSuccess)
      return e;
    if (dev >= 0 && dev < 64) opted_in[dev] = 1;
  }
  const int64_t tokens = (int64_t)cta_tokens * CG;
  const int64_t tiles = PREFIX ? (a.total_q + tokens - 1) / tokens * a.splits
                               : a.total_q / tokens + a.num_seqs;   // sum of the rounded-up counts
  const int64_t grid = tiles * a.h_kv * p.subs * CG;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, qmap, kmap, vmap);
}

template <typename IO, bool PREFIX>
static cudaError_t launch_tc_d(const GdnAttnArgs& a, int io, cudaStream_t s) {
  // Head dim 64 has no pair form: half of its 64 value channels would not fill
  // a 128-byte operand row.
  switch (a.d) {
    case 64: return launch_tc<IO, 64, 1, PREFIX>(a, io, s);
    case 128: return launch_tc<IO, 128, 2, PREFIX>(a, io, s);
    default: return launch_tc<IO, 256, 2, PREFIX>(a, io, s);
  }
}

}  // namespace attn
}  // namespace gdn

cudaError_t gdn_launch_attn_prefill(const GdnAttnArgs& a, int io, cudaStream_t s) {
  using namespace gdn::attn;
  return io == GDN_BF16 ? launch_tc_d<__nv_bfloat16, false>(a, io, s)
                        : launch_tc_d<__half, false>(a, io, s);
}

// Row blocks x head groups of the prefix pass, and the CTAs of each.
static int64_t prefix_items(int h_q, int h_kv, int d, int n, int& cg) {
  cg = d == 64 ? 1 : 2;
  int gp = 1;
  while ((h_q / h_kv) % (2 * gp) == 0 && gp < 128) gp *= 2;
  const int64_t tokens = (int64_t)gdn::attn::BM / gp * cg;
  return ((n + tokens - 1) / tokens) * (h_q / gp);
}

// The keys of the prefix are cut so that two thirds of the SMs have a share, each
// of at least two blocks: the pass over the sequences' own keys starts on the
// other third at once.  (All SMs for the one, then all for the other: 75 us instead
// of 65 for 64 rows behind 32768 tokens with up to 1024 of their own, and a
// partial output costs h_q d floats per row to write and to merge.)
int gdn_attn_prefix_splits(int h_q, int h_kv, int d, int n, int64_t shared_len) {
  // one row alone shares nothing: its own pass covers the prefix too
  if (shared_len <= 0 || n <= 1) return 0;
  int cg;
  const int64_t items = prefix_items(h_q, h_kv, d, n, cg);
  const int64_t blocks = (shared_len + gdn::attn::BN - 1) / gdn::attn::BN;
  int64_t splits = (gdn::attn::PREFIX_SMS / cg) / items;
  if (splits > (blocks + 1) / 2) splits = (blocks + 1) / 2;
  if (splits < 1) splits = 1;
  return (int)splits;
}

int gdn_attn_prefix_ctas(int h_q, int h_kv, int d, int n, int64_t shared_len) {
  int cg;
  const int64_t items = prefix_items(h_q, h_kv, d, n, cg);
  const int64_t ctas = items * gdn_attn_prefix_splits(h_q, h_kv, d, n, shared_len) * cg;
  return ctas < gdn::attn::SMS ? (int)ctas : gdn::attn::SMS;
}

cudaError_t gdn_launch_attn_prefix(const GdnAttnArgs& a, int io, cudaStream_t s) {
  using namespace gdn::attn;
  return io == GDN_BF16 ? launch_tc_d<__nv_bfloat16, true>(a, io, s)
                        : launch_tc_d<__half, true>(a, io, s);
}
