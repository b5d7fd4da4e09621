// gdn_kv8.cu -- the paged cache held in 8 bits: new tokens go in (normed, rotated
// and quantised on the way), cached tokens come out packed, and the kept tokens
// of a sequence move to other pages.  (gdn_kv8_decode.cu is the attention.)
//
// A block is KV8_BLOCK = 16 tokens of one head; its largest value decides its scale, a
// power of two.  A number of t bits of mantissa and a floating point is rounded to
// the same relative error under any scale that keeps it out of the subnormals, so
// powers of two lose nothing, and a scale that grows (a later token with a larger
// value) divides what the block holds by a power of two: exactly but for the
// subnormals.  Everything here is bound by the bytes that it moves.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_attn_device.cuh"
#include "gdn_kv8.cuh"
#include "gdn_rope.cuh"

namespace gdn {
namespace attn {

// ---- which rows a CTA has ------------------------------------------------------

// Rows of one sequence that go to one block.
struct Run {
  int64_t t0;      // first row of the call
  int64_t place;   // its place in the sequence; < 0: padding rows
  int32_t b, rows;
};

// A sequence's rows of the call and the number of its runs.
struct SequenceRuns {
  int64_t c0, len, count;
  int32_t start;
  int r;           // the first row's slot in its block
  __device__ __forceinline__ SequenceRuns(const int32_t* cu, const int32_t* starts, int num_seqs, int b)
      : c0(0), len(0), count(0), start(0), r(0) {
    if (b >= num_seqs) return;
    c0 = cu[b];
    len = (int64_t)cu[b + 1] - c0;
    start = starts ? starts[b] : 0;
    r = start < 0 ? 0 : start % KV8_BLOCK;
    if (len > 0) count = (r + len + KV8_BLOCK - 1) / KV8_BLOCK;
  }
  __device__ __forceinline__ Run run(int b, int64_t i) const {
    const int64_t i0 = max(i * KV8_BLOCK - r, (int64_t)0), i1 = min(i * KV8_BLOCK - r + KV8_BLOCK, len);
    return {c0 + i0, start < 0 ? -1 : start + i0, b, (int32_t)(i1 - i0)};
  }
};

// Run number `index` of packed sequences, by the whole CTA (WARPS warps); false: there
// is none, or cu is not a sequence of ends (reported).  starts null: places count from
// 0.  The runs before it are counted sequence by sequence, in one pass over cu that
// checks it too.
template <int WARPS>
__device__ __forceinline__ bool find_run(const int32_t* cu, const int32_t* starts, int num_seqs,
                                         int64_t n, int64_t index, int32_t* d_status, Run& run) {
  __shared__ int64_t sums[WARPS];
  __shared__ Run found;
  if (!cu) {   // a row of its own for every sequence
    run = {index, (int64_t)starts[index], (int32_t)index, 1};
    return true;
  }
  if (threadIdx.x == 0) found.rows = 0;
  bool bad = cu[0] != 0 || cu[num_seqs] != n;
  int64_t seen = 0;
  for (int base = 0; base < num_seqs; base += 32 * WARPS) {
    const int b = base + threadIdx.x;
    const SequenceRuns s(cu, starts, num_seqs, b);
    bad |= s.len < 0;
    int64_t before;
    const int64_t all = block_scan(s.count, sums, WARPS, before);
    const int64_t mine = index - seen - before;
    if (mine >= 0 && mine < s.count) found = s.run(b, mine);
    seen += all;
  }
  if (__syncthreads_or(bad)) {
    if (index == 0 && threadIdx.x == 0) set_status(d_status, GDN_DEV_BAD_CU_SEQLENS);
    return false;
  }
  run = found;
  return run.rows > 0;
}

// Number of runs; < 0: cu is not a sequence of ends.
template <int WARPS>
__device__ __forceinline__ int64_t count_runs(const int32_t* cu, const int32_t* starts, int num_seqs,
                                              int64_t n, int64_t* sums) {
  bool bad = cu[0] != 0 || cu[num_seqs] != n;
  int64_t count = 0, before;
  for (int b = threadIdx.x; b < num_seqs; b += 32 * WARPS) {
    const SequenceRuns s(cu, starts, num_seqs, b);
    bad |= s.len < 0;
    count += s.count;
  }
  count = block_scan(count, sums, WARPS, before);
  return __syncthreads_or(bad) ? -1 : count;
}

// Page of a sequence's block that starts at or before `place` (uniform over the
// CTA); < 0: none, and reported.
__device__ __forceinline__ int64_t page_of(const gdn_kv8_cache& c, int page_shift, int b,
                                           int64_t place, int32_t* d_status) {
  const int64_t pg = place >> page_shift;
  if (pg >= c.pages_per_seq) {
    set_status(d_status, GDN_DEV_BAD_LENGTH);
    return -1;
  }
  const int32_t page = __ldg(c.block_table + (int64_t)b * c.pages_per_seq + pg);
  if (page < 0 || page >= c.num_pages) {
    set_status(d_status, GDN_DEV_BAD_PAGE);
    return -1;
  }
  return page;
}

// Most runs that n rows of num_seqs sequences can be: each may start and end inside a block.
static int64_t most_runs(int64_t n, int64_t num_seqs) {
  const int64_t most = n / KV8_BLOCK + 2 * num_seqs;
  return most < n ? most : n;
}

// ---- append --------------------------------------------------------------------

// A CTA has one run at a time, of up to 16 rows, and forms its rows' cosines and sines once for all
// the heads that it has of them (all, or a share where runs are few).  A tile
// is a run's rows of one head (q, k or v), by a team of threads: eight channels
// per lane, D / 8 lanes per row, the rows at their slots of the block, so that what
// the block held before lies in the lanes of its own slots.
//
// Two kernels of the same arithmetic: few rows are loaded straight into registers, their tiles
// spread over CTAs; many go through a ring of tiles that one warp keeps filled by TMA
// (16,384 tokens of 16 + 4 heads of 256: 82 us, 117 with loads into registers).
constexpr int APPEND_THREADS = 256, FEW_TEAM = 128;

template <int TEAM>
__device__ __forceinline__ void team_bar(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TEAM) : "memory");
}

template <int D, int TEAM>
struct AppendCfg {
  static constexpr int TEAMS = APPEND_THREADS / TEAM;
  static constexpr int N = KV8_BLOCK * (D / 8) / TEAM;   // rows of a lane
  static constexpr int CS = D / 2 * 3;                   // a slot's cosines, sines, negated sines
  static constexpr uint32_t ANGLES = KV8_BLOCK * CS * 4;
};

// What a CTA knows of its run.
struct RunPlace {
  Run run;
  int64_t page;    // < 0: nothing is stored
  int r, block;    // the first row's slot; the block's place in its page
  bool padding;
};
__device__ __forceinline__ RunPlace place_of(const GdnKv8AppendArgs& p, const Run& run) {
  RunPlace w;
  w.run = run;
  w.padding = run.place < 0;
  w.r = w.padding ? 0 : (int)(run.place % KV8_BLOCK);
  w.page = w.padding ? -1 : page_of(p.cache, p.r.page_shift, run.b, run.place, p.r.d_status);
  w.block = w.padding ? 0 : (int)(run.place & ((1 << p.r.page_shift) - 1)) / KV8_BLOCK;
  return w;
}

// The runs r0 .. r1 into places[0 ..].run, by the whole CTA (cu is known to be sound).
template <int WARPS>
__device__ __forceinline__ void find_runs(const int32_t* cu, const int32_t* starts, int num_seqs,
                                          int64_t r0, int64_t r1, int64_t* sums, RunPlace* places) {
  int64_t seen = 0;
  for (int base = 0; base < num_seqs && seen < r1; base += 32 * WARPS) {
    const int b = base + threadIdx.x;
    const SequenceRuns s(cu, starts, num_seqs, b);
    int64_t before;
    const int64_t all = block_scan(s.count, sums, WARPS, before);
    const int64_t first = seen + before;
    for (int64_t i = max(first, r0); i < min(first + s.count, r1); ++i) places[i - r0].run = s.run(b, i - first);
    seen += all;
  }
  __syncthreads();
}

// The rows' cosines and sines at their slots, by the first `threads` of the CTA.
template <typename IO, int D>
__device__ __forceinline__ void put_angles(const GdnRopeArgs& a, const RunPlace& w,
                                           const uint64_t* fraction, float* cs, int threads) {
  const int half = a.rot_dim / 2;
  if (half == 0) return;
  const int per = threads / half, u0 = threadIdx.x / half, i = threadIdx.x - u0 * half;
  if (u0 >= per) return;
  const int32_t* pos = a.positions + (a.axes.count ? a.axes.pair[i] * a.n : 0) + w.run.t0;
  for (int u = u0; u < w.run.rows; u += per)
    put_angle<IO, D>(cs + (w.r + u) * AppendCfg<D, FEW_TEAM>::CS, angle_place<D>(a.interleaved, i), pos[u],
                     fraction[i], a.rope_scale);
}

// A lane's weights of the norm that a tile's rows have.
__device__ __forceinline__ void load_weights(const GdnRopeArgs& a, int tile, int nq, int part,
                                             float4 (&wt)[2]) {
  const float* wp = tile < nq ? a.q_norm : tile < nq + a.h_kv ? a.k_norm : nullptr;
  if (!wp) return;
  wt[0] = __ldg(reinterpret_cast<const float4*>(wp + 8 * part));
  wt[1] = __ldg(reinterpret_cast<const float4*>(wp + 8 * part + 4));
}

// One tile's rows x (of slots slot0 .., others zeros), normed with the weights wt, rotated and stored; by a team (the block's
// largest value passes through red).  live: false leaves the stores out.
template <typename IO, int D, int TEAM>
__device__ __forceinline__ void append_tile(const GdnKv8AppendArgs& p, const RunPlace& w,
                                            const LanePlace<D>& at, int tile, int nq, int slot0,
                                            int team, const float* cs, float (&red)[TEAM / 32],
                                            const float4 (&wt)[2], const Vec8<IO> (&x)[AppendCfg<D, TEAM>::N],
                                            bool live) {
  constexpr int N = AppendCfg<D, TEAM>::N, CS = AppendCfg<D, TEAM>::CS;
  const GdnRopeArgs& a = p.r;
  const int tt = threadIdx.x % TEAM, lane = threadIdx.x & 31;
  const Run& run = w.run;
  const int r = w.r;
  const bool is_q = tile < nq, is_v = tile >= nq + a.h_kv;
  const int head = is_q ? tile : is_v ? tile - nq - a.h_kv : tile - nq;
  uint64_t y[N][4];
  if (is_v) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float f[8];
      x[u].get(f);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[u][i] = pk(f[2 * i], f[2 * i + 1]);
    }
  } else {
    norm_rotate_fp32<IO, D, N>(at, N, (is_q ? a.q_norm : a.k_norm) != nullptr, a.interleaved, a.rot_dim > 0, a.eps, wt,
                               cs + slot0 * CS, x, y);
  }
  // the packed rows
  IO* out = reinterpret_cast<IO*>(is_q ? a.q_out : is_v ? nullptr : a.k_out);
  if (out && live) {
    const int heads = is_q ? a.h_q : a.h_kv;
    out += (run.t0 * heads + head) * D + 8 * at.part;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int row = slot0 + u - r;
      if (row < 0 || row >= run.rows) continue;
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) unpk(y[u][i], f[2 * i], f[2 * i + 1]);
      Vec8<IO> v;
      v.set(f);
      if (w.padding) v.w = make_uint4(0, 0, 0, 0);
      v.store(out + (int64_t)row * heads * D);
    }
  }
  if (is_q || w.page < 0) return;   // the same for the whole team
  const int64_t first = (w.page * a.h_kv + head) << a.page_shift;
  float* sp = (is_v ? p.cache.v_scale : p.cache.k_scale) + first / KV8_BLOCK + w.block;
  unsigned char* codes = reinterpret_cast<unsigned char*>(is_v ? p.cache.v : p.cache.k) +
                         (first + w.block * KV8_BLOCK) * D + 8 * at.part;
  const float held = r > 0 ? *sp : -1.f;   // < 0: the block begins here
  // (rows outside the run are zeros; a maximum passes over NaN)
  float top = 0.f;
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f0, f1;
      unpk(y[u][i], f0, f1);
      top = max3(top, fabsf(f0), fabsf(f1));
    }
  auto over_team = [&] {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) red[tt >> 5] = top;
    team_bar<TEAM>(team);
#pragma unroll
    for (int i = 0; i < TEAM / 32; ++i) top = fmaxf(top, red[i]);
  };
  over_team();
  if (top == INFINITY) {   // an Inf is stored as NaN and has no part in the scale; the whole team
    top = 0.f;
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f0, f1;
        unpk(y[u][i], f0, f1);
        f0 = fabsf(f0) == INFINITY ? NAN : f0;
        f1 = fabsf(f1) == INFINITY ? NAN : f1;
        y[u][i] = pk(f0, f1);
        top = max3(top, fabsf(f0), fabsf(f1));
      }
    team_bar<TEAM>(team);   // all have read red
    over_team();
  }
  if (!live) return;
  const int e = kv8_exponent(top);
  float scale = pow2(e), inv = pow2(-e);
  if (kv8_scale_ok(held)) {
    if (held >= scale) {
      scale = held;
      inv = 1.0f / held;
    } else {   // what the block holds already, at the new scale (zeros, where it stood for zeros)
      const float f = held * inv;
#pragma unroll
      for (int u = 0; u < N; ++u)
        if (slot0 + u < r) {
          uint2* c = reinterpret_cast<uint2*>(codes + (slot0 + u) * D);
          const uint2 old = *c;
          const float4 lo = from_e4m3x4(old.x), hi = from_e4m3x4(old.y);
          *c = make_uint2(to_e4m3x4(lo.x * f, lo.y * f, lo.z * f, lo.w * f),
                          to_e4m3x4(hi.x * f, hi.y * f, hi.z * f, hi.w * f));
        }
    }
  }
  if (tt == 0) *sp = scale;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int row = slot0 + u - r;
    if (row < 0 || row >= run.rows) continue;
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpk(mul2(y[u][i], pk(inv, inv)), f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint2*>(codes + (slot0 + u) * D) = make_uint2(
        to_e4m3x4(f[0], f[1], f[2], f[3]), to_e4m3x4(f[4], f[5], f[6], f[7]));
  }
}

template <typename IO, int D>
__global__ void __launch_bounds__(APPEND_THREADS)
    kv8_append_kernel(const __grid_constant__ GdnKv8AppendArgs p) {
  constexpr int TEAM = FEW_TEAM, N = AppendCfg<D, TEAM>::N, TEAMS = AppendCfg<D, TEAM>::TEAMS;
  extern __shared__ __align__(16) float cs[];     // [slot][cosines, sines, negated sines]
  __shared__ uint64_t fraction[D / 2];
  __shared__ float red[2][TEAMS][TEAM / 32];      // of every other tile: one barrier per tile
  const GdnRopeArgs& a = p.r;
  const int tid = threadIdx.x, team = tid / TEAM, tt = tid % TEAM;
  pdl_wait();
  for (int i = tid; i < a.rot_dim / 2; i += APPEND_THREADS) fraction[i] = turn_fraction(a.inv_freq[i]);
  Run run;
  if (!find_run<APPEND_THREADS / 32>(p.cu, p.starts, p.num_seqs, a.n, blockIdx.x, a.d_status, run))
    return;
  __syncthreads();
  const RunPlace w = place_of(p, run);
  put_angles<IO, D>(a, w, fraction, cs, APPEND_THREADS);
  __syncthreads();

  const LanePlace<D> at(a);
  const int slot0 = tt / (D / 8) * N;          // of this lane's rows
  const int nq = a.q.data ? a.h_q : 0, tiles = nq + 2 * a.h_kv;
  const int step = TEAMS * gridDim.y;
  auto load = [&](int tile, Vec8<IO> (&x)[N]) {
    const gdn_view& v = tile < nq ? a.q : tile < nq + a.h_kv ? a.k : a.v;
    const int head = tile < nq ? tile : (tile - nq) % a.h_kv;
    const IO* src = reinterpret_cast<const IO*>(v.data) + run.t0 * v.token_stride +
                    head * v.head_stride + 8 * at.part;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int row = slot0 + u - w.r;
      if (row >= 0 && row < run.rows && !w.padding)
        x[u].load(src + row * v.token_stride);
      else
        x[u].w = make_uint4(0, 0, 0, 0);
    }
  };
  Vec8<IO> x[N];
  for (int tile = blockIdx.y * TEAMS + team, it = 0; tile < tiles; tile += step, ++it) {
    float4 wt[2] = {};
    load(tile, x);
    load_weights(a, tile, nq, at.part, wt);
    append_tile<IO, D, TEAM>(p, w, at, tile, nq, slot0, team, cs, red[it & 1][team], wt, x, true);
  }
}

// ---- many rows: a ring of tiles -------------------------------------------------

template <int D>
struct RingCfg {
  static constexpr uint32_t TILE = KV8_BLOCK * D * 2;
  // Four rows a lane: what is done once per tile and lane is as much as a row (16,384 tokens of
  // 16 + 16 heads of 64: 56 us, 85 with one row a lane).
  static constexpr int TEAM = D / 2;
  static constexpr int STAGES = D == 256 ? 8 : 16;
  static_assert(STAGES % (APPEND_THREADS / TEAM) == 0, "each stage is one team's");
  static constexpr uint32_t ANGLES = (AppendCfg<D, TEAM>::ANGLES + 127) / 128 * 128;
  static constexpr uint32_t SMEM = ANGLES + STAGES * TILE;
  static constexpr int PER_SM = 2, CTAS = SMS * PER_SM;
};
constexpr int RING_THREADS = APPEND_THREADS + 32, RING_WARPS = RING_THREADS / 32;
constexpr int RING_RUNS = 64;   // that are looked up at a time

// All runs' tiles form one line, which the CTAs share in equal parts: a run is a CTA's from
// one tile to another.
template <typename IO, int D>
__global__ void __launch_bounds__(RING_THREADS, RingCfg<D>::PER_SM)
    kv8_append_ring_kernel(const __grid_constant__ GdnKv8AppendArgs p,
                           const __grid_constant__ CUtensorMap qmap,
                           const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap) {
  using C = RingCfg<D>;
  using namespace gdn::tc;
  constexpr int TEAM = C::TEAM, N = AppendCfg<D, TEAM>::N, TEAMS = AppendCfg<D, TEAM>::TEAMS;
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ uint64_t fraction[D / 2];
  __shared__ float red[2][TEAMS][TEAM / 32];
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES];
  __shared__ int64_t sums[RING_WARPS];
  __shared__ RunPlace places[RING_RUNS];
  float* cs = reinterpret_cast<float*>(ring_smem);
  const uint32_t ring = smem_u32(ring_smem) + C::ANGLES;
  const GdnRopeArgs& a = p.r;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], TEAM / 32);
    }
    fence_mbar_init();
  }
  pdl_wait();
  for (int i = tid; i < a.rot_dim / 2; i += RING_THREADS) fraction[i] = turn_fraction(a.inv_freq[i]);
  const int nq = a.q.data ? a.h_q : 0, tiles = nq + 2 * a.h_kv;
  const int64_t runs = count_runs<RING_WARPS>(p.cu, p.starts, p.num_seqs, a.n, sums);
  if (runs < 0) {
    if (blockIdx.x == 0 && tid == 0) set_status(a.d_status, GDN_DEV_BAD_CU_SEQLENS);
    return;
  }
  const int64_t t_end = runs * tiles * (blockIdx.x + 1) / gridDim.x;
  bool ok = true;
  int j = 0;   // tiles so far
  for (int64_t t = runs * tiles * blockIdx.x / gridDim.x; t < t_end;) {
    const int64_t r0 = t / tiles, r1 = min((t_end + tiles - 1) / tiles, r0 + RING_RUNS);
    const int64_t stop = min(t_end, r1 * tiles);
    const int x0 = (int)(t - r0 * tiles), x1 = (int)(stop - r0 * tiles);   // tiles of these runs
    find_runs<RING_WARPS>(p.cu, p.starts, p.num_seqs, r0, r1, sums, places);
    if (tid < r1 - r0) places[tid] = place_of(p, places[tid].run);
    __syncthreads();
    if (warp == APPEND_THREADS / 32) {
      // ---- loads: a tile per box; rows past the run, and past the end as zeros, come along ----
      int tile = x0;
      const RunPlace* w = places;
      for (int x = x0; x < x1 && ok; ++x, ++j) {
        const int s = j % C::STAGES;
        if (j >= C::STAGES) ok = mbar_wait(&empty[s], (j / C::STAGES - 1) & 1, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0 && !(a.withhold && blockIdx.x == 0 && j == 0)) {   // (the test's)
          mbar_expect_tx(&full[s], C::TILE);
          const int head = tile < nq ? tile : tile < nq + a.h_kv ? tile - nq : tile - nq - a.h_kv;
          tma_box_at(ring + s * C::TILE, tile < nq ? &qmap : tile < nq + a.h_kv ? &kmap : &vmap, head,
                     (int)w->run.t0, &full[s]);
        }
        __syncwarp();
        if (++tile == tiles) {
          tile = 0;
          ++w;
        }
      }
    } else {
      const int team = tid / TEAM, tt = tid % TEAM;
      const LanePlace<D> at(a);
      const int slot0 = tt / (D / 8) * N;
      for (int tile = x0, left = x1, k = 0; left > 0; left -= tiles, tile = 0, ++k) {
        const RunPlace w = places[k];
        const int last = min(left, tiles);
        if (k > 0) asm volatile("bar.sync 15, %0;" ::"n"(APPEND_THREADS) : "memory");   // the run before is done with
        put_angles<IO, D>(a, w, fraction, cs, APPEND_THREADS);
        asm volatile("bar.sync 15, %0;" ::"n"(APPEND_THREADS) : "memory");
        for (; tile < last; ++tile, ++j) {
          if (j % TEAMS != team) continue;
          const int s = j % C::STAGES;
          float4 wt[2] = {};
          load_weights(a, tile, nq, at.part, wt);
          // (a wait that ran out keeps the barriers' counts: only the stores are left out)
          if (ok) ok = mbar_wait(&full[s], (j / C::STAGES) & 1, a.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          const IO* in = reinterpret_cast<const IO*>(ring_smem + C::ANGLES + s * C::TILE) + 8 * at.part;
          Vec8<IO> v[N];
#pragma unroll
          for (int u = 0; u < N; ++u) {
            const int row = slot0 + u - w.r;
            if (row >= 0 && row < w.run.rows)
              v[u].load(in + row * D);
            else
              v[u].w = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&empty[s]);
          append_tile<IO, D, TEAM>(p, w, at, tile, nq, slot0, team, cs, red[j / TEAMS & 1][team], wt, v, ok);
        }
      }
    }
    t = stop;
    __syncthreads();   // the places are free again, the angles too
  }
  // What is in flight lands before this CTA's memory is another's.
  if (warp == APPEND_THREADS / 32)
    for (int x = max(j - C::STAGES, 0); x < j; ++x)
      mbar_wait(&full[x % C::STAGES], (x / C::STAGES) & 1, GRACE_NS);
  if (!ok) set_status(a.d_status, GDN_DEV_WAIT_TIMEOUT);
}

template <typename IO, int D>
static cudaError_t launch_append_d(const GdnKv8AppendArgs& a, cudaStream_t s) {
  const int64_t runs = a.cu ? most_runs(a.r.n, a.num_seqs) : a.r.n;
  const int tiles = (a.r.q.data ? a.r.h_q : 0) + 2 * a.r.h_kv;
  // Whole blocks for the most part, and enough of them for all SMs.  (Replayed, one sequence, 64 channels
  // rotated, registers and ring: 2400 tokens of 16 + 4 heads of 256 22 and 24 us, 2600 22 and 29, 4000 30
  // and 30, 8000 52 and 46; 32 + 8 of 128 22 and 26, 26 and 31, 35 and 32, 57 and 48; 16 + 16 of 64 15 and
  // 17, 20 and 21, 29 and 22, 47 and 32.  They meet at 4000, 3500 and 2700 tokens, above this border.)
  if (a.r.n >= 8 * runs && runs >= SMS) {
    const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(gdn_tensor_map_encoder());
    if (!enc) return cudaErrorNotSupported;
    CUtensorMap map[3] = {};
    const gdn_view* views[3] = {&a.r.q, &a.r.k, &a.r.v};
    for (int i = 0; i < 3; ++i) {   // rows of a view as (channel, head, token); a box: a tile
      if (!views[i]->data) continue;
      const int heads = i ? a.r.h_kv : a.r.h_q;
      const cuuint64_t dims[3] = {D, (cuuint64_t)heads, (cuuint64_t)a.r.n};
      // the stride of an axis of extent one is never used: any legal value does
      const cuuint64_t strides[2] = {heads > 1 ? (cuuint64_t)views[i]->head_stride * 2 : 16,
                                     (cuuint64_t)views[i]->token_stride * 2};
      const cuuint32_t box[3] = {D, 1, KV8_BLOCK};
      const cuuint32_t estr[3] = {1, 1, 1};
      if (enc(&map[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(views[i]->data), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    }
    auto kernel = kv8_append_ring_kernel<IO, D>;
    static int opted_in[64] = {};
    int dev = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !opted_in[dev]) {
      if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)RingCfg<D>::SMEM)) != cudaSuccess)
        return e;
      if (dev >= 0 && dev < 64) opted_in[dev] = 1;
    }
    const unsigned ctas = (unsigned)(runs < RingCfg<D>::CTAS ? runs : RingCfg<D>::CTAS);
    return launch_behind(kernel, dim3(ctas), RING_THREADS, RingCfg<D>::SMEM, s, a, map[0], map[1], map[2]);
  }
  // few runs: their tiles over several CTAs
  constexpr int TEAMS = AppendCfg<D, FEW_TEAM>::TEAMS;
  const int most = (tiles + TEAMS - 1) / TEAMS;
  int split = 1;
  while (split < most && runs * split < 8 * SMS) ++split;
  const size_t smem = a.r.rot_dim > 0 ? AppendCfg<D, FEW_TEAM>::ANGLES : 0;
  return launch_behind(kv8_append_kernel<IO, D>, dim3((unsigned)runs, (unsigned)split), APPEND_THREADS,
                       smem, s, a);
}

// ---- gather ---------------------------------------------------------------------

constexpr int GATHER_THREADS = 256;

// Sixteen numbers of a row: one 16-byte load, two 16-byte stores.
template <typename IO>
__device__ __forceinline__ void put_sixteen(IO* dst, uint4 w, float scale) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = from_e4m3x4(u[2 * h + i]);
      f[4 * i] = v.x * scale;
      f[4 * i + 1] = v.y * scale;
      f[4 * i + 2] = v.z * scale;
      f[4 * i + 3] = v.w * scale;
    }
    Vec8<IO> o;
    o.set(f);
    o.store(dst + 8 * h);
  }
}

template <typename IO, int D>
__global__ void __launch_bounds__(GATHER_THREADS)
    kv8_gather_kernel(const __grid_constant__ GdnKv8GatherArgs p) {
  constexpr int PARTS = D / 16, TILE = KV8_BLOCK * PARTS, UNROLL = 4;
  pdl_wait();
  Run run;
  if (!find_run<GATHER_THREADS / 32>(p.cu, nullptr, p.num_seqs, p.total, blockIdx.x, p.d_status,
                                     run))
    return;
  const int64_t page = page_of(p.cache, p.page_shift, run.b, run.place, p.d_status);
  const int block = (int)(run.place & ((1 << p.page_shift) - 1)) / KV8_BLOCK;
  const int kinds = (p.k_out ? 1 : 0) + (p.v_out ? 1 : 0), all = TILE * p.h_kv * kinds;
  for (int base = threadIdx.x; base < all; base += UNROLL * GATHER_THREADS) {
    uint4 w[UNROLL];
    float scale[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int i = base + j * GATHER_THREADS, tile = i / TILE, row = i % TILE / PARTS;
      w[j] = make_uint4(0, 0, 0, 0);
      scale[j] = 0.f;
      if (i >= all || row >= run.rows || page < 0) continue;
      const int head = tile % p.h_kv;
      const bool is_v = !p.k_out || tile >= p.h_kv;
      const int64_t first = (page * p.h_kv + head) << p.page_shift;
      w[j] = __ldcs(reinterpret_cast<const uint4*>(
          reinterpret_cast<const unsigned char*>(is_v ? p.cache.v : p.cache.k) +
          (first + block * KV8_BLOCK + row) * D + i % PARTS * 16));
      scale[j] = __ldg((is_v ? p.cache.v_scale : p.cache.k_scale) + first / KV8_BLOCK + block);
    }
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int i = base + j * GATHER_THREADS, tile = i / TILE, row = i % TILE / PARTS;
      if (i >= all || row >= run.rows) continue;
      const int head = tile % p.h_kv;
      const bool is_v = !p.k_out || tile >= p.h_kv;
      put_sixteen<IO>(reinterpret_cast<IO*>(is_v ? p.v_out : p.k_out) +
                          ((run.t0 + row) * p.h_kv + head) * D + i % PARTS * 16,
                      w[j], scale[j]);
    }
  }
}

template <typename IO, int D>
static cudaError_t launch_gather_d(const GdnKv8GatherArgs& a, cudaStream_t s) {
  return launch_behind(kv8_gather_kernel<IO, D>, dim3((unsigned)most_runs(a.total, a.num_seqs)),
                       GATHER_THREADS, 0, s, a);
}

// ---- evict ----------------------------------------------------------------------

constexpr int SELECT_THREADS = 1024, SELECT_WARPS = SELECT_THREADS / 32;
constexpr int SELECT_BINS = 2 * SELECT_THREADS;   // of eleven bits
constexpr int SELECT_KEYS = 48 * 1024;            // weights, at most, that stay in shared memory

// A weight's rank as an unsigned number from 1 to 2^31: bits of a float that is not negative,
// and 1.  Places that stay in any case are above all, places past the end below.
constexpr uint32_t RANK_SURE = 0xffffffffu, RANK_NONE = 0;
__device__ __forceinline__ uint32_t weight_rank(float w) {
  return (__float_as_uint(fmaxf(w, 0.f)) & 0x7fffffffu) + 1;   // NaN: as 0
}

__device__ __forceinline__ int64_t evict_len(const GdnKv8EvictArgs& p, int b) {
  const int64_t cap = (int64_t)p.from.pages_per_seq << p.page_shift;
  int64_t len = max(p.seq_lens[b], 0);
  if (len > cap) {
    set_status(p.d_status, GDN_DEV_BAD_LENGTH);
    len = cap;
  }
  return len;
}

struct __align__(16) SelectShared {
  uint32_t hist[SELECT_BINS];
  uint64_t sums[SELECT_WARPS];
  uint32_t sums32[2][SELECT_WARPS];
  uint32_t digit, above;
};

// Sum of v over the threads below this one, as block_scan, whose sum over the warps is one
// thread's work here times 32.  Calls that follow each other take turns of `sums`.
template <typename T>
__device__ __forceinline__ T select_scan(T v, T* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  const T mine = sums[lane];
  T sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  return __shfl_sync(0xffffffffu, sum - mine, warp) + incl - v;
}
static_assert(SELECT_WARPS == 32, "a lane per warp");

// The places of one sequence and head that are kept.  The rank of the last one that the middle
// keeps is found digit by digit, eleven bits at a time from the top (a histogram of those that
// share the digits so far), then one ordered pass writes the places: all above that rank and, of
// those equal to it, the lowest.  The ranks stay in shared memory, or are formed again for each
// pass where they do not fit.  A chain of latencies and of issue, the instructions' own
// arrival included: each runs once, so the loops are short, four places at a time
// and not unrolled (in registers, unrolled: 24 us where this takes 8, one sequence of 5120;
// with the middle's borders looked at in every pass and the scans of a CTA between them 10, and
// 19 for 15 of 32 sequences of up to 16384).
__global__ void __launch_bounds__(SELECT_THREADS, 2)
    kv8_select_kernel(const __grid_constant__ GdnKv8EvictArgs p, int room) {
  extern __shared__ __align__(16) uint32_t ranks[];   // [room]
  __shared__ SelectShared sh;
  pdl_wait();
  pdl_launch();
  const int tid = threadIdx.x;
  const int b = blockIdx.x / p.h_kv, j = blockIdx.x % p.h_kv;
  const int64_t cap = (int64_t)p.from.pages_per_seq << p.page_shift;
  const int64_t cap_to = (int64_t)p.to.pages_per_seq << p.page_shift;
  // (places are counted without a sign: a block table row holds fewer than 2^31 - 65536)
  const uint32_t len = (uint32_t)evict_len(p, b), now = min(len, (uint32_t)p.keep);
  const float* w = p.weights + ((int64_t)b * p.h_kv + j) * cap;
  float* w_out = p.weights_out ? p.weights_out + ((int64_t)b * p.h_kv + j) * cap_to : nullptr;
  int32_t* kept = p.kept + ((int64_t)b * p.h_kv + j) * p.keep;
  if (j == 0 && tid == 0) p.new_lens[b] = (int32_t)now;
  if (len <= (uint32_t)p.keep) {
    for (uint32_t i = tid; i < len; i += SELECT_THREADS) {
      kept[i] = (int32_t)i;
      if (w_out) w_out[i] = w[i];
    }
  } else {
    const uint32_t lo = p.first, hi = len - p.last;   // the middle; longer than what it keeps
    const bool here = len <= (uint32_t)room;
    // of places i .. i + 3, i a multiple of 4 below len (rows of weights are a multiple of 16 long)
    auto form = [&](uint32_t i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(w + i));
      const float x[4] = {v.x, v.y, v.z, v.w};
      uint32_t k[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        k[e] = i + e >= len ? RANK_NONE : i + e < lo || i + e >= hi ? RANK_SURE : weight_rank(x[e]);
      return make_uint4(k[0], k[1], k[2], k[3]);
    };
    if (here)
#pragma unroll 2
      for (uint32_t i = 4 * tid; i < len; i += 4 * SELECT_THREADS)
        *reinterpret_cast<uint4*>(ranks + i) = form(i);
    auto four = [&](uint32_t i) { return here ? *reinterpret_cast<const uint4*>(ranks + i) : form(i); };
    uint32_t want = (uint32_t)(p.keep - p.first - p.last);   // of those that share the digits so far
    uint32_t border = want > 0 ? 0 : RANK_SURE - 1;
#pragma unroll 1
    for (int pass = 0; pass < 3 && want > 0; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      sh.hist[2 * tid] = sh.hist[2 * tid + 1] = 0;
      __syncthreads();
#pragma unroll 1
      for (uint32_t i = 4 * tid; i < len; i += 4 * SELECT_THREADS) {
        const uint4 v = four(i);
        const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t digits = (k[e] ^ border) >> shift;   // (the border's own are still 0)
          if (digits >> bits == 0) atomicAdd(&sh.hist[digits], 1u);
        }
      }
      __syncthreads();
      // from the top: this thread's two bins (in the first pass those above 1024 are of RANK_SURE)
      const int bin = SELECT_BINS - 2 - 2 * tid;
      const bool real = pass > 0 || bin <= 1024;
      const uint32_t upper = real ? sh.hist[bin + 1] : 0, lower = real ? sh.hist[bin] : 0;
      const uint32_t before = select_scan(upper + lower, sh.sums32[pass & 1]);
      if (before < want && before + upper + lower >= want) {
        const bool first = before + upper >= want;
        sh.digit = bin + (first ? 1 : 0);
        sh.above = before + (first ? 0 : upper);
      }
      __syncthreads();
      border |= sh.digit << shift;
      want -= sh.above;
    }
    __syncthreads();
    // In order: each warp has a stretch of places.  Of each stretch the numbers of those above
    // the border (upper half) and of those equal to it, then the places behind what the warps
    // before have, no warp waiting for another.
    const int warp = tid >> 5, lane = tid & 31;
    const uint32_t per = (len + 4 * SELECT_THREADS - 1) / (4 * SELECT_THREADS) * 128;
    const uint32_t i_first = min(len, warp * per), i_end = min(len, i_first + per);
    auto count = [&](const uint4& k) {
      return (uint32_t)((k.x > border) + (k.y > border) + (k.z > border) + (k.w > border)) << 16 |
             (uint32_t)((k.x == border) + (k.y == border) + (k.z == border) + (k.w == border));
    };
    uint64_t mine = 0;
#pragma unroll 1
    for (uint32_t i = i_first + 4 * lane; i < i_end; i += 128) {
      const uint32_t c = count(four(i));
      mine += ((uint64_t)(c >> 16) << 32) | (c & 0xffffu);
    }
    uint64_t seen = __shfl_sync(0xffffffffu, select_scan(mine, sh.sums), 0);
    const bool copy = w_out != nullptr;
    uint32_t i = i_first + 4 * lane;
    float4 next = copy && i < i_end ? __ldg(reinterpret_cast<const float4*>(w + i)) : make_float4(0, 0, 0, 0);
#pragma unroll 1
    for (uint32_t base = i_first; base < i_end; base += 128, i += 128) {
      const uint4 v = i < i_end ? four(i) : make_uint4(RANK_NONE, RANK_NONE, RANK_NONE, RANK_NONE);
      const float x[4] = {next.x, next.y, next.z, next.w};
      if (copy && i + 128 < i_end) next = __ldg(reinterpret_cast<const float4*>(w + i + 128));
      const uint32_t k[4] = {v.x, v.y, v.z, v.w}, c = count(v);
      uint32_t incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      const uint32_t below = incl - c, all = __shfl_sync(0xffffffffu, incl, 31);
      uint32_t tied = (uint32_t)seen + (below & 0xffffu);
      uint32_t to = (uint32_t)(seen >> 32) + (below >> 16) + min(tied, want);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (k[e] > border || (k[e] == border && tied < want)) {
          kept[to] = (int32_t)(i + e);
          if (copy) w_out[to] = x[e];
          ++to;
        }
        tied += k[e] == border;
      }
      seen += ((uint64_t)(all >> 16) << 32) | (all & 0xffffu);
    }
  }
  for (uint32_t i = now + tid; i < (uint32_t)p.keep; i += SELECT_THREADS) kept[i] = -1;
  if (w_out)
    for (int64_t i = now + tid; i < cap_to; i += SELECT_THREADS) w_out[i] = 0.f;
}

constexpr int MOVE_WARPS = GdnKv8MoveGrid::WARPS, MOVE_BLOCKS = GdnKv8MoveGrid::BLOCKS;
static_assert(MOVE_BLOCKS * KV8_BLOCK <= 32 * MOVE_WARPS, "a thread per row");

// A CTA has some blocks of the new pages of one sequence and head.  Where their up to 16 kept rows
// each were is looked up by all threads at once, then a warp moves a block's keys or its values
// at a time.  (A look-up by each warp for its 16 rows, three dependent latencies for 4 KB: 85 us
// where this takes 70, 32 sequences of up to 16384 cut to half, 4 heads of 256.)
template <int D>
__global__ void __launch_bounds__(32 * MOVE_WARPS, D == 256 ? 4 : 5)
    kv8_move_kernel(const __grid_constant__ GdnKv8EvictArgs p, int blocks, int across) {
  constexpr int PARTS = D / 16, PASS = 32 / PARTS, N = KV8_BLOCK / PASS;   // rows of a pass, passes
  __shared__ int64_t rows[MOVE_BLOCKS * KV8_BLOCK], to_rows[MOVE_BLOCKS];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t item = blockIdx.x / across;
  const int b = (int)(item / p.h_kv), j = (int)(item % p.h_kv);
  const int block0 = (int)(blockIdx.x % across) * blocks;
  pdl_wait();   // the selection's places
  if (tid < blocks * KV8_BLOCK) {
    const int64_t i = (int64_t)block0 * KV8_BLOCK + tid;
    int64_t row = -1;
    const int32_t place = i < p.keep ? p.kept[item * p.keep + i] : -1;
    if (place >= 0) {
      const int64_t page = page_of(p.from, p.page_shift, b, place, p.d_status);
      if (page >= 0) row = ((page * p.h_kv + j) << p.page_shift) + (place & ((1 << p.page_shift) - 1));
    }
    rows[tid] = row;
    if (tid % KV8_BLOCK == 0) {   // (a block whose first row is none has none)
      const int64_t page = place >= 0 ? page_of(p.to, p.page_shift, b, i, p.d_status) : -1;
      to_rows[tid / KV8_BLOCK] = page < 0 ? -1 : ((page * p.h_kv + j) << p.page_shift) +
                                                     (i & ((1 << p.page_shift) - 1));
    }
  }
  __syncthreads();
  for (int unit = tid >> 5; unit < 2 * blocks; unit += MOVE_WARPS) {
    const bool is_v = unit & 1;
    const int64_t* const from = rows + (unit >> 1) * KV8_BLOCK;
    const int64_t to = to_rows[unit >> 1];
    const int64_t mine = from[lane % KV8_BLOCK];
    if (to < 0 || !__any_sync(0xffffffffu, mine >= 0)) continue;
    const unsigned char* src = reinterpret_cast<const unsigned char*>(is_v ? p.from.v : p.from.k);
    unsigned char* dst = reinterpret_cast<unsigned char*>(is_v ? p.to.v : p.to.k) + to * D;
    const float scale = mine >= 0 ? (is_v ? p.from.v_scale : p.from.k_scale)[mine / KV8_BLOCK] : 0.f;
    uint4 x[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int64_t at = from[u * PASS + lane / PARTS];
      if (at >= 0) x[u] = __ldcs(reinterpret_cast<const uint4*>(src + at * D + lane % PARTS * 16));
    }
    float top = scale;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ratio = top > 0.f ? scale / top : 1.f;
    const bool same = __all_sync(0xffffffffu, ratio == 1.f || mine < 0);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int s = u * PASS + lane / PARTS;
      if (!same) {
        const float f = __shfl_sync(0xffffffffu, ratio, s);
        uint32_t* v = reinterpret_cast<uint32_t*>(&x[u]);
        if (f != 1.f && from[s] >= 0)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 y = from_e4m3x4(v[e]);
            v[e] = to_e4m3x4(y.x * f, y.y * f, y.z * f, y.w * f);
          }
      }
      if (from[s] >= 0) *reinterpret_cast<uint4*>(dst + s * D + lane % PARTS * 16) = x[u];
    }
    if (lane == 0) (is_v ? p.to.v_scale : p.to.k_scale)[to / KV8_BLOCK] = top;
  }
}

template <int D>
static cudaError_t launch_move_d(const GdnKv8EvictArgs& a, cudaStream_t s) {
  const GdnKv8MoveGrid grid((int64_t)a.n * a.h_kv, a.keep);
  return launch_behind(kv8_move_kernel<D>, dim3((unsigned)grid.ctas), 32 * MOVE_WARPS, 0, s, a,
                       grid.blocks, (int)grid.across);   // (on its way while the selection ends)
}

template <typename IO>
static cudaError_t launch_append_io(const GdnKv8AppendArgs& a, cudaStream_t s) {
  return a.r.d == 64 ? launch_append_d<IO, 64>(a, s)
                     : a.r.d == 128 ? launch_append_d<IO, 128>(a, s) : launch_append_d<IO, 256>(a, s);
}
template <typename IO>
static cudaError_t launch_gather_io(const GdnKv8GatherArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_gather_d<IO, 64>(a, s)
                   : a.d == 128 ? launch_gather_d<IO, 128>(a, s) : launch_gather_d<IO, 256>(a, s);
}

}  // namespace attn
}  // namespace gdn

cudaError_t gdn_launch_kv8_append(const GdnKv8AppendArgs& a, int io, cudaStream_t s) {
  using namespace gdn::attn;
  return io == GDN_BF16 ? launch_append_io<__nv_bfloat16>(a, s) : launch_append_io<__half>(a, s);
}
cudaError_t gdn_launch_kv8_gather(const GdnKv8GatherArgs& a, int io, cudaStream_t s) {
  using namespace gdn::attn;
  return io == GDN_BF16 ? launch_gather_io<__nv_bfloat16>(a, s) : launch_gather_io<__half>(a, s);
}
cudaError_t gdn_launch_kv8_evict(const GdnKv8EvictArgs& a, cudaStream_t s) {
  using namespace gdn::attn;
  const int64_t cap = (int64_t)a.from.pages_per_seq << a.page_shift;
  const int room = cap < SELECT_KEYS ? (int)cap : SELECT_KEYS;
  cudaError_t e;
  static int opted_in[64] = {};
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !opted_in[dev]) {
    if ((e = cudaFuncSetAttribute(kv8_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  SELECT_KEYS * 4)) != cudaSuccess)
      return e;
    if (dev >= 0 && dev < 64) opted_in[dev] = 1;
  }
  if ((e = launch_behind(kv8_select_kernel, dim3((unsigned)(a.n * a.h_kv)), SELECT_THREADS,
                         (size_t)room * 4, s, a, room)) != cudaSuccess)
    return e;
  return a.d == 64 ? launch_move_d<64>(a, s)
                   : a.d == 128 ? launch_move_d<128>(a, s) : launch_move_d<256>(a, s);
}
