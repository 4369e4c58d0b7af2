// Attention of a step's rows over the paged fp8 cache, split over the context, on the
// 5th-generation tensor cores.
//
//   S[t, q] = scale * scale_t * (codes_t . q)     (token t, query q = one head of one row)
//   P[t, q] = 2^(S log2e - m_q)                   O[d, q] = sum_t codes_t[d] scale_t P[t, q]
//
// A 128-byte run of a record (a chunk: one 128-wide latent slice, or two 64-wide ones) and 128
// tokens make a tile.  Tokens are the M of the first product, dimensions that of the second, and
// queries the N of both: the heads that share a latent slice, times the rows of a request that
// share its context (1 to 96 columns, no padding beyond 16), so the cache is read once for all of
// them.  The first product takes the e4m3 tile as it lies in the cache (kind::mxf8f6f4); a bf16
// query is the exact sum of two e4m3 terms under one power-of-two scale per 32 dimensions.  The
// second takes P scale_t in f16 (the one rounding between the scores and o: 11 bits) and the tile
// widened to f16, which is exact.  m_q is chosen so that the largest P scale_t is about 2^6: what
// f16 cannot hold lies 2^-31 below it.  (Weights as two e4m3 terms under block scales would spare
// the widening, but cost each weight three times the instructions: 270 us against
// 145 at 48 rows over 8 contexts of 1K..64K when both were young; weights in bf16 took three
// instructions per two codes to widen the tile, f16 takes one.)
// O stays in TMEM over a whole run of tiles: m_q, an integer, moves only when a weight passes it
// by far (then O is rescaled, exactly).
//
// Work: the tiles of all (request, group of rows) pairs in one line, cut evenly into as many
// pieces as there are teams; a team is one CTA per chunk, so that the CTAs that read the same
// records run side by side.  Every CTA derives the cut from the step's positions and requests.
// A pair that falls into one piece is finished there; pieces of the others leave (O, m, l) in
// the workspace, which a second kernel joins.
//
// Roles: warps 0-7 softmax (TMEM lane quadrant = warp % 4: one token per thread; warp / 4: half
// of the columns), 8-11 widening, 12 the first product's MMAs, 13 the second's, 14 and 15 loads
// (every other tile each: TMA boxes through the page table, or cp.async for page sizes that are no
// multiple of 8).  What runs once per launch or item is kept short,
// in rolled loops: its instructions come from L2 or further away.
// Every mbarrier wait is bounded; a wait that runs out is reported, and from then on every role
// runs its loop without waiting, copying or issuing, so that the barriers among warps still
// complete and TMEM is freed.
#include "attend_plan.cuh"
#include "tc_common.cuh"

namespace mono {
namespace {

using namespace tc;
using namespace attend;

constexpr int TT = 128;        // tokens per tile
constexpr int NQ = 96;         // query columns at most
constexpr int MERGE = 64;      // up to here both terms of the queries are columns of one MMA
constexpr int GROUP = 16;      // rows of a group at most
constexpr int ST = 5;          // tiles in the ring
constexpr int THREADS = 24 * 32;
constexpr int SOFT_WARPS = 16, SOFT = SOFT_WARPS * 32, GROUPS = SOFT_WARPS / 4;
constexpr int WIDE_WARP = 16, WIDE_WARPS = 4, S_WARP = 20, O_WARP = 21;
constexpr int LOAD_WARP = 22, LOAD_WARPS = 2;
// registers a thread: softmax warps take what the others give up (in all, the launch's)
constexpr int REGS = 80, SOFT_REGS = 88, OTHER_REGS = 64;
static_assert(SOFT_REGS * SOFT + OTHER_REGS * 256 == REGS * THREADS, "register split");
constexpr int K_TILE = TT * 128, V_TILE = 2 * K_TILE;
constexpr int K_OFF = 0;
constexpr int V_OFF = K_OFF + ST * K_TILE;  // widened tiles [2]: dimensions 0..63, then 64..127
constexpr int P_OFF = V_OFF + 2 * V_TILE;   // weights: columns 0..63, then 64..95
constexpr int Q_OFF = P_OFF + V_TILE;       // hi rows, then lo rows
constexpr int IMG = 512;
constexpr int QIMG_OFF = Q_OFF + 2 * NQ * 128;
constexpr int ONE_OFF = QIMG_OFF + IMG;
constexpr int SC_OFF = ONE_OFF + IMG;  // the 16 bytes behind the codes, scale first [ST][128]
constexpr int PLAN_OFF = SC_OFF + ST * TT * 16;
constexpr int SMEM_BYTES = PLAN_OFF + (3 * MAX_REQ + 4) * 4 + 1024;
static_assert(V_OFF % 1024 == 0 && P_OFF % 1024 == 0 && Q_OFF % 1024 == 0 && (NQ * 128) % 1024 == 0,
              "swizzle atoms");
constexpr int CMAX = NQ / GROUPS;  // columns of a softmax warp at most
static_assert(SOFT_WARPS * CMAX * 32 * 4 <= V_TILE + 2 * NQ * 128, "the sums' scratch");

// TMEM columns
constexpr int S_COL = 0, O_COL = 256, SF_ONE = 384, SF_Q = 388;
// Instruction descriptors, M = 128; N, and the scale-byte selectors, are or-ed in.
// kind::mxf8f6f4: e4m3 x e4m3, E8M0 scales, both K-major.
constexpr uint32_t S_IDESC = (1u << 23) | ((uint32_t)(TT >> 4) << 24);
// kind::f16: f16 x f16, f32 accumulators, both MN-major.
constexpr uint32_t O_IDESC = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(TT >> 4) << 24);

struct Args {
  CUtensorMap codes, scales;  // the cache as [pages][tokens][bytes], boxes of box tokens
  int box;                    // 0: no maps
  AttendArgs a;
  Shape sh;
  float* part;    // workspace (Pieces)
  RowInfo* rows;
  int* total;
};

// Two f32 as f16, the first in the low half.
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Matrix descriptor as desc_sw128, MN-major with `lbo` bytes between 128-byte runs along MN.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lbo) {
  return (desc_sw128(saddr) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(lbo >> 4) << 16);
}
__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
template <int REGS>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int N>
__device__ __forceinline__ void bar_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}
// Barrier among 128 threads that also tells whether any of them brought a true value.
__device__ __forceinline__ bool bar_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// A wait for an mbarrier phase by a whole warp, in few instructions: some 10^7 polls (a good part
// of a second) at most, none once another wait has run out.  False if it ran out.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  uint32_t polls = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (*abort || ++polls == (1u << 23)) {
      atomicOr(status, ST_WAIT_TIMEOUT);
      *abort = 1;
      polls = ~0u;
      break;
    }
  }
  return __all_sync(0xffffffffu, polls != ~0u);
}
// How an item's columns are dealt out (see the head of the file).
struct Deal {
  int nqp, streams, bufs;  // columns; streams of softmax groups; score buffers
  __device__ explicit Deal(int cols) : nqp(cols), streams(cols <= 16 ? 4 : cols <= 48 ? 2 : 1) {
    bufs = streams == 4 ? 4 : 2;
  }
  __device__ bool merged() const { return nqp <= MERGE; }
  __device__ uint32_t s_col(int it) const { return S_COL + (256 / bufs) * (it & (bufs - 1)); }
  __device__ int flat(int stream) const { return streams == 4 ? 16 * stream : 48 * stream; }
  __device__ int slot(int it) const { return it & (bufs - 1); }
  // parity of buffer slot(i)'s phase of an item's tile i, and the phases that an item of n tiles
  // leaves (ph: the slots' parities at its start, a bit each)
  __device__ uint32_t parity(uint32_t ph, int i) const { return ((ph >> slot(i)) ^ (i / bufs)) & 1; }
  __device__ void advance(uint32_t& ph, int n) const {
    for (int b = 0; b < bufs; ++b) ph ^= (uint32_t)((n + bufs - 1 - b) / bufs & 1) << b;
  }
  // where stream k's weights lie in the rows of the weights' buffer
  __device__ int p_off(int stream) const { return streams == 4 ? 32 * stream : K_TILE * stream; }
};

// A maximum over the warp, every lane gets it (floats as ordered integers).
__device__ __forceinline__ float warp_max_any(float v) {
  int i = __float_as_int(v);
  i = i < 0 ? i ^ 0x7FFFFFFF : i;
  i = __reduce_max_sync(0xffffffffu, i);
  return __int_as_float(i < 0 ? i ^ 0x7FFFFFFF : i);
}

struct Shared {
  uint64_t full[ST], k_free[ST], s_full[4], p_full[4], pv_done[4], v_full[2], v_free[2], q_full, drain;
  float neg_m[NQ], fac[NQ], red[SOFT_WARPS][CMAX];  // m and its change: [stream][column]
  uint32_t valid[ST][4], mask[ST];  // tokens that are there; whether some row masks some token
  long long out[NQ];  // where a column's first value goes: o or the workspace
  float fin[NQ][4];   // a column's factor for each stream's O
  int slice[NQ], group_row[GROUP], group_pos[GROUP];
  uint32_t tmem;
  int cols, nrows, abort;
  Jobs start;
};
static_assert(SMEM_BYTES + sizeof(Shared) <= 227 * 1024, "shared memory");

// What a softmax warp knows of its item.
struct Soft {
  Span span;
  int t0, n, it;      // the item's first tile and tile count, the ring's next tile
  int c0, col, flat;  // this group's first column; of its stream's set: in TMEM and in m
  int first, stride;  // the group's tiles
  int nrows, cheads;  // the item's rows and the heads (columns) of each
  int min_hi, max_lo; // tokens that every row sees: [max_lo, min_hi] and the sinks
  float to_log2;
  uint32_t tmem;      // with the warp's lane quadrant
  uint32_t p_row;     // the thread's row of its stream's weights, and their first 16-byte piece
  uint32_t p_chunk;
  uint32_t ph;        // the buffers' barriers' phases at the item's start
};

// The softmax of a group's C columns over its tiles of an item, a token per thread; leaves the
// thread's share of every column's sum, in units of 2^m, in the scratch.
template <int C>
__device__ __forceinline__ void soft_tiles(const AttendArgs& a, const Soft& w, const Deal& deal,
                                           Shared& sh, uint8_t* sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, group = warp >> 2, tok = 32 * quad + lane;
  const bool merged = deal.merged();
  volatile int* abort = &sh.abort;
  float l[C], s[C];
#pragma unroll
  for (int c = 0; c < C; ++c) l[c] = 0.0f;
#pragma unroll 1
  for (int i = w.first; i < w.n; i += w.stride) {
    const int it = w.it + i, st = it % ST, b = deal.slot(i);
    const int t0 = w.span.token(w.t0 + i), t = t0 + tok;
    wait(&sh.full[st], (it / ST) & 1, a.status, abort);
    const float raw = reinterpret_cast<const float*>(sm + SC_OFF)[(st * TT + tok) * 4];
    const uint32_t ok = sh.valid[st][quad];
    const bool fin = fabsf(raw) <= 3.0e38f;
    const float ct = fin ? raw * w.to_log2 : __int_as_float(0x7FC00000);
    const float sc = fin ? raw : 0.0f;
    const float lsc = sc > 0.0f ? fmaxf(log2_of(sc), LEAST) : LEAST;
    __syncwarp();
    if (lane < w.stride) mbar_arrive(&sh.k_free[st]);  // (as many arrivals whoever takes the tile)
    // some of the tile's tokens are not every row's to see
    const bool part = ok != 0xffffffffu || t0 + TT - 1 > w.min_hi ||
                      (t0 < w.max_lo && t0 + TT > a.sinks);
    uint32_t see = 0xffffffffu;
    if (__builtin_expect(part, 0)) {  // the group's columns that see the token
#pragma unroll 1
      for (int j = 0; j < w.nrows; ++j) {
        const int hi = a.causal ? sh.group_pos[j] : w.span.hi;
        const int lo = a.window > 0 ? max(0, hi - a.window + 1) : 0;
        if (((ok >> lane) & 1) && t <= hi && (t >= lo || t < a.sinks)) continue;
        // columns [c, c + cheads) of the item, from this group's first on
        const int c = j * w.cheads - w.c0;
        const int x = min(max(c, 0), 31), y = min(max(c + w.cheads, 0), 31);
        see &= ~((1u << y) - (1u << x));
      }
    }
    wait(&sh.s_full[b], deal.parity(w.ph, i), a.status, abort);
    const uint32_t scol = w.tmem + deal.s_col(i) + w.c0;
    // weights; a second round where some query's m has to move (always in an item's first tile)
#pragma unroll 1
    for (bool moved = false;; moved = true) {
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < C; g += 8) tc_ld8(scol + g, s + g);
      if (merged) {
#pragma unroll
        for (int g = 0; g < C; g += 8) {
          float x[8];
          tc_ld8(scol + deal.nqp + g, x);
          tc_wait_ld();
          tc_loaded(x);
          tc_loaded(s + g);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[g + e] += x[e];
        }
      } else {
        tc_wait_ld();
#pragma unroll
        for (int g = 0; g < C; g += 8) tc_loaded(s + g);
      }
      const float4* nm = reinterpret_cast<const float4*>(sh.neg_m + w.flat);
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < C; c += 4) {
        const float4 m = nm[c / 4];
        fma2(s[c], s[c + 1], ct, m.x, m.y);
        fma2(s[c + 2], s[c + 3], ct, m.z, m.w);
      }
      if (__builtin_expect(part, 0)) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (!((see >> c) & 1)) s[c] = -INFINITY;
      }
#pragma unroll
      for (int c = 0; c < C; ++c) top = fmaxf(top, s[c]);
      if (__builtin_expect(!bar_any(2 + group, !moved && top + lsc > TOP), 1)) break;
      // the columns' largest weights times scales of the tile
#pragma unroll 1
      for (int g = 0; g < C; g += 8) {
        float x[8], y[8], mine = 0.0f;
        tc_ld8(scol + g, x);
        if (merged) tc_ld8(scol + deal.nqp + g, y);
        tc_wait_ld();
        tc_loaded(x);
        if (merged) tc_loaded(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float v = fmaf(merged ? x[e] + y[e] : x[e], ct, lsc);
          if (!(v > -INFINITY) || !((see >> (g + e)) & 1)) v = -INFINITY;
          const float m = warp_max_any(v);
          if (lane == e) mine = m;
        }
        if (lane < 8) sh.red[warp][g + lane] = mine;
      }
      bar_sync<128>(6 + group);
      if (quad == 0 && lane < C) {
        const float(*r)[CMAX] = sh.red + 4 * group;
        const float m = fmaxf(fmaxf(r[0][lane], r[1][lane]), fmaxf(r[2][lane], r[3][lane]));
        const float old = -sh.neg_m[w.flat + lane];
        float f = 1.0f;
        if (m - old > BASE) {
          const float now = fminf(ceilf(m) - BASE, 3.0e38f);
          f = old == UNSET ? 0.0f : ex2(old - now);
          sh.neg_m[w.flat + lane] = -now;
        }
        sh.fac[w.flat + lane] = f;
      }
      bar_sync<128>(6 + group);
#pragma unroll
      for (int c = 0; c < C; ++c) l[c] *= sh.fac[w.flat + c];
      if (i >= w.stride) {
        const int pi = i - w.stride;  // the group's tile before: its product is in O
        wait(&sh.pv_done[deal.slot(pi)], deal.parity(w.ph, pi), a.status, abort);
        tc_fence_after();
#pragma unroll 1
        for (int g = 0; g < C; g += 8) {
          float x[8];
          const uint32_t oc = w.tmem + O_COL + w.col + g;
          tc_ld8(oc, x);
          tc_wait_ld();
          tc_loaded(x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= sh.fac[w.flat + g + e];
          tc_st8(oc, x);
        }
        tc_wait_st();
      }
    }
    // weights times scales, rows of 128 bytes per token; the buffer's last reader has finished
    if (i >= w.stride) {
      const int pi = i - w.stride;
      wait(&sh.pv_done[deal.slot(pi)], deal.parity(w.ph, pi), a.status, abort);
    }
#pragma unroll
    for (int g = 0; g < C; g += 8) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float p0 = ex2(s[g + e]), p1 = ex2(s[g + e + 1]);
        add2(l[g + e], l[g + e + 1], p0, p1);
        mul2(p0, p1, sc);
        o[e / 2] = f16x2_of(p0, p1);
      }
      const int col = w.c0 + g;
      *reinterpret_cast<uint4*>(sm + w.p_row + (col >> 6) * K_TILE +
                                (((w.p_chunk + ((col & 63) >> 3)) ^ (tok & 7)) << 4)) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
    fence_proxy_async_shared();
    tc_fence_before();
    __syncwarp();
    if (lane < w.stride) mbar_arrive(&sh.p_full[b]);
  }
  // every product of the item is done: the weights' and the queries' buffers are scratch
#pragma unroll 1
  for (int i = max(0, w.n - deal.bufs); i < w.n; ++i)
    wait(&sh.pv_done[deal.slot(i)], deal.parity(w.ph, i), a.status, abort);
  tc_fence_after();
  float* scratch = reinterpret_cast<float*>(sm + P_OFF) + warp * CMAX * 32 + lane;
#pragma unroll
  for (int c = 0; c < C; ++c) scratch[32 * c] = l[c];
}

__global__ void __launch_bounds__(THREADS, 1) attend_kernel(const __grid_constant__ Args ar) {
  const AttendArgs& a = ar.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~uintptr_t(1023));
  __shared__ __align__(16) Shared ss;
  volatile int* abort = &ss.abort;
  Plan plan;
  plan.pre = reinterpret_cast<int*>(sm + PLAN_OFF);
  plan.pmax = plan.pre + MAX_REQ + 4;
  plan.pmin = plan.pmax + MAX_REQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Shape& sh = ar.sh;
  const int team = blockIdx.x / sh.chunks, chunk = blockIdx.x - team * sh.chunks;
  const int chunk_bytes = min(128, a.kv_dim - 128 * chunk);

  if (tid == 0) {
    // a tile is free when the first product, the widening and the softmax warps have read it
    for (int s = 0; s < ST; ++s)
      mbar_init(&ss.full[s], 1), mbar_init(&ss.k_free[s], 1 + WIDE_WARPS + SOFT_WARPS);
    for (int s = 0; s < 4; ++s)
      mbar_init(&ss.s_full[s], 1), mbar_init(&ss.pv_done[s], 1), mbar_init(&ss.p_full[s], SOFT_WARPS);
    for (int s = 0; s < 2; ++s) mbar_init(&ss.v_full[s], WIDE_WARPS), mbar_init(&ss.v_free[s], 1);
    mbar_init(&ss.q_full, SOFT_WARPS);
    mbar_init(&ss.drain, 2);
    ss.abort = 0;
    fence_mbar_init();
  }
  if (warp == S_WARP) tmem_alloc<512>(&ss.tmem);
  if (tid < 2 * IMG / 4) reinterpret_cast<uint32_t*>(sm + QIMG_OFF)[tid] = 0x7F7F7F7Fu;
  fence_proxy_async_shared();

  derive_plan<THREADS>(a, sh, plan, team, team < sh.teams, &ss.start, ar.total);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ss.tmem;
  Jobs items = ss.start;
  Job im;

  if (warp >= LOAD_WARP) {
    // ------------------------------------------------------- loads: a warp takes every other tile
    regs_down<OTHER_REGS>();
    int ni = warp - LOAD_WARP;
    bool more = next_job(a, sh, plan, items, im);
    // a lane per box of the next tile (of a token each without maps, four times): its page, on its
    // way while the tile before is loaded, and its first token's place in it
    const int box = ar.box ? ar.box : 1, bs = a.kv.block_size;
    const int shift = __ffs(box) - 1, boxes = TT >> shift;
    int page[4], row[4], t0 = 0;
    auto locate = [&]() {
#pragma unroll 1
      while (more && ni >= im.n) ni -= im.n, more = next_job(a, sh, plan, items, im);
      if (!more) return;
      t0 = im.span.token(im.t0 + ni);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (32 * q >= boxes) break;
        const int t = t0 + ((32 * q + lane) << shift), lb = t / bs;
        page[q] = -1;
        row[q] = t - lb * bs;
        if (32 * q + lane < boxes && lb < a.kv.max_blocks && t <= im.span.hi &&
            (t + box > im.span.lo || t < a.sinks))
          page[q] = __ldg(a.kv.table + (size_t)im.b * a.kv.max_blocks + lb);
        else
          row[q] = -1;
      }
    };
    auto mapped = [&](int q) {
      const bool m = page[q] >= 0 && page[q] < a.kv.num_blocks;
      if (row[q] >= 0 && !m) atomicOr(a.status, ST_UNMAPPED_PAGE);
      return m;
    };
    auto masks = [&](uint32_t there) {  // for some row of the request
      const int first = a.causal ? plan.pmin[im.b] : im.span.hi;
      const int last_lo = a.window > 0 ? max(0, im.span.hi - a.window + 1) : 0;
      return (uint32_t)(there != 0xffffffffu || t0 + TT - 1 > first ||
                        (t0 < last_lo && t0 + TT > a.sinks));
    };
    locate();
#pragma unroll 1
    for (int it = warp - LOAD_WARP; more; it += LOAD_WARPS) {
      const int s = it % ST;
      bool go = true;
      if (it >= ST) go = wait(&ss.k_free[s], ((it / ST) - 1) & 1, a.status, abort);
      uint8_t* st = sm + K_OFF + s * K_TILE;
      uint8_t* sc = sm + SC_OFF + s * TT * 16;
      uint32_t there = 0xffffffffu;
      if (ar.box) {
        // boxes with a token to see; their other tokens, and what the rest of the slot holds, are
        // masked
        const bool m = mapped(0);
        const uint32_t have = __ballot_sync(0xffffffffu, m);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int t = t0 + 32 * q + lane;
          const bool see = ((have >> ((32 * q + lane) >> shift)) & 1) && t <= im.span.hi &&
                           (t >= im.span.lo || t < a.sinks);
          const uint32_t w = __ballot_sync(0xffffffffu, see);
          if (lane == q) ss.valid[s][q] = w;
          there &= w;
        }
        if (lane == 0) ss.mask[s] = masks(there);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&ss.full[s], go ? __popc(have) * box * (128 + 16) : 0);
        __syncwarp();
        if (m && go) {
          tma_load_3d(st + ((lane * 128) << shift), &ar.codes, 128 * chunk, row[0], page[0], &ss.full[s]);
          tma_load_3d(sc + ((lane * 16) << shift), &ar.scales, a.kv_dim, row[0], page[0], &ss.full[s]);
        }
      } else {
        const int piece = lane & 7;
        const bool in_chunk = go && 16 * piece < chunk_bytes;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          const int pg = q == 0 ? page[0] : q == 1 ? page[1] : q == 2 ? page[2] : page[3];
          const int rw = q == 0 ? row[0] : q == 1 ? row[1] : q == 2 ? row[2] : row[3];
          const bool m = pg >= 0 && pg < a.kv.num_blocks;
          if (rw >= 0 && !m) atomicOr(a.status, ST_UNMAPPED_PAGE);
          const long long off = m ? pg * a.kv.stride_block + rw * a.kv.stride_tok : 0;
          const uint32_t w = __ballot_sync(0xffffffffu, m);
          if (lane == 0) ss.valid[s][q] = w;
          there &= w;
#pragma unroll 1
          for (int e = 0; e < 8; ++e) {
            const int k = 4 * e + (lane >> 3), r = 32 * q + k;
            const long long ro = __shfl_sync(0xffffffffu, off, k);
            if (in_chunk && ((w >> k) & 1))
              cp_async16(st + r * 128 + ((piece ^ (r & 7)) << 4), a.kv.base + ro + 128 * chunk + 16 * piece,
                         16);
          }
          if (go && m) cp_async16(sc + (32 * q + lane) * 16, a.kv.base + off + a.kv_dim, 16);
        }
        if (lane == 0) ss.mask[s] = masks(there);
        cp_async_wait_all();
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.full[s]);
      }
      ni += LOAD_WARPS;
      locate();
    }
  } else if (warp >= WIDE_WARP && warp < WIDE_WARP + WIDE_WARPS) {
    // ------------------------------------------------------------ widening: 32 tokens of every tile
    regs_down<OTHER_REGS>();
    const int lw = warp - WIDE_WARP, piece = lane & 7, r4 = lane >> 3;
    const int total = items.left;
#pragma unroll 1
    for (int it = 0; it < total; ++it) {
      const int s = it % ST, b = it & 1;
      wait(&ss.full[s], (it / ST) & 1, a.status, abort);
      if (it >= 2) wait(&ss.v_free[b], ((it >> 1) - 1) & 1, a.status, abort);
      const bool mask = ss.mask[s] != 0;
      const uint8_t* src = sm + K_OFF + s * K_TILE + 32 * lw * 128;
      uint8_t* dst = sm + V_OFF + b * V_TILE + (piece >> 2) * K_TILE + 32 * lw * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 16 * h + 4 * e + r4;
          v[e] = lds128(src + row * 128 + ((piece ^ (row & 7)) << 4));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // a NaN code that some row must not see would reach it as 0 * NaN (rows that do see the
          // token are NaN by their scores)
          if (__builtin_expect(mask, 0)) v[e] = without_nan(v[e]);
          const int row = 16 * h + 4 * e + r4, c = 2 * (piece & 3);
          uint4 x, y;
          uint32_t f[2];
          e4m3x4_to_f16x4(v[e].x, f), x.x = f[0], x.y = f[1];
          e4m3x4_to_f16x4(v[e].y, f), x.z = f[0], x.w = f[1];
          e4m3x4_to_f16x4(v[e].z, f), y.x = f[0], y.y = f[1];
          e4m3x4_to_f16x4(v[e].w, f), y.z = f[0], y.w = f[1];
          *reinterpret_cast<uint4*>(dst + row * 128 + ((c ^ (row & 7)) << 4)) = x;
          *reinterpret_cast<uint4*>(dst + row * 128 + (((c + 1) ^ (row & 7)) << 4)) = y;
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss.v_full[b]), mbar_arrive(&ss.k_free[s]);
    }
  } else if (warp == S_WARP) {
    // ------------------------------------------------------------- the first product's MMAs
    regs_down<OTHER_REGS>();
    const uint32_t k0 = smem_u32(sm + K_OFF);
    const uint64_t q0 = desc_sw128(smem_u32(sm + Q_OFF));
    int it = 0;
    uint32_t ph = 0;
    if (elect_one()) tc_cp_img(tmem + SF_ONE, sm + ONE_OFF);
    __syncwarp();
#pragma unroll 1
    for (int item = 0; next_job(a, sh, plan, items, im); ++item) {
      wait(&ss.q_full, item & 1, a.status, abort);
      const Deal deal(ss.cols);
      const bool merged = deal.merged();
      const uint32_t idesc = S_IDESC | ((uint32_t)((merged ? 2 * deal.nqp : deal.nqp) >> 3) << 17);
#pragma unroll 1
      for (int i = 0; i < im.n; ++i) {
        const int st = (it + i) % ST, b = deal.slot(i);
        bool ok = wait(&ss.full[st], ((it + i) / ST) & 1, a.status, abort);
        if (i >= deal.bufs) ok &= wait(&ss.p_full[b], deal.parity(ph, i - deal.bufs), a.status, abort);
        if (ok && elect_one()) {
          tc_fence_after();
          if (i == 0) tc_cp_img(tmem + SF_Q, sm + QIMG_OFF);
          const uint64_t kd = desc_sw128(k0 + st * K_TILE);
#pragma unroll 1
          for (int term = 0; term < (merged ? 1 : 2); ++term)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_mxf8(tmem + deal.s_col(i), kd + 2 * k, q0 + term * (NQ * 128 / 16) + 2 * k,
                          idesc | ((uint32_t)k << 4) | ((uint32_t)k << 29), tmem + SF_ONE,
                          tmem + SF_Q, term > 0 || k > 0);
          tc_commit(&ss.s_full[b]);
          tc_commit(&ss.k_free[st]);
        }
        __syncwarp();
      }
      it += im.n;
      deal.advance(ph, im.n);
    }
    if (elect_one()) tc_commit(&ss.drain);  // (what was issued has completed at this arrival)
    __syncwarp();
  } else if (warp == O_WARP) {
    // ------------------------------------------------------------ the second product's MMAs
    regs_down<OTHER_REGS>();
    const uint64_t v0 = desc_mn(smem_u32(sm + V_OFF), K_TILE);
    const uint64_t p0 = desc_mn(smem_u32(sm + P_OFF), K_TILE);
    // first, where the second kernel finds the rows' results
#pragma unroll 1
    for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
      const RowInfo info = row_info(a, sh, plan, r);
      if (lane == 0) ar.rows[r] = info;
    }
    int it = 0;
    uint32_t ph = 0;
#pragma unroll 1
    for (int item = 0; next_job(a, sh, plan, items, im); ++item) {
      wait(&ss.q_full, item & 1, a.status, abort);
      const Deal deal(ss.cols);
      const uint32_t idesc = O_IDESC | ((uint32_t)(deal.nqp >> 3) << 17);
#pragma unroll 1
      for (int i = 0; i < im.n; ++i, ++it) {
        const int b = deal.slot(i), v = it & 1, stream = i & (deal.streams - 1);
        bool ok = wait(&ss.p_full[b], deal.parity(ph, i), a.status, abort);
        ok &= wait(&ss.v_full[v], (it >> 1) & 1, a.status, abort);
        if (ok && elect_one()) {
          tc_fence_after();
          const uint64_t pd = p0 + (deal.p_off(stream) >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)  // 16 tokens each
            tc_mma_f16(tmem + O_COL + deal.flat(stream), v0 + v * (V_TILE / 16) + k * (2048 / 16),
                     pd + k * (2048 / 16), idesc, i >= deal.streams || k > 0);
          tc_commit(&ss.pv_done[b]);
          tc_commit(&ss.v_free[v]);
        }
        __syncwarp();
      }
      deal.advance(ph, im.n);
    }
    if (elect_one()) tc_commit(&ss.drain);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------------------- softmax
    regs_up<SOFT_REGS>();
    const int quad = warp & 3, group = warp >> 2;
    const int hpg = a.n_q / (a.kv_dim / a.head_dim);
    const int cheads = hpg * (chunk_bytes > a.head_dim ? 2 : 1);  // heads per row of this chunk
    const int dshift = a.head_dim == 64 ? 6 : 7;
    Soft w;
    w.it = 0;
    w.ph = 0;
    w.cheads = cheads;
    w.to_log2 = a.scale * LOG2E;
    w.tmem = tmem + ((uint32_t)(32 * quad) << 16);
#pragma unroll 1
    while (next_job(a, sh, plan, items, im)) {
      // ---- the group's rows and queries
      bar_sync<SOFT>(1);  // the previous item's columns are no longer in use
      if (warp == 0) {
        const int n = group_rows(a, sh, im.b, im.group, ss.group_row, ss.group_pos);
        const int cols = (n * cheads + 15) & ~15;
        if (lane == 0) ss.cols = cols == 80 ? 96 : cols, ss.nrows = n;
      }
      bar_sync<SOFT>(1);
      const int nrows = ss.nrows, nq = nrows * cheads;
      const Deal deal(ss.cols);
      const int nqp = deal.nqp;
      const bool merged = deal.merged();
      const bool whole = im.n == im.span.tiles;  // nobody else has tiles of this group
      const long long slot = (long long)(team * 2 + (im.t0 > 0 ? 0 : 1)) * sh.chunks + chunk;
      if (tid < NQ) {
        ss.neg_m[tid] = -UNSET;
        const int j = tid / cheads, h = tid - j * cheads, sl = h / hpg;
        const long long head = (long long)chunk * sh.heads + h;
        ss.slice[tid] = tid < nq ? sl : -1;
        if (tid < nq)
          ss.out[tid] = whole ? ss.group_row[j] * a.o_stride + head * a.head_dim
                              : (slot * NQ + tid) * PART_LD + 4;
      }
      // queries as two e4m3 terms, rows of 128 bytes: hi in row c, lo in row nqp + c (merged)
      // or NQ + c
#pragma unroll 1
      for (int i = tid; i < nqp * 16; i += SOFT) {  // first copied as they are, all at once
        const int c = i >> 4, d = (i & 15) * 8;
        const int j = c / cheads, h = c - j * cheads, sl = h / hpg;
        const bool in = c < nq && (d >> dshift) == sl;
        cp_async16(sm + P_OFF + i * 16,
                   a.q + (in ? ss.group_row[j] * a.q_stride +
                                   ((long long)chunk * sh.heads + h) * a.head_dim + (d - (sl << dshift))
                             : 0),
                   in ? 16 : 0);
      }
      cp_async_wait_all();
      // (every lane takes part in the blocks' maxima)
#pragma unroll 1
      for (int i = tid; i < ((nqp * 16 + SOFT - 1) & ~(SOFT - 1)); i += SOFT) {
        const bool live = i < nqp * 16;
        const int c = live ? i >> 4 : 0, d = (i & 15) * 8;
        float v[8];
        bf16x8_to_f32(live ? lds128(sm + P_OFF + i * 16) : make_uint4(0, 0, 0, 0), v);
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (isinf(v[e])) v[e] = __int_as_float(0x7FC00000);  // (the codes have no infinity)
          m = fmaxf(m, fabsf(v[e]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t code = e4m3_block_code(m);
        const float inv = e8m0_inverse(code);
        uint32_t hw[2] = {0, 0}, lw[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t hb, lb;
          e4m3_hilo(v[e] * inv, hb, lb);
          hw[e >> 2] |= hb << (8 * (e & 3));
          lw[e >> 2] |= lb << (8 * (e & 3));
        }
        const int rl = (merged ? nqp : NQ) + c;
        const int o = (d >> 4), x = d & 8;
        if (!live) continue;
        *reinterpret_cast<uint2*>(sm + Q_OFF + c * 128 + ((o ^ (c & 7)) << 4) + x) =
            make_uint2(hw[0], hw[1]);
        *reinterpret_cast<uint2*>(sm + Q_OFF + rl * 128 + ((o ^ (rl & 7)) << 4) + x) =
            make_uint2(lw[0], lw[1]);
        if ((d & 31) == 0) {
          sm[QIMG_OFF + (c & 31) * 16 + (c >> 5) * 4 + (d >> 5)] = (uint8_t)code;
          if (merged) sm[QIMG_OFF + (rl & 31) * 16 + (rl >> 5) * 4 + (d >> 5)] = (uint8_t)code;
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss.q_full);
      w.min_hi = 0x7FFFFFFF;
      w.max_lo = 0;
#pragma unroll 1
      for (int j = 0; j < nrows; ++j) {
        const int hi = a.causal ? ss.group_pos[j] : im.span.hi;
        w.min_hi = min(w.min_hi, hi);
        w.max_lo = max(w.max_lo, a.window > 0 ? max(0, hi - a.window + 1) : 0);
      }
      bar_sync<SOFT>(1);  // (the staged queries have been read: weights may take their place)
      w.span = im.span;
      w.t0 = im.t0;
      w.n = im.n;
      w.nrows = nrows;
      const int stream = group & (deal.streams - 1), cols = nqp * deal.streams / GROUPS;
      w.first = stream;
      w.stride = deal.streams;
      w.c0 = group / deal.streams * cols;
      w.flat = deal.flat(stream) + w.c0;
      w.col = w.flat;
      w.p_row = P_OFF + (32 * quad + lane) * 128 + (deal.streams == 2 ? K_TILE * stream : 0);
      w.p_chunk = deal.streams == 4 ? 2 * stream : 0;
      if (cols == 16)
        soft_tiles<16>(a, w, deal, ss, sm);
      else
        soft_tiles<24>(a, w, deal, ss, sm);
      w.it += im.n;
      deal.advance(w.ph, im.n);

      // ---- the item's result: the columns' sums over the tokens, then O
      const float* scratch = reinterpret_cast<const float*>(sm + P_OFF);
      __syncwarp();
      if (lane < cols) {  // this warp's share of each
        float v = 0.0f;
#pragma unroll 4
        for (int k = 0; k < 32; ++k) v += scratch[(warp * CMAX + lane) * 32 + ((k + lane) & 31)];
        ss.red[warp][lane] = v;
      }
      bar_sync<SOFT>(1);
      if (tid < nq) {
        // the streams' sums and O in the largest m (one stream: as they are)
        float m = UNSET, lt = 0.0f;
#pragma unroll 1
        for (int k = 0; k < min(deal.streams, im.n); ++k) m = fmaxf(m, -ss.neg_m[deal.flat(k) + tid]);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          float f = 0.0f;
          if (k < min(deal.streams, im.n)) {
            const int g = k + tid / cols * deal.streams, c = tid % cols;
            const float(*r)[CMAX] = ss.red + 4 * g;
            const float mk = -ss.neg_m[deal.flat(k) + tid];
            const float lk = (r[0][c] + r[1][c]) + (r[2][c] + r[3][c]);
            f = lk != lk ? 1.0f : mk == UNSET ? 0.0f : ex2(mk - m);  // (a NaN stays one)
            if (f != 0.0f) lt = fmaf(lk, f, lt);
          }
          ss.fin[tid][k] = f;
        }
        const float up = !whole ? 1.0f : lt == 0.0f ? 0.0f : 1.0f / lt;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) ss.fin[tid][k] *= up;
        if (whole) {
          const int j = tid / cheads;
          a.lse[(long long)ss.group_row[j] * a.n_q + chunk * sh.heads + tid - j * cheads] =
              lt == 0.0f ? -INFINITY : (log2f(lt) + m) * LN2;
        } else {
          ar.part[ss.out[tid] - 4] = m;
          ar.part[ss.out[tid] - 3] = lt;
        }
      }
      bar_sync<SOFT>(1);
      const int d = 32 * quad + lane;  // this thread's dimension of the chunk
      const int sl = d >> dshift, dl = d - (sl << dshift);
#pragma unroll 1
      for (int c8 = 8 * group; c8 < nqp; c8 += 8 * GROUPS) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll 1
        for (int k = 0; k < min(deal.streams, im.n); ++k) {
          float x[8];
          tc_ld8(w.tmem + O_COL + deal.flat(k) + c8, x);
          tc_wait_ld();
          tc_loaded(x);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float f = ss.fin[c8 + e][k];
            if (f != 0.0f) v[e] = fmaf(x[e], f, v[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const long long at = ss.out[c8 + e] + dl;
          const bool mine = ss.slice[c8 + e] == sl;
          if (whole) {
            if (mine) a.o[at] = __float2bfloat16_rn(v[e]);
          } else {
            if (mine) ar.part[at] = v[e];
          }
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == S_WARP) {
    (void)wait(&ss.drain, 0, a.status, abort);  // (at once unless a wait ran out before)
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

}  // namespace

cudaError_t attend_tc_prepare() {
  // the roles' register split adds up to what a block launches with
  cudaFuncAttributes f;
  cudaError_t e = cudaFuncGetAttributes(&f, attend_kernel);
  if (e == cudaSuccess && f.numRegs != REGS) e = cudaErrorInvalidConfiguration;
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
}

cudaError_t launch_attend_tc(const Launch& L, const AttendArgs& a, const attend::Pieces& ws, int sms) {
  const int chunks = (a.kv_dim + 127) / 128;
  Args ar = {{}, {}, 0, a, shape_of(a, TT, NQ, sms / chunks), ws.part, ws.rows, ws.total};
  // boxes of whole runs of a page, 8 rows (a swizzle atom) or more, that tiles are made of
  const int bs = a.kv.block_size;
  if (bs % 8 == 0) {
    const int box = std::min(bs & -bs, TT);
    if (encode_cache_map(&ar.codes, a.kv, a.kv_dim, 128, box) &&
        encode_cache_map(&ar.scales, a.kv, a.kv_dim + 16, 16, box))
      ar.box = box;
  }
  const cudaError_t e = launch_ex(L, dim3(sms), dim3(THREADS), SMEM_BYTES, attend_kernel, ar);
  return e == cudaSuccess ? attend::launch_join(L, a, ar.sh, ws) : e;
}

}  // namespace mono
