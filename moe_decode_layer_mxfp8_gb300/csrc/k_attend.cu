// Attention of a step's rows over the paged fp8 cache, split over the context, on the
// 5th-generation tensor cores.
//
//   S[t, q] = scale * scale_t * (codes_t . q)     (token t, query q = one head of one row)
//   P[t, q] = 2^(S log2e - m_q)                   O[d, q] = sum_t codes_t[d] scale_t P[t, q]
//
// A 128-byte run of a record (a chunk: one 128-wide latent slice, or two 64-wide ones) and 128
// tokens make a tile.  Tokens are the M of the first product, dimensions that of the second, and
// queries the N of both: the heads that share a latent slice, times the rows of a request that
// share its context (1 to 96 columns, padded to 16), so the cache is read once for all of them.
// The first product takes the e4m3 tile as it lies in the cache (kind::mxf8f6f4); a bf16 query is
// the sum of two e4m3 terms under one power-of-two scale per 32 dimensions: exactly, but for elements
// below 2^-9 of the 32's largest, which are off by up to 2^-17 of it.  The second one
// has two forms:
//   narrow: the same tile, transposed, against P scale_t as two e4m3 terms (together 8 bits, the
//     one rounding between scores and o) under a power-of-two scale per column and 32 tokens: the
//     tile is never rewritten, a weight costs some 14 instructions.  Both products' terms are
//     columns of one MMA, added when accumulators are read.
//   wide: the tile widened to f16 (exact) against P scale_t in f16 (11 bits): widening costs
//     shared-memory bandwidth and four warps, but a weight only some 6 instructions.
// Steps of up to 32 columns a request on average take the narrow form; the average is over the rows of
// the block table (the host does not see which of them have rows).  Measured over 8 contexts of
// 1K..64K tokens, 16 heads a slice, rows of a request 1 / 2 / 3 / 4: narrow 41 / 56 / 84 / 92 us,
// wide 69 / 73 / 78 / 82 us.
// O stays in TMEM over a whole run of tiles: m_q, an integer, is set by the run's first tile and
// moves only when a weight passes it by far (then O is rescaled, exactly).
//
// Work: the tiles of all (request, group of rows) pairs in one line, cut evenly into as many
// pieces as there are teams; a team is one CTA per chunk, so that the CTAs that read the same
// records run side by side.  Every CTA derives the cut from the step's positions and requests.
// Beginning another pair costs a team as much as ten tiles (five in the wide form), and the cut
// counts it so: without that 8 rows over 8 contexts took 45 us instead of 41, windows of 4K tokens
// for 48 rows 36 instead of 31.  A pair that falls into one piece is finished there; pieces of the
// others leave (O, m, l) in the workspace, which a second kernel joins.
//
// Roles: warps 0-15 softmax, a token per thread (TMEM lane quadrant = warp % 4) and 16 columns per
// group of four warps (24 where there are more than 64): with 16 columns the groups take every
// fourth tile each, with 32 two groups share every other tile, with more the groups share all
// tiles.  Then come the warps that make the next item's queries while the current one runs (in the
// wide form they widen tiles too), those that issue the first product's MMAs, the second's, and two
// that load (every other slot of the ring each: TMA boxes through the page table, or cp.async for
// page sizes that are no multiple of 8).  A wait for a barrier that is complete still costs a warp 100
// to 300 cycles, an MMA's issue some 60: hence two warps for each product in the narrow form, whose
// tiles take 700 cycles, and one wait per tile in the softmax.  What runs once per launch or item is kept
// short, in rolled loops: its instructions come from L2 or further away.
//
// Measured: 8 rows over 8 contexts of 1K..64K 41 us (137 MB; copy: 20 us), some 8 of them launches, the
// cut and the join; bound by HBM while tiles run, by the first tile's latency before.  48 rows 97 us,
// bound by the softmax warps' latencies (2850 cycles a tile, 0.6 instructions a cycle; its MMAs take
// 1250).  One row over 777 tokens 12.5 us: launches and latencies.
// Every mbarrier wait is bounded; a wait that runs out is reported, and from then on every role
// runs its loop without waiting, copying or issuing, so that the barriers among warps still
// complete and TMEM is freed.
#include <type_traits>

#include "attend_tc.cuh"

namespace mono {
namespace {

using namespace tc;
using namespace attend;

constexpr int THREADS = 24 * 32;
constexpr int SOFT_WARPS = 16, SOFT = SOFT_WARPS * 32, GROUPS = SOFT_WARPS / 4;
constexpr int Q_TWICE = 32;    // items of up to so many columns have their queries made ahead
constexpr int WIDE_FROM = 32;  // the wide form where requests have more columns on average (see above)
constexpr int V_TILE = 2 * K_TILE, SLOTS = 8;

// What the two forms differ in (see the head of the file).
template <bool WIDE>
struct Form {
  static constexpr int NQ = WIDE ? 96 : 64;  // query columns at most
  static constexpr int CMAX = WIDE ? 24 : 16;  // columns of a softmax warp at most
  static constexpr int ST = WIDE ? 3 : 8;    // tiles in the ring
  static constexpr int EXTRA = WIDE ? 5 : 10;  // what an item costs beside its tiles, in tiles
  // the roles' first warps
  static constexpr int PREP_WARP = SOFT_WARPS, PREP = (WIDE ? 4 : 2) * 32;
  static constexpr int MMA_WARPS = WIDE ? 1 : 2, S_WARP = PREP_WARP + PREP / 32,
                       O_WARP = S_WARP + MMA_WARPS, LOAD_WARP = O_WARP + MMA_WARPS, LOAD_WARPS = 2;
  static_assert(32 * (LOAD_WARP + LOAD_WARPS) == THREADS && PREP >= NQ, "roles");
  // shared memory
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = K_OFF + ST * K_TILE;  // widened tiles [2]: dimensions 0..63, then 64..127
  // weights [2]: tokens x (streams x columns) of 128 bytes; then those of columns from 64, of both
  static constexpr int P_OFF = V_OFF + (WIDE ? 2 * V_TILE : 0);
  // queries: hi rows, then lo rows; [2] up to Q_TWICE columns
  static constexpr int Q_OFF = P_OFF + (WIDE ? 3 : 2) * K_TILE, Q_BYTES = 2 * NQ * 128;
  static constexpr int PIMG_OFF = Q_OFF + Q_BYTES;   // scale images of the weights [SLOTS],
  static constexpr int QIMG_OFF = PIMG_OFF + (WIDE ? 0 : SLOTS * IMG);  // of the queries [2],
  static constexpr int ONE_OFF = QIMG_OFF + 2 * IMG;                   // and of ones
  static constexpr int SC_OFF = ONE_OFF + IMG;  // the 16 bytes behind the codes, scale first [ST][128]
  static constexpr int PLAN_OFF = SC_OFF + ST * TT * 16;
  static constexpr int SMEM_BYTES = PLAN_OFF + (3 * MAX_REQ + 4) * 4 + MAX_ROWS * 6 + 1024;
  static_assert(P_OFF % 1024 == 0 && Q_OFF % 1024 == 0 && Q_BYTES / 2 % 1024 == 0, "swizzle atoms");
  // TMEM columns: scores by slot, O by stream, scales (ones and the queries' per issuing warp)
  static constexpr int S_COL = 0, O_COL = 256, SF_ONE = O_COL + (WIDE ? 96 : 128),
                       SF_Q = SF_ONE + 4 * MMA_WARPS, SF_P = SF_Q + 8 * MMA_WARPS;
  static_assert(SF_P + (WIDE ? 0 : 4 * SLOTS) <= 512, "TMEM");
  // log2 of a weight times its token's scale: m puts the largest of the tile that moves it at BASE
  // or just below, and moves again when one passes 2^15 (narrow: 2^7); scales below 2^LEAST (and zeros)
  // count as that.  (What f16 cannot hold lies 2^-31 below that largest; narrow blocks have scales.)
  static constexpr float BASE = WIDE ? 6.0f : -30.0f, LEAST = WIDE ? -90.0f : -60.0f;
};
// registers a thread at launch; in the wide form softmax warps then take what the others give up (in
// all, the launch's)
constexpr int REGS = 80, SOFT_REGS = 88, OTHER_REGS = 64;
static_assert(SOFT_REGS * SOFT + OTHER_REGS * (THREADS - SOFT) == REGS * THREADS, "register split");

// Instruction descriptor, M = 128; N is or-ed in.
// kind::f16: f16 x f16, f32 accumulators, both MN-major.
constexpr uint32_t F16_IDESC = (1u << 4) | TRANS | ((uint32_t)(TT >> 4) << 24);

struct Args {
  CUtensorMap codes, scales;  // the cache as [pages][tokens][bytes], boxes of box tokens
  int box;                    // 0: no maps
  AttendArgs a;
  Shape sh;
  float* part;  // workspace (Pieces)
  RowInfo* rows;
};

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
// How an item's columns are dealt out (see the head of the file).
template <bool WIDE>
struct Deal {
  int nqp, lg, streams, bufs;  // columns; 2^lg streams of softmax groups; slots of scores, weights
  __device__ explicit Deal(int cols)
      : nqp(cols), lg(cols <= 16 ? 2 : cols <= 32 ? 1 : 0), streams(1 << lg), bufs(2 << lg) {}
  __device__ int slot(int i) const { return i & (bufs - 1); }
  __device__ int stream(int i) const { return i & (streams - 1); }
  __device__ uint32_t s_col(int i) const {
    return Form<WIDE>::S_COL + (slot(i) << (7 - lg));
  }
  // a stream's columns of O: both terms' of the weights in the narrow form
  __device__ uint32_t o_col(int stream) const { return Form<WIDE>::O_COL + (WIDE ? 1 : 2) * nqp * stream; }
  // where tile i's weights begin: their buffer, and the stream's place in its 128-byte rows
  __device__ bool p_odd(int i) const { return slot(i) >= streams; }
  __device__ int p_byte(int stream) const { return 2 * nqp * stream; }
  __device__ int q_byte(int item) const { return nqp <= Q_TWICE ? (item & 1) * (Form<WIDE>::Q_BYTES / 2) : 0; }
  // parity of slot(i)'s phase of an item's tile i, and the phases that an item of n tiles
  // leaves (ph: the slots' parities at its start, a bit each)
  __device__ uint32_t parity(uint32_t ph, int i) const { return ((ph >> slot(i)) ^ (i >> (lg + 1))) & 1; }
  __device__ void advance(uint32_t& ph, int n) const {
    for (int b = 0; b < bufs; ++b) ph ^= (uint32_t)((n + bufs - 1 - b) >> (lg + 1) & 1) << b;
  }
};

// What the softmax needs of an item beside its span, made with the item's queries.
template <bool WIDE>
struct Meta {
  static constexpr int NQ = Form<WIDE>::NQ;
  int cols, nrows;
  int row[GROUP], pos[GROUP];
  // where a column's queries are, where its first value goes, and its slice (-1: padding)
  long long query[NQ];
  alignas(16) long long out[NQ];
  alignas(16) int slice[NQ];
};
template <bool WIDE>
struct Shared {
  static constexpr int NQ = Form<WIDE>::NQ, ST = Form<WIDE>::ST, CMAX = Form<WIDE>::CMAX;
  uint64_t full[ST], k_free[ST], s_full[SLOTS], p_full[SLOTS], pv_done[SLOTS], v_full[2], v_free[2];
  uint64_t q_full[2], q_free[2], m_free[2], o_free, drain;
  alignas(16) float neg_m[NQ];
  float fac[NQ], red[SOFT_WARPS][CMAX];  // m and its change: [stream][column]
  uint32_t most[SOFT_WARPS][CMAX];  // the warp's columns' largest weights (mb)
  uint32_t valid[ST][4];  // tokens that are there
  alignas(16) float fin[4][NQ];  // a column's factor for each stream's O
  Meta<WIDE> meta[2];
  uint32_t tmem;
  int abort;
  Jobs start;
};
static_assert(Form<false>::SMEM_BYTES + sizeof(Shared<false>) <= 227 * 1024, "shared memory");
static_assert(Form<true>::SMEM_BYTES + sizeof(Shared<true>) <= 227 * 1024, "shared memory");

// Sums, or maxima, of N columns over the warp's lanes: lane k gets column k % N's.
template <int N, bool MAX>
__device__ __forceinline__ float over_lanes(float* l) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int x = N / 2; x > 0; x >>= 1) {
#pragma unroll
    for (int c = 0; c < x; ++c) {
      const bool up = lane & x;
      const float give = up ? l[c] : l[c + x], keep = up ? l[c + x] : l[c];
      const float got = __shfl_xor_sync(0xffffffffu, give, x);
      l[c] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
#pragma unroll
  for (int x = N; x < 32; x <<= 1) {
    const float got = __shfl_xor_sync(0xffffffffu, l[0], x);
    l[0] = MAX ? fmaxf(l[0], got) : l[0] + got;
  }
  return l[0];
}
// What a softmax warp knows of its item.
struct Soft {
  Span span;
  int t0, n, it;      // the item's first tile and tile count, the ring's next tile
  Clear clear;
  int c0, flat;       // this group's first column, of all and of all streams' m
  int first, stride;  // the group's tiles
  int arrive;         // arrivals of each warp at a tile's weights (SOFT_WARPS from all of them)
  int cheads;         // columns of a row
  float to_log2;
  uint32_t tmem;      // with the warp's lane quadrant
  uint32_t ph;        // the slots' barriers' phases at the item's start
};

// The softmax of a group's columns over its tiles of an item, a token per thread; leaves the
// thread's share of every column's sum, in units of 2^m.
template <bool WIDE, int C>
__device__ __forceinline__ void soft_tiles(const AttendArgs& a, const Soft& w, const Deal<WIDE>& deal,
                                           const Meta<WIDE>& meta, Shared<WIDE>& sh, uint8_t* sm,
                                           float* l) {
  using F = Form<WIDE>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, group = warp >> 2, tok = 32 * quad + lane;
  volatile int* abort = &sh.abort;
  float s[C];
#pragma unroll 1
  for (int i = w.first; i < w.n; i += w.stride) {
    const int st = (w.it + i) % F::ST, b = deal.slot(i);
    wait(&sh.s_full[b], deal.parity(w.ph, i), a.status, abort);  // (and the tile's scales)
    const float raw = reinterpret_cast<const float*>(sm + F::SC_OFF)[(st * TT + tok) * 4];
    const uint32_t ok = sh.valid[st][quad];
    // (a token that is not there has whatever was left in its place: no scale)
    const bool fin = ((ok >> lane) & 1) && fabsf(raw) <= SCALE_MAX;
    const float ct = fin ? raw * w.to_log2 : __int_as_float(0x7FC00000);
    const float sc = fin ? raw : 0.0f, size = fabsf(sc);
    const float size64 = size * 0x1p-6f;
    const float lsc = sc != 0.0f ? fmaxf(log2_of(size), F::LEAST) : F::LEAST;
    if (WIDE) {  // (as many arrivals whoever takes the tile)
      __syncwarp();
      if (lane < w.arrive) mbar_arrive(&sh.k_free[st]);
    }
    // some of the tile's tokens may not be every row's to see
    const bool part = ok != 0xffffffffu || !w.clear.has(i);
    uint32_t see = 0xffffffffu;
    if (__builtin_expect(part, 0)) {  // the group's columns that see the token
      const int t = w.span.token(w.t0 + i) + tok;
#pragma unroll 1
      for (int j = 0; j < meta.nrows; ++j) {
        const int hi = a.causal ? meta.pos[j] : w.span.hi;
        const int lo = a.window > 0 ? max(0, hi - a.window + 1) : 0;
        if (((ok >> lane) & 1) && t <= hi && (t >= lo || t < a.sinks)) continue;
        // columns [c, c + cheads) of the item, from this group's first on
        const int c = j * w.cheads - w.c0;
        const int x = min(max(c, 0), 31), y = min(max(c + w.cheads, 0), 31);
        see &= ~((1u << y) - (1u << x));
      }
    }
    if (!WIDE && __builtin_expect(part && w.c0 == 0, 0)) {
      // NaN codes that some row must not see would reach it as 0 * NaN (rows that do see the token
      // are NaN by their scores); the first product has read the tile
      uint8_t* k = sm + F::K_OFF + st * K_TILE + tok * 128;
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        uint4* at = reinterpret_cast<uint4*>(k + (((e + lane) & 7) << 4));
        *at = without_nan(*at);
      }
    }
    const uint32_t scol = w.tmem + deal.s_col(i) + w.c0;
    uint32_t mb[C];
    // weights; m moves ahead of an item's first tile, and where a weight asks for it
    bool move = i == w.first, moved = false;
#pragma unroll 1
    for (;;) {
      tc_fence_after();
      if (__builtin_expect(move, 0)) {
        // the columns' largest weights times scales of the tile
#pragma unroll 1
        for (int g = 0; g < C; g += 8) {
          float x[8], y[8];
          tc_ld8(scol + g, x);
          if (!WIDE) tc_ld8(scol + deal.nqp + g, y);
          tc_wait_ld();
          tc_loaded(x);
          if (!WIDE) tc_loaded(y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // (a score that an f32 does not hold, -inf, is not one that is not seen)
            x[e] = fmaxf(fmaf(WIDE ? x[e] : x[e] + y[e], ct, lsc), -2.0f * SCORE_MAX);
            if (!((see >> (g + e)) & 1)) x[e] = -INFINITY;
          }
          const float v = over_lanes<8, true>(x);
          if (lane < 8) sh.red[warp][g + lane] = v;
        }
        bar_sync<128>(6 + group);
        if (quad == 0 && lane < C) {
          const float(*r)[F::CMAX] = sh.red + 4 * group;
          const float m = fmaxf(fmaxf(r[0][lane], r[1][lane]), fmaxf(r[2][lane], r[3][lane]));
          const float old = -sh.neg_m[w.flat + lane];
          float f = 1.0f;
          if (m - old > F::BASE) {
            const float now = fabsf(m) <= SCORE_MAX ? ceilf(m) - F::BASE : __int_as_float(0x7FC00000);
            f = old == UNSET ? 0.0f : ex2(old - now);
            sh.neg_m[w.flat + lane] = -now;
          }
          sh.fac[w.flat + lane] = f;
        }
        bar_sync<128>(6 + group);
        if (i >= w.stride) {
#pragma unroll
          for (int c = 0; c < C; ++c) l[c] *= sh.fac[w.flat + c];
          const int pi = i - w.stride;  // the group's tile before: its product is in O
          wait(&sh.pv_done[deal.slot(pi)], deal.parity(w.ph, pi), a.status, abort);
          tc_fence_after();
#pragma unroll 1
          for (int g0 = 0; g0 < (WIDE ? C : 2 * C); g0 += 8) {  // (both terms')
            float x[8];
            const int g = g0 < C ? g0 : g0 - C;
            const uint32_t oc = w.tmem + deal.o_col(w.first) + w.c0 + g + (g0 < C ? 0 : deal.nqp);
            tc_ld8(oc, x);
            tc_wait_ld();
            tc_loaded(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= sh.fac[w.flat + g + e];
            tc_st8(oc, x);
          }
          tc_wait_st();
        }
        moved = true;
      }
      float x[WIDE ? 1 : C];
#pragma unroll
      for (int g = 0; g < C; g += 8) {
        tc_ld8(scol + g, s + g);
        if (!WIDE) tc_ld8(scol + deal.nqp + g, x + g);
      }
      tc_wait_ld();
#pragma unroll
      for (int g = 0; g < C; g += 8) {
        tc_loaded(s + g);
        if constexpr (!WIDE) {
          tc_loaded(x + g);
#pragma unroll
          for (int e = 0; e < 8; e += 2) add2(s[g + e], s[g + e + 1], x[g + e], x[g + e + 1]);
        }
      }
      const float4* nm = reinterpret_cast<const float4*>(sh.neg_m + w.flat);
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
      uint32_t ask;
      if constexpr (WIDE) {
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < C; ++c) top = fmaxf(top, s[c]);
        ask = top + lsc > 15.0f;
      } else {
        // the largest weights times scales of the warp's tokens, over 2^6, as bits; 2 and more (or
        // NaN) asks for a larger m
        uint32_t any = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          s[c] = ex2(s[c]);
          mb[c] = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaf(s[c], size64, 0x1p-124f)));
          any |= mb[c];
        }
        ask = any >> 30;
      }
      if (moved) break;  // (alike in the group's warps)
      move = bar_any(2 + group, ask);
      if (__builtin_expect(!move, 1)) break;
    }
    uint8_t* prow = sm + F::P_OFF + tok * 128;
    if constexpr (WIDE) {
      // weights times scales
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
        const int col = w.c0 + g, run = col >> 6, odd = deal.p_odd(i);
        const int ch = (deal.p_byte(w.first) + 2 * (col & 63) + (run & odd) * 64) >> 4;
        *reinterpret_cast<uint4*>(prow + (run ? 2 : odd) * K_TILE + ((ch ^ (tok & 7)) << 4)) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    } else {
      // weights times scales as two e4m3 terms, 16 + 16 bytes of the token's row; a column's largest
      // of the warp's tokens is in [2^7, 2^8).  The weight meets its scale first: a weight of 0 stays
      // 0 whatever the scale, where the block's factor, 2^125 at most, times a scale may be infinite
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int g = 0; g < C; g += 4) {
#pragma unroll
        for (int c = g; c < g + 4; c += 2) {
          add2(l[c], l[c + 1], s[c], s[c + 1]);
          mul2(s[c], s[c + 1], sc);
          // 2 / the power of two of mb
          mul2(s[c], s[c + 1], __uint_as_float(~mb[c] & 0x7F800000u), __uint_as_float(~mb[c + 1] & 0x7F800000u));
        }
        hilo_x4(s + g, hi[g / 4], lo[g / 4]);
      }
      if (lane == 0) {
#pragma unroll
        for (int g = 0; g < C; g += 4)
          *reinterpret_cast<uint4*>(&sh.most[warp][g]) = make_uint4(mb[g], mb[g + 1], mb[g + 2], mb[g + 3]);
      }
      const int ch = (deal.p_byte(w.first) + w.c0) >> 4, cl = ch + (deal.nqp >> 4);
      prow += deal.p_odd(i) * K_TILE;
      *reinterpret_cast<uint4*>(prow + ((ch ^ (tok & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(prow + ((cl ^ (tok & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      __syncwarp();
      {
        const int n = w.c0 + (lane & 15) + (lane >> 4) * deal.nqp;
        sm[F::PIMG_OFF + b * IMG + (n & 31) * 16 + (n >> 5) * 4 + quad] =
            (uint8_t)((sh.most[warp][lane & 15] >> 23) - 1);
      }
    }
    fence_proxy_async_shared();
    tc_fence_before();
    __syncwarp();
    if (lane < w.arrive) mbar_arrive(&sh.p_full[b]);
  }
}

template <bool WIDE>
__global__ void __maxnreg__(REGS) attend_kernel(const __grid_constant__ Args ar) {
  using F = Form<WIDE>;
  constexpr int NQ = F::NQ, ST = F::ST, PREP_WARP = F::PREP_WARP, PREP = F::PREP, S_WARP = F::S_WARP,
                O_WARP = F::O_WARP, MMA_WARPS = F::MMA_WARPS, LOAD_WARP = F::LOAD_WARP,
                LOAD_WARPS = F::LOAD_WARPS;
  const AttendArgs& a = ar.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + (-smem_u32(smem_raw) & 1023);  // (still a shared pointer to the compiler)
  __shared__ __align__(16) Shared<WIDE> ss;
  volatile int* abort = &ss.abort;
  Plan plan;
  plan.pre = reinterpret_cast<int*>(sm + F::PLAN_OFF);
  plan.pmax = plan.pre + MAX_REQ + 4;
  plan.pmin = plan.pmax + MAX_REQ;
  plan.pos = plan.pmin + MAX_REQ;
  plan.req = reinterpret_cast<short*>(plan.pos + MAX_ROWS);
  plan.cnt = nullptr;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Shape& sh = ar.sh;
  const int team = blockIdx.x / sh.chunks, chunk = blockIdx.x - team * sh.chunks;
  const int chunk_bytes = min(128, a.kv_dim - 128 * chunk);

  if (tid == 0) {
    // a tile is free when its second product is done, or in the wide form when the first product,
    // the widening and the softmax warps have read it
    for (int s = 0; s < ST; ++s)
      mbar_init(&ss.full[s], 1), mbar_init(&ss.k_free[s], WIDE ? 1 + PREP / 32 + SOFT_WARPS : 1);
    for (int s = 0; s < 2; ++s) mbar_init(&ss.v_full[s], PREP / 32), mbar_init(&ss.v_free[s], 1);
    for (int s = 0; s < SLOTS; ++s)
      mbar_init(&ss.s_full[s], 2), mbar_init(&ss.pv_done[s], 1), mbar_init(&ss.p_full[s], SOFT_WARPS);
    // an item's queries are free with its first products, the rest of what was made with them when
    // all that read it or wait for it are done
    for (int s = 0; s < 2; ++s)
      mbar_init(&ss.q_full[s], PREP / 32), mbar_init(&ss.q_free[s], MMA_WARPS),
          mbar_init(&ss.m_free[s], MMA_WARPS + SOFT_WARPS);
    mbar_init(&ss.o_free, SOFT_WARPS);
    mbar_init(&ss.drain, 2 * MMA_WARPS);
    ss.abort = 0;
    fence_mbar_init();
  }
  if (warp == S_WARP) tmem_alloc<512>(&ss.tmem);
  for (int i = tid; i < (F::SC_OFF - F::PIMG_OFF) / 4; i += THREADS)
    reinterpret_cast<uint32_t*>(sm + F::PIMG_OFF)[i] = 0x7F7F7F7Fu;
  fence_proxy_async_shared();

  derive_plan<THREADS>(a, sh, plan, team, team < sh.teams, &ss.start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ss.tmem;
  Jobs items = ss.start;
  Job im = {};

  // An item's rows and queries, by N threads (t: 0..N - 1, whole warps); before: the last item's one
  // buffer of queries has to be free.
  const int hpg = a.n_q / (a.kv_dim / a.head_dim);
  const int cheads = hpg * (chunk_bytes > a.head_dim ? 2 : 1);  // heads per row of this chunk
  const int dshift = a.head_dim == 64 ? 6 : 7;
  auto prepare = [&](auto threads, int item, int t, bool before) {
    constexpr int N = decltype(threads)::value, BAR = N == PREP ? 1 : 12;
    const int qb = item & 1;
    Meta<WIDE>& meta = ss.meta[qb];
    if (t < 32) {
      const int n = group_rows(a, sh, plan, im.b, im.group, meta.row, meta.pos);
      const int cols = (n * cheads + 15) & ~15;
      if (lane == 0) meta.cols = cols == 80 ? 96 : cols, meta.nrows = n;  // (four groups' columns)
    }
    bar_sync<N>(BAR);
    const int nqp = meta.cols, nq = meta.nrows * cheads;
    if (t < NQ) {  // a column per thread: its head of the chunk, and where its queries and its results are
      const bool whole = im.n == im.span.tiles;  // nobody else has tiles of this group
      const int slot = (team * 2 + (im.t0 > 0 ? 0 : 1)) * sh.chunks + chunk;
      const int j = t / cheads, h = t - j * cheads;
      const int at = (chunk * sh.heads + h) * a.head_dim, r = t < nq ? meta.row[j] : 0;
      meta.slice[t] = t < nq ? (h >= hpg ? 1 : 0) : -1;
      meta.query[t] = r * a.q_stride + at;
      meta.out[t] = whole ? r * a.o_stride + at : (long long)(slot * NQ + t) * PART_LD + 4;
    }
    const bool once = nqp > Q_TWICE;  // (the one buffer that both halves are)
    if (item > 0 && (once || before)) wait(&ss.q_free[qb ^ 1], ((item - 1) >> 1) & 1, a.status, abort);
    bar_sync<N>(BAR);
    // queries as two e4m3 terms, rows of 128 bytes: hi in row c, lo in row nqp + c.  A thread takes
    // 8 dimensions of every so-manieth column; their 16 bytes are copied to where its codes go
    const int d = (t & 15) * 8, sl = d >> dshift, o = d >> 4;
    const __nv_bfloat16* q = a.q + (d - (sl << dshift));
    uint8_t* to = sm + F::Q_OFF + (once ? 0 : qb * (F::Q_BYTES / 2)) + (d & 8);
    uint8_t* img = sm + F::QIMG_OFF + qb * IMG + (d >> 5);
    auto place = [&](int r) { return to + r * 128 + ((o ^ (r & 7)) << 4); };
#pragma unroll 1
    for (int c = t >> 4; c < nqp; c += N / 16) {
      const bool in = c < nq && meta.slice[c] == sl;
      const __nv_bfloat16* from = in ? q + meta.query[c] : a.q;
      cp_async8(place(c), from, in ? 8 : 0);
      cp_async8(place(nqp + c), from + (in ? 4 : 0), in ? 8 : 0);
    }
    cp_async_wait_all();
#pragma unroll 1
    for (int c = t >> 4; c < nqp; c += N / 16) {
      uint2* hi = reinterpret_cast<uint2*>(place(c));
      uint2* lo = reinterpret_cast<uint2*>(place(nqp + c));
      const uint32_t code = split_query(make_uint4(hi->x, hi->y, lo->x, lo->y), *hi, *lo);
      if ((d & 31) == 0) {
        img[(c & 31) * 16 + (c >> 5) * 4] = (uint8_t)code;
        if (!WIDE) img[((nqp + c) & 31) * 16 + ((nqp + c) >> 5) * 4] = (uint8_t)code;
      }
    }
    fence_proxy_async_shared();
  };
  bool more = next_job(a, sh, plan, items, im);
  // the first item's by all but the loading warps, then by their own warps, ahead of their use
  if (more && warp < LOAD_WARP) {
    prepare(std::integral_constant<int, 32 * LOAD_WARP>(), 0, tid, false);
    bar_sync<32 * LOAD_WARP>(12);
  }

  if (warp >= SOFT_WARPS) {
    if constexpr (WIDE) regs_down<OTHER_REGS>();
    if (warp >= LOAD_WARP) {
      // ---------------------- loads: each slot of the ring has one loading warp (every other slot's:
      // a wait by parity is for the phase that is meant only where the waiter saw the one before)
      const int lw = warp - LOAD_WARP;
      int ni = lw;
      TileLoader tile(ar.box);
      auto locate = [&]() {
#pragma unroll 1
        while (more && ni >= im.n) ni -= im.n, more = next_job(a, sh, plan, items, im);
        if (more) tile.locate(a, im, ni);
      };
      locate();
#pragma unroll 1
      for (int it = lw; more;) {
        const int s = it % ST;
        bool go = true;
        if (it >= ST) go = wait(&ss.k_free[s], ((it / ST) - 1) & 1, a.status, abort);
        tile.load(a, im, ar.codes, ar.scales, chunk, sm + F::K_OFF + s * K_TILE, sm + F::SC_OFF + s * TT * 16,
                  ss.valid[s], &ss.full[s], go);
        const int step = ST % LOAD_WARPS == 0 || s + LOAD_WARPS < ST ? LOAD_WARPS : ST - s + lw;
        it += step;
        ni += step;
        locate();
      }
    } else if (warp >= PREP_WARP && warp < PREP_WARP + PREP / 32) {
      // ---------------------- the items' rows and queries, and in the wide form the tiles' widening
      const int ptid = tid - 32 * PREP_WARP;
      int it = 0;
      bool before = false;  // the item before had more than Q_TWICE columns
#pragma unroll 1
      for (int item = 0; more; ++item, more = next_job(a, sh, plan, items, im)) {
        const int qb = item & 1;
        if (item >= 2) {
          wait(&ss.q_free[qb], ((item >> 1) - 1) & 1, a.status, abort);
          wait(&ss.m_free[qb], ((item >> 1) - 1) & 1, a.status, abort);
        }
        if (item > 0) prepare(std::integral_constant<int, PREP>(), item, ptid, before);
        before = ss.meta[qb].cols > Q_TWICE;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.q_full[qb]);
        const Meta<WIDE>& meta = ss.meta[qb];
        if constexpr (WIDE) {  // a warp widens 32 tokens of every tile
          const Clear clear = clear_tiles(a, im, meta);
          const int lw = warp - PREP_WARP, piece = lane & 7, r4 = lane >> 3;
#pragma unroll 1
          for (int i = 0; i < im.n; ++i, ++it) {
            const int s = it % ST, b = it & 1;
            wait(&ss.full[s], (it / ST) & 1, a.status, abort);
            if (it >= 2) wait(&ss.v_free[b], ((it >> 1) - 1) & 1, a.status, abort);
            const bool part = ss.valid[s][lw] != 0xffffffffu || !clear.has(i);
            const uint8_t* src = sm + F::K_OFF + s * K_TILE + 32 * lw * 128;
            uint8_t* dst = sm + F::V_OFF + b * V_TILE + (piece >> 2) * K_TILE + 32 * lw * 128;
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
                // a NaN code that some row must not see would reach it as 0 * NaN (rows that do see
                // the token are NaN by their scores)
                if (__builtin_expect(part, 0)) v[e] = without_nan(v[e]);
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
        }
      }
    } else if (warp >= S_WARP && warp < S_WARP + MMA_WARPS) {
      // ------------------ the first product's MMAs (two warps: each issues every other tile's)
      const int mine = warp - S_WARP;
      const uint64_t k0 = desc_sw128(smem_u32(sm + F::K_OFF)), q0 = desc_sw128(smem_u32(sm + F::Q_OFF));
      const uint32_t sf = tmem + F::SF_Q + 8 * mine, ones = tmem + F::SF_ONE + 4 * mine;
      int it = 0;
      uint32_t ph = 0;
      if (elect_one()) tc_cp_img(ones, sm + F::ONE_OFF);
      __syncwarp();
#pragma unroll 1
      for (int item = 0; more; ++item, more = next_job(a, sh, plan, items, im)) {
        const int qb = item & 1;
        wait(&ss.q_full[qb], (item >> 1) & 1, a.status, abort);
        const Deal<WIDE> deal(ss.meta[qb].cols);
        // the queries' terms: two columns of the scores each, or added up (wide)
        const int n = WIDE ? deal.nqp : 2 * deal.nqp;
        const uint32_t idesc = IDESC | ((uint32_t)(n >> 3) << 17);
        const uint64_t qd = q0 + (deal.q_byte(item) >> 4);
        if (elect_one()) {
          const uint8_t* img = sm + F::QIMG_OFF + qb * IMG;
          tc_cp_img(sf, img);
        }
        __syncwarp();
#pragma unroll 1
        for (int i = mine; i < im.n; i += MMA_WARPS) {
          const int st = (it + i) % ST, b = deal.slot(i);
          bool ok = wait(&ss.full[st], ((it + i) / ST) & 1, a.status, abort);
          // the slot's scores and weights are no longer in use
          if (i >= deal.bufs)
            ok &= wait(&ss.pv_done[b], deal.parity(ph, i - deal.bufs), a.status, abort);
          if (ok && elect_one()) {
            tc_fence_after();
            const uint64_t kd = k0 + st * (K_TILE / 16);
#pragma unroll
            for (int k = 0; k < (WIDE ? 8 : 4); ++k)
              tc_mma_mxf8(tmem + deal.s_col(i), kd + 2 * (k & 3), qd + 2 * (k & 3) + (k >> 2) * (n * 128 / 16),
                          idesc | ((uint32_t)(k & 3) << 4) | ((uint32_t)(k & 3) << 29), ones, sf, k > 0);
            tc_commit(&ss.s_full[b]);
            if (WIDE) tc_commit(&ss.k_free[st]);
            // This thread has waited for the copies, and its arrival here (a release; the commit's is
            // none) passes what they wrote on to the softmax warps, which read the scales and, to
            // clear masked codes, the tile behind this barrier alone.
            mbar_arrive(&ss.s_full[b]);
          }
          __syncwarp();
        }
        if (elect_one()) tc_commit(&ss.q_free[qb]);
#pragma unroll 1
        for (int i = max(0, im.n - MMA_WARPS); i < im.n; ++i)  // all are done when each warp's last is
          wait(&ss.pv_done[deal.slot(i)], deal.parity(ph, i), a.status, abort);
        // (neither runs ahead of the phases that the other waits for)
        if (MMA_WARPS > 1) bar_sync<32 * MMA_WARPS>(11);
        it += im.n;
        deal.advance(ph, im.n);
      }
      if (elect_one()) tc_commit(&ss.drain);  // (what was issued has completed at this arrival)
      __syncwarp();
    } else if (warp >= O_WARP && warp < O_WARP + MMA_WARPS) {
      // ------------- the second product's MMAs (two warps: each issues every other tile's, so that it
      // has its own streams' O; the first one all where there is one stream)
      const int mine = warp - O_WARP;
      const uint64_t k0 = desc_sw128(smem_u32(sm + F::K_OFF)), v0 = desc_mn(smem_u32(sm + F::V_OFF), K_TILE);
      // first, where the second kernel finds the rows' results
#pragma unroll 1
      for (int r = blockIdx.x + mine * gridDim.x; r < a.rows; r += MMA_WARPS * gridDim.x) {
        const RowInfo info = row_info(a, sh, plan, r);
        if (lane == 0) ar.rows[r] = info;
      }
      int it = 0;
      uint32_t ph = 0;
#pragma unroll 1
      for (int item = 0; more; ++item, more = next_job(a, sh, plan, items, im)) {
        wait(&ss.q_full[item & 1], (item >> 1) & 1, a.status, abort);
        const Deal<WIDE> deal(ss.meta[item & 1].cols);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.m_free[item & 1]);
        const int step = deal.streams == 1 ? 1 : MMA_WARPS;
        const int first = mine < step ? mine : im.n;
        // (only where this warp has tiles: it may miss phases of other items)
        if (item > 0 && first < im.n) wait(&ss.o_free, (item - 1) & 1, a.status, abort);
        const uint32_t idesc = WIDE ? F16_IDESC | ((uint32_t)(deal.nqp >> 3) << 17)
                                    : IDESC | TRANS | ((uint32_t)(2 * deal.nqp >> 3) << 17);
#pragma unroll 1
        for (int i = first; i < im.n; i += step) {
          const int b = deal.slot(i), stream = deal.stream(i), st = (it + i) % ST;
          bool ok = wait(&ss.p_full[b], deal.parity(ph, i), a.status, abort);
          if (WIDE) ok &= wait(&ss.v_full[(it + i) & 1], ((it + i) >> 1) & 1, a.status, abort);
          if (ok && elect_one()) {
            tc_fence_after();
            const int odd = deal.p_odd(i);
            const uint32_t p = smem_u32(sm + F::P_OFF) + odd * K_TILE + deal.p_byte(stream);
            const uint32_t oc = tmem + deal.o_col(stream);
            if constexpr (WIDE) {
              const uint64_t vd = v0 + ((it + i) & 1) * (V_TILE / 16);
              // (columns from 64: behind both buffers, the second one's 64 bytes further)
              const uint64_t pd = desc_mn(p, (2 - odd) * K_TILE + 64 * odd);
#pragma unroll
              for (int k = 0; k < 8; ++k)  // 16 tokens each
                tc_mma_f16(oc, vd + k * (2048 / 16), pd + k * (2048 / 16), idesc, i >= deal.streams || k > 0);
            } else {
              const uint32_t sf = tmem + F::SF_P + 4 * b, ones = tmem + F::SF_ONE + 4 * (i & 1);
              tc_cp_img(sf, sm + F::PIMG_OFF + b * IMG);
              const uint64_t kd = k0 + st * (K_TILE / 16), pd = desc_sw128(p);
#pragma unroll
              for (int k = 0; k < 4; ++k)  // 32 tokens each
                tc_mma_mxf8(oc, kd + k * (4096 / 16), pd + k * (4096 / 16),
                            idesc | ((uint32_t)k << 4) | ((uint32_t)k << 29), ones, sf,
                            i >= deal.streams || k > 0);
            }
            tc_commit(&ss.pv_done[b]);
            tc_commit(WIDE ? &ss.v_free[(it + i) & 1] : &ss.k_free[st]);
          }
          __syncwarp();
        }
        it += im.n;
        deal.advance(ph, im.n);
      }
      if (elect_one()) tc_commit(&ss.drain);
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------------------- softmax
    if constexpr (WIDE) regs_up<SOFT_REGS>();
    const int quad = warp & 3, group = warp >> 2;
    Soft w;
    w.it = 0;
    w.ph = 0;
    w.cheads = cheads;
    w.to_log2 = a.scale * LOG2E;
    w.tmem = tmem + ((uint32_t)(32 * quad) << 16);
#pragma unroll 1
    for (int item = 0; more; ++item, more = next_job(a, sh, plan, items, im)) {
      wait(&ss.q_full[item & 1], (item >> 1) & 1, a.status, abort);
      const Meta<WIDE>& meta = ss.meta[item & 1];
      const Deal<WIDE> deal(meta.cols);
      const int nqp = deal.nqp, nq = meta.nrows * cheads;
      const bool whole = im.n == im.span.tiles;
      w.span = im.span;
      w.t0 = im.t0;
      w.n = im.n;
      w.first = group & (deal.streams - 1);
      w.stride = deal.streams;
      const int share = WIDE && nqp > 64 ? 24 : 16;  // columns of a group
      w.c0 = (group >> deal.lg) * share;
      w.flat = nqp * w.first + w.c0;
      w.arrive = deal.streams + (nqp == 48 && group == 0 ? 1 : 0);  // (the fourth group is idle)
      w.clear = clear_tiles(a, im, meta);
      float l[F::CMAX];
#pragma unroll
      for (int c = 0; c < F::CMAX; ++c) l[c] = 0.0f;
      if (w.c0 < nqp) {
        if (quad == 0 && lane < share) ss.neg_m[w.flat + lane] = -UNSET;
        bar_sync<128>(6 + group);
        if (share == 16)
          soft_tiles<WIDE, 16>(a, w, deal, meta, ss, sm, l);
        else
          soft_tiles<WIDE, F::CMAX>(a, w, deal, meta, ss, sm, l);
      }
      // every product of the item is done when each issuing warp's last is (a group that has no part in
      // a tile may pass its barrier a phase early; the barrier below holds it until those that have are here)
#pragma unroll 1
      for (int i = max(0, w.n - MMA_WARPS); i < w.n; ++i)
        wait(&ss.pv_done[deal.slot(i)], deal.parity(w.ph, i), a.status, abort);
      tc_fence_after();
      w.it += im.n;
      deal.advance(w.ph, im.n);

      // ---- the item's result: the columns' sums over the tokens, then O
      {
        const float v = over_lanes<16, false>(l);
        if (lane < 16) ss.red[warp][lane] = v;
      }
      if constexpr (WIDE) {
        const float v = over_lanes<8, false>(l + 16);
        if (lane < 8) ss.red[warp][16 + lane] = v;
      }
      bar_sync<SOFT>(10);
      if (warp < ((nq << deal.lg) + 31) / 32) {
        // the streams' sums and O in the largest m (one stream: as they are); a lane per column and
        // stream
        const int c = tid >> deal.lg, k = tid & (deal.streams - 1);
        const bool live = c < nq && k < im.n;
        float mk = UNSET, lk = 0.0f;
        if (live) {
          const int g = k + (c / share << deal.lg), at = c % share;
          const float(*r)[F::CMAX] = ss.red + 4 * g;
          mk = -ss.neg_m[nqp * k + c];
          lk = (r[0][at] + r[1][at]) + (r[2][at] + r[3][at]);
        }
        float m = mk;
#pragma unroll 1
        for (int x = 1; x < deal.streams; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        float f = lk != lk ? 1.0f : mk == UNSET ? 0.0f : ex2(mk - m);  // (a NaN stays one)
        float lt = f != 0.0f ? lk * f : 0.0f;
#pragma unroll 1
        for (int x = 1; x < deal.streams; x <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, x);
        if (whole) f = lt == 0.0f ? 0.0f : f / lt;
        if (live) ss.fin[k][c] = f;
        if (live && k == 0) {
          if (whole) {
            const int j = c / cheads;
            a.lse[(long long)meta.row[j] * a.n_q + chunk * sh.heads + c - j * cheads] =
                lt == 0.0f ? -INFINITY : (log2f(lt) + m) * LN2;
          } else {
            ar.part[meta.out[c] - 4] = m;
            ar.part[meta.out[c] - 3] = lt;
          }
        }
      }
      bar_sync<SOFT>(10);
      tc_fence_after();
      const int d = 32 * quad + lane;  // this thread's dimension of the chunk
      const int sl = d >> dshift, dl = d - (sl << dshift);
#pragma unroll 1
      for (int c4 = 4 * group; c4 < nqp; c4 += 4 * GROUPS) {
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int k = 0; k < min(deal.streams, im.n); ++k) {
          float x[4], y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          tc_ld4(w.tmem + deal.o_col(k) + c4, x);
          if (!WIDE) tc_ld4(w.tmem + deal.o_col(k) + nqp + c4, y);
          const float4 f = *reinterpret_cast<const float4*>(&ss.fin[k][c4]);
          tc_wait_ld();
          tc_loaded4(x);
          if (!WIDE) tc_loaded4(y);
          if (f.x != 0.0f) v[0] = fmaf(x[0] + y[0], f.x, v[0]);
          if (f.y != 0.0f) v[1] = fmaf(x[1] + y[1], f.y, v[1]);
          if (f.z != 0.0f) v[2] = fmaf(x[2] + y[2], f.z, v[2]);
          if (f.w != 0.0f) v[3] = fmaf(x[3] + y[3], f.w, v[3]);
        }
        const int4 mine = *reinterpret_cast<const int4*>(&meta.slice[c4]);
        const longlong2 a0 = *reinterpret_cast<const longlong2*>(&meta.out[c4]);
        const longlong2 a1 = *reinterpret_cast<const longlong2*>(&meta.out[c4 + 2]);
        if (whole) {
          __nv_bfloat16* to = a.o + dl;
          if (mine.x == sl) to[a0.x] = __float2bfloat16_rn(v[0]);
          if (mine.y == sl) to[a0.y] = __float2bfloat16_rn(v[1]);
          if (mine.z == sl) to[a1.x] = __float2bfloat16_rn(v[2]);
          if (mine.w == sl) to[a1.y] = __float2bfloat16_rn(v[3]);
        } else {
          float* to = ar.part + dl;
          if (mine.x == sl) to[a0.x] = v[0];
          if (mine.y == sl) to[a0.y] = v[1];
          if (mine.z == sl) to[a1.x] = v[2];
          if (mine.w == sl) to[a1.y] = v[3];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss.o_free), mbar_arrive(&ss.m_free[item & 1]);
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
  // the wide form's register split adds up to what a block launches with
  cudaFuncAttributes f;
  cudaError_t e = cudaFuncGetAttributes(&f, attend_kernel<true>);
  if (e == cudaSuccess && f.numRegs != REGS) e = cudaErrorInvalidConfiguration;
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attend_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Form<true>::SMEM_BYTES);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attend_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Form<false>::SMEM_BYTES);
  return e;
}

cudaError_t launch_attend_tc(const Launch& L, const AttendArgs& a, const attend::Pieces& ws, int sms) {
  const int chunks = (a.kv_dim + 127) / 128;
  const Shape narrow = shape_of(a, TT, Form<false>::NQ, sms / chunks, Form<false>::EXTRA);
  const bool wide = (a.rows + a.n_req - 1) / a.n_req * narrow.heads > WIDE_FROM;
  Args ar = {{}, {}, 0, a, wide ? shape_of(a, TT, Form<true>::NQ, sms / chunks, Form<true>::EXTRA) : narrow,
             ws.part, ws.rows};
  ar.box = encode_cache_maps(&ar.codes, &ar.scales, a);
  const cudaError_t e =
      wide ? launch_ex(L, dim3(sms), dim3(THREADS), Form<true>::SMEM_BYTES, attend_kernel<true>, ar)
           : launch_ex(L, dim3(sms), dim3(THREADS), Form<false>::SMEM_BYTES, attend_kernel<false>, ar);
  return e == cudaSuccess ? attend::launch_join(L, a, ar.sh, ws) : e;
}

}  // namespace mono
