// Attention of a step's rows over the paged fp8 cache, split over the context, on the
// 5th-generation tensor cores.
//
//   S[t, q] = scale * scale_t * (codes_t . q)     (token t, query q = one head of one row)
//   P[t, q] = 2^(S log2e - m_q)                   O[d, q] = sum_t codes_t[d] scale_t P[t, q]
//
// A 128-byte run of a record (a chunk: one 128-wide latent slice, or two 64-wide ones) and 128
// tokens make a tile, and both products take it as it lies in the cache: e4m3, 128 bytes a
// token, is a K-major A operand of the first (M = tokens, K = dimensions) and, transposed, an
// MN-major A operand of the second (M = dimensions, K = tokens).  So queries are the MMA's N:
// the heads that share a latent slice, times the rows of a request that share its context (1 to
// 96 columns, no padding beyond 16), and the cache is read once for all of them.
// kind::mxf8f6f4 takes the other operand as e4m3 under one power-of-two scale per 32 K
// elements.  A bf16 query is the exact sum of two such terms; P scale_t gets its scale per
// (query, 32 tokens) from the largest of the 32, and two terms carry 8 bits of each and no
// less than 2^-21 of that largest.  O stays in TMEM over a whole run of tiles: m_q, an
// integer, moves only when a score passes it by 2^40 (then O is rescaled, exactly).
//
// Work: the tiles of all (request, group of rows) pairs in one line, cut evenly into as many
// pieces as there are teams; a team is one CTA per chunk, so that the CTAs that read the same
// records run side by side.  Every CTA derives the cut from the step's positions and requests.
// A pair that falls into one piece is finished there; pieces of the others leave (O, m, l) in
// the workspace, which a second kernel joins.
//
// Roles: warps 0-7 softmax (TMEM lane quadrant = warp % 4: one token per thread; warp / 4: half
// of the columns), 8-11 loads (cp.async through the page table, any page size), 12 MMA issue.
// Every mbarrier wait is bounded; a wait that runs out is reported, and from then on every role
// runs its loop without waiting, copying or issuing, so that the barriers among warps still
// complete and TMEM is freed.
#include "cache_kernels.h"
#include "tc_common.cuh"

namespace mono {
namespace {

using namespace tc;

constexpr int TT = 128;        // tokens per tile
constexpr int NQ = 96;         // query columns at most
constexpr int MERGE = 64;      // up to here both terms are columns of one MMA
constexpr int GROUP = 16;      // rows of a group at most
constexpr int ALT = 48;        // up to here the two softmax halves take turns with whole tiles
constexpr int ST = 6;          // tiles in the ring
constexpr int MAX_REQ = 1024;
constexpr int THREADS = 16 * 32;
constexpr int SOFT_WARPS = 8, LOAD_WARP = 8, LOAD_WARPS = 4, MMA_WARP = 12;
// registers a thread: softmax warps take what the others give up (in all, the launch's 128)
constexpr int SOFT_REGS = 200, OTHER_REGS = 56;
static_assert(SOFT_REGS * 256 + OTHER_REGS * 256 == 128 * THREADS, "register split");
constexpr float JUMP = 40.0f;      // log2 of how far a weight may pass 1
constexpr float UNSET = -1.0e30f;  // m_q of a query that has seen no token
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

constexpr int K_OFF = 0;
constexpr int P_BUF = 2 * TT * 128;  // hi terms, then lo terms (merged: hi and lo in the first)
constexpr int P_OFF = K_OFF + ST * TT * 128;
constexpr int Q_OFF = P_OFF + 2 * P_BUF;  // hi rows, then lo rows
constexpr int IMG = 512;
constexpr int PIMG_OFF = Q_OFF + 2 * NQ * 128;  // [2 buffers]
constexpr int QIMG_OFF = PIMG_OFF + 2 * IMG;
constexpr int ONE_OFF = QIMG_OFF + IMG;
constexpr int SC_OFF = ONE_OFF + IMG;  // token scales [ST][128]
constexpr int PLAN_OFF = SC_OFF + ST * TT * 4;
constexpr int SMEM_BYTES = PLAN_OFF + (MAX_REQ + 1) * 8 + 2 * MAX_REQ * 4 + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
static_assert(P_OFF % 1024 == 0 && Q_OFF % 1024 == 0 && (NQ * 128) % 1024 == 0, "swizzle atoms");

// TMEM columns
constexpr int S_COL = 0, O_COL = 256, O_ALT = 96, SF_ONE = 480, SF_Q = 484, SF_P = 488;
// Instruction descriptor of kind::mxf8f6f4: e4m3 x e4m3, E8M0 scales, M = 128; N, the scale-byte
// selectors and the transposes are or-ed in.
constexpr uint32_t IDESC = (1u << 23) | ((uint32_t)(TT >> 4) << 24);
constexpr uint32_t TRANS = (1u << 15) | (1u << 16);

// The step as every CTA derives it: per request its rows' largest and smallest position, and
// the units (tiles times row groups) of all requests before it.
struct Plan {
  long long* pre;  // [n_req + 1]
  int *pmax, *pmin;
};

// What the rows of a request see, in tiles: [0, head) and [body, body + tiles - head).
struct Span {
  int hi, lo, head, body, tiles;
  __device__ int token(int i) const { return (i < head ? i : body + i - head) * TT; }
};

struct Shape {
  int width;     // bytes of the chunk: 128, or 64 in the last of an odd number of 64-wide slices
  int heads;     // heads per row in a full chunk
  int rows_per;  // rows of a group
  int chunks, teams;
};

__device__ __forceinline__ Shape shape_of(const AttendArgs& a, int grid) {
  Shape s;
  const int hpg = a.n_q / (a.kv_dim / a.head_dim);
  s.heads = hpg * (a.head_dim == 64 && a.kv_dim > 64 ? 2 : 1);
  s.rows_per = min(GROUP, NQ / s.heads);
  s.chunks = (a.kv_dim + 127) / 128;
  s.teams = grid / s.chunks;
  s.width = 128;
  return s;
}

__device__ __forceinline__ Span span_of(const AttendArgs& a, int pmax, int pmin) {
  Span s;
  s.hi = pmax;
  const int first = a.causal ? pmin : pmax;
  s.lo = a.window > 0 ? max(0, first - a.window + 1) : 0;
  const long long cap = (long long)a.kv.max_blocks * a.kv.block_size;  // fits 31 bits
  const int last = min(pmax, (int)cap - 1);
  const int lo = min(s.lo, (int)cap);
  const int b0 = lo / TT, b1 = last >= lo ? last / TT + 1 : b0;
  s.head = min((min(min(a.sinks, s.lo), (int)cap) + TT - 1) / TT, b0);
  s.body = b0;
  s.tiles = s.head + b1 - b0;
  return s;
}

// One piece of work of a team: tiles [t0, t0 + n) of a row group of a request.
struct Item {
  int b, group, t0, n;
  Span span;
};

// The items of a team in order: fn(item) for each.
template <class F>
__device__ __forceinline__ void for_items(const AttendArgs& a, const Plan& p, const Shape& sh,
                                          int team, F&& fn) {
  const long long W = p.pre[a.n_req];
  long long w = W * team / sh.teams;
  const long long w1 = W * (team + 1) / sh.teams;
  if (w >= w1) return;
  int b = 0;
  for (int step = MAX_REQ / 2; step > 0; step >>= 1)  // the last request that starts at or before w
    if (b + step < a.n_req && p.pre[b + step] <= w) b += step;
  while (w < w1) {
    while (p.pre[b + 1] <= w) ++b;
    Item it;
    it.b = b;
    it.span = span_of(a, p.pmax[b], p.pmin[b]);
    const long long u = w - p.pre[b];
    it.group = (int)(u / it.span.tiles);
    it.t0 = (int)(u - (long long)it.group * it.span.tiles);
    it.n = (int)min((long long)(it.span.tiles - it.t0), w1 - w);
    fn(it);
    w += it.n;
  }
}

// Where row r's results are: its request's and group's units [g0, g0 + tiles) and its place in
// the group; tiles 0: nothing to see.
struct RowInfo {
  long long g0;
  int tiles, place;
};

struct Args {
  AttendArgs a;
  float* part;     // [teams][2 slots][chunks][NQ][128 + 2]: O, then m and l
  RowInfo* rows;   // [rows]
  long long* total;  // units of the step
};
constexpr int PART_LD = 128 + 4;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two f16 values as e4m3 hi codes and the codes of what is left (a pair each).
__device__ __forceinline__ void hilo_f16x2(uint32_t x, uint32_t& hi, uint32_t& lo) {
  asm("{\n .reg .b16 h, l;\n .reg .b32 f, r;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n cvt.rn.f16x2.e4m3x2 f, h;\n"
      " sub.rn.f16x2 r, %2, f;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 l, r;\n cvt.u32.u16 %0, h;\n cvt.u32.u16 %1, l;\n}"
      : "=r"(hi), "=r"(lo)
      : "r"(x));
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
// The whole warp's view of the abort flag.
__device__ __forceinline__ bool stopped(volatile int* abort) {
  return __any_sync(0xffffffffu, *abort != 0);
}
// A maximum over the warp, every lane gets it (floats as ordered integers).
__device__ __forceinline__ float warp_max_any(float v) {
  int i = __float_as_int(v);
  i = i < 0 ? i ^ 0x7FFFFFFF : i;
  i = __reduce_max_sync(0xffffffffu, i);
  return __int_as_float(i < 0 ? i ^ 0x7FFFFFFF : i);
}

struct Shared {
  uint64_t full[ST], empty[ST], s_full[2], p_full[2], pv_done[2], q_full, drain;
  float neg_m[2][NQ], fac[2][NQ], red[SOFT_WARPS][NQ];  // [stream] (one unless the halves take turns)
  uint32_t tmem, valid[ST][4];
  int col_hi[NQ], col_lo[NQ], group_row[GROUP], group_pos[GROUP];
  int cols, abort;
  long long warp_tot[THREADS / 32];
};

// What a softmax warp knows of its item.
struct Soft {
  Span span;
  int t0, n, it;        // the item's first tile and tile count, the ring's next tile
  int nqp, c0, stream;  // columns of the item, this half's first one, its (O, m) set
  int min_hi, max_lo;   // tokens that every row sees: [max_lo, min_hi] and the sinks
  float to_log2;
  uint32_t tmem;        // with the warp's lane quadrant
};

// The softmax of C columns over an item's tiles (TURNS: every other one), a token per thread.
// l: this thread's share of the columns' sums, in units of 2^m.
template <int C, bool TURNS, bool MERGED>
__device__ __forceinline__ void soft_tiles(const AttendArgs& a, const Soft& w, Shared& sh, uint8_t* sm,
                                           float* l_out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, half = warp >> 2, tok = 32 * quad + lane;
  volatile int* abort = &sh.abort;
  float* neg_m = sh.neg_m[w.stream];
  float* fac = sh.fac[w.stream];
  float l[C], s[C];
#pragma unroll
  for (int c = 0; c < C; ++c) l[c] = 0.0f;
  const int first = TURNS ? (half ^ (w.it & 1)) : 0, stride = TURNS ? 2 : 1;
  for (int i = first; i < w.n; i += stride) {
    const int it = w.it + i, st = it % ST, pb = it & 1;
    const int t0 = w.span.token(w.t0 + i), t = t0 + tok;
    warp_wait(&sh.full[st], (it / ST) & 1, a.status, abort);
    const float raw = reinterpret_cast<const float*>(sm + SC_OFF)[st * TT + tok];
    const uint32_t ok = sh.valid[st][quad];
    const bool fin = fabsf(raw) <= 3.0e38f;
    const float ct = fin ? raw * w.to_log2 : __int_as_float(0x7FC00000);
    const float sc = fin ? raw : 0.0f;
    // some of the tile's tokens are not every row's to see
    const bool part = __any_sync(0xffffffffu, ok != 0xffffffffu || t0 + TT - 1 > w.min_hi ||
                                                  (t0 < w.max_lo && t0 + TT > a.sinks));
    // a weight says nothing of a token of next to no scale
    const bool faint = __any_sync(0xffffffffu, !(sc > 1.0e-12f));
    warp_wait(&sh.s_full[pb], (it >> 1) & 1, a.status, abort);
    tc_fence_after();
    const uint32_t scol = w.tmem + S_COL + 128 * pb + w.c0;
    auto load = [&]() {  // the products of the tile
#pragma unroll
      for (int g = 0; g < C; g += 8) tc_ld8(scol + g, s + g);
      if (MERGED) {
#pragma unroll
        for (int g = 0; g < C; g += 16) {
          float x[16];
          tc_ld8(scol + w.nqp + g, x);
          tc_ld8(scol + w.nqp + g + 8, x + 8);
          tc_wait_ld();
          tc_loaded(x);
          tc_loaded(x + 8);
          if (g == 0)
#pragma unroll
            for (int k = 0; k < C; k += 8) tc_loaded(s + k);
#pragma unroll
          for (int e = 0; e < 16; ++e) s[g + e] += x[e];
        }
      } else {
        tc_wait_ld();
#pragma unroll
        for (int g = 0; g < C; g += 8) tc_loaded(s + g);
      }
    };
    auto mask = [&](float v, int c) {
      const bool see = ((ok >> lane) & 1) && t <= sh.col_hi[w.c0 + c] &&
                       (t >= sh.col_lo[w.c0 + c] || t < a.sinks);
      return see ? v : -INFINITY;
    };
    auto weigh = [&]() {  // s: products -> 2^(score - m)
      const float4* nm = reinterpret_cast<const float4*>(neg_m + w.c0);
#pragma unroll
      for (int c = 0; c < C; c += 4) {
        const float4 m = nm[c / 4];
        s[c] = fmaf(s[c], ct, m.x);
        s[c + 1] = fmaf(s[c + 1], ct, m.y);
        s[c + 2] = fmaf(s[c + 2], ct, m.z);
        s[c + 3] = fmaf(s[c + 3], ct, m.w);
      }
      if (part) {
#pragma unroll
        for (int c = 0; c < C; ++c) s[c] = mask(s[c], c);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) s[c] = ex2(s[c]);
    };
    uint32_t mx[C];  // exponent bits of the block's largest weight times scale
    uint32_t top = 0;
    auto blocks = [&]() {
      top = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        mx[c] = __reduce_max_sync(0xffffffffu, __float_as_uint(s[c] * sc));
        top = max(top, mx[c]);
      }
    };
    load();
    weigh();
    blocks();
    bool over = top >= (uint32_t)(127 + (int)JUMP) << 23;
    if (faint) {
#pragma unroll
      for (int c = 0; c < C; ++c) over |= s[c] > exp2f(JUMP);
    }
    if (bar_any(2 + half, over)) {
      // m moves where a weight passes 2^(JUMP / 2) (always in an item's first tile)
      load();
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float v = s[c] * ct;
        if (part) v = mask(v, c);
        const float m = warp_max_any(v > -INFINITY ? v : -INFINITY);
        if (lane == 0) sh.red[warp][w.c0 + c] = m;
      }
      bar_sync<128>(4 + half);
      if (quad == 0)
        for (int c = w.c0 + lane; c < w.c0 + C; c += 32) {
          const float(*r)[NQ] = sh.red + 4 * half;
          const float m = fmaxf(fmaxf(r[0][c], r[1][c]), fmaxf(r[2][c], r[3][c]));
          const float old = -neg_m[c];
          float f = 1.0f;
          if (m - old > 0.5f * JUMP) {
            const float now = fminf(ceilf(m), 3.0e38f);
            f = old == UNSET ? 0.0f : ex2(old - now);
            neg_m[c] = -now;
          }
          fac[c] = f;
        }
      bar_sync<128>(4 + half);
#pragma unroll
      for (int c = 0; c < C; ++c) l[c] *= fac[w.c0 + c];
      if (i > first) {
        const int prev = it - stride;  // its product is in O
        warp_wait(&sh.pv_done[prev & 1], (prev >> 1) & 1, a.status, abort);
        tc_fence_after();
        for (int term = 0; term < (MERGED ? 2 : 1); ++term)
          for (int g = 0; g < C; g += 8) {
            float x[8];
            const uint32_t oc = w.tmem + O_COL + O_ALT * w.stream + term * w.nqp + w.c0 + g;
            tc_ld8(oc, x);
            tc_wait_ld();
            tc_loaded(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= fac[w.c0 + g + e];
            tc_st8(oc, x);
          }
        tc_wait_st();
      }
      load();
      weigh();
      blocks();
    }
    if (it >= 2) warp_wait(&sh.pv_done[pb], ((it >> 1) - 1) & 1, a.status, abort);
    if (part && (TURNS || half == 0)) {
      // NaN codes of tokens that some row must not see would reach it as 0 * NaN
      uint32_t* k = reinterpret_cast<uint32_t*>(sm + K_OFF + st * TT * 128 + tok * 128);
#pragma unroll 1
      for (int e = 0; e < 32; ++e) {
        const int j = (e + 4 * lane) & 31;
        const uint32_t v = k[j];
        const uint32_t nan = (((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
        if (nan) k[j] = v & ~(nan * 0xFFu);
      }
    }
    // weights times scales under their blocks' scales, as two e4m3 terms
    uint8_t* prow = sm + P_OFF + pb * P_BUF + tok * 128;
    uint8_t* img = sm + PIMG_OFF + pb * IMG;
#pragma unroll
    for (int g = 0; g < C; g += 16) {
      uint32_t hi[4], lo[4];
      uint32_t mine = 0;
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        float y[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = g + e + k;
          // the block's largest in [2^7, 2^8); exponents 15..254
          const uint32_t mb = min(max(mx[c] & 0x7F800000u, 15u << 23), 254u << 23);
          if (lane == e + k) mine = mb;
          l[c] += s[c];
          y[k] = s[c] * sc * __uint_as_float((261u << 23) - mb);
        }
        uint32_t h, r;
        hilo_f16x2(f16x2_of(y[0], y[1]), h, r);
        if (e & 2) {
          hi[e >> 2] |= h << 16;
          lo[e >> 2] |= r << 16;
        } else {
          hi[e >> 2] = h;
          lo[e >> 2] = r;
        }
      }
      if (lane < 16) {
        const int n = w.c0 + g + lane, nl = w.nqp + n;
        const uint8_t code = (uint8_t)((mine >> 23) - 7);
        img[(n & 31) * 16 + (n >> 5) * 4 + quad] = code;
        if (MERGED) img[(nl & 31) * 16 + (nl >> 5) * 4 + quad] = code;
      }
      const int ch = (w.c0 + g) >> 4, cl = MERGED ? (w.nqp + w.c0 + g) >> 4 : ch;
      *reinterpret_cast<uint4*>(prow + ((ch ^ (tok & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(prow + (MERGED ? 0 : TT * 128) + ((cl ^ (tok & 7)) << 4)) =
          make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    fence_proxy_async_shared();
    tc_fence_before();
    __syncwarp();
    if (lane < (TURNS ? 2 : 1)) mbar_arrive(&sh.p_full[pb]);  // eight arrivals a tile either way
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const float v = warp_sum(l[c]);
    if (lane == 0) l_out[w.c0 + c] = v;
  }
}

__global__ void __launch_bounds__(THREADS, 1) attend_kernel(const Args ar) {
  const AttendArgs& a = ar.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~uintptr_t(1023));
  __shared__ __align__(16) Shared ss;
  volatile int* abort = &ss.abort;
  Plan plan;
  plan.pre = reinterpret_cast<long long*>(sm + PLAN_OFF);
  plan.pmax = reinterpret_cast<int*>(plan.pre + MAX_REQ + 1);
  plan.pmin = plan.pmax + MAX_REQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Shape sh = shape_of(a, gridDim.x);
  const int team = blockIdx.x / sh.chunks, chunk = blockIdx.x - team * sh.chunks;
  const int chunk_bytes = min(128, a.kv_dim - 128 * chunk);

  if (tid == 0) {
    // a tile lands with its copies (the loading warp's lanes) and its mask (lane 0)
    for (int s = 0; s < ST; ++s) mbar_init(&ss.full[s], 33), mbar_init(&ss.empty[s], 1);
    for (int s = 0; s < 2; ++s)
      mbar_init(&ss.s_full[s], 1), mbar_init(&ss.p_full[s], SOFT_WARPS), mbar_init(&ss.pv_done[s], 1);
    mbar_init(&ss.q_full, SOFT_WARPS);
    mbar_init(&ss.drain, 1);
    ss.abort = 0;
  }
  if (warp == MMA_WARP) tmem_alloc<512>(&ss.tmem);
  for (int i = tid; i < IMG / 4; i += THREADS)
    reinterpret_cast<uint32_t*>(sm + ONE_OFF)[i] = 0x7F7F7F7Fu;
  for (int i = tid; i < 3 * IMG / 4; i += THREADS)
    reinterpret_cast<uint32_t*>(sm + PIMG_OFF)[i] = 0x7F7F7F7Fu;
  fence_proxy_async_shared();

  // ---------------------------------------------------------------------------- the cut
  for (int b = tid; b < a.n_req; b += THREADS) {
    plan.pmax[b] = -1;
    plan.pmin[b] = 0x7FFFFFFF;
    reinterpret_cast<int*>(&plan.pre[b + 1])[0] = 0;  // rows so far
  }
  pdl_trigger();
  pdl_wait();
  __syncthreads();
  for (int r = tid; r < a.rows; r += THREADS) {
    const int p = a.positions[r], b = a.row_req[r];
    if (p < 0) continue;
    if (b < 0 || b >= a.n_req) {
      if (blockIdx.x == 0) atomicOr(a.status, ST_UNMAPPED_PAGE);
      continue;
    }
    atomicMax(&plan.pmax[b], p);
    atomicMin(&plan.pmin[b], p);
    atomicAdd(reinterpret_cast<int*>(&plan.pre[b + 1]), 1);
  }
  __syncthreads();
  long long base = 0;
  for (int b0 = 0; b0 < a.n_req; b0 += THREADS) {
    const int b = b0 + tid;
    long long u = 0;
    if (b < a.n_req) {
      const int n = reinterpret_cast<int*>(&plan.pre[b + 1])[0];
      if (n > 0) {
        u = (long long)((n + sh.rows_per - 1) / sh.rows_per) *
            span_of(a, plan.pmax[b], plan.pmin[b]).tiles;
        if (plan.pmax[b] >= (long long)a.kv.max_blocks * a.kv.block_size && blockIdx.x == 0)
          atomicOr(a.status, ST_UNMAPPED_PAGE);
      }
    }
    long long x = u;
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) ss.warp_tot[warp] = x;
    __syncthreads();
    long long before = base;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) before += ss.warp_tot[i];
      base += ss.warp_tot[i];
    }
    if (b < a.n_req) plan.pre[b + 1] = before + x;
    __syncthreads();
  }
  if (tid == 0) plan.pre[0] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ss.tmem;

  // where the second kernel finds the rows' results
  if (blockIdx.x == 0 && tid == 0) *ar.total = plan.pre[a.n_req];
  for (int r = blockIdx.x + gridDim.x * warp; r < a.rows; r += gridDim.x * (THREADS / 32)) {
    const int b = a.row_req[r];
    RowInfo info = {0, 0, 0};
    if (a.positions[r] >= 0 && b >= 0 && b < a.n_req) {
      int rank = 0;
      for (int i = lane; i < r; i += 32) rank += a.row_req[i] == b && a.positions[i] >= 0;
      rank = __reduce_add_sync(0xffffffffu, rank);
      const Span s = span_of(a, plan.pmax[b], plan.pmin[b]);
      const int group = rank / sh.rows_per;
      info = {plan.pre[b] + (long long)group * s.tiles, s.tiles, rank - group * sh.rows_per};
    }
    if (lane == 0) ar.rows[r] = info;
  }

  if (team >= sh.teams) {
    // no team: nothing to do
  } else if (warp >= LOAD_WARP && warp < LOAD_WARP + LOAD_WARPS) {
    // --------------------------------------------------- loads: a warp takes every fourth tile
    regs_down<OTHER_REGS>();
    const int lw = warp - LOAD_WARP, piece = lane & 7;
    const bool in_chunk = 16 * piece < chunk_bytes;
    int it = 0;
    for_items(a, plan, sh, team, [&](const Item& im) {
      for (int i = (lw - it) & 3; i < im.n; i += LOAD_WARPS) {
        const int j = it + i, s = j % ST, t0 = im.span.token(im.t0 + i) + lane;
        long long off[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int t = t0 + 32 * q;
          off[q] = -1;
          if (t <= im.span.hi && (t >= im.span.lo || t < a.sinks)) {
            off[q] = record_offset(a.kv, im.b, t);
            if (off[q] < 0) atomicOr(a.status, ST_UNMAPPED_PAGE);
          }
        }
        if (j >= ST) warp_wait(&ss.empty[s], ((j / ST) - 1) & 1, a.status, abort);
        const bool go = !stopped(abort);
        uint8_t* st = sm + K_OFF + s * TT * 128;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t ok = __ballot_sync(0xffffffffu, off[q] >= 0);
          if (lane == 0) ss.valid[s][q] = ok;
          if (go) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int row = 4 * e + (lane >> 3);
              const long long ro = __shfl_sync(0xffffffffu, off[q], row);
              const bool in = ro >= 0 && in_chunk;
              cp_async16(st + (32 * q + row) * 128 + ((piece ^ (row & 7)) << 4),
                         a.kv.base + (in ? ro + 128 * chunk + 16 * piece : 0), in ? 16 : 0);
            }
            cp_async4(sm + SC_OFF + (s * TT + 32 * q + lane) * 4,
                      a.kv.base + (off[q] >= 0 ? off[q] + a.kv_dim : 0), off[q] >= 0 ? 4 : 0);
          }
        }
        cp_async_arrive_noinc(&ss.full[s]);
        if (lane == 0) mbar_arrive(&ss.full[s]);
      }
      it += im.n;
    });
    cp_async_wait_all();
  } else if (warp > MMA_WARP) {
    regs_down<OTHER_REGS>();  // (idle: they complete the warpgroup)
  } else if (warp == MMA_WARP) {
    // -------------------------------------------------------------------------- MMA issue
    regs_down<OTHER_REGS>();
    const uint32_t k0 = smem_u32(sm + K_OFF), p0 = smem_u32(sm + P_OFF), q0 = smem_u32(sm + Q_OFF);
    int it = 0, item = 0;
    // tile i's second product; first: O's first of the item
    auto pv = [&](int i, int nqp, bool first) {
      warp_wait(&ss.p_full[i & 1], (i >> 1) & 1, a.status, abort);
      if (!stopped(abort) && elect_one()) {
        tc_fence_after();
        const bool merged = nqp <= MERGE;
        const uint32_t ka = k0 + (i % ST) * TT * 128, pb = p0 + (i & 1) * P_BUF;
        const uint32_t o = tmem + O_COL + (nqp <= ALT ? O_ALT * (i & 1) : 0);
        tc_cp_img(tmem + SF_P, sm + PIMG_OFF + (i & 1) * IMG);
        const uint32_t idesc = IDESC | TRANS | ((uint32_t)((merged ? 2 * nqp : nqp) >> 3) << 17);
        for (int term = 0; term < (merged ? 1 : 2); ++term)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_mxf8(o, desc_sw128(ka + 4096 * k), desc_sw128(pb + term * TT * 128 + 4096 * k),
                        idesc | ((uint32_t)k << 4) | ((uint32_t)k << 29), tmem + SF_ONE,
                        tmem + SF_P, !first || term > 0 || k > 0);
        tc_commit(&ss.empty[i % ST]);
        tc_commit(&ss.pv_done[i & 1]);
      }
      __syncwarp();
    };
    if (elect_one()) tc_cp_img(tmem + SF_ONE, sm + ONE_OFF);
    __syncwarp();
    for_items(a, plan, sh, team, [&](const Item& im) {
      warp_wait(&ss.q_full, item & 1, a.status, abort);
      const int nqp = ss.cols;
      ++item;
      const bool merged = nqp <= MERGE;
      const int firsts = nqp <= ALT ? 2 : 1;
      const uint32_t idesc = IDESC | ((uint32_t)((merged ? 2 * nqp : nqp) >> 3) << 17);
      for (int i = 0; i < im.n; ++i) {
        const int j = it + i;
        warp_wait(&ss.full[j % ST], (j / ST) & 1, a.status, abort);
        if (!stopped(abort) && elect_one()) {
          fence_proxy_async_shared();  // the copies, seen to have landed, before the MMA's reads
          tc_fence_after();
          if (i == 0) tc_cp_img(tmem + SF_Q, sm + QIMG_OFF);
          const uint32_t ka = k0 + (j % ST) * TT * 128;
          for (int term = 0; term < (merged ? 1 : 2); ++term)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_mxf8(tmem + S_COL + 128 * (j & 1), desc_sw128(ka + 32 * k),
                          desc_sw128(q0 + term * NQ * 128 + 32 * k),
                          idesc | ((uint32_t)k << 4) | ((uint32_t)k << 29), tmem + SF_ONE,
                          tmem + SF_Q, term > 0 || k > 0);
          tc_commit(&ss.s_full[j & 1]);
        }
        __syncwarp();
        if (i > 0) pv(j - 1, nqp, i - 1 < firsts);
      }
      pv(it + im.n - 1, nqp, im.n - 1 < firsts);
      it += im.n;
    });
    // after a wait that ran out: what was issued completes before TMEM is freed
    if (stopped(abort) && elect_one()) {
      tc_commit(&ss.drain);
      (void)mbar_wait(&ss.drain, 0, a.status, 100000000ull);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------------------- softmax
    regs_up<SOFT_REGS>();
    const int quad = warp & 3, half = warp >> 2;
    const int hpg = a.n_q / (a.kv_dim / a.head_dim);
    const int cheads = hpg * (chunk_bytes > a.head_dim ? 2 : 1);  // heads per row of this chunk
    const int dshift = a.head_dim == 64 ? 6 : 7;
    int it = 0;
    for_items(a, plan, sh, team, [&](const Item& im) {
      // ---- the group's rows and queries
      bar_sync<256>(1);  // the previous item's columns are no longer in use
      if (warp == 0) {
        const int first = im.group * sh.rows_per;
        int seen = 0, n = 0;
        for (int r0 = 0; r0 < a.rows && n < sh.rows_per; r0 += 32) {
          const int r = r0 + lane;
          const int p = r < a.rows && a.row_req[r] == im.b ? a.positions[r] : -1;
          const uint32_t m = __ballot_sync(0xffffffffu, p >= 0);
          const int rank = seen + __popc(m & ((1u << lane) - 1)) - first;
          if (p >= 0 && rank >= 0 && rank < sh.rows_per)
            ss.group_row[rank] = r, ss.group_pos[rank] = p;
          seen += __popc(m);
          n = max(0, min(sh.rows_per, seen - first));
        }
        if (lane == 0) ss.cols = ((n * cheads + 15) & ~15) | (n << 16);
      }
      bar_sync<256>(1);
      const int nrows = ss.cols >> 16, nqp = ss.cols & 0xFFFF, nq = nrows * cheads;
      const bool merged = nqp <= MERGE, turns = nqp <= ALT;
      if (tid < NQ) {
        int hi = 0x7FFFFFFF, lo = 0;  // padding columns see everything
        if (tid < nq) {
          hi = a.causal ? ss.group_pos[tid / cheads] : im.span.hi;
          lo = a.window > 0 ? max(0, hi - a.window + 1) : 0;
        }
        ss.col_hi[tid] = hi;
        ss.col_lo[tid] = lo;
        ss.neg_m[0][tid] = ss.neg_m[1][tid] = -UNSET;
      }
      // queries as two e4m3 terms, rows of 128 bytes: hi in row c, lo in row nqp + c (merged)
      // or NQ + c
      for (int i = tid; i < nqp * 16; i += 256) {
        const int c = i >> 4, d = (i & 15) * 8;
        const int j = c / cheads, h = c - j * cheads, sl = h / hpg;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        const bool in = c < nq && (d >> dshift) == sl;
        if (in)
          bf16x8_to_f32(*reinterpret_cast<const uint4*>(
                            a.q + ss.group_row[j] * a.q_stride +
                            ((long long)chunk * sh.heads + h) * a.head_dim + (d - (sl << dshift))),
                        v);
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
        const int o = (d >> 4), w = d & 8;
        *reinterpret_cast<uint2*>(sm + Q_OFF + c * 128 + ((o ^ (c & 7)) << 4) + w) =
            make_uint2(hw[0], hw[1]);
        *reinterpret_cast<uint2*>(sm + Q_OFF + rl * 128 + ((o ^ (rl & 7)) << 4) + w) =
            make_uint2(lw[0], lw[1]);
        if ((d & 31) == 0) {
          sm[QIMG_OFF + (c & 31) * 16 + (c >> 5) * 4 + (d >> 5)] = (uint8_t)code;
          if (merged) sm[QIMG_OFF + (rl & 31) * 16 + (rl >> 5) * 4 + (d >> 5)] = (uint8_t)code;
        }
      }
      fence_proxy_async_shared();
      Soft w;
      w.min_hi = 0x7FFFFFFF;
      w.max_lo = 0;
      for (int j = 0; j < nrows; ++j) {
        const int hi = a.causal ? ss.group_pos[j] : im.span.hi;
        w.min_hi = min(w.min_hi, hi);
        w.max_lo = max(w.max_lo, a.window > 0 ? max(0, hi - a.window + 1) : 0);
      }
      bar_sync<256>(1);
      if (tid == 0) ss.cols = nqp;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss.q_full);
      w.span = im.span;
      w.t0 = im.t0;
      w.n = im.n;
      w.it = it;
      w.nqp = nqp;
      w.to_log2 = a.scale * LOG2E;
      w.tmem = tmem + ((uint32_t)(32 * quad) << 16);
      // the halves take turns with whole tiles (their own O and m each), or share the columns
      w.stream = turns ? half : 0;
      const int half0 = (nqp / 16 + 1) / 2 * 16;  // columns of half 0 where they share
      w.c0 = turns || half == 0 ? 0 : half0;
      const int cols = turns ? nqp : half == 0 ? half0 : nqp - half0;
      float* lo = ss.red[warp];
      if (turns) {
        if (cols == 16) soft_tiles<16, true, true>(a, w, ss, sm, lo);
        else if (cols == 32) soft_tiles<32, true, true>(a, w, ss, sm, lo);
        else soft_tiles<48, true, true>(a, w, ss, sm, lo);
      } else if (merged) {
        soft_tiles<32, false, true>(a, w, ss, sm, lo);
      } else if (cols == 32) {
        soft_tiles<32, false, false>(a, w, ss, sm, lo);
      } else {
        soft_tiles<48, false, false>(a, w, ss, sm, lo);
      }
      const int first_stream = it & 1;
      it += im.n;

      // ---- the item's result
      for (int i = max(it - 2, it - im.n); i < it; ++i)
        warp_wait(&ss.pv_done[i & 1], (i >> 1) & 1, a.status, abort);
      tc_fence_after();
      bar_sync<256>(1);
      const bool whole = im.n == im.span.tiles;  // nobody else has tiles of this group
      float* pt = ar.part + ((size_t)(team * 2 + (im.t0 > 0 ? 0 : 1)) * sh.chunks + chunk) * NQ * PART_LD;
      const int d = 32 * quad + lane;  // this thread's dimension of the chunk
      for (int c8 = 8 * half; c8 < nqp; c8 += 16) {
        float acc[8], m[8], lt[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = lt[e] = 0.0f, m[e] = UNSET;
        for (int k = 0; k < (turns ? 2 : 1); ++k) {
          if (turns && im.n == 1 && k != first_stream) continue;  // a stream without a tile
          float x[8];
          const uint32_t oc = w.tmem + O_COL + O_ALT * k + c8;
          tc_ld8(oc, x);
          tc_wait_ld();
          tc_loaded(x);
          if (merged) {
            float y[8];
            tc_ld8(oc + nqp, y);
            tc_wait_ld();
            tc_loaded(y);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += y[e];
          }
          const float(*r)[NQ] = ss.red + (turns ? 4 * k : c8 < half0 ? 0 : 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = c8 + e;
            const float lk = (r[0][c] + r[1][c]) + (r[2][c] + r[3][c]);
            const float mk = -ss.neg_m[k][c], mn = fmaxf(m[e], mk);
            const float f0 = m[e] == UNSET ? 0.0f : ex2(m[e] - mn);
            const float f1 = mk == UNSET && lk == 0.0f ? 0.0f : ex2(mk - mn);
            acc[e] = acc[e] * f0 + (f1 == 0.0f ? 0.0f : x[e] * f1);
            lt[e] = lt[e] * f0 + lk * f1;
            m[e] = mn;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = c8 + e;
          if (c >= nq) continue;
          const int j = c / cheads, h = c - j * cheads, sl = h / hpg;
          const long long head = (long long)chunk * sh.heads + h;
          const bool mine = (d >> dshift) == sl;
          if (whole) {
            if (mine)
              a.o[ss.group_row[j] * a.o_stride + head * a.head_dim + (d - (sl << dshift))] =
                  __float2bfloat16_rn(lt[e] == 0.0f ? 0.0f : acc[e] / lt[e]);
            if (d == 0)
              a.lse[(long long)ss.group_row[j] * a.n_q + head] =
                  lt[e] == 0.0f ? -INFINITY : (log2f(lt[e]) + m[e]) * LN2;
          } else {
            if (mine) pt[c * PART_LD + 4 + (d - (sl << dshift))] = acc[e];
            if (d == 0) pt[c * PART_LD] = m[e], pt[c * PART_LD + 1] = lt[e];
          }
        }
      }
      tc_fence_before();
    });
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

// Joins the pieces of a (row, head): a warp each, 4 (2) dimensions a lane.  Rows that one piece
// holds are done; pad rows and rows that see nothing get zeros.
constexpr int JOIN_WARPS = 4;
__global__ void __launch_bounds__(JOIN_WARPS * 32) attend_join_kernel(const Args ar, int grid) {
  const AttendArgs& a = ar.a;
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x, h = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (h >= a.n_q) return;
  const Shape sh = shape_of(a, grid);
  const RowInfo info = ar.rows[r];
  const int per = a.head_dim / 32, d = lane * per;
  __nv_bfloat16* o = a.o + r * a.o_stride + (long long)h * a.head_dim + d;
  if (info.tiles == 0) {
    for (int e = 0; e < per; ++e) o[e] = __float2bfloat16_rn(0.0f);
    if (lane == 0) a.lse[(long long)r * a.n_q + h] = -INFINITY;
    return;
  }
  const long long W = *ar.total, g1 = info.g0 + info.tiles - 1;
  // the team that holds unit g: the last k with W k / teams <= g
  auto team_of = [&](long long g) {
    int k = (int)(g * sh.teams / W);
    while (W * (k + 1) / sh.teams <= g) ++k;
    while (W * k / sh.teams > g) --k;
    return k;
  };
  const int k0 = team_of(info.g0), k1 = team_of(g1);
  if (k0 == k1) return;  // whole in one team
  const int chunk = h / sh.heads, hpg = a.n_q / (a.kv_dim / a.head_dim);
  const int cheads = hpg * (min(128, a.kv_dim - 128 * chunk) > a.head_dim ? 2 : 1);
  const int c = info.place * cheads + (h - chunk * sh.heads);
  auto piece = [&](int k) {
    const int slot = W * k / sh.teams > info.g0 ? 0 : 1;  // began before this team, or in it
    return ar.part + (((size_t)(k * 2 + slot) * sh.chunks + chunk) * NQ + c) * PART_LD;
  };
  auto empty = [&](int k) { return W * k / sh.teams == W * (k + 1) / sh.teams; };
  float M = UNSET;
  for (int k = k0 + lane; k <= k1; k += 32)
    if (!empty(k)) M = fmaxf(M, piece(k)[0]);
  M = warp_max(M);
  float num[4] = {0.0f, 0.0f, 0.0f, 0.0f}, den = 0.0f;
  for (int k = k0; k <= k1; ++k) {
    if (empty(k)) continue;
    const float* p = piece(k);
    const float f = ex2(p[0] - M);
    den = fmaf(f, p[1], den);
    for (int e = 0; e < per; ++e) num[e] = fmaf(f, p[4 + d + e], num[e]);
  }
  for (int e = 0; e < per; ++e) o[e] = __float2bfloat16_rn(den == 0.0f ? 0.0f : num[e] / den);
  if (lane == 0)
    a.lse[(long long)r * a.n_q + h] = den == 0.0f ? -INFINITY : (log2f(den) + M) * LN2;
}

// weights[b][t] += sum over b's rows and heads of exp(s - lse): a thread per token, rows and
// heads in order.
template <int DH>
__global__ void __launch_bounds__(TT) attend_weights_kernel(AttendArgs a, int tiles) {
  pdl_wait();
  const int b = blockIdx.y, G = a.kv_dim / DH, hpg = a.n_q / G;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const long long t = (long long)tile * TT + threadIdx.x;
    float w = 0.0f;
    bool any = false;
    for (int r = 0; r < a.rows; ++r) {
      if (a.row_req[r] != b || a.positions[r] < 0) continue;
      int hi = a.positions[r];
      if (!a.causal)
        for (int i = 0; i < a.rows; ++i)
          if (a.row_req[i] == b) hi = max(hi, a.positions[i]);
      const int lo = a.window > 0 ? max(0, hi - a.window + 1) : 0;
      if (t > hi || (t < lo && t >= a.sinks)) continue;
      const long long off = record_offset(a.kv, b, (int)t);
      if (off < 0) continue;
      any = true;
      const float sc = *reinterpret_cast<const float*>(a.kv.base + off + a.kv_dim) * a.scale;
      for (int h = 0; h < a.n_q; ++h) {
        float d = 0.0f;
        for (int i = 0; i < DH; ++i) {
          uint32_t f[2];
          e4m3x4_to_f16x4(a.kv.base[off + (h / hpg) * DH + i], f);
          d = fmaf(__half2float(__ushort_as_half((unsigned short)(f[0] & 0xFFFF))),
                   __bfloat162float(a.q[r * a.q_stride + h * DH + i]), d);
        }
        w += expf(d * sc - a.lse[(size_t)r * a.n_q + h]);
      }
    }
    if (any && t < a.weights_stride) a.weights[b * a.weights_stride + t] += w;
  }
}

struct Layout {
  size_t rows, total, part, bytes;
};
Layout layout(int max_rows, int sms) {
  Layout l;
  l.total = 0;
  l.rows = 256;
  l.part = l.rows + ((size_t)max_rows * sizeof(RowInfo) + 255) / 256 * 256;
  l.bytes = l.part + (size_t)sms * 2 * NQ * PART_LD * sizeof(float);
  return l;
}

}  // namespace

size_t attend_workspace_bytes(int max_rows, int sms) { return layout(max_rows, sms).bytes; }

cudaError_t attend_prepare() {
  // the roles' register split adds up to what a block launches with: 128 a thread
  cudaFuncAttributes f;
  cudaError_t e = cudaFuncGetAttributes(&f, attend_kernel);
  if (e == cudaSuccess && f.numRegs != 128) e = cudaErrorInvalidConfiguration;
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
}

cudaError_t launch_attend(const Launch& L, const AttendArgs& a, uint8_t* ws, int max_rows, int sms) {
  const Layout l = layout(max_rows, sms);
  Args ar = {a, reinterpret_cast<float*>(ws + l.part), reinterpret_cast<RowInfo*>(ws + l.rows),
             reinterpret_cast<long long*>(ws + l.total)};
  cudaError_t e = launch_ex(L, dim3(sms), dim3(THREADS), SMEM_BYTES, attend_kernel, ar);
  if (e == cudaSuccess)
    e = launch_ex(L, dim3(a.rows, (a.n_q + JOIN_WARPS - 1) / JOIN_WARPS), dim3(JOIN_WARPS * 32), 0,
                  attend_join_kernel, ar, sms);
  const long long cap = (long long)a.kv.max_blocks * a.kv.block_size;
  const int tiles = (int)((cap + TT - 1) / TT);
  if (e == cudaSuccess && a.weights)
    e = launch_ex(L, dim3(min(tiles, 1024), a.n_req), dim3(TT), 0,
                  a.head_dim == 128 ? attend_weights_kernel<128> : attend_weights_kernel<64>, a,
                  tiles);
  return e;
}

}  // namespace mono
