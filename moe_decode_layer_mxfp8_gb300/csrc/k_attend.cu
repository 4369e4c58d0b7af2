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
constexpr int ST = 6;          // tiles in the ring
constexpr int AHEAD = 5;       // of these in flight
constexpr int MAX_REQ = 1024;
constexpr int THREADS = 13 * 32;
constexpr int SOFT_WARPS = 8, LOAD_WARP = 8, MMA_WARP = 12;
constexpr float JUMP = 40.0f;      // log2 of how far a score may pass m_q
constexpr float UNSET = -1.0e30f;  // m_q of a query that has seen no token
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

constexpr int K_OFF = 0;
constexpr int P_BUF = 2 * TT * 128;  // hi terms, then lo terms (merged: hi and lo in the first)
constexpr int P_OFF = K_OFF + ST * TT * 128;
constexpr int Q_OFF = P_OFF + 2 * P_BUF;  // hi rows, then lo rows
constexpr int IMG = 512;
constexpr int PIMG_OFF = Q_OFF + 2 * NQ * 128;  // [2 buffers][hi, lo]
constexpr int QIMG_OFF = PIMG_OFF + 4 * IMG;
constexpr int ONE_OFF = QIMG_OFF + IMG;
constexpr int SC_OFF = ONE_OFF + IMG;  // token scales [ST][128]
constexpr int PLAN_OFF = SC_OFF + ST * TT * 4;
constexpr int SMEM_BYTES = PLAN_OFF + (MAX_REQ + 1) * 8 + 2 * MAX_REQ * 4 + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
static_assert(P_OFF % 1024 == 0 && Q_OFF % 1024 == 0 && (NQ * 128) % 1024 == 0, "swizzle atoms");

// TMEM columns
constexpr int S_COL = 0, O_COL = 256, SF_ONE = 384, SF_Q = 388, SF_P = 392;  // two images each
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
// Two f16 values as e4m3 hi codes and, of 16 times what is left, lo codes (a code pair each).
__device__ __forceinline__ void hilo_f16x2(uint32_t x, uint32_t& hi, uint32_t& lo) {
  asm("{\n .reg .b16 h, l;\n .reg .b32 f, r, s;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n cvt.rn.f16x2.e4m3x2 f, h;\n"
      " sub.rn.f16x2 r, %2, f;\n mov.b32 s, 0x4C004C00;\n mul.rn.f16x2 r, r, s;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 l, r;\n cvt.u32.u16 %0, h;\n cvt.u32.u16 %1, l;\n}"
      : "=r"(hi), "=r"(lo)
      : "r"(x));
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
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

__global__ void __launch_bounds__(THREADS, 1) attend_kernel(const Args ar) {
  const AttendArgs& a = ar.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[ST], empty[ST], s_full[2], p_full[2], pv_done[2], q_full, drain;
  __shared__ uint32_t s_tmem, valid[ST][4];
  __shared__ int s_abort;
  __shared__ __align__(16) float neg_m[NQ], fac[NQ], red[4][NQ];
  __shared__ int col_hi[NQ], col_lo[NQ];
  __shared__ int group_row[GROUP], group_pos[GROUP], s_rows;
  __shared__ long long warp_tot[THREADS / 32];
  volatile int* abort = &s_abort;
  Plan plan;
  plan.pre = reinterpret_cast<long long*>(sm + PLAN_OFF);
  plan.pmax = reinterpret_cast<int*>(plan.pre + MAX_REQ + 1);
  plan.pmin = plan.pmax + MAX_REQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Shape sh = shape_of(a, gridDim.x);
  const int team = blockIdx.x / sh.chunks, chunk = blockIdx.x - team * sh.chunks;
  const int chunk_bytes = min(128, a.kv_dim - 128 * chunk);

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&full[s], 128), mbar_init(&empty[s], 1);
    for (int s = 0; s < 2; ++s)
      mbar_init(&s_full[s], 1), mbar_init(&p_full[s], SOFT_WARPS), mbar_init(&pv_done[s], 1);
    mbar_init(&q_full, SOFT_WARPS);
    mbar_init(&drain, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) tmem_alloc<512>(&s_tmem);
  for (int i = tid; i < IMG / 4; i += THREADS)
    reinterpret_cast<uint32_t*>(sm + ONE_OFF)[i] = 0x7F7F7F7Fu;
  for (int i = tid; i < 5 * IMG / 4; i += THREADS)
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
    if (lane == 31) warp_tot[warp] = x;
    __syncthreads();
    long long before = base;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) before += warp_tot[i];
      base += warp_tot[i];
    }
    if (b < a.n_req) plan.pre[b + 1] = before + x;
    __syncthreads();
  }
  if (tid == 0) plan.pre[0] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

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
  } else if (warp >= LOAD_WARP && warp < LOAD_WARP + 4) {
    // ------------------------------------------------------------------------------ loads
    const int lw = warp - LOAD_WARP, piece = lane & 7;
    int it = 0;
    auto landed = [&](int i) {
      fence_proxy_async_shared();
      mbar_arrive(&full[i % ST]);
    };
    for_items(a, plan, sh, team, [&](const Item& im) {
      for (int i = 0; i < im.n; ++i, ++it) {
        const int s = it % ST;
        const int t = im.span.token(im.t0 + i) + 32 * lw + lane;
        long long off = -1;
        if (t <= im.span.hi && (t >= im.span.lo || t < a.sinks)) {
          off = record_offset(a.kv, im.b, t);
          if (off < 0) atomicOr(a.status, ST_UNMAPPED_PAGE);
        }
        const uint32_t ok = __ballot_sync(0xffffffffu, off >= 0);
        if (it >= ST) warp_wait(&empty[s], ((it / ST) - 1) & 1, a.status, abort);
        if (!stopped(abort)) {
          uint8_t* st = sm + K_OFF + s * TT * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int row = 4 * j + (lane >> 3);
            const long long ro = __shfl_sync(0xffffffffu, off, row);
            const bool in = ro >= 0 && 16 * piece < chunk_bytes;
            cp_async16(st + (32 * lw + row) * 128 + ((piece ^ (row & 7)) << 4),
                       a.kv.base + (in ? ro + 128 * chunk + 16 * piece : 0), in ? 16 : 0);
          }
          cp_async4(sm + SC_OFF + (s * TT + 32 * lw + lane) * 4,
                    a.kv.base + (off >= 0 ? off + a.kv_dim : 0), off >= 0 ? 4 : 0);
        }
        if (lane == 0) valid[s][lw] = ok;
        cp_async_commit();
        if (it >= AHEAD - 1) {
          cp_async_wait<AHEAD - 1>();
          landed(it - (AHEAD - 1));
        }
      }
    });
    cp_async_wait<0>();
    for (int i = max(0, it - (AHEAD - 1)); i < it; ++i) landed(i);
  } else if (warp == MMA_WARP) {
    // -------------------------------------------------------------------------- MMA issue
    const uint32_t k0 = smem_u32(sm + K_OFF), p0 = smem_u32(sm + P_OFF), q0 = smem_u32(sm + Q_OFF);
    int it = 0, item = 0;
    auto pv = [&](int i, int nqp, bool first) {  // tile i's second product
      warp_wait(&p_full[i & 1], (i >> 1) & 1, a.status, abort);
      if (!stopped(abort) && elect_one()) {
        tc_fence_after();
        const bool merged = nqp <= MERGE;
        const uint32_t ka = k0 + (i % ST) * TT * 128, pb = p0 + (i & 1) * P_BUF;
        const uint8_t* img = sm + PIMG_OFF + (i & 1) * 2 * IMG;
        tc_cp_img(tmem + SF_P, img);
        if (!merged) tc_cp_img(tmem + SF_P + 4, img + IMG);
        const uint32_t idesc = IDESC | TRANS | ((uint32_t)((merged ? 2 * nqp : nqp) >> 3) << 17);
        for (int term = 0; term < (merged ? 1 : 2); ++term)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_mxf8(tmem + O_COL, desc_sw128(ka + 4096 * k),
                        desc_sw128(pb + term * TT * 128 + 4096 * k),
                        idesc | ((uint32_t)k << 4) | ((uint32_t)k << 29), tmem + SF_ONE,
                        tmem + SF_P + 4 * term, !first || term > 0 || k > 0);
        tc_commit(&empty[i % ST]);
        tc_commit(&pv_done[i & 1]);
      }
      __syncwarp();
    };
    if (elect_one()) tc_cp_img(tmem + SF_ONE, sm + ONE_OFF);
    __syncwarp();
    for_items(a, plan, sh, team, [&](const Item& im) {
      warp_wait(&q_full, item & 1, a.status, abort);
      const int nqp = s_rows;  // columns of the item, published before q_full
      ++item;
      const bool merged = nqp <= MERGE;
      const uint32_t idesc = IDESC | ((uint32_t)((merged ? 2 * nqp : nqp) >> 3) << 17);
      for (int i = 0; i < im.n; ++i) {
        const int j = it + i;
        warp_wait(&full[j % ST], (j / ST) & 1, a.status, abort);
        if (!stopped(abort) && elect_one()) {
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
          tc_commit(&s_full[j & 1]);
        }
        __syncwarp();
        if (i > 0) pv(j - 1, nqp, i == 1);
      }
      pv(it + im.n - 1, nqp, im.n == 1);
      it += im.n;
    });
    // after a wait that ran out: what was issued completes before TMEM is freed
    if (stopped(abort) && elect_one()) {
      tc_commit(&drain);
      (void)mbar_wait(&drain, 0, a.status, 100000000ull);
    }
    __syncwarp();
  } else if (warp < SOFT_WARPS) {
    // ---------------------------------------------------------------------------- softmax
    const int quad = warp & 3, half = warp >> 2, tok = 32 * quad + lane;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const int hpg = a.n_q / (a.kv_dim / a.head_dim);
    const int cheads = hpg * (chunk_bytes > a.head_dim ? 2 : 1);  // heads per row of this chunk
    const int dshift = a.head_dim == 64 ? 6 : 7;
    const float to_log2 = a.scale * LOG2E;
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
          if (p >= 0 && rank >= 0 && rank < sh.rows_per) group_row[rank] = r, group_pos[rank] = p;
          seen += __popc(m);
          n = max(0, min(sh.rows_per, seen - first));
        }
        if (lane == 0) s_rows = ((n * cheads + 15) & ~15) | (n << 16);
      }
      bar_sync<256>(1);
      const int nrows = s_rows >> 16, nqp = s_rows & 0xFFFF, nq = nrows * cheads;
      const bool merged = nqp <= MERGE;
      if (tid < NQ) {
        int hi = 0x7FFFFFFF, lo = 0;  // padding columns see everything
        if (tid < nq) {
          hi = a.causal ? group_pos[tid / cheads] : im.span.hi;
          lo = a.window > 0 ? max(0, hi - a.window + 1) : 0;
        }
        col_hi[tid] = hi;
        col_lo[tid] = lo;
        neg_m[tid] = -UNSET;
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
                            a.q + group_row[j] * a.q_stride +
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
      bar_sync<256>(1);
      if (tid == 0) s_rows = nqp;
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
      int min_hi = 0x7FFFFFFF, max_lo = 0;
      for (int j = 0; j < nrows; ++j) {
        const int hi = a.causal ? group_pos[j] : im.span.hi;
        min_hi = min(min_hi, hi);
        max_lo = max(max_lo, a.window > 0 ? max(0, hi - a.window + 1) : 0);
      }

      const int ng = nqp / 16;          // groups of 8 columns of this half
      const int c0 = half * 8 * ng;     // its first column
      float l[NQ / 2], s[NQ / 2];
#pragma unroll
      for (int c = 0; c < NQ / 2; ++c) l[c] = 0.0f;

      for (int i = 0; i < im.n; ++i, ++it) {
        const int st = it % ST, pb = it & 1;
        const int t0 = im.span.token(im.t0 + i), t = t0 + tok;
        warp_wait(&full[st], (it / ST) & 1, a.status, abort);
        const float raw = reinterpret_cast<const float*>(sm + SC_OFF)[st * TT + tok];
        const uint32_t ok = valid[st][quad];
        const bool fin = fabsf(raw) <= 3.0e38f;
        const float ct = fin ? raw * to_log2 : __int_as_float(0x7FC00000);
        const float sc = fin ? raw : 0.0f;
        // some of the tile's tokens are not every row's to see
        const bool part = ok != 0xffffffffu || t0 + TT - 1 > min_hi ||
                          (t0 < max_lo && t0 + TT > a.sinks);
        warp_wait(&s_full[pb], (it >> 1) & 1, a.status, abort);
        tc_fence_after();
        const uint32_t scol = tmem + lanes + S_COL + 128 * pb + c0;
        // scores in log2 units, masked ones -inf
        auto load_scores = [&]() {
#pragma unroll
          for (int g = 0; g < NQ / 16; ++g)
            if (g < ng) tc_ld8(scol + 8 * g, s + 8 * g);
          tc_wait_ld();
#pragma unroll
          for (int g = 0; g < NQ / 16; ++g)
            if (g < ng) tc_loaded(s + 8 * g);
          if (merged) {
#pragma unroll
            for (int g = 0; g < MERGE / 16; ++g)
              if (g < ng) {
                float x[8];
                tc_ld8(scol + nqp + 8 * g, x);
                tc_wait_ld();
                tc_loaded(x);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[8 * g + e] += x[e];
              }
          }
#pragma unroll
          for (int c = 0; c < NQ / 2; ++c)
            if (c < 8 * ng) s[c] *= ct;
          if (part) {
            const bool mapped = (ok >> lane) & 1;
#pragma unroll
            for (int c = 0; c < NQ / 2; ++c)
              if (c < 8 * ng) {
                const bool see = mapped && t <= col_hi[c0 + c] &&
                                 (t >= col_lo[c0 + c] || t < a.sinks);
                if (!see) s[c] = -INFINITY;
              }
          }
        };
        load_scores();
        bool over = false;
#pragma unroll
        for (int c = 0; c < NQ / 2; ++c)
          if (c < 8 * ng) over |= s[c] + neg_m[c0 + c] > JUMP;
        if (bar_any(2 + half, over)) {
          // m_q moves where a score passes it (always in an item's first tile)
#pragma unroll
          for (int c = 0; c < NQ / 2; ++c)
            if (c < 8 * ng) {
              const float m = warp_max_any(s[c] > -INFINITY ? s[c] : -INFINITY);
              if (lane == 0) red[quad][c0 + c] = m;
            }
          bar_sync<128>(4 + half);
          if (quad == 0)
            for (int c = c0 + lane; c < c0 + 8 * ng; c += 32) {
              const float m = fmaxf(fmaxf(red[0][c], red[1][c]), fmaxf(red[2][c], red[3][c]));
              const float old = -neg_m[c];
              float f = 1.0f;
              if (m - old > JUMP) {
                const float now = fminf(ceilf(m), 3.0e38f);
                f = old == UNSET ? 0.0f : ex2(old - now);
                neg_m[c] = -now;
              }
              fac[c] = f;
            }
          bar_sync<128>(4 + half);
#pragma unroll
          for (int c = 0; c < NQ / 2; ++c)
            if (c < 8 * ng) l[c] *= fac[c0 + c];
          if (i > 0) {
            warp_wait(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, a.status, abort);
            tc_fence_after();
            for (int term = 0; term < (merged ? 2 : 1); ++term)
              for (int g = 0; g < ng; ++g) {
                float x[8];
                const uint32_t oc = tmem + lanes + O_COL + term * nqp + c0 + 8 * g;
                tc_ld8(oc, x);
                tc_wait_ld();
                tc_loaded(x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= fac[c0 + 8 * g + e];
                tc_st8(oc, x);
              }
            tc_wait_st();
          }
        }
        if (it >= 2) warp_wait(&pv_done[pb], ((it >> 1) - 1) & 1, a.status, abort);
        if (part && half == 0) {
          // NaN codes of tokens that some row must not see would reach it as 0 * NaN
          for (int j = 0; j < 8; ++j) {
            uint32_t* w = reinterpret_cast<uint32_t*>(sm + K_OFF + st * TT * 128 + tok * 128 + 16 * j);
            for (int e = 0; e < 4; ++e) {
              const uint32_t v = w[e], x = v & 0x7F7F7F7Fu;
              const uint32_t nan = ((x + 0x01010101u) & 0x80808080u) >> 7;  // bytes equal to 0x7F
              if (nan) w[e] = v & ~(nan * 0xFFu);
            }
          }
        }
        // weights: P scale_t under its block's scale, as two e4m3 terms
        uint8_t* prow = sm + P_OFF + pb * P_BUF + tok * 128;
        uint8_t* img = sm + PIMG_OFF + pb * 2 * IMG;
#pragma unroll
        for (int g = 0; g < NQ / 16; ++g)
          if (g < ng) {
            float w[8], mul[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int c = 8 * g + e;
              const float p = ex2(s[c] + neg_m[c0 + c]);
              l[c] += p;
              w[e] = p * sc;
            }
            int mine = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t mx = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(w[e])));
              const int code = max((int)(mx >> 23) - 7, 8);
              mul[e] = __uint_as_float((uint32_t)(254 - code) << 23);
              if (lane == e) mine = code;
            }
            if (lane < 8) {
              const int n = c0 + 8 * g + lane;
              img[(n & 31) * 16 + (n >> 5) * 4 + quad] = (uint8_t)mine;
              const int nl = merged ? nqp + n : n;
              (merged ? img : img + IMG)[(nl & 31) * 16 + (nl >> 5) * 4 + quad] = (uint8_t)(mine - 4);
            }
            uint32_t hb[4], lb[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              hilo_f16x2(f16x2_of(w[2 * e] * mul[2 * e], w[2 * e + 1] * mul[2 * e + 1]), hb[e], lb[e]);
            const int ch = c0 + 8 * g, cl = merged ? nqp + ch : ch;
            uint8_t* rl = merged ? prow : prow + TT * 128;
            *reinterpret_cast<uint2*>(prow + (((ch >> 4) ^ (tok & 7)) << 4) + (ch & 15)) =
                make_uint2(hb[0] | hb[1] << 16, hb[2] | hb[3] << 16);
            *reinterpret_cast<uint2*>(rl + (((cl >> 4) ^ (tok & 7)) << 4) + (cl & 15)) =
                make_uint2(lb[0] | lb[1] << 16, lb[2] | lb[3] << 16);
          }
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[pb]);
      }

      // ---- the item's result: sums over the tokens, then O
#pragma unroll
      for (int c = 0; c < NQ / 2; ++c)
        if (c < 8 * ng) {
          const float v = warp_sum(l[c]);
          if (lane == 0) red[quad][c0 + c] = v;
        }
      const int last = it - 1;
      warp_wait(&pv_done[last & 1], (last >> 1) & 1, a.status, abort);
      tc_fence_after();
      bar_sync<256>(1);
      const bool whole = im.n == im.span.tiles;  // nobody else has tiles of this group
      float* pt = ar.part + ((size_t)(team * 2 + (im.t0 > 0 ? 0 : 1)) * sh.chunks + chunk) * NQ * PART_LD;
      const int d = tok;  // this thread's dimension of the chunk
      for (int g = 0; g < ng; ++g) {
        float x[8];
        tc_ld8(tmem + lanes + O_COL + c0 + 8 * g, x);
        tc_wait_ld();
        tc_loaded(x);
        if (merged) {
          float y[8];
          tc_ld8(tmem + lanes + O_COL + nqp + c0 + 8 * g, y);
          tc_wait_ld();
          tc_loaded(y);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] += y[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = c0 + 8 * g + e;
          if (c >= nq) continue;
          const int j = c / cheads, h = c - j * cheads, sl = h / hpg;
          const float lt = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
          const long long head = (long long)chunk * sh.heads + h;
          if (whole) {
            const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
            if ((d >> dshift) == sl)
              a.o[group_row[j] * a.o_stride + head * a.head_dim + (d - (sl << dshift))] =
                  __float2bfloat16_rn(lt == 0.0f ? 0.0f : x[e] * inv);
            if (d == 0)
              a.lse[(long long)group_row[j] * a.n_q + head] =
                  lt == 0.0f ? -INFINITY : (log2f(lt) - neg_m[c]) * LN2;
          } else {
            if ((d >> dshift) == sl) pt[c * PART_LD + 4 + (d - (sl << dshift))] = x[e];
            if (d == 0) pt[c * PART_LD] = -neg_m[c], pt[c * PART_LD + 1] = lt;
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
