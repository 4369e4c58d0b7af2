// Attention over the paged fp8 cache for few query columns (a row or so per request), and the
// gathering of attention weights.
//
// Attention.  The rows of a group times the heads that share a 128-byte chunk of the record make
// at most 16 columns: the M of m16n8k16 MMAs (f16, f32 accumulation), which run here at the rate
// that 16 columns need -- 16 tokens of a chunk take 32 of them, 550 cycles of an SM per 128 tokens
// against 690 of HBM -- while a tcgen05 tile would leave seven eighths of its rows empty or widen
// every tile in shared memory.  A warp owns a chunk and every n-th block of 16 tokens; its blocks
// come by TMA (or cp.async where pages are no multiple of 16) into a ring of its own, eight blocks
// deep, so warps meet only at an item's end.  Queries stay in registers as f16, scaled by a power
// of two per column (exact for every element down to 2^-24 of a column's largest); codes are
// widened to f16 in registers, once as tokens x dimensions for the scores and once, read
// transposed, for the sums; scores, weights and their sums are f32, weights times scales are f16
// for the second product under a reference m per column that moves only when a weight outgrows
// it (attend_plan.cuh).
//
// Weights.  With lse known, weights[t] += sum over rows and heads of 2^(s log2e - lse): the score
// half of the above, all chunks of a token in one warp, no exchange but a shuffle, one writer per
// token.
#include "attend_plan.cuh"

namespace mono {
namespace {

using namespace attend;

constexpr int WARPS = 8, THREADS = (WARPS + 1) * 32;  // and a warp that loads
constexpr int BLOCK = 32, NB = BLOCK / 8;  // tokens of a warp's step, and MMA columns of 8
constexpr int ST = 4;                // tiles in the ring
constexpr int TILE_BYTES = 32768;    // codes of a tile: tokens x chunks x 128, at most
constexpr int MAX_TILE = WARPS * BLOCK, COLS = 16;
constexpr int RING_OFF = 0;                                // [ST] chunks of tile x 128 (1 KB atoms)
constexpr int SCALE_OFF = RING_OFF + ST * TILE_BYTES;      // [ST][tile] 16-byte runs, scale first
constexpr int SUM_LD = 128 + 4;                            // a column's O, m, l
constexpr int SUM_OFF = SCALE_OFF + ST * MAX_TILE * 16;    // [WARPS / 2][COLS][SUM_LD]
constexpr int QLD = 128 + 8;
constexpr int Q_OFF = SUM_OFF;                              // [chunks][COLS][QLD] f16, before that
constexpr int SUM_WARPS = 5;  // (subs that hand their sums over at once, or the queries)
constexpr int PLAN_OFF = SUM_OFF + SUM_WARPS * COLS * SUM_LD * 4;
static_assert(8 * COLS * QLD * 2 <= SUM_WARPS * COLS * SUM_LD * 4, "queries under the sums");
constexpr int SMEM_BYTES = PLAN_OFF + (3 * MAX_REQ + 4) * 4 + 1024;
static_assert(SMEM_BYTES + 2048 <= 227 * 1024, "shared memory");

struct Args {
  CUtensorMap codes, scales;
  int box;  // rows of a box; 0: no maps
  int subs; // warps per chunk
  AttendArgs a;
  Shape sh;
  Pieces ws;
};

struct Shared {
  uint64_t full[ST], empty[ST];
  uint32_t valid[ST][MAX_TILE / 32];
  int group_row[16], group_pos[16], rows, abort;
  float qs[8][COLS];
  Jobs start;
};

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Bounded wait by every lane (some 10^7 polls), none once another has run out; the data behind one
// that ran out is whatever it is.
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  uint32_t polls = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (*abort || ++polls == (1u << 23)) {
      atomicOr(status, ST_WAIT_TIMEOUT);
      *abort = 1;
      break;
    }
  __syncwarp();
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
__device__ __forceinline__ void workers_sync() {  // the warps that do not load
  asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
}
// Eight elements from dimension d of a head as f16, times up, in the order in which lanes hold codes:
// dimension 64 p + 16 j + 4 u + e at K step 4 p + u, MMA column 2 j + e (e < 2) or 2 j + 6 + e.
__device__ __forceinline__ void store_query(__half* row, int d, const float (&v)[8], float up) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int dd = d + 4 * t, p = dd >> 6, j = (dd >> 4) & 3, u = (dd >> 2) & 3;
    uint32_t* at = reinterpret_cast<uint32_t*>(row + (4 * p + u) * 16 + 2 * j);
    at[0] = f16x2(v[4 * t] * up, v[4 * t + 1] * up);
    at[4] = f16x2(v[4 * t + 2] * up, v[4 * t + 3] * up);
  }
}
// The exponent that brings a largest magnitude m to [2^8, 2^9) (within f32's reach).
__device__ __forceinline__ int query_exponent(float m) {
  return m > 0.0f ? min(max((int)(__float_as_uint(m) >> 23) - 127 - 8, -100), 100) : 0;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// Two words of four codes (tokens x, y; the same four dimensions) as f16 pairs (x, y) per dimension.
__device__ __forceinline__ void pair_codes(uint32_t x, uint32_t y, uint32_t (&h)[4]) {
  uint32_t f[2];
  e4m3x4_to_f16x4(__byte_perm(x, y, 0x5140), f);
  h[0] = f[0], h[1] = f[1];
  e4m3x4_to_f16x4(__byte_perm(x, y, 0x7362), f);
  h[2] = f[0], h[3] = f[1];
}

__global__ void __launch_bounds__(THREADS, 1) attend_few_kernel(const __grid_constant__ Args ar) {
  const AttendArgs& a = ar.a;
  const Shape& sh = ar.sh;
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
  const int chunks = sh.chunks, subs = ar.subs, tile = sh.tile;
  if (tid == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&ss.full[s], 1), mbar_init(&ss.empty[s], chunks * subs);
    ss.abort = 0;
    fence_mbar_init();
  }
  derive_plan<THREADS>(a, sh, plan, blockIdx.x, true, &ss.start, ar.ws.total);
  __syncthreads();
  Jobs items = ss.start;
  Job im;

  if (warp == WARPS) {
    // ------------------------------------------------------------------------------- loads
    const int box = ar.box ? ar.box : 1, bs = a.kv.block_size, shift = __ffs(box) - 1;
    const int runs = tile >> shift;
    uint32_t it = 0;
#pragma unroll 1
    while (next_job(a, sh, plan, items, im)) {
      // lane per run of a tile (of a token where there are no maps): its page, looked up a tile ahead
      int page[8], row[8], t0 = 0;
      auto locate = [&](int i) {
        if (i >= im.n) return;
        t0 = im.span.token(im.t0 + i);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (32 * q >= runs) break;
          const int t = t0 + ((32 * q + lane) << shift), lb = t / bs;
          row[q] = t - lb * bs;
          page[q] = -1;
          const bool in = 32 * q + lane < runs && t <= im.span.hi && (t + box > im.span.lo || t < a.sinks);
          if (!in) row[q] = -1;
          else if (lb < a.kv.max_blocks) page[q] = __ldg(a.kv.table + (size_t)im.b * a.kv.max_blocks + lb);
        }
      };
      locate(0);
#pragma unroll 1
      for (int i = 0; i < im.n; ++i, ++it) {
        const int s = it % ST;
        if (it >= ST) wait(&ss.empty[s], ((it / ST) - 1) & 1, a.status, abort);
        uint8_t* st = sm + RING_OFF + s * TILE_BYTES;
        uint8_t* sc = sm + SCALE_OFF + s * MAX_TILE * 16;
        if (ar.box) {
          const bool m = page[0] >= 0 && page[0] < a.kv.num_blocks;
          if (row[0] >= 0 && !m) atomicOr(a.status, ST_UNMAPPED_PAGE);
          const uint32_t have = __ballot_sync(0xffffffffu, m);
#pragma unroll 1
          for (int q = 0; 32 * q < tile; ++q) {
            const int k = 32 * q + lane, t = t0 + k;
            const bool see = k < tile && ((have >> (k >> shift)) & 1) && t <= im.span.hi &&
                             (t >= im.span.lo || t < a.sinks);
            const uint32_t w = __ballot_sync(0xffffffffu, see);
            if (lane == 0) ss.valid[s][q] = w;
          }
          if (lane == 0) mbar_arrive_expect_tx(&ss.full[s], __popc(have) * box * (128 * chunks + 16));
          __syncwarp();
          if (m) {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c)
              tma_load_3d(st + ((c * tile + (lane << shift)) << 7), &ar.codes, 128 * c, row[0], page[0],
                          &ss.full[s]);
            tma_load_3d(sc + ((lane << shift) << 4), &ar.scales, a.kv_dim, row[0], page[0], &ss.full[s]);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            if (32 * q >= tile) break;
            const bool m = page[q] >= 0 && page[q] < a.kv.num_blocks;
            if (row[q] >= 0 && !m) atomicOr(a.status, ST_UNMAPPED_PAGE);
            const uint32_t w = __ballot_sync(0xffffffffu, m);
            if (lane == 0) ss.valid[s][q] = w;
            const long long off = m ? page[q] * a.kv.stride_block + row[q] * a.kv.stride_tok : 0;
            const int pieces = a.kv_dim / 16;
#pragma unroll 1
            for (int r = 0; r < 32; ++r) {
              const long long ro = __shfl_sync(0xffffffffu, off, r);
              if (!((w >> r) & 1)) continue;
              const int k = 32 * q + r;
#pragma unroll 1
              for (int p = lane; p <= 8 * chunks; p += 32) {
                if (p == 8 * chunks)
                  cp_async16(sc + k * 16, a.kv.base + ro + a.kv_dim, 16);
                else  // (zeros behind the last of an odd number of 64-wide slices)
                  cp_async16(st + (((p >> 3) * tile + k) << 7) + (((p & 7) ^ (k & 7)) << 4),
                             a.kv.base + ro + (p < pieces ? 16 * p : 0), p < pieces ? 16 : 0);
              }
            }
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&ss.full[s]);
        }
        locate(i + 1);
      }
    }
    return;
  }

  // ------------------------------------------------------------------------------ workers
  const int i4 = lane >> 2, j4 = lane & 3;  // fragment row and column group
  const int chunk = warp % chunks, sub = warp / chunks;
  const bool works = sub < subs;
  const int hpg = a.n_q / (a.kv_dim / a.head_dim);
  const int dshift = a.head_dim == 64 ? 6 : 7;
  auto heads_of = [&](int ch) { return hpg * (min(128, a.kv_dim - 128 * ch) > a.head_dim ? 2 : 1); };
  const int cheads = heads_of(chunk);
  if (warp == WARPS - 1)
#pragma unroll 1
    for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
      const RowInfo info = row_info(a, sh, plan, r);
      if (lane == 0) ar.ws.rows[r] = info;
    }
  __half* sq = reinterpret_cast<__half*>(sm + Q_OFF);
  uint32_t it = 0;
#pragma unroll 1
  while (next_job(a, sh, plan, items, im)) {
    workers_sync();  // the previous item's columns are no longer in use
    if (warp == 0) {
      const int n = group_rows(a, sh, im.b, im.group, ss.group_row, ss.group_pos);
      if (lane == 0) ss.rows = n;
    }
    workers_sync();
    const int nrows = ss.rows, nq = nrows * cheads;
    // queries: 16 lanes a column of a chunk
#pragma unroll 1
    for (int i = tid; i < chunks * COLS * 16; i += WARPS * 32) {
      const int d = (i & 15) * 8, c = (i >> 4) % COLS, ch = i / (16 * COLS), heads = heads_of(ch);
      const int jr = c / heads, h = c - jr * heads, sl = h / hpg;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (c < nrows * heads && (d >> dshift) == sl)
        x = *reinterpret_cast<const uint4*>(a.q + ss.group_row[jr] * a.q_stride +
                                            ((long long)ch * sh.heads + h) * a.head_dim + d - (sl << dshift));
      float v[8], m = 0.0f;
      bf16x8_to_f32(x, v);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (fabsf(v[e]) <= 3.4e38f) m = fmaxf(m, fabsf(v[e]));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int e = query_exponent(m);
      if (d == 0) ss.qs[ch][c] = pow2(e) * a.scale * LOG2E;
      store_query(sq + (ch * COLS + c) * QLD, d, v, pow2(-e));
    }
    // what the thread's two rows (columns i4 and i4 + 8 of the chunk) see
    int hi[2], lo[2], min_hi = 0x7FFFFFFF, max_lo = 0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int c = i4 + 8 * r;
      hi[r] = !a.causal || c >= nq ? im.span.hi : ss.group_pos[c / cheads];
      lo[r] = a.window > 0 ? max(0, hi[r] - a.window + 1) : 0;
      min_hi = min(min_hi, hi[r]);
      max_lo = max(max_lo, lo[r]);
    }
    workers_sync();
    const float qs[2] = {ss.qs[chunk][i4], ss.qs[chunk][i4 + 8]};
    uint32_t q[8][4];  // the chunk's queries stay in registers
#pragma unroll
    for (int u = 0; u < 8; ++u)
      ldsm_x4(q[u], sq + (chunk * COLS + (lane & 15)) * QLD + (lane >> 4) * 8 + 16 * u);
    float o[16][4], l[2] = {0.0f, 0.0f}, nm[2] = {-UNSET, -UNSET};
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;

    if (works) {
#pragma unroll 1
      for (int i = 0; i < im.n; ++i) {
        const int s = (it + i) % ST, t0 = im.span.token(im.t0 + i) + sub * BLOCK;
        const uint8_t* codes = sm + RING_OFF + s * TILE_BYTES + ((chunk * tile + sub * BLOCK) << 7);
        wait(&ss.full[s], ((it + i) / ST) & 1, a.status, abort);
        // ---- scores
        float c[NB][4];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint4 x = lds128(codes + (8 * n + i4) * 128 + (((j4 + 4 * p) ^ i4) << 4));
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t b[2];
              e4m3x4_to_f16x4(xs[u], b);
              mma_f16_acc(c[n], q[4 * p + u], b[0], b[1]);
            }
          }
        }
        // ---- weights: tokens 8n + 2j, 8n + 2j + 1
        const float* scp = reinterpret_cast<const float*>(sm + SCALE_OFF + s * MAX_TILE * 16) + 4 * sub * BLOCK;
        float ct[2 * NB], sc[2 * NB];
        bool odd = false;  // a scale that is no ordinary number
#pragma unroll
        for (int e = 0; e < 2 * NB; ++e) {
          sc[e] = ct[e] = scp[4 * (2 * j4 + (e & 1) + 8 * (e >> 1))];
          odd |= !(sc[e] >= 8.077935669463161e-28f && sc[e] <= 3.0e38f);  // 2^LEAST
        }
        const uint32_t ok = ss.valid[s][sub];
        const bool mask = ok != 0xFFFFFFFFu || t0 + BLOCK - 1 > min_hi || (t0 < max_lo && t0 + BLOCK > a.sinks);
        const uint32_t rare = __ballot_sync(0xffffffffu, odd || mask);
        if (__builtin_expect(rare != 0, 0)) {
#pragma unroll
          for (int e = 0; e < 2 * NB; ++e) {
            const bool fin = fabsf(sc[e]) <= 3.0e38f;
            ct[e] = fin ? sc[e] : __int_as_float(0x7FC00000);
            sc[e] = fmaxf(fin ? sc[e] : 0.0f, 8.077935669463161e-28f);
          }
        }
        uint32_t pa[2 * NB];
        float w[NB][4];
#pragma unroll 1
        for (bool moved = false;; moved = true) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[n][e] = fmaf(c[n][e] * ct[2 * n + (e & 1)], qs[e >> 1], nm[e >> 1]);
          if (__builtin_expect(rare != 0, 0)) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int k = 8 * n + 2 * j4 + (e & 1), t = t0 + k, r = e >> 1;
                if (!((ok >> k) & 1) || t > hi[r] || (t < lo[r] && t >= a.sinks)) w[n][e] = -INFINITY;
              }
          }
#pragma unroll
          for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[n][e] = ex2(w[n][e]);
            pa[2 * n] = f16x2(w[n][0] * sc[2 * n], w[n][1] * sc[2 * n + 1]);
            pa[2 * n + 1] = f16x2(w[n][2] * sc[2 * n], w[n][3] * sc[2 * n + 1]);
          }
          // (f16 has infinities from 65520 on; NaN is no reason)
          uint32_t top = pa[0];
#pragma unroll
          for (int n = 1; n < 2 * NB; ++n) asm("max.f16x2 %0, %0, %1;" : "+r"(top) : "r"(pa[n]));
          const bool over = (top & 0x7FFFu) > 0x7800u || (top >> 16) > 0x7800u;  // 2^15
          if (moved || !__any_sync(0xffffffffu, over)) break;
          // m moves: each row's largest weight times scale of the block, over the row's four lanes
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float m = -INFINITY;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int e = 2 * r; e < 2 * r + 2; ++e) {
                const int k = 8 * n + 2 * j4 + (e & 1), t = t0 + k;
                const float v = fmaf(c[n][e] * ct[2 * n + (e & 1)], qs[r], log2_of(sc[2 * n + (e & 1)]));
                const bool see = ((ok >> k) & 1) && t <= hi[r] && (t >= lo[r] || t < a.sinks);
                if (see && v > m) m = v;
              }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const float old = -nm[r];
            float f = 1.0f;
            if (m - old > BASE) {
              const float now = fminf(ceilf(m) - BASE, 3.0e38f);
              f = old == UNSET ? 0.0f : ex2(old - now);
              nm[r] = -now;
            }
            l[r] *= f;
#pragma unroll
            for (int n = 0; n < 16; ++n) o[n][2 * r] *= f, o[n][2 * r + 1] *= f;
          }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          l[0] += w[n][0] + w[n][1];
          l[1] += w[n][2] + w[n][3];
        }
        // ---- sums: dimension 16 i + n is MMA n's column i
#pragma unroll
        for (int z = 0; z < BLOCK / 16; ++z) {
          uint4 v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 2 * j4 + (e & 1) + 8 * (e >> 1);
            v[e] = lds128(codes + (16 * z + r) * 128 + ((i4 ^ (r & 7)) << 4));
          }
          if (__builtin_expect(rare != 0, 0)) {
            // a NaN code that a row must not see would reach it as 0 * NaN
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = without_nan(v[e]);
          }
          const uint32_t az[4] = {pa[4 * z], pa[4 * z + 1], pa[4 * z + 2], pa[4 * z + 3]};
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t x0 = g == 0 ? v[0].x : g == 1 ? v[0].y : g == 2 ? v[0].z : v[0].w;
            const uint32_t x1 = g == 0 ? v[1].x : g == 1 ? v[1].y : g == 2 ? v[1].z : v[1].w;
            const uint32_t x2 = g == 0 ? v[2].x : g == 1 ? v[2].y : g == 2 ? v[2].z : v[2].w;
            const uint32_t x3 = g == 0 ? v[3].x : g == 1 ? v[3].y : g == 2 ? v[3].z : v[3].w;
            uint32_t b0[4], b1[4];
            pair_codes(x0, x1, b0);
            pair_codes(x2, x3, b1);
#pragma unroll
            for (int e = 0; e < 4; ++e) mma_f16_acc(o[4 * g + e], az, b0[e], b1[e]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.empty[s]);
      }
    }
    it += im.n;
    // ---- the subs' results come together, halving their number: m, l and O by column
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    float* sums = reinterpret_cast<float*>(sm + SUM_OFF);
    workers_sync();  // (where the queries were)
#pragma unroll 1
    for (int half = subs / 2; half >= 1; half /= 2) {
      float* mine = sums + ((sub % half) * chunks + chunk) * COLS * SUM_LD;
      if (sub >= half && sub < 2 * half) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float* col = mine + (i4 + 8 * r) * SUM_LD;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < 16; n += 4)
              *reinterpret_cast<float4*>(col + 16 * (2 * j4 + h) + n) =
                  make_float4(o[n][2 * r + h], o[n + 1][2 * r + h], o[n + 2][2 * r + h], o[n + 3][2 * r + h]);
          if (j4 == 0) col[128] = -nm[r], col[129] = l[r];
        }
      }
      workers_sync();
      if (sub < half) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float* col = mine + (i4 + 8 * r) * SUM_LD;
          const float m1 = col[128], l1 = col[129], m0 = -nm[r], m = fmaxf(m0, m1);
          // (a side that has seen nothing but a NaN keeps it)
          const float f0 = l[r] != l[r] ? 1.0f : m0 == UNSET ? 0.0f : ex2(m0 - m);
          const float f1 = l1 != l1 ? 1.0f : m1 == UNSET ? 0.0f : ex2(m1 - m);
          nm[r] = -m;
          l[r] = l[r] * f0 + l1 * f1;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < 16; n += 4) {
              const float4 x = *reinterpret_cast<const float4*>(col + 16 * (2 * j4 + h) + n);
              o[n][2 * r + h] = o[n][2 * r + h] * f0 + x.x * f1;
              o[n + 1][2 * r + h] = o[n + 1][2 * r + h] * f0 + x.y * f1;
              o[n + 2][2 * r + h] = o[n + 2][2 * r + h] * f0 + x.z * f1;
              o[n + 3][2 * r + h] = o[n + 3][2 * r + h] * f0 + x.w * f1;
            }
        }
      }
      workers_sync();
    }
    if (sub == 0) {
      const bool whole = im.n == im.span.tiles;  // nobody else has tiles of this group
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int c = i4 + 8 * r;
        if (c >= nq) continue;
        const int jr = c / cheads, h = c - jr * cheads, sl = h / hpg;
        const long long head = (long long)chunk * sh.heads + h;
        const float inv = !whole ? 1.0f : l[r] == 0.0f ? 0.0f : 1.0f / l[r];
        float* part = ar.ws.part +
                      ((((size_t)blockIdx.x * 2 + (im.t0 > 0 ? 0 : 1)) * chunks + chunk) * COLS + c) * PART_LD;
        __nv_bfloat16* out = a.o + ss.group_row[jr] * a.o_stride + head * a.head_dim;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int d = 16 * (2 * j4 + hh), dl = d - (sl << dshift);
          if ((d >> dshift) != sl) continue;
#pragma unroll
          for (int n = 0; n < 16; n += 8) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = o[n + e][2 * r + hh] * inv;
            if (whole) {
              *reinterpret_cast<uint4*>(out + dl + n) =
                  make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                             pack_bf16x2(x[6], x[7]));
            } else {
              *reinterpret_cast<float4*>(part + 4 + dl + n) = make_float4(x[0], x[1], x[2], x[3]);
              *reinterpret_cast<float4*>(part + 8 + dl + n) = make_float4(x[4], x[5], x[6], x[7]);
            }
          }
        }
        if (j4 == 0) {
          if (whole)
            a.lse[(long long)ss.group_row[jr] * a.n_q + head] =
                l[r] == 0.0f ? -INFINITY : (log2f(l[r]) - nm[r]) * LN2;
          else
            part[0] = -nm[r], part[1] = l[r];
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------- weights
constexpr int W_WARPS = 8, W_THREADS = W_WARPS * 32;
constexpr int W_ROWS = 6;   // rows of a pass, while their queries fit the shared memory
constexpr int W_TILE = 128; // tokens of a unit: 16 a warp
constexpr int W_PLAN = (3 * MAX_REQ + 4) * 4;
constexpr int W_SMEM_MAX = 110 * 1024;  // two CTAs an SM

// Bytes of a row's queries (rows of a slice's heads padded to 16, f16, 8 elements of padding each)
__host__ __device__ __forceinline__ int w_row_bytes(const AttendArgs& a) {
  return a.kv_dim / a.head_dim * 16 * (a.head_dim + 8) * 2;
}

template <int DH>
__global__ void __launch_bounds__(W_THREADS, 2) attend_weights_kernel(const AttendArgs a, const Shape sh,
                                                                    int* total, int rows_fit) {
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ Jobs s_start;
  __shared__ int s_row[W_ROWS], s_pos[W_ROWS], s_n;
  __shared__ float s_lse[W_ROWS * 256], s_qs[W_ROWS * 256];  // by (row, head), up to 256 heads
  Plan plan;
  plan.pre = reinterpret_cast<int*>(sm);
  plan.pmax = plan.pre + MAX_REQ + 4;
  plan.pmin = plan.pmax + MAX_REQ;
  __half* sq = reinterpret_cast<__half*>(sm + W_PLAN);
  constexpr int QLD = DH + 8, STEPS = DH / 16, PIECES = DH / 64;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i4 = lane >> 2, j4 = lane & 3;
  const int G = a.kv_dim / DH, hpg = a.n_q / G;
  derive_plan<W_THREADS>(a, sh, plan, blockIdx.x, true, &s_start, total);
  __syncthreads();
  Jobs items = s_start;
  Job im;
#pragma unroll 1
  while (next_job(a, sh, plan, items, im)) {
    // every row of the request in turn, rows_fit at a time
#pragma unroll 1
    for (int first = 0;; first += rows_fit) {
      __syncthreads();
      if (warp == 0) {
        int seen = 0, n = 0;
#pragma unroll 1
        for (int r0 = 0; r0 < a.rows && n < rows_fit; r0 += 32) {
          const int r = r0 + lane;
          const int qb = r < a.rows ? a.row_req[r] : -1, p0 = r < a.rows ? a.positions[r] : -1;
          const int p = qb == im.b ? p0 : -1;
          const uint32_t m = __ballot_sync(0xffffffffu, p >= 0);
          const int rank = seen + __popc(m & ((1u << lane) - 1)) - first;
          if (p >= 0 && rank >= 0 && rank < rows_fit) s_row[rank] = r, s_pos[rank] = p;
          seen += __popc(m);
          n = max(0, min(rows_fit, seen - first));
        }
        if (lane == 0) s_n = n;
      }
      __syncthreads();
      const int n = s_n;
      if (n == 0) break;
      // queries as f16 under a power of two per head
      constexpr int LN = DH / 8;  // lanes of a head
#pragma unroll 1
      for (int i0 = 0; i0 < n * G * 16 * LN; i0 += W_THREADS) {
        const int i = i0 + tid, c = i / LN, d = (i % LN) * 8;
        const int h16 = c % 16, g = (c / 16) % G, r = c / (16 * G);
        const bool in = r < n && h16 < hpg;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (in)
          x = *reinterpret_cast<const uint4*>(a.q + s_row[r] * a.q_stride + (g * hpg + h16) * DH + d);
        float v[8], m = 0.0f;
        bf16x8_to_f32(x, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (fabsf(v[e]) <= 3.4e38f) m = fmaxf(m, fabsf(v[e]));
#pragma unroll
        for (int o = 1; o < LN; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int ex = query_exponent(m);
        const float up = pow2(-ex);
        if (r >= n) continue;
        if (d == 0) {
          const int k = (r * G + g) * 16 + h16;
          s_qs[k] = pow2(ex) * a.scale * LOG2E;
          s_lse[k] = in ? a.lse[(long long)s_row[r] * a.n_q + g * hpg + h16] * LOG2E : INFINITY;
        }
        store_query(sq + (size_t)c * QLD, d, v, up);
      }
      __syncthreads();
#pragma unroll 1
      for (int k = 0; k < im.n; ++k) {
        // a warp's 16 tokens: lanes of a quad share tokens i4 and i4 + 8
        const int t0 = im.span.token(im.t0 + k) + 16 * warp;
        if (t0 > im.span.hi) continue;
        const uint8_t* rec[2];
        float sc[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = t0 + i4 + 8 * e;
          const long long off = t <= im.span.hi && (t >= im.span.lo || t < a.sinks)
                                    ? record_offset(a.kv, im.b, t) : -1;
          rec[e] = off >= 0 ? a.kv.base + off : nullptr;
        }
        float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // tokens 2j, 2j + 1, 2j + 8, 2j + 9
        float ct[4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          sc[e] = rec[e] ? *reinterpret_cast<const float*>(rec[e] + a.kv_dim) : 0.0f;
        const uint32_t there0 = __ballot_sync(0xffffffffu, rec[0] != nullptr);
        const uint32_t there1 = __ballot_sync(0xffffffffu, rec[1] != nullptr);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ct[e] = __shfl_sync(0xffffffffu, sc[e >> 1], 4 * (2 * j4 + (e & 1)));
        uint4 nx[2][PIECES];
        auto fetch = [&](int g) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
              nx[e][p] = rec[e] ? __ldg(reinterpret_cast<const uint4*>(rec[e] + g * DH + 64 * p + 16 * j4))
                                : make_uint4(0, 0, 0, 0);
        };
        fetch(0);
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
          uint32_t b[2][STEPS][2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
              e4m3x4_to_f16x4(nx[e][p].x, b[e][4 * p]);
              e4m3x4_to_f16x4(nx[e][p].y, b[e][4 * p + 1]);
              e4m3x4_to_f16x4(nx[e][p].z, b[e][4 * p + 2]);
              e4m3x4_to_f16x4(nx[e][p].w, b[e][4 * p + 3]);
            }
          if (g + 1 < G) fetch(g + 1);
#pragma unroll 1
          for (int r = 0; r < n; ++r) {
            const int hi = a.causal ? s_pos[r] : im.span.hi;
            const int lo = a.window > 0 ? max(0, hi - a.window + 1) : 0;
            float c[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[0][e] = c[1][e] = 0.0f;
            const __half* src = sq + ((size_t)(r * G + g) * 16 + (lane & 15)) * QLD + (lane >> 4) * 8;
#pragma unroll
            for (int k16 = 0; k16 < STEPS; ++k16) {
              uint32_t qf[4];
              ldsm_x4(qf, src + 16 * k16);
              mma_f16_acc(c[0], qf, b[0][k16][0], b[0][k16][1]);
              mma_f16_acc(c[1], qf, b[1][k16][0], b[1][k16][1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int at = (r * G + g) * 16 + i4 + 8 * h;
              const float qs = s_qs[at], ls = s_lse[at];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int t = t0 + 2 * j4 + (e & 1) + 8 * (e >> 1);
                const bool see = t <= hi && (t >= lo || t < a.sinks) &&
                                 (((e >> 1 ? there1 : there0) >> (4 * (2 * j4 + (e & 1)))) & 1);
                const float p = ex2(fmaf(c[e >> 1][2 * h + (e & 1)] * ct[e], qs, -ls));
                if (see) w[e] += p;
              }
            }
          }
        }
        // the heads' sums, over the lanes that share tokens; in a fixed order
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] += __shfl_xor_sync(0xffffffffu, w[e], 4);
          w[e] += __shfl_xor_sync(0xffffffffu, w[e], 8);
          w[e] += __shfl_xor_sync(0xffffffffu, w[e], 16);
        }
        if (lane < 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = t0 + 2 * j4 + (e & 1) + 8 * (e >> 1);
            const bool there = ((e >> 1 ? there1 : there0) >> (4 * (2 * j4 + (e & 1)))) & 1;
            if (there && t < a.weights_stride) a.weights[im.b * a.weights_stride + t] += w[e];
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t attend_few_prepare() {
  cudaError_t e = cudaFuncSetAttribute(attend_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attend_weights_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, W_SMEM_MAX);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attend_weights_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, W_SMEM_MAX);
  return e;
}

// Warps per chunk, and with them the tokens of a tile.
static int subs_of(int chunks) {
  int subs = 1;
  while (2 * subs * chunks <= WARPS) subs *= 2;
  return subs;
}

bool attend_few_fits(const AttendArgs& a) {
  // at most a row or so per request, and its columns of a chunk within 16
  const Shape sh = shape_of(a, BLOCK, COLS, 1);
  const int rows = (a.rows + a.n_req - 1) / a.n_req;
  return sh.heads <= COLS && sh.chunks <= 8 && rows <= sh.rows_per;
}

cudaError_t launch_attend_few(const Launch& L, const AttendArgs& a, const attend::Pieces& ws, int sms) {
  const int chunks = (a.kv_dim + 127) / 128, subs = subs_of(chunks);
  Args ar = {{}, {}, 0, subs, a, shape_of(a, subs * BLOCK, COLS, sms), ws};
  const int bs = a.kv.block_size;
  if (bs % 8 == 0) {
    const int box = std::min(bs & -bs, subs * BLOCK);
    if (encode_cache_map(&ar.codes, a.kv, a.kv_dim, 128, box) &&
        encode_cache_map(&ar.scales, a.kv, a.kv_dim + 16, 16, box))
      ar.box = box;
  }
  const cudaError_t e = launch_ex(L, dim3(sms), dim3(THREADS), SMEM_BYTES, attend_few_kernel, ar);
  return e == cudaSuccess ? attend::launch_join(L, a, ar.sh, ws) : e;
}

cudaError_t launch_attend_weights(const Launch& L, const AttendArgs& a, const attend::Pieces& ws, int sms) {
  Shape sh = shape_of(a, W_TILE, COLS, 2 * sms);
  sh.rows_per = 1024;  // a unit is a tile with all its request's rows
  const int row = w_row_bytes(a);
  const int fit = std::max(1, std::min(W_ROWS, (W_SMEM_MAX - W_PLAN) / row));
  const int smem = W_PLAN + fit * row;
  return launch_ex(L, dim3(2 * sms), dim3(W_THREADS), smem,
                   a.head_dim == 128 ? attend_weights_kernel<128> : attend_weights_kernel<64>, a, sh,
                   ws.total, fit);
}

}  // namespace mono
