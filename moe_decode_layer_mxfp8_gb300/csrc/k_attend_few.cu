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

constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int BLOCK = 16;             // tokens of a warp's step
constexpr int TILE = 64;              // tokens of a unit of work
constexpr int ST = 8;                 // blocks in a warp's ring
constexpr int CODES = BLOCK * 128, BLOCK_BYTES = CODES + BLOCK * 16;  // codes, then scale runs
constexpr int COLS = 16;
constexpr int RING_OFF = 0;                                  // [WARPS][ST] codes (1 KB atoms)
constexpr int SCALE_OFF = RING_OFF + WARPS * ST * CODES;     // [WARPS][ST] scale runs
constexpr int SUM_OFF = SCALE_OFF + WARPS * ST * BLOCK * 16; // [WARPS][COLS][SUM_LD]: O, m, l
constexpr int SUM_LD = 128 + 4;
constexpr int PLAN_OFF = SUM_OFF + WARPS * COLS * SUM_LD * 4;
constexpr int SMEM_BYTES = PLAN_OFF + (3 * MAX_REQ + 4) * 4 + 1024;
static_assert(SMEM_BYTES + 2048 <= 227 * 1024, "shared memory");

struct Args {
  CUtensorMap codes, scales;
  int tma;
  AttendArgs a;
  Shape sh;
  Pieces ws;
};

struct Shared {
  uint64_t full[WARPS][ST];
  uint32_t valid[WARPS][ST];
  int group_row[16], group_pos[16], rows;
  float fac[COLS][WARPS];
  Jobs start;
};

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Bounded wait by every lane (some 10^7 polls); after a timeout the data is whatever it is.
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, int* status) {
  uint32_t polls = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (++polls == (1u << 23)) {
      atomicOr(status, ST_WAIT_TIMEOUT);
      break;
    }
  __syncwarp();
}
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
  Plan plan;
  plan.pre = reinterpret_cast<int*>(sm + PLAN_OFF);
  plan.pmax = plan.pre + MAX_REQ + 4;
  plan.pmin = plan.pmax + MAX_REQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i4 = lane >> 2, j4 = lane & 3;  // fragment row and column group
  const int chunks = sh.chunks, subs = WARPS / chunks;  // warps per chunk
  const int chunk = warp % chunks, sub = warp / chunks;
  const bool works = sub < subs;
  if (lane == 0)
    for (int s = 0; s < ST; ++s) mbar_init(&ss.full[warp][s], ar.tma ? 1 : 32);
  fence_mbar_init();
  derive_plan<THREADS>(a, sh, plan, blockIdx.x, true, &ss.start, ar.ws.total);
  __syncthreads();
  Jobs items = ss.start;
  Job im;
  if (warp == WARPS - 1)
#pragma unroll 1
    for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
      const RowInfo info = row_info(a, sh, plan, r);
      if (lane == 0) ar.ws.rows[r] = info;
    }

  const int chunk_bytes = min(128, a.kv_dim - 128 * chunk);
  const int hpg = a.n_q / (a.kv_dim / a.head_dim);
  const int cheads = hpg * (chunk_bytes > a.head_dim ? 2 : 1);
  const int dshift = a.head_dim == 64 ? 6 : 7;
  uint8_t* ring = sm + RING_OFF + warp * ST * CODES;
  uint8_t* runs = sm + SCALE_OFF + warp * ST * BLOCK * 16;
  uint32_t used = 0;  // blocks taken from the ring since the start (mod 2^32)

#pragma unroll 1
  while (next_job(a, sh, plan, items, im)) {
    __syncthreads();  // the previous item's columns are no longer in use
    if (warp == 0) {
      const int n = group_rows(a, sh, im.b, im.group, ss.group_row, ss.group_pos);
      if (lane == 0) ss.rows = n;
    }
    // this warp's blocks of the item: every subs-th of its tiles' blocks
    constexpr int PER = TILE / BLOCK;
    const int blocks = works ? (im.n * PER - sub + subs - 1) / subs : 0;
    auto token = [&](int k) {  // first token of the warp's k-th block
      const int g = sub + k * subs;
      return im.span.token(im.t0 + g / PER) + (g % PER) * BLOCK;
    };
    // pages: of block kb + lane of the warp, looked up 32 blocks at a time; or, where pages are no
    // multiple of 16, of a lane's token of block kb.  -2: nothing there to see, -1: unmapped.
    auto lookup = [&](int kb) {
      const int k = ar.tma ? kb + lane : kb;
      if (k >= blocks) return -2;
      const int t = token(k) + (ar.tma ? 0 : lane >> 1), lb = t / a.kv.block_size;
      const bool in = ar.tma ? t <= im.span.hi && (t + BLOCK > im.span.lo || t < a.sinks)
                             : t <= im.span.hi && (t >= im.span.lo || t < a.sinks);
      if (!in) return -2;
      return lb < a.kv.max_blocks ? max(-1, __ldg(a.kv.table + (size_t)im.b * a.kv.max_blocks + lb)) : -1;
    };
    int pages = -2, pages_next = -2;
    auto request = [&](int k, uint32_t at) {  // block k into ring slot at % ST
      const int s = at % ST;
      int page = pages;
      if (ar.tma) {
        if (k > 0 && (k & 31) == 0) pages = pages_next, pages_next = lookup(k + 32);
        page = __shfl_sync(0xffffffffu, pages, k & 31);
      }
      const int tk = token(k) + (ar.tma ? 0 : lane >> 1), row = tk % a.kv.block_size;
      const bool mapped = page >= 0 && page < a.kv.num_blocks;
      if (page != -2 && !mapped) atomicOr(a.status, ST_UNMAPPED_PAGE);
      uint8_t* dst = ring + s * CODES;
      uint8_t* sc = runs + s * BLOCK * 16;
      if (ar.tma) {
        const int t = token(k) + (lane & 15);
        const uint32_t v = __ballot_sync(0xffffffffu, mapped && t <= im.span.hi &&
                                                          (t >= im.span.lo || t < a.sinks));
        if (lane == 0) {
          ss.valid[warp][s] = v;
          mbar_arrive_expect_tx(&ss.full[warp][s], mapped ? BLOCK_BYTES : 0);
          if (mapped) {
            tma_load_3d(dst, &ar.codes, 128 * chunk, row, page, &ss.full[warp][s]);
            tma_load_3d(sc, &ar.scales, a.kv_dim, row, page, &ss.full[warp][s]);
          }
        }
      } else {
        const uint32_t m = __ballot_sync(0xffffffffu, mapped);
        uint32_t v = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) v |= ((m >> (2 * e)) & 1) << e;
        if (lane == 0) ss.valid[warp][s] = v;
        const int r = lane >> 1;
        const uint8_t* src = a.kv.base;
        if (mapped) src += page * a.kv.stride_block + row * a.kv.stride_tok;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int p = 4 * (lane & 1) + e;
          const bool in = mapped && 16 * p < chunk_bytes;
          cp_async16(dst + r * 128 + ((p ^ (r & 7)) << 4), in ? src + 128 * chunk + 16 * p : a.kv.base,
                     in ? 16 : 0);
        }
        if (!(lane & 1)) cp_async16(sc + r * 16, mapped ? src + a.kv_dim : a.kv.base, mapped ? 16 : 0);
        cp_async_arrive_noinc(&ss.full[warp][s]);
      }
    };
    pages = lookup(0);
    if (ar.tma) pages_next = lookup(32);
#pragma unroll 1
    for (int k = 0; k < min(blocks, ST); ++k) {
      request(k, used + k);
      if (!ar.tma) pages = lookup(k + 1);
    }
    __syncthreads();
    const int nrows = ss.rows, nq = nrows * cheads;

    // queries: column c = 16 rows of the MMA's A; this thread's rows i4 and i4 + 8.  K step (p, u)
    // pairs MMA columns 2j, 2j + 1, 2j + 8, 2j + 9 with dimensions 64 p + 16 j + 4 u + 0..3, as a
    // lane holds codes.
    uint32_t q[2][4][4];
    float qs[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int c = i4 + 8 * r, jr = c / cheads, h = c - jr * cheads, sl = h / hpg;
      const bool in = works && c < nq;
      const __nv_bfloat16* src =
          a.q + (in ? ss.group_row[jr] * a.q_stride + ((long long)chunk * sh.heads + h) * a.head_dim : 0);
      float v[2][16], m = 0.0f;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int d = 64 * p + 16 * j4;
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (in && (d >> dshift) == sl) {
          const uint4* s4 = reinterpret_cast<const uint4*>(src + d - (sl << dshift));
          x = s4[0], y = s4[1];
        }
        float f[8];
        bf16x8_to_f32(x, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[p][e] = f[e];
        bf16x8_to_f32(y, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[p][8 + e] = f[e];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (fabsf(v[p][e]) <= 3.4e38f) m = fmaxf(m, fabsf(v[p][e]));
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      // the column's largest to [2^8, 2^9); exponents far from one stay in reach of f32
      const int e = m > 0.0f ? min(max((int)(__float_as_uint(m) >> 23) - 127 - 8, -100), 100) : 0;
      const float up = __uint_as_float((uint32_t)(127 - e) << 23);
      qs[r] = __uint_as_float((uint32_t)(127 + e) << 23) * a.scale * LOG2E;
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          q[p][u][r] = f16x2(v[p][4 * u] * up, v[p][4 * u + 1] * up);
          q[p][u][2 + r] = f16x2(v[p][4 * u + 2] * up, v[p][4 * u + 3] * up);
        }
    }
    // what the two rows see
    int hi[2], lo[2], min_hi = 0x7FFFFFFF, max_lo = 0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int c = i4 + 8 * r;
      hi[r] = !a.causal || c >= nq ? im.span.hi : ss.group_pos[c / cheads];
      lo[r] = a.window > 0 ? max(0, hi[r] - a.window + 1) : 0;
      min_hi = min(min_hi, hi[r]);
      max_lo = max(max_lo, lo[r]);
    }
    float o[16][4], l[2] = {0.0f, 0.0f}, nm[2] = {-UNSET, -UNSET};
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;

#pragma unroll 1
    for (int k = 0; k < blocks; ++k) {
      const uint32_t at = used + k;
      const int s = at % ST, t0 = token(k);
      const uint8_t* codes = ring + s * CODES;
      wait(&ss.full[warp][s], (at / ST) & 1, a.status);
      const uint32_t ok = ss.valid[warp][s];
      // ---- scores of 16 tokens
      float c[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
        const int r = 8 * n + i4;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 w = lds128(codes + r * 128 + (((j4 + 4 * p) ^ (r & 7)) << 4));
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t b[2];
            e4m3x4_to_f16x4(ws[u], b);
            mma_f16_acc(c[n], q[p][u], b[0], b[1]);
          }
        }
      }
      // ---- weights
      const float* scp = reinterpret_cast<const float*>(runs + s * BLOCK * 16);
      const bool part = (ok & 0xFFFFu) != 0xFFFFu;
      const bool mask = __any_sync(0xffffffffu, part || t0 + BLOCK - 1 > min_hi ||
                                                    (t0 < max_lo && t0 + BLOCK > a.sinks));
      float sc[4], ct[4];  // tokens 2j, 2j + 1, 2j + 8, 2j + 9
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float raw = scp[4 * (2 * j4 + (e & 1) + 8 * (e >> 1))];
        const bool fin = fabsf(raw) <= 3.0e38f;
        ct[e] = fin ? raw : __int_as_float(0x7FC00000);
        sc[e] = fmaxf(fin ? raw : 0.0f, 8.077935669463161e-28f);  // 2^LEAST
      }
      uint32_t pa[4];
      float w[2][4];
#pragma unroll 1
      for (bool moved = false;; moved = true) {
        float top = 0.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = e >> 1, tk = 2 * n + (e & 1);
            float x = fmaf(c[n][e] * ct[tk], qs[r], nm[r]);
            if (mask) {
              const int t = t0 + 8 * n + 2 * j4 + (e & 1);
              if (!((ok >> (t - t0)) & 1) || t > hi[r] || (t < lo[r] && t >= a.sinks)) x = -INFINITY;
            }
            const float p = ex2(x);
            w[n][e] = p;
            const float v = p * sc[tk];
            top = fmaxf(top, v);
          }
        if (moved || !__any_sync(0xffffffffu, top > 32768.0f)) break;
        // m moves: each row's largest weight times scale of the block, over the row's four lanes
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float m = -INFINITY;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 2 * r; e < 2 * r + 2; ++e) {
              const int tk = 2 * n + (e & 1), t = t0 + 8 * n + 2 * j4 + (e & 1);
              const float v = fmaf(c[n][e] * ct[tk], qs[r], log2_of(sc[tk]));
              const bool see = ((ok >> (t - t0)) & 1) && t <= hi[r] && (t >= lo[r] || t < a.sinks);
              if (see && v > m) m = v;
            }
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const float old = -nm[r];
          if (m - old > BASE) {
            const float now = fminf(ceilf(m) - BASE, 3.0e38f);
            const float f = old == UNSET ? 0.0f : ex2(old - now);
            nm[r] = -now;
            l[r] *= f;
#pragma unroll
            for (int n = 0; n < 16; ++n) {
              o[n][2 * r] = f == 0.0f ? 0.0f : o[n][2 * r] * f;
              o[n][2 * r + 1] = f == 0.0f ? 0.0f : o[n][2 * r + 1] * f;
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        l[0] += w[n][0] + w[n][1];
        l[1] += w[n][2] + w[n][3];
        pa[2 * n] = f16x2(w[n][0] * sc[2 * n], w[n][1] * sc[2 * n + 1]);
        pa[2 * n + 1] = f16x2(w[n][2] * sc[2 * n], w[n][3] * sc[2 * n + 1]);
      }
      // ---- sums: dimension 16 i + n is MMA n's column i
      uint4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 2 * j4 + (e & 1) + 8 * (e >> 1);
        v[e] = lds128(codes + r * 128 + ((i4 ^ (r & 7)) << 4));
        if (__builtin_expect(mask, 0)) {
          // a NaN code that a row must not see would reach it as 0 * NaN
          uint32_t* x = reinterpret_cast<uint32_t*>(&v[e]);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t nan = (((x[g] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
            x[g] &= ~(nan * 0xFFu);
          }
        }
      }
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
        for (int e = 0; e < 4; ++e) mma_f16_acc(o[4 * g + e], pa, b0[e], b1[e]);
      }
      __syncwarp();
      if (k + ST < blocks) {
        request(k + ST, at + ST);
        if (!ar.tma) pages = lookup(k + ST + 1);
      }
    }
    used += blocks;
    // ---- the warps' results, to shared memory: each column's O, m and l
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    float* sums = reinterpret_cast<float*>(sm + SUM_OFF) + warp * COLS * SUM_LD;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float* row_sum = sums + (i4 + 8 * r) * SUM_LD;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < 16; n += 4)
          *reinterpret_cast<float4*>(row_sum + 16 * (2 * j4 + h) + n) =
              make_float4(o[n][2 * r + h], o[n + 1][2 * r + h], o[n + 2][2 * r + h], o[n + 3][2 * r + h]);
      if (j4 == 0) row_sum[128] = -nm[r], row_sum[129] = l[r];
    }
    __syncthreads();
    // a thread per (chunk, column, 16 dimensions): the subs' sums in the largest m
    const bool whole = im.n == im.span.tiles;
#pragma unroll 1
    for (int i = tid; i < chunks * COLS * 8; i += THREADS) {
      const int g = i & 7, c = (i >> 3) % COLS, ch = i / (8 * COLS);
      const int bytes = min(128, a.kv_dim - 128 * ch);
      const int heads = hpg * (bytes > a.head_dim ? 2 : 1);
      if (c >= nrows * heads) continue;
      const int jr = c / heads, h = c - jr * heads, sl = h / hpg;
      if (((16 * g) >> dshift) != sl) continue;
      const float* base = reinterpret_cast<const float*>(sm + SUM_OFF) + (ch * COLS + c) * SUM_LD;
      const int step = chunks * COLS * SUM_LD;
      float m = UNSET;
#pragma unroll 1
      for (int k = 0; k < subs; ++k) m = fmaxf(m, base[k * step + 128]);
      float acc[16], lt = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
#pragma unroll 1
      for (int k = 0; k < subs; ++k) {
        const float* p = base + k * step;
        const float lk = p[129], f = lk != lk ? 1.0f : p[128] == UNSET ? 0.0f : ex2(p[128] - m);
        if (f == 0.0f) continue;
        lt = fmaf(lk, f, lt);
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 x = *reinterpret_cast<const float4*>(p + 16 * g + e);
          acc[e] = fmaf(x.x, f, acc[e]), acc[e + 1] = fmaf(x.y, f, acc[e + 1]);
          acc[e + 2] = fmaf(x.z, f, acc[e + 2]), acc[e + 3] = fmaf(x.w, f, acc[e + 3]);
        }
      }
      const long long head = (long long)ch * sh.heads + h;
      const int dl = 16 * g - (sl << dshift);
      if (whole) {
        const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
        uint4* dst = reinterpret_cast<uint4*>(a.o + ss.group_row[jr] * a.o_stride + head * a.head_dim + dl);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          dst[e] = make_uint4(pack_bf16x2(acc[8 * e] * inv, acc[8 * e + 1] * inv),
                              pack_bf16x2(acc[8 * e + 2] * inv, acc[8 * e + 3] * inv),
                              pack_bf16x2(acc[8 * e + 4] * inv, acc[8 * e + 5] * inv),
                              pack_bf16x2(acc[8 * e + 6] * inv, acc[8 * e + 7] * inv));
        if (dl == 0)
          a.lse[(long long)ss.group_row[jr] * a.n_q + head] =
              lt == 0.0f ? -INFINITY : (log2f(lt) + m) * LN2;
      } else {
        float* dst = ar.ws.part +
                     ((((size_t)blockIdx.x * 2 + (im.t0 > 0 ? 0 : 1)) * chunks + ch) * COLS + c) * PART_LD;
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<float4*>(dst + 4 + dl + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
        if (dl == 0) dst[0] = m, dst[1] = lt;
      }
    }
  }
}

// ------------------------------------------------------------------------------- weights
constexpr int W_ROWS = 6;   // rows of a pass, while their queries fit the shared memory
constexpr int W_TILE = 128; // tokens of a unit: 16 a warp
constexpr int W_PLAN = (3 * MAX_REQ + 4) * 4;
constexpr int W_SMEM_MAX = 110 * 1024;  // two CTAs an SM

// Bytes of a row's queries (rows of a slice's heads padded to 16, f16, 8 elements of padding each)
__host__ __device__ __forceinline__ int w_row_bytes(const AttendArgs& a) {
  return a.kv_dim / a.head_dim * 16 * (a.head_dim + 8) * 2;
}

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}

template <int DH>
__global__ void __launch_bounds__(THREADS, 2) attend_weights_kernel(const AttendArgs a, const Shape sh,
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
  derive_plan<THREADS>(a, sh, plan, blockIdx.x, true, &s_start, total);
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
      // queries as f16 under a power of two per head, in the order in which lanes hold codes:
      // dimension 64 p + 16 j + 4 u + e at step 4 p + u, column 2 j + e (e < 2) or 2 j + 6 + e
      constexpr int LN = DH / 8;  // lanes of a head
#pragma unroll 1
      for (int i0 = 0; i0 < n * G * 16 * LN; i0 += THREADS) {
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
        const int ex = m > 0.0f ? min(max((int)(__float_as_uint(m) >> 23) - 127 - 8, -100), 100) : 0;
        const float up = __uint_as_float((uint32_t)(127 - ex) << 23);
        if (r >= n) continue;
        if (d == 0) {
          const int k = (r * G + g) * 16 + h16;
          s_qs[k] = __uint_as_float((uint32_t)(127 + ex) << 23) * a.scale * LOG2E;
          s_lse[k] = in ? a.lse[(long long)s_row[r] * a.n_q + g * hpg + h16] * LOG2E : INFINITY;
        }
        __half* dst = sq + (size_t)c * QLD;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int dd = d + 4 * t, p = dd >> 6, j = (dd >> 4) & 3, u = (dd >> 2) & 3;
          uint32_t* at = reinterpret_cast<uint32_t*>(dst + (4 * p + u) * 16 + 2 * j);
          at[0] = f16x2(v[4 * t] * up, v[4 * t + 1] * up);
          at[4] = f16x2(v[4 * t + 2] * up, v[4 * t + 3] * up);
        }
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

bool attend_few_fits(const AttendArgs& a) {
  // at most a row or so per request, and its columns of a chunk within 16
  const Shape sh = shape_of(a, TILE, COLS, 1);
  const int rows = (a.rows + a.n_req - 1) / a.n_req;
  return sh.heads <= COLS && sh.chunks <= WARPS && rows <= sh.rows_per;
}

cudaError_t launch_attend_few(const Launch& L, const AttendArgs& a, const attend::Pieces& ws, int sms) {
  Args ar = {{}, {}, 0, a, shape_of(a, TILE, COLS, sms), ws};
  if (a.kv.block_size % BLOCK == 0)
    ar.tma = encode_cache_map(&ar.codes, a.kv, a.kv_dim, 128, BLOCK) &&
             encode_cache_map(&ar.scales, a.kv, a.kv_dim + 16, 16, BLOCK);
  const cudaError_t e = launch_ex(L, dim3(sms), dim3(THREADS), SMEM_BYTES, attend_few_kernel, ar);
  return e == cudaSuccess ? attend::launch_join(L, a, ar.sh, ws) : e;
}

cudaError_t launch_attend_weights(const Launch& L, const AttendArgs& a, const attend::Pieces& ws, int sms) {
  Shape sh = shape_of(a, W_TILE, COLS, 2 * sms);
  sh.rows_per = 1024;  // a unit is a tile with all its request's rows
  const int row = w_row_bytes(a);
  const int fit = std::max(1, std::min(W_ROWS, (W_SMEM_MAX - W_PLAN) / row));
  const int smem = W_PLAN + fit * row;
  return launch_ex(L, dim3(2 * sms), dim3(THREADS), smem,
                   a.head_dim == 128 ? attend_weights_kernel<128> : attend_weights_kernel<64>, a, sh,
                   ws.total, fit);
}

}  // namespace mono
