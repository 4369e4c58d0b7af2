// Gathering of attention weights: with the attention's lse known,
//
//   weights[b][t] += sum over b's rows that see t, and over heads, of 2^(s log2e - lse log2e)
//
// the first product of the attention alone (k_attend.cu has its operands): 128 tokens of a 128-byte
// chunk of the record are the M of a kind::mxf8f6f4 MMA, the two e4m3 terms of the chunk's heads, times
// the rows of a pass, its N.  The queries of all chunks stay in shared memory over a run of tiles; a
// group of four softmax warps, a token per thread, takes a tile through all its chunks, so that a
// token's sum stays in one register, in a fixed order, with one writer.  The four groups work on four
// tiles at a time, whose chunks come in turn.  Requests with more rows than a pass holds are read once
// per pass.
// Measured: 8 rows over 8 contexts of 1K..32K tokens 27 us (71 MB; copy: 10 us), bound by HBM while
// tiles run; m16n8k16 MMAs on codes widened in registers took 50.
#include "attend_tc.cuh"

namespace mono {
namespace {

using namespace tc;
using namespace attend;

constexpr int SOFT_WARPS = 16, SOFT = SOFT_WARPS * 32, GROUPS = SOFT_WARPS / 4;
constexpr int S_WARP = SOFT_WARPS, S_WARPS = 2, LOAD_WARP = S_WARP + S_WARPS, LOAD_WARPS = 4;
constexpr int THREADS = 32 * (LOAD_WARP + LOAD_WARPS);
constexpr int ST = 6;                  // tiles in the ring
constexpr int NQ = 48;                 // query columns of a pass at most
constexpr int CHUNKS = 8;              // chunks of a record at most
constexpr int Q_BYTES = 96 * 1024;     // queries of a pass at most: [chunk] hi rows, then lo rows
constexpr int K_OFF = 0, Q_OFF = ST * K_TILE, QIMG_OFF = Q_OFF + Q_BYTES;
constexpr int ONE_OFF = QIMG_OFF + CHUNKS * IMG, SC_OFF = ONE_OFF + IMG;
constexpr int PLAN_OFF = SC_OFF + ST * TT * 16;
constexpr int SMEM_BYTES = PLAN_OFF + (3 * MAX_REQ + 4) * 4 + MAX_ROWS * 6 + MAX_REQ * 2 + 1024;
// TMEM: scores by slot (a group has two of 32 columns, or one of 96), scales (ones and the queries' of
// every chunk, for either issuing warp)
constexpr int S_COL = 0, SF_ONE = 384, SF_Q = SF_ONE + 4 * S_WARPS;
static_assert(SF_Q + 4 * CHUNKS * S_WARPS <= 512, "TMEM");

struct Args {
  CUtensorMap codes, scales;  // the cache as [pages][tokens][bytes], boxes of box tokens
  int box;                    // 0: no maps
  int pad, pass;              // columns of a row (of a chunk, padded to 16); rows of a pass
  AttendArgs a;
  Shape sh;
};

struct Rows {
  int nrows, row[GROUP], pos[GROUP];
};
struct Shared {
  uint64_t full[ST], k_free[ST], s_full[2 * GROUPS], s_free[2 * GROUPS], q_full, drain;
  alignas(16) float neg_lse[CHUNKS][NQ];  // log2; -infinity: padding
  uint32_t valid[ST][4];                  // tokens that are there
  Rows rows;
  uint32_t tmem;
  int abort;
  Jobs start;
};
static_assert(SMEM_BYTES + sizeof(Shared) <= 227 * 1024, "shared memory");

// The order of a pass over an item's n tiles: four at a time, a group each, all their chunks in turn
// (fewer tiles at the end).
struct Walk {
  int n, chunks, i, tile, chunk, width;
  __device__ Walk(int tiles, int c) : n(tiles), chunks(c), i(0), tile(0), chunk(0), width(min(GROUPS, tiles)) {}
  __device__ bool more() const { return i < n; }
  __device__ int at() const { return i + tile; }
  __device__ void next() {
    if (++tile < width) return;
    tile = 0;
    if (++chunk < chunks) return;
    chunk = 0;
    i += width;
    width = min(GROUPS, n - i);
  }
};

__global__ void __launch_bounds__(THREADS, 1) attend_weights_kernel(const __grid_constant__ Args ar) {
  const AttendArgs& a = ar.a;
  const Shape& sh = ar.sh;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + (-smem_u32(smem_raw) & 1023);  // (still a shared pointer to the compiler)
  __shared__ __align__(16) Shared ss;
  volatile int* abort = &ss.abort;
  Plan plan;
  plan.pre = reinterpret_cast<int*>(sm + PLAN_OFF);
  plan.pmax = plan.pre + MAX_REQ + 4;
  plan.pmin = plan.pmax + MAX_REQ;
  plan.pos = plan.pmin + MAX_REQ;
  plan.req = reinterpret_cast<short*>(plan.pos + MAX_ROWS);
  plan.cnt = plan.req + MAX_ROWS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunks = sh.chunks, cols = ar.pad * ar.pass, tail = a.kv_dim - 128 * (chunks - 1);
  const int lg = cols <= 16 ? 1 : 0;  // 2^lg slots of scores a group
  if (tid == 0) {
    // a tile is free when the product and a group's warps have read it, and the other issuing warp has
    // seen it
    for (int s = 0; s < ST; ++s) mbar_init(&ss.full[s], 1), mbar_init(&ss.k_free[s], S_WARPS + 4);
    for (int s = 0; s < 2 * GROUPS; ++s) mbar_init(&ss.s_full[s], 2), mbar_init(&ss.s_free[s], 4);
    mbar_init(&ss.q_full, SOFT_WARPS);
    mbar_init(&ss.drain, S_WARPS);
    ss.abort = 0;
    fence_mbar_init();
  }
  if (warp == S_WARP) tmem_alloc<512>(&ss.tmem);
  for (int i = tid; i < (CHUNKS + 1) * IMG / 4; i += THREADS)
    reinterpret_cast<uint32_t*>(sm + QIMG_OFF)[i] = 0x7F7F7F7Fu;
  fence_proxy_async_shared();
  derive_plan<THREADS>(a, sh, plan, blockIdx.x, true, &ss.start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ss.tmem;
  Jobs items = ss.start;
  Job im;
  auto passes = [&](const Job& j) { return (plan.cnt[j.b] + ar.pass - 1) / ar.pass; };

  if (warp >= LOAD_WARP) {
    // ---------------- loads: each slot of the ring has one loading warp (a wait by parity is for the
    // phase that is meant only where the waiter saw the one before)
    int it = 0;
    TileLoader tile(ar.box);
#pragma unroll 1
    while (next_job(a, sh, plan, items, im)) {
#pragma unroll 1
      for (int p = passes(im); p > 0; --p) {
#pragma unroll 1
        for (Walk w(im.n, chunks); w.more(); w.next(), ++it) {
          if (it % ST % LOAD_WARPS != warp - LOAD_WARP) continue;
          const int s = it % ST;
          tile.locate(a, im, w.at());
          bool go = true;
          if (it >= ST) go = wait(&ss.k_free[s], ((it / ST) - 1) & 1, a.status, abort);
          tile.load(a, im, ar.codes, ar.scales, w.chunk, sm + K_OFF + s * K_TILE, sm + SC_OFF + s * TT * 16,
                    ss.valid[s], &ss.full[s], go);
        }
      }
    }
  } else if (warp >= S_WARP) {
    // -------------------------------------------- the product's MMAs: a warp issues two groups' tiles
    const int mine = warp - S_WARP;
    const uint32_t ones = tmem + SF_ONE + 4 * mine, sf = tmem + SF_Q + 4 * CHUNKS * mine;
    const uint64_t k0 = desc_sw128(smem_u32(sm + K_OFF)), q0 = desc_sw128(smem_u32(sm + Q_OFF));
    const uint32_t idesc = IDESC | ((uint32_t)(2 * cols >> 3) << 17);
    uint32_t it = 0, pass = 0, used[2] = {0, 0};  // tiles of either group so far
    if (elect_one()) tc_cp_img(ones, sm + ONE_OFF);
    __syncwarp();
#pragma unroll 1
    while (next_job(a, sh, plan, items, im)) {
#pragma unroll 1
      for (int p = passes(im); p > 0; --p, ++pass) {
        wait(&ss.q_full, pass & 1, a.status, abort);
        bar_sync<32 * S_WARPS>(2);  // (neither runs ahead of the phase that the other waits for)
        if (elect_one()) {
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) tc_cp_img(sf + 4 * c, sm + QIMG_OFF + c * IMG);
        }
        __syncwarp();
#pragma unroll 1
        for (Walk w(im.n, chunks); w.more(); w.next(), ++it) {
          const int st = it % ST, hi = w.tile >> 1;
          // (the other warp's tiles too, and before they may go: a wait by parity is for the phase that
          // is meant only where the waiter saw the one before)
          bool ok = wait(&ss.full[st], (it / ST) & 1, a.status, abort);
          if ((w.tile & 1) != mine) {
            if (lane == 0) mbar_arrive(&ss.k_free[st]);
            continue;
          }
          const uint32_t k = hi ? used[1]++ : used[0]++;
          const int b = w.tile + (k & lg) * GROUPS;  // the group's slot
          if ((k >> lg) > 0) ok &= wait(&ss.s_free[b], ((k >> lg) - 1) & 1, a.status, abort);
          if (ok && elect_one()) {
            tc_fence_after();
            const uint64_t kd = k0 + st * (K_TILE / 16), qd = q0 + w.chunk * (2 * cols * 128 / 16);
            const uint32_t d = tmem + S_COL + b * (lg ? 32 : 96);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              tc_mma_mxf8(d, kd + 2 * e, qd + 2 * e, idesc | ((uint32_t)e << 4) | ((uint32_t)e << 29), ones,
                          sf + 4 * w.chunk, e > 0);
            tc_commit(&ss.s_full[b]);
            tc_commit(&ss.k_free[st]);
            mbar_arrive(&ss.s_full[b]);  // (see k_attend.cu)
          }
          __syncwarp();
        }
      }
    }
    if (elect_one()) tc_commit(&ss.drain);  // (what was issued has completed at this arrival)
    __syncwarp();
  } else {
    // ------------------------------------------------------------------------- queries, weights
    const int quad = warp & 3, group = warp >> 2, tok = 32 * quad + lane;
    const int hpg = a.n_q / (a.kv_dim / a.head_dim), dshift = a.head_dim == 64 ? 6 : 7;
    const float to_log2 = a.scale * LOG2E;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    Shape by_pass = sh;
    by_pass.rows_per = ar.pass;
    uint32_t it = 0, k = 0;  // the ring's next tile; this group's tiles so far
#pragma unroll 1
    while (next_job(a, sh, plan, items, im)) {
      const int np = passes(im);
#pragma unroll 1
      for (int p = 0; p < np; ++p) {
        bar_sync<SOFT>(1);  // the pass before has been read
        if (warp == 0) {
          const int n = group_rows(a, by_pass, plan, im.b, p, ss.rows.row, ss.rows.pos);
          if (lane == 0) ss.rows.nrows = n;
        }
        bar_sync<SOFT>(1);
        const int nrows = ss.rows.nrows;
        // queries as two e4m3 terms, rows of 128 bytes by chunk: hi in row c, lo in row cols + c
        const int d = (tid & 15) * 8, sl = d >> dshift, o = d >> 4;
#pragma unroll 1
        for (int x = tid >> 4; x < chunks * cols; x += SOFT / 16) {
          const int chunk = x / cols, c = x - chunk * cols, j = c / ar.pad, h = c - j * ar.pad;
          const int heads = hpg * ((chunk == chunks - 1 ? tail : 128) > a.head_dim ? 2 : 1);
          const bool in = j < nrows && h < heads;
          const int head = chunk * sh.heads + h;
          uint4 q = make_uint4(0, 0, 0, 0);
          if (in && (h >= hpg ? 1 : 0) == sl)
            q = __ldg(reinterpret_cast<const uint4*>(a.q + ss.rows.row[j] * a.q_stride +
                                                     (long long)head * a.head_dim + (d - (sl << dshift))));
          if (d == 0)
            ss.neg_lse[chunk][c] =
                in ? -LOG2E * a.lse[(long long)ss.rows.row[j] * a.n_q + head] : -INFINITY;
          uint2 hi, lo;
          const uint32_t code = split_query(q, hi, lo);
          uint8_t* at = sm + Q_OFF + chunk * (2 * cols * 128) + (d & 8);
          const int rl = cols + c;
          *reinterpret_cast<uint2*>(at + c * 128 + ((o ^ (c & 7)) << 4)) = hi;
          *reinterpret_cast<uint2*>(at + rl * 128 + ((o ^ (rl & 7)) << 4)) = lo;
          if ((d & 31) == 0) {
            uint8_t* img = sm + QIMG_OFF + chunk * IMG + (d >> 5);
            img[(c & 31) * 16 + (c >> 5) * 4] = (uint8_t)code;
            img[(rl & 31) * 16 + (rl >> 5) * 4] = (uint8_t)code;
          }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.q_full);
        bar_sync<SOFT>(1);  // (neg_lse)
        const Clear clear = clear_tiles(a, im, ss.rows);
#pragma unroll 1
        for (int i = group; i < im.n; i += GROUPS) {
          const int width = min(GROUPS, im.n - i + group), t = im.span.token(im.t0 + i) + tok;
          float ct = 0.0f, sum = 0.0f, old = 0.0f;
          uint32_t see = 0;  // rows of the pass that see the token
          bool there = false;
#pragma unroll 1
          for (int chunk = 0; chunk < chunks; ++chunk, ++k) {
            const uint32_t at = it + chunk * width + group, st = at % ST;
            const int b = group + (k & lg) * GROUPS;
            wait(&ss.s_full[b], (k >> lg) & 1, a.status, abort);  // (and the tile's scales)
            if (chunk == 0) {
              const float raw = reinterpret_cast<const float*>(sm + SC_OFF)[(st * TT + tok) * 4];
              const uint32_t ok = ss.valid[st][quad];
              ct = fabsf(raw) <= SCALE_MAX ? raw * to_log2 : __int_as_float(0x7FC00000);
              there = (ok >> lane) & 1;
              see = there ? (1u << nrows) - 1 : 0u;  // (no padding columns: a NaN score would count)
              if (__builtin_expect(!clear.has(i), 0)) {
#pragma unroll 1
                for (int j = 0; j < nrows; ++j) {
                  const int hi = a.causal ? ss.rows.pos[j] : im.span.hi;
                  const int lo = a.window > 0 ? max(0, hi - a.window + 1) : 0;
                  if (!(t <= hi && (t >= lo || t < a.sinks))) see &= ~(1u << j);
                }
              }
              there = there && t < a.weights_cols;
              if (there) old = a.weights[im.b * a.weights_stride + t];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ss.k_free[st]);
            const uint32_t scol = lanes + S_COL + b * (lg ? 32 : 96);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < cols; c += 16) {
              float s[16], x[16];
#pragma unroll
              for (int g = 0; g < 16; g += 8) tc_ld8(scol + c + g, s + g), tc_ld8(scol + cols + c + g, x + g);
              tc_wait_ld();
              tc_loaded(s), tc_loaded(s + 8), tc_loaded(x), tc_loaded(x + 8);
              const float4* nl = reinterpret_cast<const float4*>(&ss.neg_lse[chunk][c]);
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 m = nl[e / 4];
                add2(s[e], s[e + 1], x[e], x[e + 1]);
                add2(s[e + 2], s[e + 3], x[e + 2], x[e + 3]);
                fma2(s[e], s[e + 1], ct, m.x, m.y);
                fma2(s[e + 2], s[e + 3], ct, m.z, m.w);
              }
              float u = 0.0f, v = 0.0f;
#pragma unroll
              for (int e = 0; e < 16; e += 2) add2(u, v, ex2(s[e]), ex2(s[e + 1]));
              if ((see >> (c / ar.pad)) & 1) sum += u + v;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ss.s_free[b]);
          }
          if (there) a.weights[im.b * a.weights_stride + t] = old + sum;
          it += chunks * width;
        }
        // (a last row of fewer tiles that this group had no part in)
        if (im.n % GROUPS && im.n % GROUPS <= group) it += chunks * (im.n % GROUPS);
      }
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

cudaError_t attend_weights_prepare() {
  return cudaFuncSetAttribute(attend_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
}

cudaError_t launch_attend_weights(const Launch& L, const AttendArgs& a, int sms) {
  Args ar = {{}, {}, 0, 0, 0, a, shape_of(a, TT, NQ, sms, 4)};
  ar.sh.rows_per = MAX_ROWS;  // a unit is a tile with all its request's rows
  ar.pad = (ar.sh.heads + 15) & ~15;
  // rows of a pass: as many as requests have on average, while columns and queries fit
  const int row_bytes = ar.sh.chunks * 2 * ar.pad * 128;
  ar.pass = std::min({(a.rows + a.n_req - 1) / a.n_req, NQ / ar.pad, Q_BYTES / row_bytes, GROUP});
  ar.box = encode_cache_maps(&ar.codes, &ar.scales, a);
  return launch_ex(L, dim3(sms), dim3(THREADS), SMEM_BYTES, attend_weights_kernel, ar);
}

}  // namespace mono
