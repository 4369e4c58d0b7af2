// Attention of a batch whose requests share prefixes, on the 5th-generation tensor cores: a prefix is
// read once for the rows of all its requests, every request's own tokens for its rows.
//
//   S[q, t] = codes_t . q        (query q = one head of one row, token t)
//   P[q, t] = 2^(a_t S - m_q) scale_t,  a_t = scale scale_t log2e     O[q, :] = sum_t P[q, t] codes_t
//
// Queries are the M of both products, 128 of them a block: the heads that read a latent slice, times as
// many rows as fit.  Tokens are the N of the first product, 128 a tile, and its K operand is the V
// operand of the second: the tile is widened from e4m3 to f16 (exact) once, and serves both.  A query
// is f16 too, off by at most 2^-24 of its largest element (those out of f16's reach are scaled by a
// power of two).  P is f16 (11 bits; the one rounding between scores and o) under m_q, an integer that
// follows the weights times scales, so that the largest of the tile that set it is in (2^5, 2^6], and
// moves when one passes 2^15; O is rescaled then, exactly.  P takes its scores' place in TMEM.
//
// Work: groups (a prefix with its requests' rows; a request's own tokens with its rows), slices and
// pairs of blocks make items; the tiles of all items lie in one line, cut evenly over the CTAs, every
// CTA deriving the cut for itself.  A CTA has two streams of softmax: those of the two blocks of a pair
// over the same tiles, or of one block over every other tile.  What a CTA has of an item leaves (O, m, l)
// in the workspace; a second kernel joins them.
//
// Roles: warps 0-3 and 4-7 softmax, a query per thread; 8-11 widen tiles; 12 issues MMAs; 13 loads; 14
// makes the items' rows; 15 tells the join where pieces are.
// Every mbarrier wait is bounded; a wait that runs out is reported, and from then on every role runs its
// loop without waiting, copying or issuing.
#include "attend_tc.cuh"

namespace mono {
namespace {

using namespace tc;
using namespace attend;

constexpr int THREADS = 512, SOFT = 256;
constexpr int WIDEN_WARP = 8, MMA_WARP = 12, LOAD_WARP = 13, ROWS_WARP = 14;
constexpr int MAX_GROUPS = MAX_PREFIX + MAX_REQ;
constexpr int BLOCK = 128;       // queries
constexpr int EXTRA = 3;         // what an item costs a CTA beside its steps, in steps
constexpr int HALF = TT * 128;   // bytes of 64 dimensions of a tile, or a block, in f16
constexpr float BASE = 6.0f, LEAST = -90.0f;  // log2 of the weights times scales that m puts at most; scales below
constexpr uint32_t TOO_LARGE = 0x7800;        // f16 of 2^15
// registers a thread at launch, and as the roles divide them
constexpr int REGS = 128, SOFT_REGS = 192, OTHER_REGS = 64;
static_assert(SOFT_REGS * SOFT + OTHER_REGS * (THREADS - SOFT) == REGS * THREADS, "register split");

template <int DH>
struct Form {
  static constexpr int WIDE = DH / 64 * HALF, NARROW = TT * DH;  // a tile in f16, in e4m3
  static constexpr int NS = DH == 128 ? 3 : 5, ST = DH == 128 ? 2 : 4;  // rings of wide and narrow tiles
  static constexpr int Q_OFF = 0, V_OFF = Q_OFF + 2 * WIDE, K_OFF = V_OFF + NS * WIDE;
  static constexpr int SC_OFF = K_OFF + ST * NARROW;      // the 16 bytes behind the codes [ST][TT]
  static constexpr int TOK_OFF = SC_OFF + ST * TT * 16;   // a_t, scale_t, log2 scale_t [NS][3][TT]
  static constexpr int PLAN_OFF = TOK_OFF + NS * 3 * TT * 4;
  static constexpr int PLAN_BYTES = MAX_GROUPS * (4 + 4 + 4 + 2) + 16 + MAX_ROWS * 6 + MAX_REQ * 2;
  static constexpr int SMEM_BYTES = PLAN_OFF + PLAN_BYTES + 1024;
  static constexpr int O_COL = 256;  // TMEM: scores (and weights) of stream u at 128 u, its O at O_COL + DH u
};

struct Args {
  CUtensorMap codes, scales;
  int box;  // 0: no maps
  int slices, hps, rows_per;  // latent slices, heads of one, rows of a block
  SharedArgs a;
  float* home;   // pieces: [2][max_rows][n_q], of those that begin an item; prefixes', then own tokens'
  float* over;   // [CTAs][2 * BLOCK], of a CTA's item that began before it
  int* info;     // [rows][8]
  int max_rows;
};

// The step as every CTA derives it.  Groups: prefixes, then requests.
struct Plan {
  int* pre;    // [groups + 1] the line's steps of all groups before
  int* end;    // [groups] one behind the last token that a row sees
  int* first;  // [groups] the first
  short* cnt;  // [groups] rows
  int* hi;     // [rows] a row's last token
  short* req;  // [rows] its request; -1: nothing to see
  short* pfx;  // [n_req] its prefix; -1: none, -2: bad
};

struct Item {  // of a group: a slice, and a pair of blocks (or the last one)
  int g, slice, pair;
};
struct Shape2 {  // of a group's items
  int tiles, blocks, whole, half;  // a pair's and a single block's lengths in the line
  __device__ int slice_len() const { return (blocks >> 1) * whole + (blocks & 1) * half; }
  __device__ bool pairs(int pair) const { return 2 * pair + 1 < blocks; }
  __device__ int len(int pair) const { return pairs(pair) ? whole : half; }
};
__device__ __forceinline__ Shape2 shape_of_group(const Args& ar, const Plan& p, int g) {
  Shape2 s = {0, 0, 0, 0};
  const int n = p.cnt[g], lo = p.first[g], end = p.end[g];
  if (n == 0 || end <= lo) return s;
  s.tiles = ((end - 1) >> 7) - (lo >> 7) + 1;
  s.blocks = (n + ar.rows_per - 1) / ar.rows_per;
  s.whole = EXTRA + s.tiles;
  s.half = EXTRA + (s.tiles + 1) / 2;
  return s;
}

// A CTA's part of an item: steps [s0, s1), of one tile for both streams or of two.
struct Job {
  Item at;
  bool pairs;
  int tile0, tiles, s0, n[2];  // the group's first tile and number; first step; the streams' tiles
  __device__ int count() const { return pairs ? n[0] : n[0] + n[1]; }
  // the i-th tile of the ring, and which it is for stream u's j-th
  __device__ int token(int i) const { return (tile0 + (pairs ? s0 + i : 2 * s0 + i)) * TT; }
  __device__ int ring(int u, int j) const { return pairs ? j : 2 * j + u; }
};
struct Cursor {
  Item at;
  int unit, left;
};
__device__ __forceinline__ bool next_job(const Args& ar, const Plan& p, Cursor& c, Job& job) {
  const int groups = ar.a.n_prefix + ar.a.n_req;
#pragma unroll 1
  while (c.left > 0) {
    const Shape2 s = shape_of_group(ar, p, c.at.g);
    const int len = s.len(c.at.pair), n = min(len - c.unit, c.left);
    job.at = c.at;
    job.pairs = s.pairs(c.at.pair);
    job.tile0 = p.first[c.at.g] >> 7;
    job.tiles = s.tiles;
    job.s0 = max(0, c.unit - EXTRA);
    const int s1 = c.unit + n - EXTRA;
    job.n[0] = s1 - job.s0;
    job.n[1] = job.pairs ? job.n[0] : min(2 * s1, s.tiles) - 2 * job.s0 - job.n[0];
    c.left -= n;
    c.unit = 0;
    if (++c.at.pair >= (s.blocks + 1) >> 1) {
      c.at.pair = 0;
      if (++c.at.slice >= ar.slices) {
        c.at.slice = 0;
        do ++c.at.g;
        while (c.at.g < groups && p.pre[c.at.g + 1] <= p.pre[c.at.g]);
      }
    }
    if (job.n[0] > 0) return true;
  }
  return false;
}

struct Shared {
  uint64_t full[4], k_free[4], v_full[5], v_free[5];
  uint64_t s_full[2], p_full[2], o_full[2], q_full[2], m_full[2], m_free[2], drain;
  uint32_t valid[4][4];                // tokens that are there, of a narrow tile
  alignas(16) uint32_t see[5][4];      // and of a wide one
  int part[5];                         // not every row of the item sees all its tokens
  short row[2][2 * BLOCK];             // an item's rows (-1: none), its blocks' one after another
  int least[2];                        // the smallest of their last tokens
  float2 ml[2][BLOCK];
  uint32_t tmem;
  int abort;
  Cursor start;
};
static_assert(Form<128>::SMEM_BYTES + sizeof(Shared) <= 227 * 1024, "shared memory");
static_assert(Form<64>::SMEM_BYTES + sizeof(Shared) <= 227 * 1024, "shared memory");

// x a + b, two tokens of a query
__device__ __forceinline__ void fma2t(float& x, float& y, float ax, float ay, float b) {
  asm("{\n .reg .b64 s, m, b;\n mov.b64 s, {%0, %1};\n mov.b64 m, {%2, %3};\n mov.b64 b, {%4, %4};\n"
      " fma.rn.f32x2 s, s, m, b;\n mov.b64 {%0, %1}, s;\n}"
      : "+f"(x), "+f"(y)
      : "f"(ax), "f"(ay), "f"(b));
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void loaded32(uint32_t (&r)[32]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
               "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
  asm volatile("" : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
               "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
               "+r"(r[31]));
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// f16 x f16, f32 accumulators; A in shared memory, or in TMEM
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Matrix descriptor as desc_sw128, MN-major with `lbo` bytes between 128-byte runs along MN.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lbo) {
  return (desc_sw128(saddr) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(lbo >> 4) << 16);
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Fills the plan (every thread of the block) and finds the CTA's first item; the results are behind the
// caller's next barrier.  Waits for the kernels before.
__device__ __forceinline__ void derive_plan(const Args& ar, const Plan& plan, Cursor* start) {
  const SharedArgs& a = ar.a;
  const int tid = threadIdx.x, lane = tid & 31, np = a.n_prefix, groups = np + a.n_req;
  const bool tell = blockIdx.x == 0;
  const int cap = a.kv.max_blocks * a.kv.block_size, pcap = a.pre.max_blocks * a.kv.block_size;  // (fit 31 bits)
#pragma unroll 1
  for (int g = tid; g < groups; g += THREADS) plan.end[g] = 0, plan.cnt[g] = 0, plan.first[g] = 0;
  pdl_trigger();
  pdl_wait();
#pragma unroll 1
  for (int b = tid; b < a.n_req; b += THREADS) {
    int g = a.prefix_of ? a.prefix_of[b] : 0;
    if (g < -1 || g >= np) g = -2;
    plan.pfx[b] = (short)g;
  }
  __syncthreads();
#pragma unroll 1
  for (int b = tid; b < a.n_req; b += THREADS) {
    const int g = plan.pfx[b];
    plan.first[np + b] = g >= 0 ? max(0, a.prefix_lengths[g]) : 0;
  }
  // a request's rows and their largest position
#pragma unroll 1
  for (int r = tid; r < a.rows; r += THREADS) {
    const int p = min(a.positions[r], 0x7FFFFFFE), b = a.row_req[r];
    const bool in = b >= 0 && b < a.n_req, live = p >= 0 && in && plan.pfx[b] >= -1;
    if (p >= 0 && !live && tell) atomicOr(a.status, ST_UNMAPPED_PAGE);
    plan.req[r] = (short)(live ? b : -1);
    plan.hi[r] = live ? p : -1;
    if (live) atomicMax(&plan.end[np + b], p + 1);
  }
  __syncthreads();
#pragma unroll 1
  for (int r = tid; r < a.rows; r += THREADS) {
    const int b = plan.req[r];
    if (b < 0) continue;
    const int hi = a.causal ? plan.hi[r] : plan.end[np + b] - 1, g = plan.pfx[b], len = plan.first[np + b];
    plan.hi[r] = hi;
    // (16-bit counters: the words that hold them)
    auto count = [&](int k) { atomicAdd(reinterpret_cast<int*>(plan.cnt) + (k >> 1), k & 1 ? 1 << 16 : 1); };
    count(np + b);
    if (g >= 0) {
      count(g);
      atomicMax(&plan.end[g], min(min(hi + 1, len), pcap));
      if (min(hi + 1, len) > pcap && tell) atomicOr(a.status, ST_UNMAPPED_PAGE);
    }
    if (hi >= cap && hi >= len && tell) atomicOr(a.status, ST_UNMAPPED_PAGE);
  }
  __syncthreads();
  if (tid < 32) {
    int W = 0;
#pragma unroll 1
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const int g = g0 + lane;
      int u = 0;
      if (g < groups) {
        if (g >= np) plan.end[g] = min(plan.end[g], cap);
        u = shape_of_group(ar, plan, g).slice_len() * ar.slices;
      }
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, u, o);
        if (lane >= o) u += y;
      }
      if (g < groups) plan.pre[g + 1] = W + u;
      W += __shfl_sync(0xffffffffu, u, 31);
    }
    __syncwarp();
    if (lane == 0) {
      plan.pre[0] = 0;
      const Cut cut(W, gridDim.x);
      Cursor c = {{0, 0, 0}, 0, cut.size(blockIdx.x)};
      if (c.left > 0) {
        const int w0 = cut.start(blockIdx.x);
        int lo = 0, hi = groups;  // the last group that starts by w0 (and is not empty: the next starts later)
#pragma unroll 1
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (plan.pre[mid] <= w0) lo = mid; else hi = mid;
        }
        const Shape2 s = shape_of_group(ar, plan, lo);
        int u = w0 - (lo ? plan.pre[lo] : 0);
        c.at.g = lo;
        c.at.slice = u / s.slice_len();
        u -= c.at.slice * s.slice_len();
        c.at.pair = min(u / s.whole, s.blocks >> 1);
        c.unit = u - c.at.pair * s.whole;
      }
      *start = c;
    }
  }
}

// The rows of an item's blocks into `rows`, in row order, by a whole warp; returns the smallest of their
// last tokens.
__device__ __forceinline__ int item_rows(const Args& ar, const Plan& plan, const Job& job, short* rows) {
  const int lane = threadIdx.x & 31, np = ar.a.n_prefix, g = job.at.g;
  const int first = 2 * job.at.pair * ar.rows_per, most = (job.pairs ? 2 : 1) * ar.rows_per;
#pragma unroll 1
  for (int i = lane; i < 2 * BLOCK; i += 32) rows[i] = -1;
  __syncwarp();
  int seen = 0, least = 0x7FFFFFFF;
#pragma unroll 1
  for (int r0 = 0; r0 < ar.a.rows && seen - first < most; r0 += 32) {
    const int r = r0 + lane, b = r < ar.a.rows ? plan.req[r] : -1;
    const bool in = b >= 0 && (g < np ? plan.pfx[b] == g : b == g - np);
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    const int rank = seen + __popc(m & ((1u << lane) - 1)) - first;
    if (in && rank >= 0 && rank < most) {
      rows[rank < ar.rows_per ? rank : BLOCK + rank - ar.rows_per] = (short)r;
      least = min(least, plan.hi[r]);
    }
    seen += __popc(m);
  }
  return __reduce_min_sync(0xffffffffu, least);
}

// Loads narrow tiles, a warp: TMA boxes through the page table, or cp.async where there are no maps.
// A lane per box of the tile (of a token each without maps, four times), looked up ahead of the load.
template <int DH>
struct Loader {
  int box, shift, boxes, t0, lo, end;
  int page[4], row[4];
  __device__ explicit Loader(int b) {
    box = b ? b : 1;
    shift = __ffs(box) - 1;
    boxes = TT >> shift;
  }
  __device__ __forceinline__ void locate(const Args& ar, const Plan& plan, const Job& job, int i) {
    const int lane = threadIdx.x & 31, np = ar.a.n_prefix, g = job.at.g, bs = ar.a.kv.block_size;
    const PagedView& v = g < np ? ar.a.pre : ar.a.kv;
    const int* table = v.table + (size_t)(g < np ? g : g - np) * v.max_blocks;
    t0 = job.token(i);
    lo = plan.first[g];
    end = plan.end[g];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (32 * q >= boxes) break;
      const int t = t0 + ((32 * q + lane) << shift), lb = t / bs;
      page[q] = row[q] = -1;
      if (32 * q + lane < boxes && t < end && t + box > lo) {
        row[q] = t - lb * bs;
        if (lb < v.max_blocks) page[q] = __ldg(table + lb);
      }
    }
  }
  __device__ __forceinline__ void load(const Args& ar, int slice, uint8_t* st, uint8_t* sc, uint32_t* valid,
                                       uint64_t* full, bool go) {
    const SharedArgs& a = ar.a;
    const int lane = threadIdx.x & 31;
    if (box > 1) {
      const bool m = page[0] >= 0 && page[0] < a.kv.num_blocks;
      if (row[0] >= 0 && !m) atomicOr(a.status, ST_UNMAPPED_PAGE);
      if (m && go) {
        tma_load_3d(st + ((lane * DH) << shift), &ar.codes, DH * slice, row[0], page[0], full);
        tma_load_3d(sc + ((lane * 16) << shift), &ar.scales, a.kv_dim, row[0], page[0], full);
      }
      const uint32_t have = __ballot_sync(0xffffffffu, m);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int t = t0 + 32 * q + lane;
        const bool see = ((have >> ((32 * q + lane) >> shift)) & 1) && t >= lo && t < end;
        const uint32_t w = __ballot_sync(0xffffffffu, see);
        if (lane == q) valid[q] = w;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(full, go ? __popc(have) * box * (DH + 16) : 0);
      __syncwarp();
    } else {
      constexpr int PIECES = DH / 16, ROWS = 32 / PIECES;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const int pg = q == 0 ? page[0] : q == 1 ? page[1] : q == 2 ? page[2] : page[3];
        const int rw = q == 0 ? row[0] : q == 1 ? row[1] : q == 2 ? row[2] : row[3];
        const bool m = pg >= 0 && pg < a.kv.num_blocks;
        if (rw >= 0 && !m) atomicOr(a.status, ST_UNMAPPED_PAGE);
        const long long off = m ? pg * a.kv.stride_block + rw * a.kv.stride_tok : 0;
        const uint32_t w = __ballot_sync(0xffffffffu, m);
        if (lane == 0) valid[q] = w;
#pragma unroll 1
        for (int e = 0; e < 32 / ROWS; ++e) {
          const int k = ROWS * e + lane / PIECES, piece = lane & (PIECES - 1);
          const long long ro = __shfl_sync(0xffffffffu, off, k);
          if (go && ((w >> k) & 1))
            cp_async16(st + (32 * q + k) * DH + 16 * piece, a.kv.base + ro + DH * slice + 16 * piece, 16);
        }
        if (go && m) cp_async16(sc + (32 * q + lane) * 16, a.kv.base + off + a.kv_dim, 16);
      }
      cp_async_wait_all();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
  }
};

// What a softmax thread knows of its item and query.
struct Soft {
  uint32_t s_at, o_at;  // TMEM: the stream's scores and O, with the warp's lane quadrant
  int hi;               // the row's last token
  float factor;         // of the scores
  bool scaled;          // some of the warp's factors are not 1
  float m, l;
};

// The largest weight times scale (log2) of the thread's query in a tile.
template <bool PART>
__device__ __forceinline__ float tile_max(const Soft& w, const float* tok, const uint32_t* see, int t0) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t s[32];
    tc_ld32(w.s_at + 32 * c, s);
    uint32_t sees = 0xffffffffu;
    if (PART) {
      const int n = w.hi - (t0 + 32 * c) + 1;
      sees = see[c] & (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1);
    }
    tc_wait_ld();
    loaded32(s);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      float x = fmaf(__uint_as_float(s[e]) * w.factor, tok[32 * c + e], tok[2 * TT + 32 * c + e]);
      if (PART && !((sees >> e) & 1)) x = -INFINITY;
      top = fmaxf(top, x);
    }
  }
  return top;
}

// The tile's weights times scales as packed f16, their sum (without scales), and the largest pair.
template <bool PART>
__device__ __forceinline__ void tile_weights(const Soft& w, const float* tok, const uint32_t* see, int t0,
                                             uint32_t (&p)[64], float& l0, float& l1, uint32_t& top) {
  uint32_t s[2][32];
  tc_ld32(w.s_at, s[0]);
  l0 = l1 = 0.0f;
  top = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    tc_wait_ld();
    loaded32(s[c & 1]);
    if (c < 3) tc_ld32(w.s_at + 32 * (c + 1), s[(c + 1) & 1]);
    float* x = reinterpret_cast<float*>(s[c & 1]);
    if (w.scaled) {
#pragma unroll
      for (int e = 0; e < 32; e += 2) mul2(x[e], x[e + 1], w.factor);
    }
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const float4 a = *reinterpret_cast<const float4*>(tok + 32 * c + e);
      fma2t(x[e], x[e + 1], a.x, a.y, -w.m);
      fma2t(x[e + 2], x[e + 3], a.z, a.w, -w.m);
    }
    if (PART) {
      const int n = w.hi - (t0 + 32 * c) + 1;
      const uint32_t sees = see[c] & (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (!((sees >> e) & 1)) x[e] = -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const float4 sc = *reinterpret_cast<const float4*>(tok + TT + 32 * c + e);
      float p0 = ex2(x[e]), p1 = ex2(x[e + 1]), p2 = ex2(x[e + 2]), p3 = ex2(x[e + 3]);
      add2(l0, l1, p0, p1);
      add2(l0, l1, p2, p3);
      mul2(p0, p1, sc.x, sc.y);
      mul2(p2, p3, sc.z, sc.w);
      p[16 * c + e / 2] = f16x2_of(p0, p1);
      p[16 * c + e / 2 + 1] = f16x2_of(p2, p3);
      top = max_u16x2(top, max_u16x2(p[16 * c + e / 2], p[16 * c + e / 2 + 1]));
    }
  }
}

// Moves the query's reference to the tile's weights, and what was summed under the old one with it.
template <int DH, bool PART>
__device__ __forceinline__ void move_reference(Soft& w, const float* tok, const uint32_t* see, int t0, bool first) {
  const float top = tile_max<PART>(w, tok, see, t0);
  float f = 1.0f;
  if (top - w.m > BASE) {
    const float now = fabsf(top) <= SCORE_MAX ? ceilf(top) - BASE : __int_as_float(0x7FC00000);
    f = w.m == UNSET ? 0.0f : ex2(w.m - now);
    w.m = now;
  }
  if (first) return;
  w.l *= f;
#pragma unroll 1
  for (int c = 0; c < DH; c += 32) {
    uint32_t o[32];
    tc_ld32(w.o_at + c, o);
    tc_wait_ld();
    loaded32(o);
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
    st32(w.o_at + c, o);
  }
  tc_wait_st();
}

template <int DH>
__global__ void __maxnreg__(REGS) attend_shared_kernel(const __grid_constant__ Args ar) {
  using F = Form<DH>;
  constexpr int NS = F::NS, ST = F::ST;
  const SharedArgs& a = ar.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + (-smem_u32(smem_raw) & 1023);
  __shared__ __align__(16) Shared ss;
  volatile int* abort = &ss.abort;
  Plan plan;
  plan.pre = reinterpret_cast<int*>(sm + F::PLAN_OFF);
  plan.end = plan.pre + MAX_GROUPS + 4;
  plan.first = plan.end + MAX_GROUPS;
  plan.hi = plan.first + MAX_GROUPS;
  plan.cnt = reinterpret_cast<short*>(plan.hi + MAX_ROWS);
  plan.req = plan.cnt + MAX_GROUPS;
  plan.pfx = plan.req + MAX_ROWS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&ss.full[s], 1), mbar_init(&ss.k_free[s], 4);
    for (int s = 0; s < NS; ++s) mbar_init(&ss.v_full[s], 4), mbar_init(&ss.v_free[s], 1);
    for (int u = 0; u < 2; ++u) {
      mbar_init(&ss.s_full[u], 2), mbar_init(&ss.p_full[u], 4), mbar_init(&ss.o_full[u], 1);
      mbar_init(&ss.q_full[u], 4), mbar_init(&ss.m_full[u], 1), mbar_init(&ss.m_free[u], 12);
    }
    mbar_init(&ss.drain, 1);
    ss.abort = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) tmem_alloc<512>(&ss.tmem);
  derive_plan(ar, plan, &ss.start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ss.tmem;
  Cursor cur = ss.start;
  Job job;

  if (warp >= WIDEN_WARP) {
    regs_down<OTHER_REGS>();
    if (warp < MMA_WARP) {
      // -------------------------------------------- tiles from e4m3 to f16, 32 tokens a warp
      constexpr int PIECES = DH / 16, ROWS = 32 / PIECES;  // of 16 codes; rows at a time
      const int q = warp - WIDEN_WARP, piece = lane & (PIECES - 1), r0 = lane / PIECES;
      const float to_log2 = a.scale * LOG2E;
      int it = 0;
#pragma unroll 1
      for (int item = 0; next_job(ar, plan, cur, job); ++item) {
        wait(&ss.m_full[item & 1], (item >> 1) & 1, a.status, abort);
        const int least = ss.least[item & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.m_free[item & 1]);
        const int n = job.count();
#pragma unroll 1
        for (int i = 0; i < n; ++i, ++it) {
          const int st = it % ST, s = it % NS;
          wait(&ss.full[st], (it / ST) & 1, a.status, abort);
          if (it >= NS) wait(&ss.v_free[s], (it / NS - 1) & 1, a.status, abort);
          const uint32_t ok = ss.valid[st][q];
          const bool late = least < job.token(i) + TT - 1;  // some row does not see the last token
          const bool part = late || (ss.valid[st][0] & ss.valid[st][1] & ss.valid[st][2] & ss.valid[st][3]) != 0xffffffffu;
          const uint8_t* src = sm + F::K_OFF + st * F::NARROW + 32 * q * DH;
          uint8_t* dst = sm + F::V_OFF + s * F::WIDE + 32 * q * 128 + (piece >> 2) * HALF;
          uint32_t nan = 0;  // tokens with NaN codes
#pragma unroll
          for (int h = 0; h < 32; h += 4 * ROWS) {
            uint4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = lds128(src + (h + e * ROWS) * DH + lane * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // a NaN code that some row must not see would reach it as 0 * NaN: it is a 0 here, and the
              // token's factor is NaN
              if (__builtin_expect(part, 0)) {
                const uint4 c = without_nan(v[e]);
                const uint32_t bad =
                    __ballot_sync(0xffffffffu, c.x != v[e].x || c.y != v[e].y || c.z != v[e].z || c.w != v[e].w);
#pragma unroll 1
                for (int k = 0; k < ROWS; ++k)
                  if ((bad >> (k * PIECES)) & ((1u << PIECES) - 1)) nan |= 1u << (h + e * ROWS + k);
                v[e] = c;
              }
              const int row = h + e * ROWS + r0, c = 2 * (piece & 3);
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
          {  // a token per lane
            const float raw = *reinterpret_cast<const float*>(sm + F::SC_OFF + (st * TT + 32 * q + lane) * 16);
            const bool fin = ((ok >> lane) & 1) && fabsf(raw) <= SCALE_MAX;
            const float sc = fin ? raw : 0.0f;
            float* tok = reinterpret_cast<float*>(sm + F::TOK_OFF) + s * 3 * TT + 32 * q + lane;
            tok[0] = fin && !((nan >> lane) & 1) ? raw * to_log2 : __int_as_float(0x7FC00000);
            tok[TT] = sc;
            tok[2 * TT] = sc != 0.0f ? fmaxf(log2_of(fabsf(sc)), LEAST) : LEAST;
            if (lane == 0) ss.see[s][q] = ok;
            if (q == 0 && lane == 0) ss.part[s] = part;
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ss.v_full[s]), mbar_arrive(&ss.k_free[st]);
        }
      }
    } else if (warp == MMA_WARP) {
      // ------------------------------------------------------------------------------- MMAs
      constexpr uint32_t IS = (1u << 4) | ((uint32_t)(TT >> 3) << 17) | ((uint32_t)(BLOCK >> 4) << 24);
      constexpr uint32_t IO = (1u << 4) | (1u << 16) | ((uint32_t)(DH >> 3) << 17) | ((uint32_t)(BLOCK >> 4) << 24);
      const uint64_t q0 = desc_sw128(smem_u32(sm + F::Q_OFF)), k0 = desc_sw128(smem_u32(sm + F::V_OFF)),
                     v0 = desc_mn(smem_u32(sm + F::V_OFF), HALF);
      int it = 0;              // the ring's tiles of the items before
      uint32_t pc[2] = {0, 0};  // the streams' tiles so far
      auto scores = [&](int u, int j) {
        const int i = it + job.ring(u, j), s = i % NS;
        bool ok = wait(&ss.v_full[s], (i / NS) & 1, a.status, abort);
        if (ok && elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < DH / 16; ++k)
            mma_ss(tmem + 128 * u, q0 + u * (F::WIDE / 16) + (k >> 2) * (HALF / 16) + 2 * (k & 3),
                   k0 + s * (F::WIDE / 16) + (k >> 2) * (HALF / 16) + 2 * (k & 3), IS, k > 0);
          tc_commit(&ss.s_full[u]);
          // (the commit is no release: this arrival passes on what the widening warps wrote)
          mbar_arrive(&ss.s_full[u]);
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int item = 0; next_job(ar, plan, cur, job); ++item) {
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          wait(&ss.q_full[u], item & 1, a.status, abort);
          if ((u ? job.n[1] : job.n[0]) > 0) scores(u, 0);
          else if (lane == 0) mbar_arrive(&ss.o_full[u]);
          __syncwarp();
        }
#pragma unroll 1
        for (int j = 0; j < job.n[0]; ++j) {
#pragma unroll 1
          for (int u = 0; u < 2; ++u) {
            const int n = u ? job.n[1] : job.n[0];
            if (j >= n) break;
            const int s = (it + job.ring(u, j)) % NS;
            const bool ok = wait(&ss.p_full[u], (u ? pc[1] : pc[0]) & 1, a.status, abort);
            if (u) ++pc[1]; else ++pc[0];
            if (ok && elect_one()) {
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < TT / 16; ++k)
                mma_ts(tmem + F::O_COL + DH * u, tmem + 128 * u + 8 * k, v0 + s * (F::WIDE / 16) + k * (2048 / 16), IO,
                       j > 0 || k > 0);
              if (!job.pairs || u == 1) tc_commit(&ss.v_free[s]);
              if (j + 1 == n) tc_commit(&ss.o_full[u]);
            }
            __syncwarp();
            if (j + 1 < n) scores(u, j + 1);
          }
        }
        it += job.count();
      }
      if (elect_one()) tc_commit(&ss.drain);
      __syncwarp();
    } else if (warp == LOAD_WARP) {
      // ------------------------------------------------------------------------------ loads
      Loader<DH> tile(ar.box);
      int it = 0;
      bool more = next_job(ar, plan, cur, job);
      int i = 0, n = more ? job.count() : 0;
      if (more) tile.locate(ar, plan, job, 0);
#pragma unroll 1
      while (more) {
        const int st = it % ST;
        bool go = true;
        if (it >= ST) go = wait(&ss.k_free[st], (it / ST - 1) & 1, a.status, abort);
        tile.load(ar, job.at.slice, sm + F::K_OFF + st * F::NARROW, sm + F::SC_OFF + st * TT * 16, ss.valid[st],
                  &ss.full[st], go);
        ++it;
        if (++i == n) {
          more = next_job(ar, plan, cur, job);
          i = 0;
          n = more ? job.count() : 0;
        }
        if (more) tile.locate(ar, plan, job, i);
      }
    } else if (warp == ROWS_WARP) {
      // ------------------------------------------------------------------- the items' rows
#pragma unroll 1
      for (int item = 0; next_job(ar, plan, cur, job); ++item) {
        const int b = item & 1;
        if (item >= 2) wait(&ss.m_free[b], ((item >> 1) - 1) & 1, a.status, abort);
        const int least = item_rows(ar, plan, job, ss.row[b]);
        if (lane == 0) ss.least[b] = least;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.m_full[b]);
      }
    } else {
      // ------------------------- where the join finds a row's pieces: per kind of group, its first unit in
      // the line, tiles, blocks and the row's rank (tiles 0: none)
#pragma unroll 1
      for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int b = plan.req[r];
        int rank[2] = {0, 0};
        const int g = b < 0 ? -1 : plan.pfx[b];
        if (b >= 0) {
#pragma unroll 1
          for (int i = lane; i < r; i += 32) {
            const int c = plan.req[i];
            rank[1] += c == b;
            rank[0] += c >= 0 && plan.pfx[c] == g;
          }
        }
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          const int n = __reduce_add_sync(0xffffffffu, k ? rank[1] : rank[0]);
          const int at = b < 0 ? -1 : k ? a.n_prefix + b : g;
          int4 v = {0, 0, 0, n};
          if (at >= 0) {
            const Shape2 s = shape_of_group(ar, plan, at);
            v.x = plan.pre[at], v.y = s.tiles, v.z = s.blocks;
          }
          if (lane == 0) reinterpret_cast<int4*>(ar.info)[2 * r + k] = v;
        }
        if (lane == 0 && r == 0) ar.info[8 * a.rows] = plan.pre[a.n_prefix + a.n_req];
      }
    }
  } else {
    // ------------------------------------------------------------------------------- softmax
    regs_up<SOFT_REGS>();
    const int u = warp >> 2, quad = warp & 3, q = 32 * quad + lane;
    Soft w;
    w.s_at = tmem + 128 * u + ((uint32_t)(32 * quad) << 16);
    w.o_at = tmem + F::O_COL + DH * u + ((uint32_t)(32 * quad) << 16);
    const int j_row = q / ar.hps, head = q - j_row * ar.hps;
    int it = 0;
    uint32_t sc = 0;
#pragma unroll 1
    for (int item = 0; next_job(ar, plan, cur, job); ++item) {
      wait(&ss.m_full[item & 1], (item >> 1) & 1, a.status, abort);
      const int row = j_row < ar.rows_per ? ss.row[item & 1][(job.pairs ? u * BLOCK : 0) + j_row] : -1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss.m_free[item & 1]);
      w.hi = row >= 0 ? plan.hi[row] : -1;
      w.m = UNSET;
      w.l = 0.0f;
      w.factor = 1.0f;
      {  // the query
        uint4 v[DH / 8];
        if (row >= 0) {
          const uint4* src = reinterpret_cast<const uint4*>(a.q + row * a.q_stride + (job.at.slice * ar.hps + head) * DH);
#pragma unroll
          for (int e = 0; e < DH / 8; ++e) v[e] = src[e];
        } else {
#pragma unroll
          for (int e = 0; e < DH / 8; ++e) v[e] = make_uint4(0u, 0u, 0u, 0u);
        }
        // its largest finite element, as bf16 bits
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < DH / 8; ++e) {
          const uint32_t x[4] = {v[e].x & 0x7FFF7FFFu, v[e].y & 0x7FFF7FFFu, v[e].z & 0x7FFF7FFFu, v[e].w & 0x7FFF7FFFu};
          top = max_u16x2(top, max_u16x2(max_u16x2(x[0], x[1]), max_u16x2(x[2], x[3])));
        }
        top = max(top >> 16, top & 0xFFFFu);
        float up = 1.0f;
        // (in f16's reach as it is: 2^-1 to 2^15; NaN and infinities make the row NaN either way)
        if (top != 0 && top < 0x7F80u && (top < 0x3F00u || top >= 0x4700u)) {
          const int e = max((int)(top >> 7), 1);  // the largest element is 2^(e - 127) or more: to 2^4, or as near as an f32 goes
          const int k = min(max(131 - e, -126), 126);
          up = __uint_as_float((uint32_t)(127 + k) << 23);
          w.factor = __uint_as_float((uint32_t)(127 - k) << 23);
        }
        uint8_t* dst = sm + F::Q_OFF + u * F::WIDE + q * 128;
#pragma unroll
        for (int e = 0; e < DH / 8; ++e) {
          float f[8];
          bf16x8_to_f32(v[e], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] *= up;
          if (__builtin_expect(top >= 0x7F80u, 0)) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (isinf(f[k])) f[k] = __int_as_float(0x7FC00000);
          }
          *reinterpret_cast<uint4*>(dst + (e >> 3) * HALF + (((e & 7) ^ (q & 7)) << 4)) =
              make_uint4(f16x2_of(f[0], f[1]), f16x2_of(f[2], f[3]), f16x2_of(f[4], f[5]), f16x2_of(f[6], f[7]));
        }
      }
      w.scaled = __any_sync(0xffffffffu, w.factor != 1.0f);
      const bool idle = !__any_sync(0xffffffffu, row >= 0);  // no queries in this warp
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss.q_full[u]);

      const int n = u ? job.n[1] : job.n[0];
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++sc) {
        const int i = job.ring(u, j), s = (it + i) % NS, t0 = job.token(i);
        wait(&ss.s_full[u], sc & 1, a.status, abort);
        if (!idle) {
          tc_fence_after();
          const float* tok = reinterpret_cast<const float*>(sm + F::TOK_OFF) + s * 3 * TT;
          const uint32_t* see = ss.see[s];
          const bool part = ss.part[s];
          uint32_t p[64], top;
          float l0, l1;
          bool moved = false, move = j == 0;
#pragma unroll 1
          for (;;) {
            if (move) {
              if (part) move_reference<DH, true>(w, tok, see, t0, j == 0);
              else move_reference<DH, false>(w, tok, see, t0, j == 0);
              moved = true;
            }
            if (part) tile_weights<true>(w, tok, see, t0, p, l0, l1, top);
            else tile_weights<false>(w, tok, see, t0, p, l0, l1, top);
            if (moved) break;
            move = __any_sync(0xffffffffu, (top & 0xFFFFu) > TOO_LARGE || (top >> 16) > TOO_LARGE);
            if (!move) break;
          }
          w.l += l0 + l1;
          st32(w.s_at, p);
          st32(w.s_at + 32, p + 32);
          tc_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.p_full[u]);
      }
      wait(&ss.o_full[u], item & 1, a.status, abort);
      tc_fence_after();
      it += job.count();

      // ---- the piece: where it goes, then O
      float* to = nullptr;
      if (row >= 0) {
        const int kind = job.at.g < a.n_prefix ? 0 : 1;
        const size_t k = job.s0 == 0 ? ((size_t)kind * ar.max_rows + row) * a.n_q + job.at.slice * ar.hps + head
                                     : (size_t)blockIdx.x * (2 * BLOCK) + (job.pairs ? u * BLOCK : 0) + q;
        to = (job.s0 == 0 ? ar.home : ar.over) + k * (DH + 4);
      }
      if (job.pairs) {
        if (to) *reinterpret_cast<float2*>(to) = make_float2(w.m, w.l);
#pragma unroll 1
        for (int c = 0; c < DH; c += 32) {
          uint32_t o[32];
          tc_ld32(w.o_at + c, o);
          tc_wait_ld();
          loaded32(o);
          if (to)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(to + 4 + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      } else {  // both streams' O in the larger m, half of the dimensions each
        ss.ml[u][q] = make_float2(w.m, w.l);
        bar_sync<SOFT>(1);
        const float2 x = ss.ml[0][q], y = ss.ml[1][q];
        const float m = fmaxf(x.x, y.x);
        // (a NaN stays one)
        const float fx = x.y != x.y ? 1.0f : x.x == UNSET ? 0.0f : ex2(x.x - m);
        const float fy = y.y != y.y ? 1.0f : y.x == UNSET ? 0.0f : ex2(y.x - m);
        const float l = (fx != 0.0f ? x.y * fx : 0.0f) + (fy != 0.0f ? y.y * fy : 0.0f);
        if (to && u == 0) *reinterpret_cast<float2*>(to) = make_float2(m, l);
        const uint32_t o0 = tmem + F::O_COL + ((uint32_t)(32 * quad) << 16);
#pragma unroll 1
        for (int c = u * (DH / 2); c < (u + 1) * (DH / 2); c += 32) {
          uint32_t v[32], z[32];
          tc_ld32(o0 + c, v);
          tc_ld32(o0 + DH + c, z);
          tc_wait_ld();
          loaded32(v);
          loaded32(z);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float p0 = fx != 0.0f ? __uint_as_float(v[e]) * fx : 0.0f;
            const float p1 = fy != 0.0f ? __uint_as_float(z[e]) * fy : 0.0f;
            v[e] = __float_as_uint(p0 + p1);
          }
          if (to)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(to + 4 + c + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        tc_fence_before();
        bar_sync<SOFT>(1);  // (the next item's products go over both)
        tc_fence_after();
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    (void)wait(&ss.drain, 0, a.status, abort);
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

// Joins the pieces of a (row, head), of its prefix and its own tokens: a warp each, 4 dimensions a lane
// (64 wide: the half warps take every other piece).
constexpr int JOIN_WARPS = 4, AHEAD = 4;
__global__ void __launch_bounds__(JOIN_WARPS * 32) join_shared_kernel(const __grid_constant__ Args ar, int ctas) {
  const SharedArgs& a = ar.a;
  const int r = blockIdx.x, h = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int dh = a.head_dim, d = 4 * lane & (dh - 1), step = 128 / dh, own = lane * 4 / dh;
  const int slice = h / ar.hps, ld = dh + 4;
  pdl_trigger();
  pdl_wait();
  if (h >= a.n_q) return;
  const Cut cut(ar.info[8 * a.rows], ctas);
  int n[2], over[2];  // a kind's pieces; its second one's place
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int4 v = reinterpret_cast<const int4*>(ar.info)[2 * r + k];
    n[k] = 0, over[k] = 0;
    if (v.y == 0) continue;
    Shape2 s = {v.y, v.z, EXTRA + v.y, EXTRA + (v.y + 1) / 2};
    const int block = v.w / ar.rows_per, pair = block >> 1;
    const int from = v.x + slice * s.slice_len() + pair * s.whole;
    const int k0 = cut.team_of(from + EXTRA), k1 = cut.team_of(from + s.len(pair) - 1);
    n[k] = k1 - k0 + 1;
    over[k] = (k0 + 1) * (2 * BLOCK) + (s.pairs(pair) ? (block & 1) * BLOCK : 0) + (v.w - block * ar.rows_per) * ar.hps +
              (h - slice * ar.hps);
  }
  const int all = n[0] + n[1];
  auto piece = [&](int i) -> const float* {
    const int k = i < n[0] ? 0 : 1, x = k ? i - n[0] : i;
    return x == 0 ? ar.home + (((size_t)k * ar.max_rows + r) * a.n_q + h) * ld
                  : ar.over + ((size_t)over[k] + (size_t)(x - 1) * (2 * BLOCK)) * ld;
  };
  auto fetch = [&](int i) { return *reinterpret_cast<const float4*>(piece(i) + 4 + d); };
  float m = UNSET, den = 0.0f;
  float4 num = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int b = 0; b < all; b += 32) {
    const int in = min(32, all - b);
    float2 ml = {UNSET, 0.0f};
    if (lane < in) ml = *reinterpret_cast<const float2*>(piece(b + lane));
    float4 x[AHEAD];
#pragma unroll
    for (int e = 0; e < AHEAD; ++e)
      if (own + step * e < in) x[e] = fetch(b + own + step * e);
    const float to = fmaxf(m, warp_max(ml.x)), old = m == to ? 1.0f : ex2(m - to);
    // (a piece that saw nothing has no part; a NaN stays one)
    const float f = ml.y != ml.y ? 1.0f : ml.y == 0.0f ? 0.0f : ex2(ml.x - to);
    m = to;
    den = fmaf(den, old, warp_sum(f != 0.0f ? f * ml.y : 0.0f));
    num.x *= old, num.y *= old, num.z *= old, num.w *= old;
#pragma unroll 1
    for (int i = 0; i < in; i += step * AHEAD) {
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        const int at = i + own + step * e;
        const float g = __shfl_sync(0xffffffffu, f, at & 31);
        if (at < in && g != 0.0f) {
          num.x = fmaf(g, x[e].x, num.x), num.y = fmaf(g, x[e].y, num.y);
          num.z = fmaf(g, x[e].z, num.z), num.w = fmaf(g, x[e].w, num.w);
        }
        if (at + step * AHEAD < in) x[e] = fetch(b + at + step * AHEAD);
      }
    }
  }
  if (dh == 64) {
    num.x += __shfl_xor_sync(0xffffffffu, num.x, 16), num.y += __shfl_xor_sync(0xffffffffu, num.y, 16);
    num.z += __shfl_xor_sync(0xffffffffu, num.z, 16), num.w += __shfl_xor_sync(0xffffffffu, num.w, 16);
  }
  const float inv = den == 0.0f ? 0.0f : 1.0f / den;
  if (den == 0.0f) num = {0.0f, 0.0f, 0.0f, 0.0f};
  *reinterpret_cast<uint2*>(a.o + r * a.o_stride + (long long)h * dh + d) =
      make_uint2(pack_bf16x2(num.x * inv, num.y * inv), pack_bf16x2(num.z * inv, num.w * inv));
  if (lane == 0 && a.lse) a.lse[(long long)r * a.n_q + h] = den == 0.0f ? -INFINITY : (log2f(den) + m) * LN2;
}

template <int DH>
cudaError_t prepare() {
  // the register split adds up to what a block launches with
  cudaFuncAttributes f;
  cudaError_t e = cudaFuncGetAttributes(&f, attend_shared_kernel<DH>);
  if (e == cudaSuccess && f.numRegs != REGS) e = cudaErrorInvalidConfiguration;
  return e == cudaSuccess ? cudaFuncSetAttribute(attend_shared_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 Form<DH>::SMEM_BYTES)
                          : e;
}

struct Layout {
  size_t info, home, over, bytes;
};
Layout layout(int max_rows, int n_q, int head_dim, int sms) {
  Layout l;
  const size_t piece = (size_t)(head_dim + 4) * 4;
  l.info = 0;
  l.home = ((size_t)max_rows * 32 + 16 + 255) / 256 * 256;
  l.over = l.home + 2 * (size_t)max_rows * n_q * piece;
  l.bytes = l.over + (size_t)sms * 2 * BLOCK * piece;
  return l;
}

}  // namespace

size_t shared_workspace_bytes(int max_rows, int n_q, int head_dim, int sms) {
  return layout(max_rows, n_q, head_dim, sms).bytes;
}

cudaError_t shared_prepare() {
  const cudaError_t e = prepare<128>();
  return e == cudaSuccess ? prepare<64>() : e;
}

bool shared_fits(int rows, int slices, long long tokens) {
  return 2 * (long long)rows * slices * ((tokens + TT - 1) / TT + 1 + EXTRA) <= INT32_MAX;
}

cudaError_t launch_attend_shared(const Launch& L, const SharedArgs& a, uint8_t* ws, int max_rows, int sms) {
  const Layout l = layout(max_rows, a.n_q, a.head_dim, sms);
  Args ar = {};
  ar.a = a;
  ar.slices = a.kv_dim / a.head_dim;
  ar.hps = a.n_q / ar.slices;
  ar.rows_per = BLOCK / ar.hps;
  ar.info = reinterpret_cast<int*>(ws + l.info);
  ar.home = reinterpret_cast<float*>(ws + l.home);
  ar.over = reinterpret_cast<float*>(ws + l.over);
  ar.max_rows = max_rows;
  ar.box = encode_shared_maps(&ar.codes, &ar.scales, a);
  cudaError_t e = a.head_dim == 128
                      ? launch_ex(L, dim3(sms), dim3(THREADS), Form<128>::SMEM_BYTES, attend_shared_kernel<128>, ar)
                      : launch_ex(L, dim3(sms), dim3(THREADS), Form<64>::SMEM_BYTES, attend_shared_kernel<64>, ar);
  if (e == cudaSuccess)
    e = launch_ex(L, dim3(a.rows, (a.n_q + JOIN_WARPS - 1) / JOIN_WARPS), dim3(JOIN_WARPS * 32), 0, join_shared_kernel,
                  ar, sms);
  return e;
}

}  // namespace mono
