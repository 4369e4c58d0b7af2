// Attention of a batch whose requests share prefixes, on the 5th-generation tensor cores: a prefix is
// read once for the rows of all its requests, every request's own tokens for its rows.
//
//   S[q, t] = codes_t . q        (query q = one head of one row, token t)
//   P[q, t] = 2^(a_t S - m_q) a_t,  a_t = scale scale_t log2e         O[q, :] = sum_t P[q, t] codes_t
//
// Queries are the M of both products, 128 of them a block: the heads that read a latent slice, times as
// many rows as fit.  Tokens are the N of the first product, 128 a tile, and its K operand is the V
// operand of the second: the tile is widened from e4m3 to f16 (exact) once, and serves both.  A query
// is f16 too, off by at most 2^-24 of its largest element (those out of f16's reach are scaled by a
// power of two).  P is f16 (11 bits; the one rounding between scores and o) under m_q, an integer that
// follows them, so that the largest of the tokens that set it (an item's first 32, or a tile's 128) is in
// (2^5, 2^6], and moves when one passes 2^15; O is rescaled then, exactly.  P takes its scores' place in TMEM.
//
// Work: groups (a prefix with its requests' rows; a request's own tokens with its rows), slices and
// pairs of blocks make items; the tiles of all items lie in one line, cut evenly over the CTAs, every
// CTA deriving the cut for itself.  A CTA has two streams of softmax: those of two blocks over the same
// tiles, of two slices of one block, or of every other tile of one block and slice.  What a CTA has of an item
// leaves (O, m, l) in the workspace; a second kernel joins them.
//
// Roles: warps 0-7 and 8-15 softmax; 16-19 widen tiles; 20 issues MMAs; 21 loads; 22 makes the items and their
// rows, and tells the join where pieces are (23 makes the registers' split come out).
// Every wait is for an mbarrier, and bounded; one that runs out is reported and ends its role, and with it
// the others' waits.  Copies and products on their way are waited for before the CTA ends.
//
// Bound by the chain of a stream's tile: the second product and the next first one (1040 cycles, of which the
// other stream's fill some), their barriers (700) and the softmax (1550); a step of two tiles takes 3150 to
// 3600 cycles where the MMAs alone would take 2050.  An item costs some 6 us beside its tiles (queries 1.5,
// first scores 0.7, first softmax 2, last product and piece 1.5), the plan and the first item 3, the join 2 to 8.
// Measured in a graph, 64 heads of 128: one question behind 777 tokens 13.0 us; eight requests behind 32K
// tokens 22, with five drafts each 54.6 (975 TFLOP/s of 1904 measured); 256 behind 8K tokens with up to 1K of
// their own 111; 8 x 128 prompt rows behind 32K tokens 835 (1320 TFLOP/s), behind 4K 167.  Beside the attention
// of whole contexts (k_attend.cu), whose queries are the N and need not fill 128: eight requests behind 32K
// tokens 22 us, 38 there, behind 1K 14.0 and 13.6; 64 behind 1K with 500 of their own 25 and 28, behind 256 23.4
// and 21.9; one question behind 777 tokens 13.0 and 12.0, behind 8K 14.1 and 21.3; 256 requests that share nothing, 127 tokens
// each 32 and 46, 511 54 and 55, 1023 76 and 67.
#include <cfloat>
#include <cstddef>

#include "attend_tc.cuh"

namespace mono {
namespace {

using namespace tc;
using namespace attend;

constexpr int SOFT_WARPS = 16, STREAM_WARPS = SOFT_WARPS / 2, WIDEN_WARPS = 4, WIDEN_TOKENS = TT / WIDEN_WARPS;
constexpr int WIDEN_WARP = SOFT_WARPS, MMA_WARP = WIDEN_WARP + WIDEN_WARPS, LOAD_WARP = MMA_WARP + 1, ROWS_WARP = LOAD_WARP + 1;
constexpr int THREADS = 32 * (ROWS_WARP + 2), SOFT = 32 * WIDEN_WARP;
constexpr int MAX_GROUPS = MAX_PREFIX + MAX_REQ;
constexpr int BLOCK = 128;       // queries
// What an item costs a CTA beside its steps, in steps (2: 48 rows behind 32K tokens 58.9 us instead of 54.5; 4: 256
// requests 115 instead of 111).
constexpr int EXTRA = 3;
constexpr int HALF = TT * 128;   // bytes of 64 dimensions of a tile, or a block, in f16
// Tiles from which on a lone block's slices are an item each (eight requests behind 32K tokens 22 us, 25 with
// two slices to an item; 256 requests of 1K tokens 80 us with two to an item, 97 with one each).
constexpr int LONG = 16;
constexpr int JOBS = 4;          // items whose rows are made ahead
constexpr float BASE = 6.0f, LEAST = -90.0f;  // log2 of the weights times a_t that m puts at most; a_t below
constexpr float TOO_LARGE = 0x1p15f;           // m moves when a weight times a_t may be larger (f16 ends at 2^16)
// The least reference: tokens below it have no weight beside those that come later, and a head whose tokens are all
// below it (as large as scores have to be for a NaN, and negative) is NaN.
constexpr float LOWEST = -SCORE_MAX;
// queries are taken times 2^6: the largest element of most is then between 2^-1 and 2^15 (bf16 bits of the limits)
constexpr float Q_SCALE = 64.0f;
constexpr uint32_t Q_LOW = 0x3C00, Q_HIGH = 0x4400;
// registers a thread at launch, and as the roles divide them
constexpr int REGS = 80, SOFT_REGS = 88, OTHER_REGS = 64;
static_assert(SOFT_REGS * SOFT + OTHER_REGS * (THREADS - SOFT) == REGS * THREADS, "register split");

// The step as every CTA derives it.  Groups: prefixes, then requests.
struct Plan {
  int pre[MAX_GROUPS + 4];  // [groups + 1] the line's steps of all groups before
  int end[MAX_GROUPS];      // one behind the last token that a row sees
  int first[MAX_GROUPS];    // the first
  int tiles[MAX_GROUPS];    // from the one's to the other's
  int len[MAX_PREFIX];      // tokens of a prefix
  int hi[MAX_ROWS];         // a row's last token
  short cnt[MAX_GROUPS];    // rows
  short req[MAX_ROWS];      // a row's request; -1: nothing to see
  short pfx[MAX_REQ];       // a request's prefix; -1: none, -2: bad
};

template <int DH>
struct Form {
  static constexpr int WIDE = DH / 64 * HALF, NARROW = TT * DH;  // a tile in f16, in e4m3
  static constexpr int NS = DH == 128 ? 3 : 5, ST = DH == 128 ? 2 : 4;  // rings of wide and narrow tiles
  // a stream's queries; its pieces go through the same place, eight rows of a warp at a time
  static constexpr int PART_LD = DH + 8;  // a piece: m, l, six words of padding, O
  static constexpr int Q_BYTES = WIDE + 16 * BLOCK;
  static_assert(Q_BYTES == 8 * 8 * PART_LD * 4, "eight rows a warp");
  static constexpr int Q_OFF = 0, V_OFF = Q_OFF + 2 * Q_BYTES, K_OFF = V_OFF + NS * WIDE;
  static constexpr int SC_OFF = K_OFF + ST * NARROW;      // the 16 bytes behind the codes [ST][TT]
  static constexpr int TOK_OFF = SC_OFF + ST * TT * 16;   // a_t [NS][TT], in the order of token_slot
  static constexpr int PLAN_OFF = TOK_OFF + NS * TT * 4;
  static constexpr int SMEM_BYTES = PLAN_OFF + (int)sizeof(Plan) + 1024;
  static constexpr int O_COL = 256;  // TMEM: scores (and weights) of stream u at 128 u, its O at O_COL + DH u
};

// Division of numbers below 2^31 by one that the host knows: n mul / 2^shift, mul = 2^(31 + l) / d rounded up,
// 2^l >= d (Granlund and Montgomery's theorem).
struct Divisor {
  uint32_t mul;
  int shift;
  static Divisor of(int d) {
    int l = 0;
    while ((1ll << l) < d) ++l;
    return {(uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
  }
  __device__ int operator()(int n) const { return (int)((uint64_t)(uint32_t)n * mul >> shift); }
};

struct Args {
  CUtensorMap codes, scales;
  int box;  // 0: no maps
  int slices, hps, rows_per;  // latent slices, heads of one, rows of a block
  Divisor by_page, by_hps, by_rows, by_grid;  // block_size, hps, rows_per, CTAs
  SharedArgs a;
  float* home;   // pieces: [2][max_rows][n_q], of those that begin an item; prefixes', then own tokens'
  float* over;   // [CTAs][2 * BLOCK], of a CTA's item that began before it
  int* info;     // [rows][slices][2][2]: pieces, and the second one's place, of a prefix and of own tokens
  int max_rows;
};

// (tokens behind what the requests' table holds are nobody's; a prefix's end was cut to its table)
__device__ __forceinline__ int end_of(const SharedArgs& a, const Plan& p, int g) {
  return g < a.n_prefix ? p.end[g] : min(p.end[g], a.kv.max_blocks * a.kv.block_size);
}

// A softmax lane has the tokens 8 k + 2 (lane & 3), and the next one, of a tile: where a token's factor is,
// so that 16 bytes hold a lane's of two k.
__device__ __forceinline__ int token_slot(int t) {
  return (t >> 4) * 16 + ((t >> 1) & 3) * 4 + ((t >> 3) & 1) * 2 + (t & 1);
}

// A group's items.  First those of two blocks: for every slice the pairs of blocks.  Then those of an odd
// last block: of two slices each, and if a slice is left, one whose streams take every other tile; in a long
// group all slices are such items, since these have half as many pieces.
enum { TWO_BLOCKS, TWO_SLICES, TWO_TILES };
struct Items {
  int tiles, blocks, len, half;  // lengths in the line of an item, and of one of TWO_TILES
  __device__ Items(const Args& ar, int tiles, int rows)
      : tiles(tiles), blocks(ar.by_rows(rows + ar.rows_per - 1)), len(EXTRA + tiles), half(EXTRA + (tiles + 1) / 2) {}
  __device__ int of_pairs(const Args& ar) const { return ar.slices * (blocks >> 1); }
  // slices of a lone block that are two to an item
  __device__ int joint(const Args& ar) const { return tiles < LONG ? ar.slices & ~1 : 0; }
  __device__ int whole(const Args& ar) const { return of_pairs(ar) + (blocks & 1) * (joint(ar) >> 1); }
  __device__ int count(const Args& ar) const { return whole(ar) + (blocks & 1) * (ar.slices - joint(ar)); }
  __device__ int at(const Args& ar, int item) const {  // an item's place
    const int n = whole(ar);
    return min(item, n) * len + max(item - n, 0) * half;
  }
  __device__ int units(const Args& ar) const { return tiles ? at(ar, count(ar)) : 0; }
};
__device__ __forceinline__ Items items_of(const Args& ar, const Plan& p, int g) {
  return Items(ar, p.tiles[g], p.cnt[g]);
}

// A CTA's part of an item: the steps from s0 on, of a tile for each stream.
struct Job {
  int g, mode, slice, block;  // of stream 0 (the other one: the next slice, or the next block)
  int tile, n[2];             // stream 0's first tile; the streams' tiles
  bool begins;                // the item's first step is here
  int least;                  // the smallest of its rows' last tokens
  alignas(16) short row[2 * BLOCK];  // its rows (-1: none), its blocks' one after another
  // tiles of the ring, and stream u's j-th among them
  __device__ int count() const { return mode == TWO_BLOCKS ? n[0] : n[0] + n[1]; }
  __device__ int ring(int u, int j) const { return mode == TWO_BLOCKS ? j : 2 * j + u; }
  // the ring's i-th
  __device__ int token(int i) const { return (tile + (mode == TWO_SLICES ? i >> 1 : i)) * TT; }
  __device__ int slice_of(int u) const { return slice + (mode == TWO_SLICES ? u : 0); }
};
struct Cursor {
  int g, item, unit, left;
};
// The CTA's next part of an item, into job but for its rows.
__device__ __forceinline__ bool next_job(const Args& ar, const Plan& p, Cursor& c, Job& job) {
  const int groups = ar.a.n_prefix + ar.a.n_req;
#pragma unroll 1
  while (c.left > 0) {
    const Items it = items_of(ar, p, c.g);
    const int of_pairs = it.of_pairs(ar), whole = it.whole(ar);
    const int len = c.item < whole ? it.len : it.half, n = min(len - c.unit, c.left);
    const int s0 = max(0, c.unit - EXTRA), s1 = c.unit + n - EXTRA;
    job.g = c.g;
    job.n[0] = job.n[1] = s1 - s0;
    job.begins = s0 == 0;
    job.tile = (p.first[c.g] >> 7) + s0;
    if (c.item < of_pairs) {
      const int pairs = it.blocks >> 1;
      job.mode = TWO_BLOCKS;
      job.slice = c.item / pairs;
      job.block = 2 * (c.item - job.slice * pairs);
    } else {
      job.block = it.blocks - 1;
      job.mode = c.item < whole ? TWO_SLICES : TWO_TILES;
      job.slice = c.item < whole ? 2 * (c.item - of_pairs) : it.joint(ar) + c.item - whole;
      if (job.mode == TWO_TILES) {
        job.tile += s0;
        job.n[1] = min(2 * s1, it.tiles) - 2 * s0 - job.n[0];
      }
    }
    c.left -= n;
    c.unit = 0;
    if (++c.item >= it.count(ar)) {
      c.item = 0;
      do ++c.g;
      while (c.g < groups && p.pre[c.g + 1] <= p.pre[c.g]);
    }
    if (job.n[0] > 0) return true;
  }
  job.n[0] = job.n[1] = 0;
  return false;
}

struct Shared {
  // barriers, and the arrivals that complete their phases
  uint64_t full[4], k_free[4], v_full[5], v_free[5], s_full[2], p_full[2], o_full[2], o_out[2], q_full[2], merge, drain;
  uint64_t j_full[JOBS], j_free[JOBS];
  uint32_t valid[4][4];                // tokens that are there, of a narrow tile
  alignas(16) uint32_t see[5][4];      // and of a wide one
  int part[5];                         // not every row of the item sees all its tokens
  alignas(16) float most[5][WIDEN_WARPS];  // its largest |a_t| (NaN: one is), of a warp's tokens each
  Job job[JOBS];
  float2 ml[2][BLOCK];
  uint32_t tmem;
  int abort;
};
// (an item is read by the softmax, widening, issuing and loading warps)
constexpr int BARRIERS = 30 + 2 * JOBS;
__device__ __forceinline__ int arrivals(int i) {
  if (i >= 30) return i < 30 + JOBS ? 1 : SOFT_WARPS + WIDEN_WARPS + 2;
  if (i >= 28) return i < 29 ? SOFT_WARPS : 1;
  if (i >= 20) return i == 22 || i == 23 ? 1 : STREAM_WARPS;
  if (i >= 18) return 2;
  return i < 4 || i >= 13 ? 1 : WIDEN_WARPS;
}
static_assert(offsetof(Shared, valid) == 8 * BARRIERS, "barriers");
static_assert(Form<128>::SMEM_BYTES + sizeof(Shared) <= 227 * 1024, "shared memory");
static_assert(Form<64>::SMEM_BYTES + sizeof(Shared) <= 227 * 1024, "shared memory");

// wait() by a thread alone
__device__ __forceinline__ bool wait_alone(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  uint32_t polls = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (*abort || ++polls == (1u << 20)) {
      atomicOr(status, ST_WAIT_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  return true;
}
// x a + b, two tokens of a query
__device__ __forceinline__ void fma2t(float& x, float& y, float ax, float ay, float b) {
  asm("{\n .reg .b64 s, m, b;\n mov.b64 s, {%0, %1};\n mov.b64 m, {%2, %3};\n mov.b64 b, {%4, %4};\n"
      " fma.rn.f32x2 s, s, m, b;\n mov.b64 {%0, %1}, s;\n}"
      : "+f"(x), "+f"(y)
      : "f"(ax), "f"(ay), "f"(b));
}
// The larger magnitudes of two pairs of bf16 (with whatever sign).
__device__ __forceinline__ uint32_t larger_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 16 rows x 32 columns: registers 4 k + 2 h + b are row lane / 4 + 8 h, column 8 k + 2 (lane & 3) + b.
__device__ __forceinline__ void ld_rows(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void loaded16(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
               "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void put_rows(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 rows x 16 columns of packed pairs: registers 2 k + h are row lane / 4 + 8 h, column 4 k + (lane & 3).
__device__ __forceinline__ void st_rows(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// A bulk copy from shared to global memory, in a group with this thread's others until they are waited for.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
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

// Fills the plan (every thread of the block); the results are behind the caller's next barrier.  Waits for the
// kernels before.  `sums`: an int per warp.
__device__ __forceinline__ void derive_plan(const Args& ar, Plan& plan, int* sums) {
  const SharedArgs& a = ar.a;
  const int tid = threadIdx.x, np = a.n_prefix, groups = np + a.n_req;
  const bool tell = blockIdx.x == 0;
  const int cap = a.kv.max_blocks * a.kv.block_size, pcap = a.pre.max_blocks * a.kv.block_size;  // (fit 31 bits)
#pragma unroll 1
  for (int g = tid; g < groups; g += THREADS) plan.end[g] = 0, plan.cnt[g] = 0, plan.first[g] = 0;
  pdl_trigger();
  pdl_wait();
  static_assert(MAX_REQ <= THREADS && MAX_PREFIX <= THREADS, "a request a thread");
  int g = -1, len = 0;  // (fetched ahead of the first use of any)
  if (tid < a.n_req) g = a.prefix_of ? a.prefix_of[tid] : 0;
  if (tid < np) len = a.prefix_lengths[tid];
  // (loops that most steps run once are kept small: this code runs once, and comes from memory)
#pragma unroll 1
  for (int r = tid; r < a.rows; r += THREADS) {
    const int p = a.positions[r], b = a.row_req[r];
    plan.hi[r] = min(p, 0x7FFFFFFE);
    plan.req[r] = (short)(b < 0 || b >= a.n_req ? -1 : b);
  }
  if (tid < a.n_req) {
    if (g < -1 || g >= np) g = -2;
    plan.pfx[tid] = (short)g;
  }
  if (tid < np) plan.len[tid] = max(0, len);
  __syncthreads();
  if (g >= 0) plan.first[np + tid] = plan.len[g];
  // a request's rows and their largest position
#pragma unroll 1
  for (int r = tid; r < a.rows; r += THREADS) {
    const int p = plan.hi[r], b = plan.req[r];
    if (p >= 0 && b >= 0 && plan.pfx[b] >= -1) {
      atomicMax(&plan.end[np + b], p + 1);
    } else {
      plan.req[r] = -1;
      if (p >= 0 && tell) atomicOr(a.status, ST_UNMAPPED_PAGE);
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int r = tid; r < a.rows; r += THREADS) {
    const int b = plan.req[r];
    if (b < 0) continue;
    const int hi = a.causal ? plan.hi[r] : plan.end[np + b] - 1, of = plan.pfx[b], len = plan.first[np + b];
    plan.hi[r] = hi;
    bool beyond = hi >= cap && hi >= len;
    // (16-bit counters: the words that hold them)
#pragma unroll 1
    for (int i = np + b, k = 0; k < 2 && i >= 0; ++k, i = of)
      atomicAdd(reinterpret_cast<int*>(plan.cnt) + (i >> 1), i & 1 ? 1 << 16 : 1);
    if (of >= 0) {
      const int end = min(hi + 1, len);
      beyond |= end > pcap;
      atomicMax(&plan.end[of], min(end, pcap));
    }
    if (beyond && tell) atomicOr(a.status, ST_UNMAPPED_PAGE);
  }
  __syncthreads();
  // the groups' places in the line
  int units = 0;
  if (tid < groups) {
    const int lo = plan.first[tid], end = end_of(a, plan, tid);
    plan.tiles[tid] = plan.cnt[tid] == 0 || end <= lo ? 0 : ((end - 1) >> 7) - (lo >> 7) + 1;
    units = items_of(ar, plan, tid).units(ar);
  }
  static_assert(MAX_GROUPS <= THREADS, "a group a thread");
  int upto = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if ((tid & 31) >= o) upto += y;
  }
  if ((tid & 31) == 31) sums[tid >> 5] = upto;
  __syncthreads();
  if (tid < groups) {
#pragma unroll 1
    for (int w = 0; w < tid >> 5; ++w) upto += sums[w];
    plan.pre[tid + 1] = upto;
  }
  if (tid == 0) plan.pre[0] = 0;
}

// The cut of a line of W.
__device__ __forceinline__ Cut cut_of(const Args& ar, int W) {
  const int n = gridDim.x;
  Cut cut(min(W, 1), 1);
  cut.teams = min(W, n);
  cut.each = W >= n ? ar.by_grid(W) : min(W, 1);
  cut.more = W - cut.each * cut.teams;
  return cut;
}

// The CTA's first item, by a whole warp.
__device__ __forceinline__ Cursor cut_line(const Args& ar, const Plan& plan) {
  const int lane = threadIdx.x & 31, groups = ar.a.n_prefix + ar.a.n_req;
  const Cut cut = cut_of(ar, plan.pre[groups]);
  Cursor c = {0, 0, 0, cut.size(blockIdx.x)};
  if (c.left > 0) {
    // the last group that starts by w0 (and is not empty: the next starts later), a lane a run of groups, then a group
    const int w0 = cut.start(blockIdx.x), each = (groups + 31) >> 5;
    static_assert(MAX_GROUPS <= 32 * 32, "a run's groups are a warp's");
    c.g = each * (__popc(__ballot_sync(0xffffffffu, lane * each < groups && plan.pre[min(lane * each, groups)] <= w0)) - 1);
    const int g = c.g + lane;
    c.g += __popc(__ballot_sync(0xffffffffu, lane < each && g < groups && plan.pre[min(g, groups)] <= w0)) - 1;
    const Items it = items_of(ar, plan, c.g);
    const int u = w0 - plan.pre[c.g], whole = it.whole(ar), more = u - whole * it.len, len = more < 0 ? it.len : it.half;
    const int n = (more < 0 ? u : more) / len;
    c.item = more < 0 ? n : whole + n;
    c.unit = (more < 0 ? u : more) - n * len;
  }
  return c;
}

// The rows of an item's blocks, in row order, by a whole warp, and the smallest of their last tokens.
__device__ __forceinline__ void item_rows(const Args& ar, const Plan& plan, Job& job) {
  const int lane = threadIdx.x & 31, np = ar.a.n_prefix, g = job.g;
  const int first = job.block * ar.rows_per, most = (job.mode == TWO_BLOCKS ? 2 : 1) * ar.rows_per;
#pragma unroll
  for (int i = 0; i < 2 * BLOCK / 8; i += 32) reinterpret_cast<uint4*>(job.row)[i + lane] = make_uint4(~0u, ~0u, ~0u, ~0u);
  __syncwarp();
  int seen = 0, least = 0x7FFFFFFF;
  constexpr int AT_ONCE = 4;  // (a group's rows are anywhere: 256 rows, 32 at a time, took 1900 cycles)
#pragma unroll 1
  for (int r0 = 0; r0 < ar.a.rows && seen - first < most; r0 += 32 * AT_ONCE) {
    int b[AT_ONCE];
    bool in[AT_ONCE];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) b[k] = r0 + 32 * k + lane < ar.a.rows ? plan.req[r0 + 32 * k + lane] : -1;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) in[k] = b[k] >= 0 && (g < np ? plan.pfx[b[k]] == g : b[k] == g - np);
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const uint32_t m = __ballot_sync(0xffffffffu, in[k]);
      const int r = r0 + 32 * k + lane, rank = seen + __popc(m & ((1u << lane) - 1)) - first;
      if (in[k] && rank >= 0 && rank < most) {
        job.row[rank < ar.rows_per ? rank : BLOCK + rank - ar.rows_per] = (short)r;
        least = min(least, plan.hi[r]);
      }
      seen += __popc(m);
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  if (lane == 0) job.least = least;
}

// Loads narrow tiles, a warp: TMA boxes through the page table, a lane each, looked up ahead of the load; or
// cp.async, a token a lane, where there are no maps.
template <int DH>
struct Loader {
  int box, shift, t0, lo, end, page, row;
  const int* table;
  int max_blocks;
  __device__ explicit Loader(int b) {
    box = b ? b : 1;
    shift = __ffs(box) - 1;
  }
  // The page and the place in it of token t (page -1: not mapped; row -1: not needed).
  __device__ __forceinline__ void look_up(const Args& ar, int t, bool needed) {
    const int lb = ar.by_page(t);
    page = row = -1;
    if (needed && t < end && t + box > lo) {
      row = t - lb * ar.a.kv.block_size;
      if (lb < max_blocks) page = __ldg(table + lb);
    }
  }
  // (asked where it is needed, so that nothing waits for a lookup before)
  __device__ __forceinline__ bool mapped(const Args& ar) const { return page >= 0 && page < ar.a.kv.num_blocks; }
  __device__ __forceinline__ void locate(const Args& ar, const Plan& plan, const Job& job, int i) {
    const int lane = threadIdx.x & 31, np = ar.a.n_prefix, g = job.g;
    const PagedView& v = g < np ? ar.a.pre : ar.a.kv;
    max_blocks = v.max_blocks;
    table = v.table + (size_t)(g < np ? g : g - np) * max_blocks;
    t0 = job.token(i);
    lo = plan.first[g];
    end = end_of(ar.a, plan, g);
    if (box > 1) look_up(ar, t0 + (lane << shift), lane < TT >> shift);
  }
  __device__ __forceinline__ void load(const Args& ar, int slice, uint8_t* st, uint8_t* sc, uint32_t* valid,
                                       uint64_t* full) {
    const SharedArgs& a = ar.a;
    const int lane = threadIdx.x & 31;
    if (box > 1) {
      const bool there = mapped(ar);
      if (there) {
        tma_load_3d(st + ((lane * DH) << shift), &ar.codes, DH * slice, row, page, full);
        tma_load_3d(sc + ((lane * 16) << shift), &ar.scales, a.kv_dim, row, page, full);
      } else if (row >= 0) {
        atomicOr(a.status, ST_UNMAPPED_PAGE);
      }
      const uint32_t have = __ballot_sync(0xffffffffu, there);
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const int t = t0 + 32 * q + lane;
        const uint32_t w =
            __ballot_sync(0xffffffffu, ((have >> ((32 * q + lane) >> shift)) & 1) && t >= lo && t < end);
        if (lane == q) valid[q] = w;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(full, __popc(have) * box * (DH + 16));
    } else {
      constexpr int PIECES = DH / 16, ROWS = 32 / PIECES;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        look_up(ar, t0 + 32 * q + lane, true);
        const bool there = mapped(ar);
        if (row >= 0 && !there) atomicOr(a.status, ST_UNMAPPED_PAGE);
        const long long off = page * a.kv.stride_block + row * a.kv.stride_tok;
        const uint32_t w = __ballot_sync(0xffffffffu, there);
        if (lane == 0) valid[q] = w;
#pragma unroll 1
        for (int e = 0; e < 32 / ROWS; ++e) {
          const int k = ROWS * e + lane / PIECES, piece = lane & (PIECES - 1);
          const long long ro = __shfl_sync(0xffffffffu, off, k);
          if ((w >> k) & 1)
            cp_async16(st + (32 * q + k) * DH + 16 * piece, a.kv.base + ro + DH * slice + 16 * piece, 16);
        }
        if (there) cp_async16(sc + (32 * q + lane) * 16, a.kv.base + off + a.kv_dim, 16);
      }
      cp_async_wait_all();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
    __syncwarp();
  }
};

// O of 16 rows times the lane's two rows' factors.
__device__ __forceinline__ void scale_rows(uint32_t at, int columns, const float (&f)[2]) {
#pragma unroll 1
  for (int c = 0; c < columns; c += 8) {
    float x[4];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                 : "r"(at + c));
    tc_wait_ld();
    tc_loaded4(x);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= f[e >> 1];
    asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + c), "f"(x[0]), "f"(x[1]),
                 "f"(x[2]), "f"(x[3])
                 : "memory");
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
  Plan& plan = *reinterpret_cast<Plan*>(sm + F::PLAN_OFF);
  // (the warp from one lane: the compiler then knows the roles to be whole warps, and leaves out a fifth of
  // the code, that for lanes apart; 256 requests 152 -> 144 us)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid < BARRIERS) {
    mbar_init(ss.full + tid, arrivals(tid));
    fence_mbar_init();
  }
  if (tid == 0) {
    ss.abort = 0;
    if (ar.box) prefetch_tmap(&ar.codes), prefetch_tmap(&ar.scales);
  }
  if (warp == MMA_WARP) tmem_alloc<512>(&ss.tmem);
  derive_plan(ar, plan, reinterpret_cast<int*>(ss.ml));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ss.tmem;

  // The next item (null: there is none, or a wait ran out), and that it is no longer needed; by whole warps.
  int item = 0;
  auto next_item = [&]() -> const Job* {
    const Job* job = &ss.job[item % JOBS];
    if (!wait(&ss.j_full[item % JOBS], (item / JOBS) & 1, a.status, abort)) return nullptr;
    return job->n[0] > 0 ? job : nullptr;
  };
  auto item_done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&ss.j_free[item % JOBS]);
    ++item;
  };

  if (warp >= WIDEN_WARP) {
    regs_down<OTHER_REGS>();
    if (warp < MMA_WARP) [&] {
      // ------------------------------------------------------------- tiles from e4m3 to f16
      constexpr int PIECES = DH / 16, ROWS = 32 / PIECES, N = WIDEN_TOKENS / ROWS;  // of 16 codes; rows at a time
      const int t0 = WIDEN_TOKENS * (warp - WIDEN_WARP), piece = lane & (PIECES - 1), r0 = lane / PIECES;
      const float to_log2 = a.scale * (LOG2E / Q_SCALE);
      const int odd = (piece >> 2) & 1;  // (such lanes store the other half first: no bank twice)
      int it = 0;
#pragma unroll 1
      while (const Job* job = next_item()) {
        const int n = job->count(), least = job->least;
#pragma unroll 1
        for (int i = 0; i < n; ++i, ++it) {
          const int st = it % ST, s = it % NS;
          if (!wait(&ss.full[st], (it / ST) & 1, a.status, abort)) return;
          const uint32_t ok = ss.valid[st][t0 >> 5];
          // some row does not see all its tokens
          const bool part = least < job->token(i) + TT - 1 ||
                            (ss.valid[st][0] & ss.valid[st][1] & ss.valid[st][2] & ss.valid[st][3]) != 0xffffffffu;
          const float raw = *reinterpret_cast<const float*>(sm + F::SC_OFF + (st * TT + t0 + lane) * 16);
          if (it >= NS && !wait(&ss.v_free[s], (it / NS - 1) & 1, a.status, abort)) return;
          const uint8_t* src = sm + F::K_OFF + st * F::NARROW + t0 * DH + lane * 16;
          uint8_t* dst = sm + F::V_OFF + s * F::WIDE + (piece >> 2) * HALF;
          uint32_t nan = 0;
          bool check = false;
          if (__builtin_expect(part && ok != 0, 0)) {
#pragma unroll 4
            for (int e = 0; e < N; ++e) {
              const uint4 v = lds128(src + e * ROWS * DH), c = without_nan(v);
              check |= c.x != v.x || c.y != v.y || c.z != v.z || c.w != v.w;
            }
            check = __any_sync(0xffffffffu, check);
          }
          if (__builtin_expect(check, 0)) {
            // a NaN code that some row must not see would reach it as 0 * NaN: it is a 0 then, and the token's
            // factor is NaN
#pragma unroll 1
            for (int e = 0; e < N; ++e) {
              uint4* at = reinterpret_cast<uint4*>(const_cast<uint8_t*>(src) + e * ROWS * DH);
              const uint4 v = *at, c = without_nan(v);
              const uint32_t bad = __ballot_sync(0xffffffffu, c.x != v.x || c.y != v.y || c.z != v.z || c.w != v.w);
              if (__builtin_expect(bad, 0)) {
                *at = c;
#pragma unroll 1
                for (int k = 0; k < ROWS; ++k)
                  if ((bad >> (k * PIECES)) & ((1u << PIECES) - 1)) nan |= 1u << (e * ROWS + k);
              }
            }
            fence_proxy_async_shared();  // (ahead of the next copy to this place)
          }
          if (__builtin_expect(ok == 0, 0)) {  // no tokens: zeros
#pragma unroll 1
            for (int e = 0; e < N; ++e) {
              const int row = t0 + e * ROWS + r0, c = 2 * (piece & 3) + odd;
              *reinterpret_cast<uint4*>(dst + row * 128 + ((c ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(dst + row * 128 + (((c ^ 1) ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            }
          } else {
#pragma unroll 1
            for (int e0 = 0; e0 < N; e0 += 4) {
              uint4 v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = lds128(src + (e0 + e) * ROWS * DH);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int row = t0 + (e0 + e) * ROWS + r0, c = 2 * (piece & 3) + odd;
                uint4 x, y;
                uint32_t f[2];
                e4m3x4_to_f16x4(odd ? v[e].z : v[e].x, f), x.x = f[0], x.y = f[1];
                e4m3x4_to_f16x4(odd ? v[e].w : v[e].y, f), x.z = f[0], x.w = f[1];
                e4m3x4_to_f16x4(odd ? v[e].x : v[e].z, f), y.x = f[0], y.y = f[1];
                e4m3x4_to_f16x4(odd ? v[e].y : v[e].w, f), y.z = f[0], y.w = f[1];
                *reinterpret_cast<uint4*>(dst + row * 128 + ((c ^ (row & 7)) << 4)) = x;
                *reinterpret_cast<uint4*>(dst + row * 128 + (((c ^ 1) ^ (row & 7)) << 4)) = y;
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ss.k_free[st]);
          {  // a token a lane
            static_assert(WIDEN_TOKENS == 32, "a token a lane");
            const bool there = (ok >> lane) & 1, fin = fabsf(raw) <= SCALE_MAX && !((nan >> lane) & 1);
            float f = !there ? 0.0f : fin ? raw * to_log2 : __int_as_float(0x7FC00000);
            if (f == 0.0f) f = FLT_MIN;  // (as good as 0, and infinity times it is infinity)
            reinterpret_cast<float*>(sm + F::TOK_OFF)[s * TT + token_slot(t0 + lane)] = f;
            const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(f)));  // (a NaN stays one)
            if (lane == 0) ss.most[s][warp - WIDEN_WARP] = __uint_as_float(most);
          }
          if (lane == 0) {
            ss.see[s][t0 >> 5] = ok;
            if (t0 == 0) ss.part[s] = part;
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ss.v_full[s]);
        }
        item_done();
      }
    }();
    else if (warp == MMA_WARP) {
      // ------------------------------------------- MMAs: a stream's second product, then its next first one, in
      // turns, so that one stream's run while the other's softmax does.  (Issued by a warp per stream they
      // mixed, both streams' scores came at once, and MMAs and softmax took turns.)  By one thread, in few
      // instructions: between two turns the other warps' push these out of the instruction cache, and each 128
      // bytes of them cost some 90 cycles again.
      constexpr uint32_t IS = (1u << 4) | ((uint32_t)(TT >> 3) << 17) | ((uint32_t)(BLOCK >> 4) << 24);
      constexpr uint32_t IO = (1u << 4) | (1u << 16) | ((uint32_t)(DH >> 3) << 17) | ((uint32_t)(BLOCK >> 4) << 24);
      if (elect_one()) {
        const uint64_t q0 = desc_sw128(smem_u32(sm + F::Q_OFF)), k0 = desc_sw128(smem_u32(sm + F::V_OFF)),
                       v0 = desc_mn(smem_u32(sm + F::V_OFF), HALF);
        auto await = [&](uint64_t* bar, uint32_t parity) {
          const bool there = wait_alone(bar, parity, a.status, abort);
          tc_fence_after();
          return there;
        };
        int s1 = 0, s2 = 0;           // the wide ring's places of the next first product, and second one
        uint32_t phase = 0, pc = 0;   // parities: of s1's place, of the streams' tiles so far
        bool ok = true;
#pragma unroll 1
        for (; ok; ++item) {
          const Job* job = &ss.job[item % JOBS];
          ok = await(&ss.j_full[item % JOBS], (item / JOBS) & 1);
          if (!ok || job->n[0] <= 0) break;
          const int n0 = job->n[0], n1 = job->n[1];
          const bool both = job->mode == TWO_BLOCKS;  // streams' tiles are the same
#pragma unroll 1
          for (int x = -2; x < 2 * n0; ++x) {  // stream x & 1
            const int u = x & 1, n = u ? n1 : n0, left = n - (x >> 1);
            const bool next = !both || u;  // (the last one that needs the place)
            if (x >= 0 && left <= 0) continue;
            // (streams of the same tiles: the next one, there long since, is seen ahead of the weights, for both)
            if (both && !u && left > 1 && !(ok = await(&ss.v_full[s1], phase))) break;
            ok = await(x < 0 ? &ss.q_full[u] : &ss.p_full[u], x < 0 ? item & 1 : (pc >> u) & 1);
            if (!ok) break;
            if (x >= 0) {
              pc ^= 1u << u;
              uint64_t vd = v0 + s2 * (F::WIDE / 16);
              uint32_t pcol = tmem + 128 * u, accumulate = x > 1;
#pragma unroll 2
              for (int k = 0; k < TT / 16; ++k, pcol += 8, vd += 2048 / 16, accumulate = 1)
                mma_ts(tmem + F::O_COL + DH * u, pcol, vd, IO, accumulate);
              if (next) {
                tc_commit(&ss.v_free[s2]);
                if (++s2 == NS) s2 = 0;
              }
              if (left == 1) tc_commit(&ss.o_full[u]);
            } else if (n == 0) {
              mbar_arrive(&ss.o_full[u]);
            }
            if (left <= 1) continue;
            if (!both && !(ok = await(&ss.v_full[s1], phase))) break;
            uint64_t qd = q0 + u * (F::Q_BYTES / 16), kd = k0 + s1 * (F::WIDE / 16);
#pragma unroll 2
            for (int k = 0; k < DH / 16; ++k) {
              mma_ss(tmem + 128 * u, qd, kd, IS, k > 0);
              const int on = k == 3 ? HALF / 16 - 6 : 2;
              qd += on, kd += on;
            }
            tc_commit(&ss.s_full[u]);
            // (the commit is no release: this arrival passes on what the widening warps wrote)
            mbar_arrive(&ss.s_full[u]);
            if (next && ++s1 == NS) s1 = 0, phase ^= 1;
          }
          if (ok) mbar_arrive(&ss.j_free[item % JOBS]);
        }
        tc_commit(&ss.drain);
      }
      __syncwarp();
    } else if (warp == LOAD_WARP) {
      // ------------------------------------------------------------------------------ loads
      // A tile's pages are looked up while the one before waits for its place.
      Loader<DH> tile(ar.box), next(ar.box);
      int it = -1, i = 0, n = 0, slice = 0;
      const Job* job = nullptr;
#pragma unroll 1
      for (;;) {
        const int of = slice;
        if (++i >= n) {
          if (job) item_done();
          job = next_item();
          i = 0;
          n = job ? job->count() : 0;
        }
        if (job) next.locate(ar, plan, *job, i), slice = job->slice_of(i & 1);
        if (it >= 0) {
          const int st = it % ST;
          if (it >= ST && !wait(&ss.k_free[st], (it / ST - 1) & 1, a.status, abort)) break;
          tile.load(ar, of, sm + F::K_OFF + st * F::NARROW, sm + F::SC_OFF + st * TT * 16, ss.valid[st], &ss.full[st]);
        }
        ++it;
        if (!job) break;
        tile = next;
      }
      // (what is on its way lands in this CTA's shared memory)
#pragma unroll 1
      for (int k = max(0, it - ST); k < it; ++k) mbar_wait(&ss.full[k % ST], (k / ST) & 1, a.status);
    } else if (warp == ROWS_WARP) {
      // ------------------------------------------------------------------ the items and their rows
      Cursor cur = cut_line(ar, plan);
#pragma unroll 1
      for (;; ++item) {
        const int k = item % JOBS;
        if (item >= JOBS && !wait(&ss.j_free[k], (item / JOBS - 1) & 1, a.status, abort)) break;
        Job& job = ss.job[k];
        bool more = false;
        if (lane == 0) more = next_job(ar, plan, cur, job);
        more = __shfl_sync(0xffffffffu, more, 0);
        __syncwarp();  // (the item that lane 0 wrote, to all lanes: a shuffle orders no memory)
        if (more) item_rows(ar, plan, job);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.j_full[k]);
        if (!more) break;
      }
      // where the join finds the pieces of a row's queries in a slice: how many of its prefix's tokens, and of its
      // own, and the place of the second of each
      const Cut cut = cut_of(ar, plan.pre[a.n_prefix + a.n_req]);
#pragma unroll 1
      for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int b = plan.req[r], g = b < 0 ? -1 : plan.pfx[b];
        int own = 0, pre = 0;  // the row's rank among those of its groups
        if (b >= 0) {
#pragma unroll 1
          for (int i = lane; i < r; i += 32) {
            const int c = plan.req[i];
            own += c == b;
            pre += c >= 0 && plan.pfx[c] == g;
          }
        }
        own = __reduce_add_sync(0xffffffffu, own);
        pre = __reduce_add_sync(0xffffffffu, pre);
#pragma unroll 1
        for (int i = lane; i < 2 * ar.slices; i += 32) {
          const int at = b < 0 ? -1 : i & 1 ? a.n_prefix + b : g, rank = i & 1 ? own : pre, slice = i >> 1;
          int2 v = {0, 0};
          if (at >= 0) {
            const Items it = items_of(ar, plan, at);
            const int block = ar.by_rows(rank), pairs = it.blocks >> 1;
            int item, len = it.len, first = 0;
            if (block < 2 * pairs) {
              item = slice * pairs + (block >> 1);
              first = (block & 1) * BLOCK;
            } else {
              const int joint = it.joint(ar);
              if (slice < joint) item = it.of_pairs(ar) + (slice >> 1), first = (slice & 1) * BLOCK;
              else item = it.whole(ar) + slice - joint, len = it.half;
            }
            if (it.tiles) {
              const int from = plan.pre[at] + it.at(ar, item), k = cut.team_of(from + EXTRA);
              v = make_int2(cut.team_of(from + len - 1) - k + 1,
                            (k + 1) * (2 * BLOCK) + first + (rank - block * ar.rows_per) * ar.hps);
            }
          }
          reinterpret_cast<int2*>(ar.info)[(size_t)r * 2 * ar.slices + i] = v;
        }
      }
    }
  } else [&] {
    // ------------------------------------------------------------------------------- softmax
    // A warp has 16 rows of its lane quadrant; of their scores and weights a lane has the rows lane / 4 and lane
    // / 4 + 8, and a quarter of the tokens (token_slot).  (With a row a lane, the loads of the tokens' factors
    // took as long as both products; with 32 rows a warp, its chain of latencies took twice as long.)
    regs_up<SOFT_REGS>();
    const int u = warp / STREAM_WARPS, quad = warp & 3, half = (warp >> 2) & 1;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16), rows16 = (uint32_t)(16 * half) << 16;
    const uint32_t s_at = lanes + 128 * u + rows16, o_at = lanes + F::O_COL + DH * u;
    const int q16 = 32 * quad + 16 * half;  // the warp's first query of the block
    int it = 0;
    uint32_t sc = 0, mc = 0;  // the stream's tiles, and phases of the merging barrier, so far
#pragma unroll 1
    while (const Job* at = next_item()) {
      const Job& job = *at;
      const int n = u ? job.n[1] : job.n[0], mode = job.mode;
      // the row and the head of query lane & 15, its row's last token, where its piece goes
      const int ql = q16 + (lane & 15), jr = ar.by_hps(ql), head = job.slice_of(u) * ar.hps + ql - jr * ar.hps;
      const int row = jr < ar.rows_per ? job.row[(mode == TWO_BLOCKS ? u * BLOCK : 0) + jr] : -1;
      const int hi = row >= 0 ? plan.hi[row] : -1;
      const bool idle = !__any_sync(0xffffffffu, row >= 0);  // no queries in this warp
      float factor = 1.0f;
      // the stream's warps have the last item's O out of the queries' place
      if (item > 0 && !wait(&ss.o_out[u], (item - 1) & 1, a.status, abort)) return;
      {  // the warp's queries as f16, 16 bytes a lane
        constexpr int PIECES = DH / 8, ROWS = 32 / PIECES, N = 16 / ROWS;  // lanes of a query; queries at a time
        const int piece = lane & (PIECES - 1), r0 = lane / PIECES;
        const long long from = row >= 0 ? row * a.q_stride + head * DH : -1;
        uint8_t* dst = sm + F::Q_OFF + u * F::Q_BYTES + q16 * 128 + (piece >> 3) * HALF;
        auto place = [&](int e) {
          const int r = e * ROWS + r0;
          return reinterpret_cast<uint4*>(dst + r * 128 + (((piece & 7) ^ (r & 7)) << 4));
        };
        auto fetch = [&](int e) {
          const long long at = __shfl_sync(0xffffffffu, from, e * ROWS + r0);
          return at >= 0 ? *reinterpret_cast<const uint4*>(a.q + at + piece * 8) : make_uint4(0, 0, 0, 0);
        };
        auto largest = [](const uint4& v) {  // as bf16 bits
          const uint32_t t = larger_bf16x2(larger_bf16x2(v.x, v.y), larger_bf16x2(v.z, v.w)) & 0x7FFF7FFFu;
          return max(t >> 16, t & 0xFFFFu);
        };
        auto rewrite = [&](uint4* at, const uint4& v, float by) {
          float f[8];
          bf16x8_to_f32(v, f);
#pragma unroll
          for (int k = 0; k < 8; k += 2) mul2(f[k], f[k + 1], by);
          *at = make_uint4(f16x2_of(f[0], f[1]), f16x2_of(f[2], f[3]), f16x2_of(f[4], f[5]), f16x2_of(f[6], f[7]));
        };
        uint4 v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = fetch(e);
        uint32_t fine = 0, high = 0;  // a bit per e: its largest element here is Q_LOW or more; the largest of all
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const uint32_t top = largest(v[e]);
          high = max(high, top);
          fine |= (uint32_t)(top >= Q_LOW) << e;
          rewrite(place(e), v[e], Q_SCALE);
        }
#pragma unroll
        for (int x = PIECES / 2; x > 0; x >>= 1) fine |= __shfl_xor_sync(0xffffffffu, fine, x);
        fine = __shfl_sync(0xffffffffu, fine, (lane & (ROWS - 1)) * PIECES);  // (query lane & 15's is its bit e)
        if (__builtin_expect(__any_sync(0xffffffffu, high >= Q_HIGH ||
                                                         (row >= 0 && !((fine >> ((lane & 15) / ROWS)) & 1))),
                             0)) {
          // some are out of f16's reach, or not finite, or zeros: again, scaled
#pragma unroll 1
          for (int e = 0; e < N; ++e) {
            const uint4 v = fetch(e);
            uint32_t top = largest(v);
#pragma unroll 1
            for (int x = PIECES / 2; x > 0; x >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
            float up = Q_SCALE, back = 1.0f;
            if (top >= 0x7F80u) {  // not finite: the query's weights are NaN
              up = back = __int_as_float(0x7FC00000);
            } else if (top != 0 && (top < Q_LOW || top >= Q_HIGH)) {
              // the largest element is in [2^(k - 127), 2^(k - 126)): to 2^4, or as near as an f32 goes
              const int k = min(max(131 - max((int)(top >> 7), 1), -120), 126);
              up = __uint_as_float((uint32_t)(127 + k) << 23);
              back = __uint_as_float((uint32_t)(127 - k) << 23) * Q_SCALE;
            }
            rewrite(place(e), v, up);
            back = __shfl_sync(0xffffffffu, back, (lane & (ROWS - 1)) * PIECES);
            if ((lane & 15) / ROWS == e) factor = back;
          }
        }
      }
      const bool scaled = __any_sync(0xffffffffu, factor != 1.0f);
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss.q_full[u]);

      float m[2] = {UNSET, UNSET}, l[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++sc) {
        const int i = job.ring(u, j), s = (it + i) % NS;
        if (!wait(&ss.s_full[u], sc & 1, a.status, abort)) return;
        if (!idle) {
          tc_fence_after();
          uint32_t raw[2][16];
          ld_rows(s_at, raw[0]);
          const bool part = ss.part[s];
          const float4 most4 = *reinterpret_cast<const float4*>(ss.most[s]);
          const float most = fmaxf(fmaxf(most4.x, most4.y), fmaxf(most4.z, most4.w));
          const bool bad = part && isnan((most4.x + most4.y) + (most4.z + most4.w));  // some factor is NaN
          const float4* tok = reinterpret_cast<const float4*>(sm + F::TOK_OFF) + s * TT / 4 + (lane & 3);
          // Exponents, weights, their sums and the weights times a_t, of 32 tokens.
          auto factors = [&](int c, float2(&t)[4]) {
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const float4 v = tok[8 * c + 2 * k];
              t[k] = make_float2(v.x, v.y), t[k + 1] = make_float2(v.z, v.w);
            }
          };
          auto exponents = [&](float* x, const float2(&t)[4]) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) fma2t(x[e], x[e + 1], t[e >> 2].x, t[e >> 2].y, -m[(e >> 1) & 1]);
          };
          auto weights = [&](float* x, const float2(&t)[4], float(&sum)[2][2]) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              x[e] = ex2(x[e]), x[e + 1] = ex2(x[e + 1]);
              add2(sum[(e >> 1) & 1][0], sum[(e >> 1) & 1][1], x[e], x[e + 1]);
              mul2(x[e], x[e + 1], t[e >> 2].x, t[e >> 2].y);
            }
          };
          // The references to the largest of some of the tile's weights times a_t (the first of them that is above
          // by BASE), and what was summed under the old ones with them.
          auto move = [&](float(&top)[2]) {
            float by[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
              top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
              by[r] = 1.0f;
              if (top[r] - m[r] > BASE) {
                const float now = top[r] <= SCORE_MAX ? fmaxf(ceilf(top[r]) - BASE, LOWEST) : __int_as_float(0x7FC00000);
                by[r] = m[r] == UNSET ? 0.0f : ex2(m[r] - now);
                m[r] = now;
              }
              l[r][0] *= by[r];
              l[r][1] *= by[r];
            }
            if (j > 0 && __any_sync(0xffffffffu, by[0] != 1.0f || by[1] != 1.0f)) scale_rows(o_at + rows16, DH, by);
          };
          // log2 of weights times a_t, under no reference
          auto logs = [&](float* x, const float2(&t)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float gx = fmaxf(log2_of(fabsf(t[k].x)), LEAST), gy = fmaxf(log2_of(fabsf(t[k].y)), LEAST);
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                x[4 * k + 2 * r] = fmaf(x[4 * k + 2 * r], t[k].x, gx);
                x[4 * k + 2 * r + 1] = fmaf(x[4 * k + 2 * r + 1], t[k].y, gy);
              }
            }
          };
          auto largest = [&](const float* x, float(&top)[2]) {
#pragma unroll
            for (int e = 0; e < 16; ++e) top[(e >> 1) & 1] = fmaxf(top[(e >> 1) & 1], x[e]);
          };
          // of tokens 32 c on, those that row r sees
          auto sees = [&](int r, int c) -> uint32_t {
            const int t = __shfl_sync(0xffffffffu, hi, (lane >> 2) + 8 * r) - (job.token(i) + 32 * c) + 1;
            return ss.see[s][c] & (t >= 32 ? ~0u : t <= 0 ? 0u : (1u << t) - 1);
          };
          auto seen = [&](const uint32_t(&w)[2], int e) { return (w[(e >> 1) & 1] >> (8 * (e >> 2) + 2 * (lane & 3) + (e & 1))) & 1; };
          // Most tiles, under the references as they are (an item's first one: those that its first 32 tokens ask
          // for, or all where some are hidden).  (32 tokens at a time, the next ones' scores fetched meanwhile; the
          // weights take the scores' place when none was too large.)
          bool plain = !scaled && !bad;
          if (__builtin_expect(!plain || part || j == 0, 0)) {
            tc_wait_ld();
            loaded16(raw[0]);
            if (plain) {
              // scores that their rows do not see: what makes their exponents -inf; an item's first references
              float top[2] = {-INFINITY, -INFINITY};
              const int chunks = part ? 4 : 1;
#pragma unroll 1
              for (int c = 0; c < chunks; ++c) {
                uint32_t w[2] = {~0u, ~0u};
                if (part) w[0] = sees(0, c), w[1] = sees(1, c);
                const bool all = __all_sync(0xffffffffu, (w[0] & w[1]) == ~0u);
                if (all && j > 0) continue;
                float2 t[4];
                ld_rows(s_at + 32 * c, raw[0]);
                factors(c, t);
                tc_wait_ld();
                loaded16(raw[0]);
                if (!all) {
                  const uint32_t mine[2] = {w[0] >> (2 * (lane & 3)), w[1] >> (2 * (lane & 3))};
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    if (!(mine[(e >> 1) & 1] & (1u << (8 * (e >> 2) + (e & 1)))))
                      raw[0][e] = 0xFF800000u ^ (__float_as_uint(e & 1 ? t[e >> 2].y : t[e >> 2].x) & 0x80000000u);
                  put_rows(s_at + 32 * c, raw[0]);
                }
                if (j == 0 && __any_sync(0xffffffffu, w[0] | w[1])) {
                  logs(reinterpret_cast<float*>(raw[0]), t);
                  largest(reinterpret_cast<float*>(raw[0]), top);
                }
              }
              if (j == 0) move(top);
              tc_wait_st();
              ld_rows(s_at, raw[0]);
            }
          }
          if (__builtin_expect(plain, 1)) {
            uint32_t p[4][8];
            float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float* x = reinterpret_cast<float*>(raw[c & 1]);
              float2 t[4];
              factors(c, t);
              tc_wait_ld();
              loaded16(raw[c & 1]);
              if (c < 3) ld_rows(s_at + 32 * (c + 1), raw[(c + 1) & 1]);
              exponents(x, t);
              weights(x, t, sum);
#pragma unroll
              for (int e = 0; e < 16; e += 2) p[c][e / 2] = f16x2_of(x[e], x[e + 1]);
            }
            // (no weight is above its sum; infinity times 0 asks, too)
            plain = __all_sync(0xffffffffu, fmaxf(fmaxf(sum[0][0], sum[0][1]), fmaxf(sum[1][0], sum[1][1])) * most <=
                                                TOO_LARGE);
            if (__builtin_expect(plain, 1)) {
#pragma unroll
              for (int c = 0; c < 4; ++c) st_rows(s_at + 16 * c, p[c]);
#pragma unroll
              for (int r = 0; r < 2; ++r) add2(l[r][0], l[r][1], sum[r][0], sum[r][1]);
            }
          }
          if (__builtin_expect(!plain, 0)) {
            // Any tile: first the references.
            float f[2] = {1.0f, 1.0f};
            if (scaled) {
#pragma unroll
              for (int r = 0; r < 2; ++r) f[r] = __shfl_sync(0xffffffffu, factor, (lane >> 2) + 8 * r);
            }
            auto load = [&](int c, uint32_t(&raw)[16], uint32_t(&w)[2]) {
              ld_rows(s_at + 32 * c, raw);
              w[0] = w[1] = ~0u;
              if (part) w[0] = sees(0, c), w[1] = sees(1, c);
              tc_wait_ld();
              loaded16(raw);
              if (scaled) {
#pragma unroll
                for (int e = 0; e < 16; e += 2)
                  mul2(reinterpret_cast<float*>(raw)[e], reinterpret_cast<float*>(raw)[e + 1], f[(e >> 1) & 1]);
              }
            };
            auto hide = [&](float* x, const uint32_t(&w)[2], float to) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (!seen(w, e)) x[e] = to;
            };
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {  // the references; the weights
              if (c == 4) move(top);
              uint32_t raw[16], w[2], p[8];
              float* x = reinterpret_cast<float*>(raw);
              float2 t[4];
              factors(c & 3, t);
              load(c & 3, raw, w);
              if (c < 4) {
                logs(x, t);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = fmaxf(x[e], LOWEST);  // (scaled ones may be -inf)
              } else {
                exponents(x, t);
              }
              if (part) hide(x, w, -INFINITY);
              if (c < 4) {
                largest(x, top);
                continue;
              }
              weights(x, t, l);
              if (bad) hide(x, w, 0.0f);
#pragma unroll
              for (int e = 0; e < 16; e += 2) p[e / 2] = f16x2_of(x[e], x[e + 1]);
              st_rows(s_at + 16 * (c & 3), p);  // (over scores that were read)
            }
          }
          tc_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.p_full[u]);
      }
      if (!wait(&ss.o_full[u], item & 1, a.status, abort)) return;
      tc_fence_after();
      it += job.count();

      // ---- the piece: the references and sums of the rows, a lane each; then O
      float m_row = UNSET, l_row = 0.0f;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float t = l[r][0] + l[r][1];
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        const float from = __shfl_sync(0xffffffffu, m[r], (lane & 7) * 4);
        t = __shfl_sync(0xffffffffu, t, (lane & 7) * 4);
        if (((lane >> 3) & 1) == r) m_row = from, l_row = t;
      }
      long long to = 0;  // where the piece goes (0: there is no such query)
      if (row >= 0)
        to = reinterpret_cast<long long>(
            (job.begins ? ar.home : ar.over) +
            (job.begins ? ((size_t)(job.g < a.n_prefix ? 0 : ar.max_rows) + row) * a.n_q + head
                        : (size_t)blockIdx.x * (2 * BLOCK) + (mode == TWO_TILES ? 0 : u * BLOCK) + ql) *
                F::PART_LD);
      if (mode != TWO_TILES) {
        if (!idle) {
          // whole pieces through shared memory, eight rows at a time, by a copy for every run of them (stored from
          // registers, or by a copy each, they took 4500 cycles)
          const long long prev = __shfl_up_sync(0xffffffffu, to, 1);
          const bool head_of_run = to && ((lane & 7) == 0 || prev + F::PART_LD * 4 != to);
          const uint32_t ends = __ballot_sync(0xffffffffu, head_of_run || !to);
          uint8_t* out = sm + F::Q_OFF + u * F::Q_BYTES + (4 * half + quad) * (F::Q_BYTES / 8);
          float* mine = reinterpret_cast<float*>(out) + (lane >> 2) * F::PART_LD + 2 * (lane & 3);
          float2 later[DH / 8];
#pragma unroll
          for (int c = 0; c < DH; c += 32) {
            uint32_t o[16];
            ld_rows(o_at + rows16 + c, o);
            tc_wait_ld();
            loaded16(o);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              *reinterpret_cast<uint2*>(mine + 8 + c + 8 * k) = make_uint2(o[4 * k], o[4 * k + 1]);
              later[c / 8 + k] = make_float2(__uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
            }
          }
#pragma unroll 1
          for (int r = 0; r < 2; ++r) {
            if (r > 0) {
              bulk_wait_read();
              __syncwarp();
#pragma unroll
              for (int k = 0; k < DH / 8; ++k) *reinterpret_cast<float2*>(mine + 8 + 8 * k) = later[k];
            }
            if (lane >> 3 == r)
              *reinterpret_cast<float2*>(reinterpret_cast<float*>(out) + (lane & 7) * F::PART_LD) = make_float2(m_row, l_row);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane >> 3 == r && head_of_run) {
              const int first = lane & 7, n = __ffs((ends >> (lane + 1) | 1u << (7 - first)));
              bulk_store(reinterpret_cast<void*>(to), reinterpret_cast<float*>(out) + first * F::PART_LD, n * F::PART_LD * 4);
            }
            bulk_commit();
          }
          bulk_wait_read();
        }
      } else {  // both streams' O in the larger m, half of the dimensions a stream
        auto meet = [&] {  // (a stream's warps read the other one's O, and leave theirs to it)
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ss.merge);
          const bool met = wait(&ss.merge, mc++ & 1, a.status, abort);
          tc_fence_after();
          return met;
        };
        if (lane < 16) ss.ml[u][ql] = make_float2(m_row, l_row);
        if (!meet()) return;
        const float2 x = ss.ml[0][ql], y = ss.ml[1][ql];
        m_row = fmaxf(x.x, y.x);
        // (a NaN stays one)
        const float fx = x.y != x.y ? 1.0f : x.x == UNSET ? 0.0f : ex2(x.x - m_row);
        const float fy = y.y != y.y ? 1.0f : y.x == UNSET ? 0.0f : ex2(y.x - m_row);
        l_row = (fx != 0.0f ? x.y * fx : 0.0f) + (fy != 0.0f ? y.y * fy : 0.0f);
        if (to && u == 0 && lane < 16) *reinterpret_cast<float2*>(to) = make_float2(m_row, l_row);
        if (!idle) {
#pragma unroll 1
          for (int c = u * (DH / 2); c < (u + 1) * (DH / 2); c += 32) {
            uint32_t v[16], z[16];
            ld_rows(o_at - DH * u + rows16 + c, v);
            ld_rows(o_at - DH * u + rows16 + DH + c, z);
            tc_wait_ld();
            loaded16(v);
            loaded16(z);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int of = (lane >> 2) + 8 * r;
              const float gx = __shfl_sync(0xffffffffu, fx, of), gy = __shfl_sync(0xffffffffu, fy, of);
              float* at = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, to, of));
              if (!at) continue;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float o[2];
#pragma unroll
                for (int b = 0; b < 2; ++b)
                  o[b] = (gx != 0.0f ? __uint_as_float(v[4 * k + 2 * r + b]) * gx : 0.0f) +
                         (gy != 0.0f ? __uint_as_float(z[4 * k + 2 * r + b]) * gy : 0.0f);
                *reinterpret_cast<float2*>(at + 8 + c + 8 * k + 2 * (lane & 3)) = make_float2(o[0], o[1]);
              }
            }
          }
        }
        if (!meet()) return;  // (the next item's products go over both)
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss.o_out[u]);
      item_done();
    }
  }();
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // (a softmax thread's rows)
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    mbar_wait(&ss.drain, 0, a.status);  // (whatever ran out before)
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

// Joins the pieces of a (row, head), of its prefix and its own tokens: `team` warps each, which take them in
// turn; 4 dimensions a lane (64 wide: the half warps take every other piece).
constexpr int JOIN_WARPS = 4, MAX_TEAM = 8, AHEAD = 6, TEAM_WARPS = 32, FEW = 3;
__global__ void __launch_bounds__(MAX_TEAM * 32) join_shared_kernel(const __grid_constant__ Args ar, int team_log2) {
  __shared__ float2 ml_of[MAX_TEAM];
  __shared__ float4 num_of[MAX_TEAM][32];
  const SharedArgs& a = ar.a;
  const int team = 1 << team_log2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mate = warp & (team - 1);
  const int r = blockIdx.x, h = (blockIdx.y * (blockDim.x >> 5) + warp) >> team_log2;
  const int dh = a.head_dim, d = 4 * lane & (dh - 1), step = dh == 128 ? 1 : 2, own = dh == 128 ? 0 : lane >> 4;
  const int slice = ar.by_hps(h), ld = dh + 8;
  pdl_trigger();
  pdl_wait();
  const int4 info = h < a.n_q ? reinterpret_cast<const int4*>(ar.info)[r * ar.slices + slice] : make_int4(0, 0, 0, 0);
  // where the pieces are, in floats behind `home` (which `over` is behind): the first ones, of its prefix and of
  // its own tokens, and the others
  const int home = (r * a.n_q + (h < a.n_q ? h : 0)) * ld, own_home = home + ar.max_rows * a.n_q * ld, next = 2 * BLOCK * ld;
  const int over = (int)(ar.over - ar.home) + (h - slice * ar.hps) * ld;
  float m = UNSET, den = 0.0f;
  float4 num = {0.0f, 0.0f, 0.0f, 0.0f};
  auto part_of = [&](const float2& ml) {  // (a piece that saw nothing has no part; a NaN stays one)
    return ml.y != ml.y ? 1.0f : ml.y == 0.0f ? 0.0f : ex2(ml.x - m);
  };
  auto add = [&](float f, const float4& x) {
    num.x = fmaf(f, x.x, num.x), num.y = fmaf(f, x.y, num.y);
    num.z = fmaf(f, x.z, num.z), num.w = fmaf(f, x.w, num.w);
  };
  if (mate == 0) {  // the first ones, fetched before it is known that they are there
    float2 p = *reinterpret_cast<const float2*>(ar.home + home), q = *reinterpret_cast<const float2*>(ar.home + own_home);
    const float4 x = *reinterpret_cast<const float4*>(ar.home + home + 8 + d),
                 y = *reinterpret_cast<const float4*>(ar.home + own_home + 8 + d);
    if (info.x <= 0) p = {UNSET, 0.0f};
    if (info.z <= 0) q = {UNSET, 0.0f};
    m = fmaxf(p.x, q.x);
    const float f = part_of(p), g = part_of(q);
    den = (f != 0.0f ? f * p.y : 0.0f) + (g != 0.0f ? g * q.y : 0.0f);
    if (f != 0.0f && own == 0) add(f, x);
    if (g != 0.0f && own == step - 1) add(g, y);
  }
  // this warp's others (from one lane, so that the compiler knows the loops to be the whole warp's)
  const int of_prefix = max(info.x - 1, 0);
  const int all = __shfl_sync(0xffffffffu, (of_prefix + max(info.z - 1, 0) - mate + team - 1) >> team_log2, 0);
  auto place = [&](int i) { return over + (i < of_prefix ? info.y * ld + i * next : info.w * ld + (i - of_prefix) * next); };
  if (all > 0 && all <= FEW) {
    // (as most are where there are many to join: of 500 instructions a warp half went into the general way)
    float2 ml[FEW];
    float4 x[FEW];
#pragma unroll
    for (int e = 0; e < FEW; ++e) {
      ml[e] = {UNSET, 0.0f};
      if (e >= all) continue;
      const float* at = ar.home + place((e << team_log2) + mate);
      ml[e] = *reinterpret_cast<const float2*>(at);
      if ((e & (step - 1)) == own) x[e] = *reinterpret_cast<const float4*>(at + 8 + d);
    }
    const float old_m = m;
#pragma unroll
    for (int e = 0; e < FEW; ++e) m = fmaxf(m, ml[e].x);
    const float old = old_m == m ? 1.0f : ex2(old_m - m);
    den *= old;
    num.x *= old, num.y *= old, num.z *= old, num.w *= old;
#pragma unroll
    for (int e = 0; e < FEW; ++e) {
      const float f = part_of(ml[e]);
      if (e >= all || f == 0.0f) continue;
      den = fmaf(f, ml[e].y, den);
      if ((e & (step - 1)) == own) add(f, x[e]);
    }
  } else
#pragma unroll 1
  for (int b = 0; b < all; b += 32) {
    const int in = min(32, all - b);
    int at = home;  // a piece a lane
    float2 ml = {UNSET, 0.0f};
    if (lane < in) {
      at = place(((b + lane) << team_log2) + mate);
      ml = *reinterpret_cast<const float2*>(ar.home + at);
    }
    float4 x[AHEAD];
    auto fetch = [&](int i) {  // (those behind the last: the last again, without a part)
#pragma unroll
      for (int e = 0; e < AHEAD; ++e)
        x[e] = *reinterpret_cast<const float4*>(
            ar.home + __shfl_sync(0xffffffffu, at, min(i + own + step * e, in - 1)) + 8 + d);
    };
    fetch(0);
    const float old_m = m;
    m = fmaxf(m, warp_max(ml.x));
    const float old = old_m == m ? 1.0f : ex2(old_m - m), f = part_of(ml);
    den = fmaf(den, old, warp_sum(f != 0.0f ? f * ml.y : 0.0f));
    num.x *= old, num.y *= old, num.z *= old, num.w *= old;
#pragma unroll 1
    for (int i = 0;;) {
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        const int k = i + own + step * e;
        const float g = __shfl_sync(0xffffffffu, f, k & 31);
        if (k < in && g != 0.0f) add(g, x[e]);
      }
      i += step * AHEAD;
      if (i >= in) break;
      fetch(i);
    }
  }
  if (dh == 64) {
    num.x += __shfl_xor_sync(0xffffffffu, num.x, 16), num.y += __shfl_xor_sync(0xffffffffu, num.y, 16);
    num.z += __shfl_xor_sync(0xffffffffu, num.z, 16), num.w += __shfl_xor_sync(0xffffffffu, num.w, 16);
  }
  if (team > 1) {
    if (lane == 0) ml_of[warp] = make_float2(m, den);
    num_of[warp][lane] = num;
    __syncthreads();
    if (mate != 0) return;
    float to = m;
#pragma unroll 1
    for (int w = 1; w < team; ++w) to = fmaxf(to, ml_of[warp + w].x);
    den = 0.0f;
    num = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int w = 0; w < team; ++w) {
      const float2 ml = ml_of[warp + w];
      const float4 x = num_of[warp + w][lane];
      const float f = ml.y != ml.y ? 1.0f : ml.y == 0.0f ? 0.0f : ex2(ml.x - to);
      if (f == 0.0f) continue;
      den = fmaf(f, ml.y, den);
      num.x = fmaf(f, x.x, num.x), num.y = fmaf(f, x.y, num.y);
      num.z = fmaf(f, x.z, num.z), num.w = fmaf(f, x.w, num.w);
    }
    m = to;
  }
  if (h >= a.n_q) return;
  if (m == LOWEST) den = __int_as_float(0x7FC00000);
  // (O was summed with a_t in the scales' place)
  const float inv = den == 0.0f ? 0.0f : 1.0f / (den * (a.scale * (LOG2E / Q_SCALE)));
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
  const size_t piece = (size_t)(head_dim + 8) * 4;  // (Form::PART_LD)
  l.info = 0;
  l.home = ((size_t)max_rows * n_q * 16 + 255) / 256 * 256;  // (as many slices as heads at most)
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
  ar.by_page = Divisor::of(a.kv.block_size);
  ar.by_hps = Divisor::of(ar.hps);
  ar.by_rows = Divisor::of(ar.rows_per);
  ar.by_grid = Divisor::of(sms);
  ar.info = reinterpret_cast<int*>(ws + l.info);
  ar.home = reinterpret_cast<float*>(ws + l.home);
  ar.over = reinterpret_cast<float*>(ws + l.over);
  ar.max_rows = max_rows;
  ar.box = encode_shared_maps(&ar.codes, &ar.scales, a);
  cudaError_t e = a.head_dim == 128
                      ? launch_ex(L, dim3(sms), dim3(THREADS), Form<128>::SMEM_BYTES, attend_shared_kernel<128>, ar)
                      : launch_ex(L, dim3(sms), dim3(THREADS), Form<64>::SMEM_BYTES, attend_shared_kernel<64>, ar);
  // Few queries have many pieces each: teams of warps, as many as the GPU holds at once (up to 20 an SM: eight
  // requests behind 32K tokens 23.1 us instead of 21.9; up to 44: 33 requests of a narrow model 21.2, not 19.8).
  int log2 = 0;
  while ((1 << log2) < MAX_TEAM && (2LL << log2) * a.rows * a.n_q <= TEAM_WARPS * sms) ++log2;
  const int team = 1 << log2, warps = team > JOIN_WARPS ? team : JOIN_WARPS;
  if (e == cudaSuccess)
    e = launch_ex(L, dim3(a.rows, (a.n_q * team + warps - 1) / warps), dim3(warps * 32), 0, join_shared_kernel, ar, log2);
  return e;
}

}  // namespace mono
