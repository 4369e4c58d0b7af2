// What the kernels of the attention over the cache share: how a step's work is cut into pieces,
// found alike by every CTA, and how the pieces are joined.
#pragma once

#include <algorithm>
#include <cfloat>

#include "cache_kernels.h"

namespace mono {
namespace attend {

constexpr int MAX_REQ = 512;
constexpr int MAX_COLS = 96;  // query columns of a row group at most
constexpr float UNSET = -FLT_MAX;  // the reference m_q of a query that has seen no token, below every score
// Token scales above this (and infinite ones) count as NaN.  The reference follows weights times scales,
// so that a weight itself lies as far below 2^-30 as its scale lies above 1: beyond this scale, weights
// that count would be lost to an f32, and their sum with them.
constexpr float SCALE_MAX = 0x1p64f;
// A reference beyond this makes its column NaN: rounded to an f32 it could miss the weight that it is
// made for by more than 2^8, and f16 weights pass 2^16.
constexpr float SCORE_MAX = 0x1p27f;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// How a kernel deals the work out: a tile of `tile` tokens, row groups of rows_per rows (cols query
// columns at most, `heads` per row in a full 128-byte chunk of the record), teams of CTAs; beginning
// another group costs a team as much as `extra` tiles.
struct Shape {
  int tile, cols, heads, rows_per, chunks, teams, extra;
};
inline Shape shape_of(const AttendArgs& a, int tile, int cols, int teams, int extra) {
  Shape s;
  s.tile = tile;
  s.cols = cols;
  s.heads = a.n_q / (a.kv_dim / a.head_dim) * (a.head_dim == 64 && a.kv_dim > 64 ? 2 : 1);
  s.rows_per = std::min(16, cols / s.heads);
  s.chunks = (a.kv_dim + 127) / 128;
  s.teams = teams;
  s.extra = extra;
  return s;
}

// The step as every CTA derives it: per request its rows' largest and smallest position, and
// the units (its row groups times the extra and their tiles) of all requests before it.
struct Plan {
  int* pre;  // [n_req + 1]
  int *pmax, *pmin;
  int* pos;    // [rows] the rows' positions, -1 for those that see nothing, and
  short* req;  // their requests
  short* cnt;  // [n_req] rows that see something; may be null
};

// What the rows of a request see, in tiles: [0, head) and [body, body + tiles - head).
struct Span {
  int hi, lo, head, body, tiles, tile;
  __device__ int token(int i) const { return (i < head ? i : body + i - head) * tile; }
};

__device__ __forceinline__ Span span_of(const AttendArgs& a, const Shape& sh, int pmax, int pmin) {
  const int TT = sh.tile;  // (a power of two)
  Span s;
  s.tile = TT;
  s.hi = pmax;
  const int first = a.causal ? pmin : pmax;
  s.lo = a.window > 0 ? max(0, first - a.window + 1) : 0;
  const long long cap = (long long)a.kv.max_blocks * a.kv.block_size;  // fits 31 bits
  const int last = min(pmax, (int)cap - 1);
  const int lo = min(s.lo, (int)cap);
  const int shift = __ffs(TT) - 1;
  const int b0 = lo >> shift, b1 = last >= lo ? (last >> shift) + 1 : b0;
  s.head = min((int)(((uint32_t)min(min(a.sinks, s.lo), (int)cap) + TT - 1) >> shift), b0);
  s.body = b0;
  s.tiles = s.head + b1 - b0;
  return s;
}

// The cut: a line of W units, the first group's extra left out, over the teams, no team (of those that
// get any) more than one unit above
// another.
struct Cut {
  int teams, each, more;  // team k starts at each * k + min(k, more)
  __device__ Cut(int W, int n) : teams(min(n, W)) {
    each = teams ? W / teams : 0;
    more = W - each * teams;
  }
  __device__ int start(int k) const { return each * k + min(k, more); }
  __device__ int size(int k) const { return k < teams ? each + (k < more ? 1 : 0) : 0; }
  __device__ int team_of(int g) const {
    const int big = (each + 1) * more;
    return g < big ? g / (each + 1) : more + (g - big) / each;
  }
};

// One piece of work of a team: tiles [t0, t0 + n) of a row group of a request.
struct Job {
  int b, group, t0, n;
  Span span;
};

// The items of a team in order, from the place that the plan found for its first unit.
struct Jobs {
  int b, group, at, left;  // at: the unit of the group
};
__device__ __forceinline__ bool next_job(const AttendArgs& a, const Shape& sh, const Plan& p, Jobs& w, Job& it) {
  it.n = 0;
#pragma unroll 1
  while (w.left > 0 && it.n <= 0) {
    it.b = w.b;
    it.group = w.group;
    it.span = span_of(a, sh, p.pmax[w.b], p.pmin[w.b]);
    const int units = it.span.tiles + sh.extra, n = min(units - w.at, w.left);
    it.t0 = max(0, w.at - sh.extra);
    it.n = w.at + n - sh.extra - it.t0;  // (none where only the extra is this team's)
    w.left -= n;
    w.at = 0;
    ++w.group;
    if (w.left > 0 && p.pre[w.b] + w.group * units >= p.pre[w.b + 1]) {
      w.group = 0;
      do ++w.b;
      while (p.pre[w.b + 1] <= p.pre[w.b]);  // (units are left, so there is such a request)
    }
  }
  return it.n > 0;
}

// Where row r's results are: in the pieces of teams [k0, k1] (one: whole, and done), at its place in
// the group; k0 -1: nothing to see.  A team's first slot is for a group that began before it, its
// second for one that begins in it.
struct RowInfo {
  int k0, k1, place;
};

__device__ __forceinline__ float log2_of(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Codes with the NaN ones as zeros.
__device__ __forceinline__ uint32_t without_nan(uint32_t v) {
  const uint32_t nan = (((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
  return v & ~(nan * 0xFFu);
}
__device__ __forceinline__ uint4 without_nan(uint4 v) {
  return make_uint4(without_nan(v.x), without_nan(v.y), without_nan(v.z), without_nan(v.w));
}

// Fills the plan in shared memory and finds the team's first item (every thread of the block calls
// it; the results are behind the caller's next barrier).  Waits for the kernels before.
template <int NT>
__device__ __forceinline__ void derive_plan(const AttendArgs& a, const Shape& sh, const Plan& plan,
                                            int team, bool live, Jobs* start) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#pragma unroll 1
  for (int b = tid; b < a.n_req; b += NT) {
    plan.pmax[b] = -1;
    plan.pmin[b] = 0x7FFFFFFF;
    plan.pre[b + 1] = 0;  // rows so far
  }
  pdl_trigger();
  pdl_wait();
  __syncthreads();
#pragma unroll 1
  for (int r = tid; r < a.rows; r += NT) {
    const int p = a.positions[r], b = a.row_req[r];
    const bool live = p >= 0 && b >= 0 && b < a.n_req;
    plan.pos[r] = live ? p : -1, plan.req[r] = (short)(live ? b : -1);
    if (p < 0) continue;
    if (b < 0 || b >= a.n_req) {
      if (blockIdx.x == 0) atomicOr(a.status, ST_UNMAPPED_PAGE);
      continue;
    }
    atomicMax(&plan.pmax[b], p);
    atomicMin(&plan.pmin[b], p);
    atomicAdd(&plan.pre[b + 1], 1);
  }
  __syncthreads();
  if (warp == 0) {
    int W = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.n_req; b0 += 32) {
      const int b = b0 + lane;
      const int n = b < a.n_req ? plan.pre[b + 1] : 0;
      int u = 0;
      if (plan.cnt && b < a.n_req) plan.cnt[b] = (short)n;
      if (n > 0) {
        const int tiles = span_of(a, sh, plan.pmax[b], plan.pmin[b]).tiles;
        if (tiles > 0) u = (n + sh.rows_per - 1) / sh.rows_per * (tiles + sh.extra);
        if (plan.pmax[b] >= (long long)a.kv.max_blocks * a.kv.block_size && blockIdx.x == 0)
          atomicOr(a.status, ST_UNMAPPED_PAGE);
      }
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, u, o);
        if (lane >= o) u += y;
      }
      if (b < a.n_req) plan.pre[b + 1] = W + u;
      W += __shfl_sync(0xffffffffu, u, 31);
    }
    __syncwarp();
    if (lane == 0) {  // the team's first unit
      plan.pre[0] = 0;
      const Cut cut(max(0, W - sh.extra), sh.teams);
      const int w0 = cut.start(team) + sh.extra;
      Jobs w = {0, 0, 0, live ? cut.size(team) : 0};
      if (w.left > 0) {
        int hi = a.n_req;  // the last request that starts by w0
#pragma unroll 1
        while (hi - w.b > 1) {
          const int mid = (w.b + hi) >> 1;
          if (plan.pre[mid] <= w0) w.b = mid; else hi = mid;
        }
        const int u = w0 - (w.b ? plan.pre[w.b] : 0);
        const int units = span_of(a, sh, plan.pmax[w.b], plan.pmin[w.b]).tiles + sh.extra;
        w.group = u / units;
        w.at = u - w.group * units;
      }
      *start = w;
    }
  }
}

// Row r's place, by a whole warp.
__device__ __forceinline__ RowInfo row_info(const AttendArgs& a, const Shape& sh, const Plan& plan,
                                            int r) {
  const int b = plan.req[r], lane = threadIdx.x & 31;
  RowInfo info = {-1, -1, 0};
  if (b >= 0) {
    int rank = 0;
#pragma unroll 1
    for (int i = lane; i < r; i += 32) rank += plan.req[i] == b;
    rank = __reduce_add_sync(0xffffffffu, rank);
    const int tiles = span_of(a, sh, plan.pmax[b], plan.pmin[b]).tiles;
    const int group = rank / sh.rows_per;
    if (tiles > 0) {
      const Cut cut(plan.pre[a.n_req] - sh.extra, sh.teams);
      const int g0 = plan.pre[b] + group * (tiles + sh.extra);  // (in the cut: without the first extra)
      info = {cut.team_of(g0), cut.team_of(g0 + tiles - 1), rank - group * sh.rows_per};
    }
  }
  return info;
}

// The rows of group `group` of request b, in row order, by a whole warp: their number.
__device__ __forceinline__ int group_rows(const AttendArgs& a, const Shape& sh, const Plan& plan, int b,
                                          int group, int* rows, int* pos) {
  const int first = group * sh.rows_per, lane = threadIdx.x & 31;
  int seen = 0, n = 0;
#pragma unroll 1
  for (int r0 = 0; r0 < a.rows && n < sh.rows_per; r0 += 32) {
    const int r = r0 + lane;
    const bool in = r < a.rows && plan.req[r] == b;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    const int rank = seen + __popc(m & ((1u << lane) - 1)) - first;
    if (in && rank >= 0 && rank < sh.rows_per) rows[rank] = r, pos[rank] = plan.pos[r];
    seen += __popc(m);
    n = max(0, min(sh.rows_per, seen - first));
  }
  return n;
}

// A piece in the workspace: [team][2 slots][chunk][column]: m, l, two words of padding, O.
constexpr int PART_LD = 128 + 4;
struct Pieces {
  float* part;
  RowInfo* rows;  // [rows]
};

cudaError_t launch_join(const Launch&, const AttendArgs&, const Shape&, const Pieces&);
// The records' codes and the 16 bytes behind them as tensor maps with boxes of whole runs of a page, 8
// rows (a swizzle atom) or more, that tiles are made of: the box's tokens; 0 where they cannot be maps.
int encode_cache_maps(CUtensorMap* codes, CUtensorMap* scales, const AttendArgs& a);
// The same with boxes of one latent slice, as they lie.
int encode_shared_maps(CUtensorMap* codes, CUtensorMap* scales, const SharedArgs& a);

}  // namespace attend

// The attention's kernel (k_attend.cu) and the gathering of its weights (k_attend_weights.cu).
cudaError_t attend_tc_prepare();
cudaError_t launch_attend_tc(const Launch&, const AttendArgs&, const attend::Pieces&, int sms);
cudaError_t attend_weights_prepare();
cudaError_t launch_attend_weights(const Launch&, const AttendArgs&, int sms);

}  // namespace mono
