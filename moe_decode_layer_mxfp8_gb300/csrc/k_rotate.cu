// Rotary positions on the way into the cache: a step's latents rotated, quantised and stored as
// records, its queries rotated beside them; and heads rotated on their own, forwards or back.
//
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin     per pair (x1, x2) of a head's rotated dimensions
//   s = max |y| / 448,     code = e4m3(y / s)       over a row's latent
//
// Every product and sum is rounded to f32 by itself (no fused multiply-add), the result once, to the
// output's type or to the codes; cosines and sines come from a table, so that the angles of far
// positions, scaled frequencies and several axes are the caller's.  A thread owns 8 neighbouring
// dimensions of a head: neighbours pair up within them, halves with the lane that owns the others' 8
// (rotated dimensions come in whole runs of 8).  It keeps its cosines and sines over all its heads of a
// row.  A latent is a warp's, so that its largest element is one reduction away from its codes.
#include "cache_kernels.h"

namespace mono {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int AHEAD = 4;       // a thread's loads in flight
constexpr int LATENT_RUNS = 4;  // runs of 8 that a lane has of a latent at most (1024 wide)

template <typename T>
struct Run;  // 8 elements as they lie
template <>
struct Run<float> {
  float4 a, b;
  __device__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]), b = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <>
struct Run<__nv_bfloat16> {
  uint4 a;
  __device__ void get(float (&f)[8]) const { bf16x8_to_f32(a, f); }
  __device__ void set(const float (&f)[8]) {
    a = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Run<__half> {
  uint4 a;
  __device__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = v.x, f[2 * i + 1] = v.y;
    }
  }
  __device__ void set(const float (&f)[8]) {
    a = make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]),
                   pack_f16x2(f[6], f[7]));
  }
};
template <typename T>
__device__ __forceinline__ Run<T> load_run(const T* p) {
  return *reinterpret_cast<const Run<T>*>(p);
}
template <typename T>
__device__ __forceinline__ void store_run(T* p, const Run<T>& v) {
  *reinterpret_cast<Run<T>*>(p) = v;
}

// What a thread knows of its 8 dimensions: whether they are rotated, with which lane's, and a
// position's cosines and sines (interleaved: of its four pairs).
struct Turn {
  bool in, first;  // rotated; the first half of the pairs
  int partner;     // lane
  float c[8], s[8];
  __device__ Turn(const Rope& r, int head_dim) {
    const int lane = threadIdx.x & 31, i = (lane & (head_dim / 8 - 1)) * 8 - r.offset, half = r.dim / 2;
    in = i >= 0 && i < r.dim;  // (dim 0: no rotation)
    first = i < half;
    partner = !in || r.interleaved ? lane : first ? lane + half / 8 : lane - half / 8;
  }
  __device__ __forceinline__ void load(const Rope& r, int head_dim, int position) {
    const int half = r.dim / 2, i = ((threadIdx.x & 31) & (head_dim / 8 - 1)) * 8 - r.offset;
    if (!in) return;
    const float* t = r.table + position * r.stride + (r.interleaved ? i / 2 : first ? i : i - half);
    const int n = r.interleaved ? 1 : 2;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k >= n) break;
      const float4 x = __ldg(reinterpret_cast<const float4*>(t) + k);
      const float4 y = __ldg(reinterpret_cast<const float4*>(t + half) + k);
      c[4 * k] = x.x, c[4 * k + 1] = x.y, c[4 * k + 2] = x.z, c[4 * k + 3] = x.w;
      s[4 * k] = y.x, s[4 * k + 1] = y.y, s[4 * k + 2] = y.z, s[4 * k + 3] = y.w;
    }
    if (r.inverse)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] = -s[k];
  }
  // Every lane of the warp calls it (halves pair up across lanes).
  __device__ __forceinline__ void apply(const Rope& r, float (&f)[8]) const {
    if (r.interleaved) {
      if (!in) return;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = f[2 * k], b = f[2 * k + 1];
        f[2 * k] = __fsub_rn(__fmul_rn(a, c[k]), __fmul_rn(b, s[k]));
        f[2 * k + 1] = __fadd_rn(__fmul_rn(b, c[k]), __fmul_rn(a, s[k]));
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float o = __shfl_sync(0xffffffffu, f[k], partner);
      if (!in) continue;
      const float x = __fmul_rn(f[k], c[k]), y = __fmul_rn(o, s[k]);
      f[k] = first ? __fsub_rn(x, y) : __fadd_rn(x, y);
    }
  }
};

// The position that row r is rotated by, -1 where there is nothing to do: a pad row, or a position
// outside the table.
__device__ __forceinline__ int rope_position(const RotateArgs& a, int r, bool& outside) {
  const int p = a.positions[r];
  int t = p;
  if (p >= 0 && a.rope_positions) t = a.rope_positions[r];
  outside = p >= 0 && a.rope.dim > 0 && (t < 0 || t >= a.rope.positions);
  return p < 0 || outside ? -1 : t;
}

// Heads of rows, or latents where there are any (the first kv_blocks CTAs).  Heads: a thread's 8
// dimensions of a slot of heads; as many rows a CTA as its threads hold.
template <typename T>
__global__ void __launch_bounds__(THREADS) rotate_kernel(const RotateArgs a) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int runs = a.head_dim / 8;
  Turn turn(a.rope, a.head_dim);
  pdl_trigger();
  pdl_wait();
  bool outside;
  if (blockIdx.x < a.kv_blocks) {
    // --------------------------------------------------------------------------- a latent per warp
    const int r = blockIdx.x * WARPS + warp;
    if (r >= a.rows) return;
    const T* kv = static_cast<const T*>(a.kv) + r * a.kv_stride;
    Run<T> v[LATENT_RUNS];
#pragma unroll
    for (int k = 0; k < LATENT_RUNS; ++k)
      if ((lane + 32 * k) * 8 < a.kv_dim) v[k] = load_run(kv + (lane + 32 * k) * 8);
    const int p = a.positions[r], t = rope_position(a, r, outside);
    if (outside && lane == 0) atomicOr(a.status, ST_POSITION);
    if (t < 0) return;
    const int b = a.row_req[r];
    const long long at = b < 0 || b >= a.n_req ? -1 : record_offset(a.cache, b, p);
    turn.load(a.rope, a.head_dim, t);
    float f[LATENT_RUNS][8], amax = 0.0f;
#pragma unroll
    for (int k = 0; k < LATENT_RUNS; ++k) {
      if (32 * 8 * k >= a.kv_dim) break;
      const bool live = (lane + 32 * k) * 8 < a.kv_dim;
      if (live)
        v[k].get(f[k]);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) f[k][e] = 0.0f;
      if (a.rope.dim > 0) turn.apply(a.rope, f[k]);
      if (live)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[k][e]));
    }
    amax = warp_max(amax);
    if (at < 0) {
      if (lane == 0) atomicOr(a.status, ST_UNMAPPED_PAGE);
      return;
    }
    // (0 / 0 otherwise; the smallest f32 over 448 are 0 too)
    float s = amax / 448.0f;
    if (s == 0.0f) s = 1.0f;
    uint8_t* rec = const_cast<uint8_t*>(a.cache.base) + at;
#pragma unroll
    for (int k = 0; k < LATENT_RUNS; ++k) {
      if ((lane + 32 * k) * 8 >= a.kv_dim) break;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = __nv_cvt_float2_to_fp8x2(make_float2(f[k][2 * e] / s, f[k][2 * e + 1] / s),
                                        __NV_SATFINITE, __NV_E4M3);
      *reinterpret_cast<uint2*>(rec + (lane + 32 * k) * 8) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
    if (lane == 0) *reinterpret_cast<float*>(rec + a.kv_dim) = s;
    return;
  }
  // ------------------------------------------------------------------------------------------ heads
  const int slot = tid / runs, slots = THREADS / runs;
  const int across = min(a.heads, slots), rows = slots / across;  // slots of a row, rows of a CTA
  const int j = slot / across, h0 = slot - j * across;
  const long long r = (long long)(blockIdx.x - a.kv_blocks) * rows + j;
  const bool live = j < rows && r < a.rows;
  const T* x = static_cast<const T*>(a.x) + r * a.x_stride + (tid % runs) * 8;
  T* out = static_cast<T*>(a.out) + r * a.out_stride + (tid % runs) * 8;
  // (what is not rotated is where it belongs already in place)
  const bool move = live && (turn.in || x != out);
  Run<T> v[AHEAD];
  auto fetch = [&](int h) {
#pragma unroll
    for (int e = 0; e < AHEAD; ++e)
      if (move && h + e * across < a.heads) v[e] = load_run(x + (h + e * across) * a.head_dim);
  };
  fetch(h0);  // (ahead of the chain from the position to the table)
  const int t = live ? rope_position(a, (int)r, outside) : -1;
  if (live && outside && h0 == 0 && tid % runs == 0) atomicOr(a.status, ST_POSITION);
  if (t >= 0) turn.load(a.rope, a.head_dim, t);
  const bool todo = move && t >= 0;
#pragma unroll 1
  for (int h = h0;; fetch(h)) {  // (as often in all lanes)
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) {
      if (h - h0 + e * across >= a.heads) break;
      float f[8] = {};
      const bool mine = todo && h + e * across < a.heads;
      if (mine) v[e].get(f);
      turn.apply(a.rope, f);
      if (!mine) continue;
      if (turn.in) v[e].set(f);
      store_run(out + (h + e * across) * a.head_dim, v[e]);
    }
    h += across * AHEAD;
    if (h - h0 >= a.heads) break;
  }
}

template <typename T>
cudaError_t launch(const Launch& L, const RotateArgs& a, unsigned grid) {
  return launch_ex(L, dim3(grid), dim3(THREADS), 0, rotate_kernel<T>, a);
}

}  // namespace

cudaError_t launch_rotate(const Launch& L, const RotateArgs& args, int dtype) {
  RotateArgs a = args;
  a.kv_blocks = a.kv ? (unsigned)((a.rows + WARPS - 1) / WARPS) : 0;
  unsigned grid = a.kv_blocks;
  if (a.x) {
    const int slots = THREADS / (a.head_dim / 8), rows = slots / (a.heads < slots ? a.heads : slots);
    grid += (unsigned)((a.rows + rows - 1) / rows);
  }
  return dtype == 0 ? launch<float>(L, a, grid)
         : dtype == 1 ? launch<__nv_bfloat16>(L, a, grid)
                      : launch<__half>(L, a, grid);
}

}  // namespace mono
