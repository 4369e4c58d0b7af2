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
// row: the fewer threads share a row, the fewer chains from a position to the table's row there are to
// wait for, as long as the threads fill the GPU.  A latent has the threads of its runs: halving its part
// of a warp, or whole warps, its largest element one reduction away from its codes.
//
// Bound by DRAM where steps are large, by latency (launch, position, table) where they are small.  Measured
// in a graph: one request's token 2.6 us; 48 rows of 64 heads 2.8, back 2.7; 20001 rows of 16 heads of 64 in
// f16 15.5 (5.4 TB/s of 6.8 measured), bf16 15.2, f32 26.0 (6.4 TB/s); 22K prompt rows of 64 heads of 128 with
// their latents in bf16 134 (5.7 TB/s), f32 228 (6.6 TB/s), their heads alone 109 (6.7 TB/s); 14K narrow f32
// latents 5.2 (a warp each: 8.5), with 16 heads of queries 21.7 (6.0 TB/s; bf16 14.0).  With CTAs of 256 threads
// the prompts take 138 and 232.
#include "cache_kernels.h"

namespace mono {
namespace {

constexpr int THREADS = 128, WARPS = THREADS / 32;
constexpr int AHEAD = 4;  // a thread's loads in flight (2: prompts 142 us, 48 rows 3.2; 8: prompts 142)
// Heads of a thread where there are rows enough to fill the GPU (20001 rows of 16 heads 15.5 us; 1: 34.3, 4: 16.7,
// 16: 17.6), which takes so many threads an SM (512 and 2048: no change where rows are many).
constexpr int PER = 8, FULL = 1024;
static_assert(WARPS * 256 >= 1024, "the widest latent a CTA");

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
// The same of what is read or written once: heads (20001 rows of 16 heads 15.5 us, with plain loads and stores 17.0;
// narrow f32 prompts with queries 21.7 and 24.4).
template <typename T>
__device__ __forceinline__ Run<T> load_once(const T* p) {
  Run<T> v;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(v) / 16); ++i)
    reinterpret_cast<uint4*>(&v)[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  return v;
}
template <typename T>
__device__ __forceinline__ void store_run(T* p, const Run<T>& v) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(v) / 16); ++i)
    __stcs(reinterpret_cast<uint4*>(p) + i, reinterpret_cast<const uint4*>(&v)[i]);
}

// What a thread knows of its 8 dimensions: whether they are rotated, with which lane's, and a position's
// cosines and sines, a sine's sign that of its product (y1 takes x2 times -sin).
struct Turn {
  bool in, first;  // rotated; the first half of the pairs
  int partner;     // lane
  float c[8], s[8];
  __device__ Turn(const Rope& r, int head_dim) {
    const int lane = threadIdx.x & 31, i = (lane & (head_dim / 8 - 1)) * 8 - r.offset, half = r.dim / 2;
    in = i >= 0 && i < r.dim;  // (dim 0: no rotation)
    first = i < half;
    partner = !in || r.interleaved ? lane : first ? lane + half / 8 : lane - half / 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) c[k] = s[k] = 0.0f;
  }
  __device__ __forceinline__ void load(const Rope& r, int head_dim, int position) {
    const int half = r.dim / 2, i = ((threadIdx.x & 31) & (head_dim / 8 - 1)) * 8 - r.offset;
    if (!in) return;
    const float4* t = reinterpret_cast<const float4*>(
        r.table + position * r.stride + (r.interleaved ? i / 2 : first ? i : i - half));
    const float4 x = __ldg(t), y = __ldg(t + half / 4);
    const uint32_t turned = r.inverse ? 0x80000000u : 0u;
    auto signed_by = [](float v, uint32_t sign) { return __uint_as_float(__float_as_uint(v) ^ sign); };
    const float cx[4] = {x.x, x.y, x.z, x.w}, sx[4] = {y.x, y.y, y.z, y.w};
    if (r.interleaved) {
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = cx[k / 2], s[k] = signed_by(sx[k / 2], turned ^ (k & 1 ? 0u : 0x80000000u));
    } else {
      const float4 z = __ldg(t + 1), w = __ldg(t + half / 4 + 1);
      const float cz[4] = {z.x, z.y, z.z, z.w}, sz[4] = {w.x, w.y, w.z, w.w};
      const uint32_t sign = turned ^ (first ? 0x80000000u : 0u);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        c[k] = cx[k], c[k + 4] = cz[k];
        s[k] = signed_by(sx[k], sign), s[k + 4] = signed_by(sz[k], sign);
      }
    }
  }
  // Every lane of the warp calls it (halves pair up across lanes); the result is one where `in`.
  __device__ __forceinline__ void apply(const Rope& r, float (&f)[8]) const {
    float o[8];
    if (r.interleaved) {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = f[k ^ 1];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = __shfl_sync(0xffffffffu, f[k], partner);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __fadd_rn(__fmul_rn(f[k], c[k]), __fmul_rn(o[k], s[k]));
  }
};

// Row r's position and rotary position, fetched at once.
__device__ __forceinline__ int2 row_positions(const RotateArgs& a, int r) {
  const int p = a.positions[r];
  return make_int2(p, a.rope_positions ? a.rope_positions[r] : p);
}
// The position that a row is rotated by, -1 where there is nothing to do: a pad row, or a position outside
// the table.
__device__ __forceinline__ int rope_position(const RotateArgs& a, int p, int t, bool& outside) {
  outside = p >= 0 && a.rope.dim > 0 && (t < 0 || t >= a.rope.positions);
  return p < 0 || outside ? -1 : t;
}

// Heads of rows, or latents where there are any (kv_blocks CTAs among the others, so that their chains of latencies
// and the heads' bandwidth overlap: 22K prompt rows 134 us, 140 with the latents first; in f32 228 and 246; without
// heads all, in fewer registers).  Heads: a thread's 8 dimensions of a slot of heads; as many rows a CTA as its threads hold.
template <typename T, bool HEADS>
__global__ void __launch_bounds__(THREADS) rotate_kernel(const RotateArgs a) {
  // (the warp, and what loops depend on, from one lane: the compiler then knows the shuffles to be whole warps')
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int runs = a.head_dim / 8;
  Turn turn(a.rope, a.head_dim);
  pdl_trigger();
  pdl_wait();
  bool outside;
  // latents' CTAs are every 2^apart-th one, until there are no more
  const unsigned nth = blockIdx.x >> a.apart;
  if (!HEADS || (nth < a.kv_blocks && nth << a.apart == blockIdx.x)) {
    // -------------------------------------------------------------------- latents, 8 elements a thread
    __shared__ float largest[WARPS];
    const int of = tid / a.span, i = (tid - of * a.span) * 8, r = (HEADS ? nth : blockIdx.x) * (THREADS / a.span) + of;
    const bool live = of < THREADS / a.span && r < a.rows && i < a.kv_dim;
    Run<T> v;
    if (live) v = load_run(static_cast<const T*>(a.kv) + r * a.kv_stride + i);
    int2 at_row = {-1, -1};
    int b = -1;
    if (live) at_row = row_positions(a, r), b = a.row_req[r];
    const int p = at_row.x, t = rope_position(a, p, at_row.y, outside);
    if (live && outside && i == 0) atomicOr(a.status, ST_POSITION);
    const long long at = t < 0 || b < 0 || b >= a.n_req ? -1 : record_offset(a.cache, b, p);
    if (t >= 0) turn.load(a.rope, a.head_dim, t);
    float f[8] = {}, amax = 0.0f;
    if (live) v.get(f);
    if (a.rope.dim > 0) {
      turn.apply(a.rope, f);
      if (!turn.in && live) v.get(f);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(0xffffffffu, amax, o);
      if (o < a.span) amax = fmaxf(amax, x);
    }
    if (a.span > 32) {
      if (lane == 0) largest[warp] = amax;
      __syncthreads();
      if (t < 0) return;
#pragma unroll 1
      for (int w = 0; w < a.span / 32; ++w) amax = fmaxf(amax, largest[of * (a.span / 32) + w]);
    }
    if (t < 0) return;
    if (at < 0) {
      if (i == 0) atomicOr(a.status, ST_UNMAPPED_PAGE);
      return;
    }
    // (0 / 0 otherwise; the smallest f32 over 448 are 0 too)
    float s = amax / 448.0f;
    if (s == 0.0f) s = 1.0f;
    uint8_t* rec = const_cast<uint8_t*>(a.cache.base) + at;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * e] / s, f[2 * e + 1] / s), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint2*>(rec + i) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    if (i == 0) *reinterpret_cast<float*>(rec + a.kv_dim) = s;
    return;
  }
  // ------------------------------------------------------------------------------------------ heads
  const int slot = tid / runs, slots = THREADS / runs;
  const int across = a.across, rows = slots / across;  // slots of a row, rows of a CTA
  const int j = slot / across, h0 = slot - j * across;
  const long long r = (long long)(blockIdx.x - (nth < a.kv_blocks ? nth + 1 : a.kv_blocks)) * rows + j;
  const bool live = j < rows && r < a.rows;
  const T* x = static_cast<const T*>(a.x) + r * a.x_stride + (tid % runs) * 8;
  T* out = static_cast<T*>(a.out) + r * a.out_stride + (tid % runs) * 8;
  // (what is not rotated is where it belongs already in place)
  const bool move = live && (turn.in || x != out);
  Run<T> v[AHEAD];
  auto fetch = [&](int h) {
#pragma unroll
    for (int e = 0; e < AHEAD; ++e)
      if (move && h + e * across < a.heads) v[e] = load_once(x + (h + e * across) * a.head_dim);
  };
  int2 at_row = {-1, -1};
  if (live) at_row = row_positions(a, (int)r);
  fetch(h0);  // (ahead of the chain from the position to the table)
  const int t = rope_position(a, at_row.x, at_row.y, outside);
  if (live && outside && h0 == 0 && tid % runs == 0) atomicOr(a.status, ST_POSITION);
  if (t >= 0) turn.load(a.rope, a.head_dim, t);
  const bool todo = move && t >= 0;
#pragma unroll 1
  for (int k = 0;;) {  // (as often in all lanes)
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) {
      if (k + e * across >= a.heads) break;
      const int h = h0 + k + e * across;
      float f[8] = {};
      const bool mine = todo && h < a.heads;
      if (mine) v[e].get(f);
      turn.apply(a.rope, f);
      if (!mine) continue;
      if (turn.in) v[e].set(f);
      store_run(out + h * a.head_dim, v[e]);
    }
    k += across * AHEAD;
    if (k >= a.heads) break;
    fetch(h0 + k);
  }
}

template <typename T>
cudaError_t launch(const Launch& L, const RotateArgs& a, unsigned grid) {
  return launch_ex(L, dim3(grid), dim3(THREADS), 0, a.x ? rotate_kernel<T, true> : rotate_kernel<T, false>, a);
}

}  // namespace

cudaError_t launch_rotate(const Launch& L, const RotateArgs& args, int dtype, int sms) {
  RotateArgs a = args;
  a.span = 32, a.kv_blocks = 0, a.apart = 0;
  if (a.kv) {
    // a latent's threads: whole warps, or the least part of one that halving leads to
    if (a.kv_dim > 256) a.span = (a.kv_dim + 255) / 256 * 32;
    while (a.span <= 32 && a.span > 1 && a.span / 2 * 8 >= a.kv_dim) a.span /= 2;
    a.kv_blocks = (unsigned)((a.rows + THREADS / a.span - 1) / (THREADS / a.span));
  }
  unsigned grid = a.kv_blocks;
  if (a.x) {
    const int slots = THREADS / (a.head_dim / 8);
    int across = a.heads < slots ? a.heads : slots;
    while (across > 1 && (a.heads + across - 1) / across < PER &&
           (long long)a.rows * across * (a.head_dim / 8) > (long long)FULL * sms)
      across /= 2;
    a.across = across;
    const int rows = slots / across;
    grid += (unsigned)((a.rows + rows - 1) / rows);
    while (a.kv_blocks && (unsigned long long)a.kv_blocks << (a.apart + 1) <= grid) ++a.apart;
  }
  return dtype == 0 ? launch<float>(L, a, grid)
         : dtype == 1 ? launch<__nv_bfloat16>(L, a, grid)
                      : launch<__half>(L, a, grid);
}

}  // namespace mono
