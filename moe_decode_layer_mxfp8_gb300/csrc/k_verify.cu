// Verification of drafted tokens against the target's probabilities (rejection sampling).
//
//   draft x_j stands while u_j q_j(x_j) < p_j(x_j); at the first that falls the token is drawn from
//   w = max(p - q, 0), else from w = p in the last row: the smallest v with
//   sum_{i <= v} w_i > r sum_i w_i
//
// A request is a cluster of up to 16 CTAs, each with a run of the vocabulary, cut once more into a
// run per warp and that into blocks: one pass sums the lanes' shares of the blocks (16-byte loads),
// the CTAs exchange their sums through distributed shared memory, and the one warp whose run holds
// the threshold finds the block and reads it again, in order.  A request whose residual is empty
// takes a second pass over p.
// Bound by reading the one row pair that the token is drawn from; small ones by latencies.
// Measured: 192 requests of 3 drafts, 100003 bf16 entries, a quarter of them greedy 30.5 us (77 MB; copy:
// 11 us), 8 of 5 drafts, 131072 f32 entries 10.8 us, 4 of 2 table drafts, 32000 f16 entries 7.6 us.
// Sums decide which token is drawn, so they are carried as pairs of f32 (error-free additions and
// products, and p - q as a pair) for every type: with 10^5 tokens, what an f32 sum of a large entry and
// three small ones loses can move as much as one draw in a thousand by a token.  FP64 runs at a 64th of
// the FP32 rate here, and a search in f64 took 40 us of a CTA's 45.
#include <cuda_fp16.h>

#include <type_traits>

#include "cache_kernels.h"
#include "f32x2.cuh"

namespace mono {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int MAX_CS = 16;
constexpr int BLOCKS = 8;  // of a warp's run

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float positive(float v) { return v > 0.0f ? v : 0.0f; }

// A number as h + l, |l| at most half a unit of h's last place.
struct Pair {
  float h = 0.0f, l = 0.0f;
  __device__ Pair operator-() const {
    Pair r;
    r.h = -h, r.l = -l;
    return r;
  }
  __device__ bool operator<=(Pair b) const { return h < b.h || (h == b.h && l <= b.l); }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const float s = a.h + b.h, v = s - a.h;
  const float e = ((a.h - (s - v)) + (b.h - v)) + (a.l + b.l);
  Pair r;
  r.h = s + e;
  r.l = e - (r.h - s);
  return r;
}
__device__ __forceinline__ Pair operator*(float r, Pair a) {
  const float s = r * a.h, e = fmaf(r, a.h, -s) + r * a.l;
  Pair p;
  p.h = s + e;
  p.l = e - (p.h - s);
  return p;
}
__device__ __forceinline__ Pair shfl(Pair a, int from) {
  Pair r;
  r.h = __shfl_sync(0xffffffffu, a.h, from);
  r.l = __shfl_sync(0xffffffffu, a.l, from);
  return r;
}
__device__ __forceinline__ Pair shfl_xor(Pair a, int o) {
  Pair r;
  r.h = __shfl_xor_sync(0xffffffffu, a.h, o);
  r.l = __shfl_xor_sync(0xffffffffu, a.l, o);
  return r;
}
// Inclusive prefix sums over the lanes.
__device__ __forceinline__ Pair warp_scan(Pair a) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Pair b;
    b.h = __shfl_up_sync(0xffffffffu, a.h, o);
    b.l = __shfl_up_sync(0xffffffffu, a.l, o);
    if (lane >= o) a = b + a;
  }
  return a;
}
// The value before this lane's of a scan.
__device__ __forceinline__ Pair shfl_before(Pair incl) {
  Pair b;
  b.h = __shfl_up_sync(0xffffffffu, incl.h, 1);
  b.l = __shfl_up_sync(0xffffffffu, incl.l, 1);
  if ((threadIdx.x & 31) == 0) b.h = b.l = 0.0f;
  return b;
}
// Sums of f32 in the making, two side by side: s, and the rounding errors of the additions to it.
struct Sum2 {
  float s0 = 0.0f, s1 = 0.0f, e0 = 0.0f, e1 = 0.0f;
  __device__ void add(float x0, float x1) {
    float t0 = s0, t1 = s1;
    add2(t0, t1, x0, x1);
    float b0 = t0, b1 = t1;  // what of x went into t
    sub2(b0, b1, s0, s1);
    float a0 = t0, a1 = t1;  // what of s did
    sub2(a0, a1, b0, b1);
    sub2(s0, s1, a0, a1);
    sub2(x0, x1, b0, b1);
    add2(e0, e1, s0, s1);
    add2(e0, e1, x0, x1);
    s0 = t0;
    s1 = t1;
  }
  __device__ void error(float x0, float x1) { add2(e0, e1, x0, x1); }
  __device__ Pair pair() const {
    Pair a, b;
    a.h = s0 + e0, a.l = e0 - (a.h - s0);
    b.h = s1 + e1, b.l = e1 - (b.h - s1);
    return a + b;
  }
};

template <class T>
struct Row {  // a row of the vocabulary as 16-byte vectors from its first aligned address on
  static constexpr int VEC = 16 / sizeof(T);
  const T* p;
  int lead;  // elements of vector 0 that lie before the row
  __device__ explicit Row(const T* q) : p(q) {
    lead = (int)((reinterpret_cast<uintptr_t>(q) & 15) / sizeof(T));
  }
};

// VEC elements from v0 on, as loaded.
template <class T>
struct Vec {
  static constexpr int VEC = 16 / sizeof(T);
  uint4 x;
  __device__ float operator[](int e) const {  // (e a constant)
    const uint32_t w = e * sizeof(T) / 4 == 0 ? x.x : e * sizeof(T) / 4 == 1 ? x.y
                       : e * sizeof(T) / 4 == 2 ? x.z : x.w;
    if (sizeof(T) == 4) return __uint_as_float(w);
    const unsigned short h = (unsigned short)(e & 1 ? w >> 16 : w & 0xFFFF);
    if (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(h));
    return __uint_as_float((uint32_t)h << 16);
  }
  // The largest of the elements from v0 on that lie in [0, V), a NaN as -infinity.
  __device__ float largest(int v0, int V) const {
    float m;
    if (v0 < 0 || v0 + VEC > V) {
      m = -INFINITY;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (v0 + e >= 0 && v0 + e < V) m = fmaxf(m, (*this)[e]);
    } else if (sizeof(T) == 4) {
      m = fmaxf(fmaxf((*this)[0], (*this)[1]), fmaxf((*this)[2], (*this)[3]));
    } else {
      Vec w = *this;
      w.x.x = max2(max2(x.x, x.y), max2(x.z, x.w));
      m = fmaxf(w[0], w[1]);
    }
    return m == m ? m : -INFINITY;
  }
  // Every element at least the other vector's (a NaN is less than all).
  __device__ Vec above(const Vec& o) const {
    Vec r;
    if (sizeof(T) == 4) {
      r.x = make_uint4(max1(x.x, o.x.x), max1(x.y, o.x.y), max1(x.z, o.x.z), max1(x.w, o.x.w));
    } else {
      r.x = make_uint4(max2(x.x, o.x.x), max2(x.y, o.x.y), max2(x.z, o.x.z), max2(x.w, o.x.w));
    }
    return r;
  }
  // Negative elements and NaN as 0, infinities as the largest number.
  __device__ Vec counted() const {
    Vec r;
    if (sizeof(T) == 4) {
      r.x = make_uint4(most1(max1(x.x, 0)), most1(max1(x.y, 0)), most1(max1(x.z, 0)), most1(max1(x.w, 0)));
    } else {
      r.x = make_uint4(most2(max2(x.x, 0)), most2(max2(x.y, 0)), most2(max2(x.z, 0)), most2(max2(x.w, 0)));
    }
    return r;
  }
  __device__ static uint32_t max1(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  __device__ static uint32_t most1(uint32_t a) {
    return __float_as_uint(fminf(__uint_as_float(a), 3.402823466e38f));
  }
  __device__ static uint32_t most2(uint32_t a) {
    uint32_t r;
    if (std::is_same<T, __half>::value)
      asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x7BFF7BFFu));
    else
      asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x7F7F7F7Fu));
    return r;
  }
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {  // (a NaN loses)
    uint32_t r;
    if (std::is_same<T, __half>::value)
      asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
      asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
// Elements outside [0, V) are 0.
template <class T>
__device__ __forceinline__ Vec<T> load_vec(const T* p, int v0, int V, bool aligned) {
  constexpr int VEC = 16 / sizeof(T);
  Vec<T> r;
  if (aligned && v0 >= 0 && v0 + VEC <= V) {
    r.x = __ldg(reinterpret_cast<const uint4*>(p + v0));
  } else {  // a row's ends, or all of a q out of step with p (192 requests: 61 us instead of 30)
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll 1
    for (int e = 0; e < VEC; ++e) {
      if (v0 + e < 0 || v0 + e >= V) continue;
      uint32_t bits;
      if (sizeof(T) == 4) bits = reinterpret_cast<const uint32_t*>(p)[v0 + e];
      else bits = (uint32_t)reinterpret_cast<const unsigned short*>(p)[v0 + e] << (e & 1 ? 16 : 0);
      const int i = e * (int)sizeof(T) / 4;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i == k) w[k] |= bits;
    }
    r.x = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

template <class T>
struct Draw {  // what a token is drawn from
  static constexpr int VEC = 16 / sizeof(T);
  const T *p, *q;  // q null: nothing is taken off (but `certain`, all of it)
  int V, certain, lead;
  bool q_aligned;
  __device__ Draw(const T* p_, const T* q_, int V_, int certain_)
      : p(p_), q(q_), V(V_), certain(certain_), lead(Row<T>(p_).lead) {
    q_aligned = q && Row<T>(q).lead == lead;
  }
  __device__ int vectors() const { return (V + lead + VEC - 1) / VEC; }
  // The weights of a loaded vector, in two f32: what is counted of p - q, and what rounding took off
  // it (the difference of x >= y >= 0: exactly (x - d) - y).
  __device__ void weights(const Vec<T>& a, const Vec<T>& b, int v0, float (&w)[VEC], float (&err)[VEC]) const {
    if (q) {
      const Vec<T> y = b.counted(), x = a.above(y);  // (nothing for a negative or NaN p)
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        w[e] = x[e], w[e + 1] = x[e + 1];
        sub2(w[e], w[e + 1], y[e], y[e + 1]);
        err[e] = x[e], err[e + 1] = x[e + 1];
        sub2(err[e], err[e + 1], w[e], w[e + 1]);
        sub2(err[e], err[e + 1], y[e], y[e + 1]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = positive(a[e]), err[e] = 0.0f;
      if (certain >= v0 && certain < v0 + VEC) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if (v0 + e != certain) continue;
          const float x = fmaxf(w[e], 1.0f);
          w[e] = x - 1.0f;
          err[e] = (x - w[e]) - 1.0f;
        }
      }
    }
  }
  // The same, added up.
  __device__ void add(const Vec<T>& a, const Vec<T>& b, int v0, Sum2& sum) const {
    float w[VEC], err[VEC];
    weights(a, b, v0, w, err);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      sum.add(w[e], w[e + 1]);
      sum.error(err[e], err[e + 1]);
    }
  }
  __device__ void load(int vec, Vec<T>& a, Vec<T>& b) const {
    const int v0 = vec * VEC - lead;
    a = load_vec(p, v0, V, true);
    if (q) b = load_vec(q, v0, V, q_aligned);
  }
};

// x y < z, exactly.
__device__ __forceinline__ bool product_below(float x, float y, float z) {
  const float s = x * y;
  if (!(s > 1.0e-30f && s < 1.0e30f)) return (double)x * (double)y < (double)z;
  return s < z || (s == z && fmaf(x, y, -s) < 0.0f);
}
// The last lane of those below n whose weight is positive and whose prefix is at most x.
__device__ __forceinline__ int lane_of(Pair before, Pair own, int n, Pair x) {
  const int lane = threadIdx.x & 31;
  const bool some = lane < n && own.h > 0.0f;
  const uint32_t below = __ballot_sync(0xffffffffu, some && before <= x);
  const uint32_t any = __ballot_sync(0xffffffffu, some);
  return below ? 31 - __clz(below) : __ffs(any) - 1;
}
__device__ __forceinline__ uint64_t ld_dsmem_u64(uint32_t cluster_addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Larger value first, then lower index: as an integer that orders so (values by their bits made
// monotonic; a NaN as -inf).
__device__ __forceinline__ uint64_t arg_key(float v, int i) {
  if (v != v) v = -INFINITY;
  uint32_t b = __float_as_uint(v + 0.0f);
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((uint64_t)b << 32) | (uint32_t)~i;
}

template <class T>
__global__ void __launch_bounds__(THREADS, 3) verify_kernel(VerifyArgs a, int cs) {
  constexpr int VEC = 16 / sizeof(T);
  // sums: of the lanes' shares of blocks, of warps' runs, of the CTA's (for two passes)
  __shared__ Pair s_block[WARPS][BLOCKS][32], s_warp[WARPS], s_cta[2];
  __shared__ uint64_t s_best[2][WARPS + 1];   // first maxima, by the row's parity
  __shared__ int s_row, s_tok;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x / cs, rank = blockIdx.x - b * cs;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, V = a.vocab;
  const int r0 = min(max(a.row_start[b], 0), a.rows);
  const int r1 = min(max(a.row_start[b + 1], r0), a.rows);
  if (r1 == r0) {
    if (tid == 0 && rank == 0) a.accepted[b] = 0;
    return;  // (the whole cluster)
  }
  const T* tp = reinterpret_cast<const T*>(a.target);
  const T* dp = reinterpret_cast<const T*>(a.draft);
  const bool greedy = a.greedy && a.greedy[b] != 0;
  const int runs = cs * WARPS, run = rank * WARPS + warp;
  int j = r0, tok = -1;
  bool writer = false;  // this CTA knows the token
  if (greedy) {
    // row by row: the first maximum of the CTAs' runs, exchanged by the cluster
    for (;; ++j) {
      const T* p = tp + (long long)j * a.target_stride;
      const Draw<T> d(p, nullptr, V, -1);
      const int nv = (d.vectors() + runs - 1) / runs, first = run * nv;
      const int last = min(first + nv, d.vectors());
      // a lane's first largest vector, kept as it was loaded
      constexpr int U = 10;  // (loaded at a time)
      float top = -INFINITY;
      int at = -1;
      Vec<T> kept = {};
#pragma unroll 1
      for (int k0 = first + lane; k0 < last; k0 += 32 * U) {
        Vec<T> f[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k0 + 32 * u < last) f[u] = load_vec(p, (k0 + 32 * u) * VEC - d.lead, V, true);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (k0 + 32 * u >= last) break;
          const float m = f[u].largest((k0 + 32 * u) * VEC - d.lead, V);
          if (at < 0 || m > top) top = m, at = k0 + 32 * u, kept = f[u];
        }
      }
      const int v0 = at * VEC - d.lead;
      if (at >= 0) {
#pragma unroll
        for (int e = VEC - 1; e >= 0; --e) {
          const float y = kept[e];
          if (v0 + e >= 0 && v0 + e < V && ((y != y && top == -INFINITY) || y == top)) at = v0 + e;
        }
      }
      uint64_t best = at >= 0 ? arg_key(top, at) : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
      uint64_t* sb = s_best[(j - r0) & 1];
      if (lane == 0) sb[warp] = best;
      __syncthreads();
      if (tid == 0) {
#pragma unroll 1
        for (int w = 1; w < WARPS; ++w) best = max(best, sb[w]);
        sb[WARPS] = best;
      }
      if (cs > 1) cluster_sync_all(); else __syncthreads();
      best = lane < cs ? ld_dsmem_u64(mapa_shared(smem_u32(&sb[WARPS]), lane)) : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
      tok = (int)~(uint32_t)best;
      if (j == r1 - 1 || a.draft_tokens[j] != tok) break;
    }
    writer = rank == 0;
    if (cs > 1) cluster_sync_all();  // (nobody leaves while its shared memory is read)
  } else {
    // the first draft that falls: a lane per draft
    if (warp == 0) {
      int fall = r1 - 1;
      for (int k0 = r0; k0 < r1 - 1; k0 += 32) {
        const int k = k0 + lane;
        bool falls = false;
        if (k < r1 - 1) {
          const int x = a.draft_tokens[k];
          falls = true;
          if (x >= 0 && x < V) {
            const float px = positive(as_f32(tp[(long long)k * a.target_stride + x]));
            const float qx = dp ? positive(as_f32(dp[(long long)k * a.draft_stride + x])) : 1.0f;
            falls = !product_below(a.u[k], qx, px);
          }
        }
        const uint32_t m = __ballot_sync(0xffffffffu, falls);
        if (m) {
          fall = k0 + __ffs(m) - 1;
          break;
        }
      }
      if (lane == 0) s_row = fall;
    }
    __syncthreads();
    j = s_row;
    const T* p = tp + (long long)j * a.target_stride;
    const int x = a.draft_tokens[j];
    // (in [0, 1), whatever comes)
    const float r = fminf(fmaxf(a.r[b], 0.0f), 1.0f - 1.0f / 16777216.0f);
    int pass = j == r1 - 1 ? 1 : 0;  // 0: the residual, 1: the row itself
#pragma unroll 1
    for (;; ++pass) {
      const Draw<T> d(p, pass == 0 && dp ? dp + (long long)j * a.draft_stride : nullptr, V,
                      pass == 0 && !dp ? x : -1);
      const int nv = (d.vectors() + runs - 1) / runs, first = run * nv;
      const int last = min(first + nv, d.vectors());
      // rounds of a vector per lane, `per` of them a block
      // loaded at a time (192 requests of 100003 bf16 entries 30.5 us; four at a time 31.6)
      constexpr int U = 2;
      const int rounds = max(1, (last - first + 31) / 32);
      const int per = ((rounds + BLOCKS - 1) / BLOCKS + U - 1) / U * U;
      Pair mine;
      int blk = 0;
#pragma unroll 1
      for (int q = 0; q < rounds; q += per, ++blk) {
        Sum2 sum;
#pragma unroll 1
        for (int i = q; i < min(q + per, rounds); i += U) {
          Vec<T> fa[U], fb[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int k = first + (i + u) * 32 + lane;
            if (i + u < q + per && k < last) d.load(k, fa[u], fb[u]);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int k = first + (i + u) * 32 + lane;
            if (i + u < q + per && k < last) {
              d.add(fa[u], fb[u], k * VEC - d.lead, sum);
            }
          }
        }
        const Pair t = sum.pair();
        s_block[warp][blk][lane] = t;
        mine = mine + t;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mine = mine + shfl_xor(mine, o);
      if (lane == 0) s_warp[warp] = mine;
      __syncthreads();
      Pair own = lane < WARPS ? s_warp[lane] : Pair(), incl = warp_scan(own);
      if (tid == WARPS - 1) s_cta[pass] = incl;
      if (cs > 1) cluster_sync_all(); else __syncthreads();
      // every warp: the CTAs' sums, their total, and whose run holds the threshold
      Pair cta;
      if (lane < cs) {
        const uint64_t v = ld_dsmem_u64(mapa_shared(smem_u32(&s_cta[pass]), lane));
        cta.h = __uint_as_float((uint32_t)v);
        cta.l = __uint_as_float((uint32_t)(v >> 32));
      }
      const Pair to = warp_scan(cta);
      const Pair total = shfl(to, 31);
      const bool sound = total.h > 0.0f && total.h <= 3.4e38f;  // (else there is nothing to draw from)
      if (!sound && pass == 0) continue;
      const Pair want = r * total;
      const int owner = sound ? lane_of(shfl_before(to), cta, cs, want) : 0;
      writer = owner == rank;
      if (tid == 0) s_tok = -1;
      __syncthreads();
      if (sound && writer) {
        const Pair in_cta = want + -shfl(shfl_before(to), owner);
        const Pair before = shfl_before(incl);
        const int w = lane_of(before, own, WARPS, in_cta);
        if (warp == w) {
          const Pair in_warp = in_cta + -shfl(before, w);
          // the blocks' sums, four lanes each, then a lane each
          static_assert(BLOCKS * 4 == 32, "a quarter of a block's lanes per lane");
          own = Pair();
          if (lane / 4 < blk)
#pragma unroll 1
            for (int i = 0; i < 8; ++i) own = own + s_block[warp][lane / 4][(lane & 3) * 8 + i];
          own = own + shfl_xor(own, 1);
          own = own + shfl_xor(own, 2);
          own = shfl(own, lane * 4 & 31);
          if (lane >= blk) own = Pair();
          const Pair b0 = shfl_before(warp_scan(own));
          const int bl = lane_of(b0, own, blk, in_warp);
          Pair goal = in_warp + -shfl(b0, bl);
          // the round that passes the goal, in order; or else (should roundings leave the sum at the
          // threshold) the block's last with a weight
          int at = -1, i = bl * per;
          bool found = false;
          const int end = min((bl + 1) * per, rounds);
          Pair incl_run;
          float wt[VEC], err[VEC];
          auto weigh = [&](int i) {
            const int k = first + i * 32 + lane;
            Vec<T> fa, fb;
            Sum2 sum;
            if (k < last) {
              d.load(k, fa, fb);
              d.weights(fa, fb, k * VEC - d.lead, wt, err);
            } else {
#pragma unroll
              for (int e = 0; e < VEC; ++e) wt[e] = err[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
              sum.add(wt[e], wt[e + 1]);
              sum.error(err[e], err[e + 1]);
            }
            return sum.pair();
          };
          int pick = -1;
#pragma unroll 1
          for (bool again = false;;) {
            const Pair share = weigh(i);
            incl_run = warp_scan(share);
            const uint32_t some = __ballot_sync(0xffffffffu, share.h > 0.0f);
            const uint32_t past = __ballot_sync(0xffffffffu, share.h > 0.0f && !(incl_run <= goal));
            if (again) {
              pick = some ? 31 - __clz(some) : -1;
              break;
            }
            if (past) {
              found = true;
              pick = __ffs(past) - 1;
              break;
            }
            if (some) at = i;
            if (++i < end) {
              goal = goal + -shfl(incl_run, 31);
              continue;
            }
            if (at < 0) break;
            again = true;
            i = at;
          }
          // the last element that begins by the goal (of all, without one).  Where the goal is a border,
          // the sums of lanes without a weight may pass it by a rounding: then the lane's first
          Pair begin = shfl_before(incl_run);
          int hit = -1;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            if (wt[e] > 0.0f && (!found || hit < 0 || begin <= goal)) hit = (first + i * 32 + lane) * VEC - d.lead + e;
            Pair x;
            x.h = wt[e], x.l = err[e];
            begin = begin + x;
          }
          hit = __shfl_sync(0xffffffffu, hit, max(pick, 0));
          if (lane == 0) s_tok = pick >= 0 ? hit : -1;
        }
      }
      __syncthreads();
      tok = s_tok;
      if (cs > 1) cluster_sync_all();  // (nobody leaves while its shared memory is read)
      break;
    }
  }
  if (writer) {
    if (tid == 0) a.accepted[b] = j - r0;
#pragma unroll 1
    for (int i = r0 + tid; i < r1; i += THREADS)
      a.tokens[i] = i < j ? a.draft_tokens[i] : i == j ? tok : -1;
  }
}

template <class T>
cudaError_t launch(const Launch& L, const VerifyArgs& a, int sms) {
  // as many CTAs a request as give the GPU three an SM (four, with fewer registers each: 36 us instead of
  // 29 for 192 requests), at least one vector a lane (two and four: 8.5 and 9.4 us instead of 7.4 for 4
  // requests of 32000)
  int cs = 1;
  const int vectors = (a.vocab + Row<T>::VEC - 1) / Row<T>::VEC;
  while (cs < MAX_CS && (long long)a.n_req * cs * 2 <= 3 * sms && cs * 2 * THREADS <= vectors) cs *= 2;
  cudaError_t e = cudaSuccess;
  if (cs > 8) e = cudaFuncSetAttribute(verify_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_req * cs);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = L.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a, cs);
}

}  // namespace

cudaError_t launch_verify(const Launch& L, const VerifyArgs& a, int dtype, int sms) {
  if (dtype == 0) return launch<float>(L, a, sms);
  if (dtype == 1) return launch<__nv_bfloat16>(L, a, sms);
  return launch<__half>(L, a, sms);
}

}  // namespace mono
