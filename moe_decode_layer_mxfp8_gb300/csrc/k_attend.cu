// Attention of a step's rows over the paged fp8 cache, split over the context.
//
// CTA = (row, latent slice, split): the split's tokens in tiles of 128, a thread per token for
// the scores and a thread per output dimension for the weighted sum, a running maximum and sum
// per head; the splits of a row are joined by a second kernel.  All arithmetic in f32.
#include "cache_kernels.h"

namespace mono {
namespace {

constexpr int TT = 128;      // tokens per tile = threads
constexpr int SPLITS = 16;
constexpr int MAXH = 16;     // heads per slice at most
constexpr int PART_HEAD = 4;

__device__ __forceinline__ int row_hi(const AttendArgs& a, int r) {
  int hi = a.positions[r];
  if (!a.causal)
    for (int i = 0; i < a.rows; ++i)
      if (a.row_req[i] == a.row_req[r]) hi = max(hi, a.positions[i]);
  return hi;
}

// Visible token i of a row: the sinks below the window first, then the window.
struct Seen {
  int lo, hi, ns;
  __device__ int count() const { return ns + hi + 1 - lo; }
  __device__ int token(int i) const { return i < ns ? i : lo + i - ns; }
};
__device__ __forceinline__ Seen seen_of(const AttendArgs& a, int hi) {
  Seen s;
  s.hi = hi;
  s.lo = a.window > 0 ? max(0, hi - a.window + 1) : 0;
  s.ns = min(a.sinks, s.lo);
  return s;
}

template <int DH>
__global__ void __launch_bounds__(TT) attend_kernel(AttendArgs a) {
  __shared__ float qs[MAXH][DH], ps[MAXH][TT], red[32];
  __shared__ __align__(16) uint8_t ks[TT][DH];
  pdl_wait();
  const int r = blockIdx.x, g = blockIdx.y, sp = blockIdx.z;
  const int G = a.kv_dim / DH, hpg = a.n_q / G, tid = threadIdx.x;
  const int b = a.row_req[r];
  float m[MAXH], l[MAXH], acc[MAXH];
  for (int h = 0; h < MAXH; ++h) m[h] = -INFINITY, l[h] = 0.0f, acc[h] = 0.0f;
  const bool live = a.positions[r] >= 0 && b >= 0 && b < a.n_req;
  if (live) {
    for (int i = tid; i < hpg * DH; i += TT)
      qs[i / DH][i % DH] = __bfloat162float(a.q[r * a.q_stride + (g * hpg) * DH + i]) * a.scale;
    const Seen s = seen_of(a, row_hi(a, r));
    const int n = s.count(), per = (n + SPLITS - 1) / SPLITS;
    const int i1 = min(n, (sp + 1) * per);
    for (int i0 = sp * per; i0 < i1; i0 += TT) {
      __syncthreads();
      const int i = i0 + tid;
      long long off = -1;
      if (i < i1) {
        off = record_offset(a.kv, b, s.token(i));
        if (off < 0) atomicOr(a.status, ST_UNMAPPED_PAGE);
      }
      float sc = 0.0f;
      uint4 v[DH / 16];
      for (int c = 0; c < DH / 16; ++c) v[c] = make_uint4(0, 0, 0, 0);
      if (off >= 0) {
        sc = *reinterpret_cast<const float*>(a.kv.base + off + a.kv_dim);
        for (int c = 0; c < DH / 16; ++c)
          v[c] = *reinterpret_cast<const uint4*>(a.kv.base + off + g * DH + 16 * c);
      }
      for (int c = 0; c < DH / 16; ++c) *reinterpret_cast<uint4*>(&ks[tid][16 * c]) = v[c];
      for (int h = 0; h < hpg; ++h) {
        float d = 0.0f;
        for (int c = 0; c < DH / 16; ++c) {
          const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
          for (int j = 0; j < 4; ++j) {
            uint32_t f[2];
            e4m3x4_to_f16x4(w[j], f);
            for (int e = 0; e < 2; ++e) {
              const float2 x = __half22float2(*reinterpret_cast<__half2*>(&f[e]));
              d = fmaf(x.x, qs[h][16 * c + 4 * j + 2 * e], d);
              d = fmaf(x.y, qs[h][16 * c + 4 * j + 2 * e + 1], d);
            }
          }
        }
        const float score = off >= 0 ? d * sc : -INFINITY;
        const float mt = fmaxf(block_max(score, red), m[h]);
        const float p = off >= 0 ? expf(score - mt) : 0.0f;
        const float f = m[h] == -INFINITY ? 0.0f : expf(m[h] - mt);
        l[h] = l[h] * f + block_sum(p, red);
        acc[h] *= f;
        if (mt > -INFINITY) m[h] = mt;
        ps[h][tid] = off >= 0 ? p * sc : 0.0f;
      }
      __syncthreads();
      if (tid < DH)
        for (int t = 0; t < TT; ++t) {
          uint32_t f[2];
          e4m3x4_to_f16x4(ks[t][tid], f);
          const float x = __half2float(__ushort_as_half((unsigned short)(f[0] & 0xFFFF)));
          for (int h = 0; h < hpg; ++h) acc[h] = fmaf(ps[h][t], x, acc[h]);
        }
    }
  }
  for (int h = 0; h < hpg; ++h) {
    float* part = a.part + (((size_t)r * a.n_q + g * hpg + h) * SPLITS + sp) * (DH + PART_HEAD);
    if (tid == 0) part[0] = m[h], part[1] = l[h];
    if (tid < DH) part[PART_HEAD + tid] = acc[h];
  }
}

template <int DH>
__global__ void __launch_bounds__(DH) attend_join_kernel(AttendArgs a) {
  pdl_wait();
  const int r = blockIdx.x, h = blockIdx.y, d = threadIdx.x;
  const float* part = a.part + ((size_t)r * a.n_q + h) * SPLITS * (DH + PART_HEAD);
  float M = -INFINITY, num = 0.0f, den = 0.0f;
  for (int s = 0; s < SPLITS; ++s) M = fmaxf(M, part[s * (DH + PART_HEAD)]);
  for (int s = 0; s < SPLITS; ++s) {
    const float* p = part + s * (DH + PART_HEAD);
    const float f = p[0] == -INFINITY ? 0.0f : expf(p[0] - M);
    den = fmaf(f, p[1], den);
    num = fmaf(f, p[PART_HEAD + d], num);
  }
  a.o[r * a.o_stride + h * DH + d] = __float2bfloat16_rn(den == 0.0f ? 0.0f : num / den);
  if (d == 0 && a.lse) a.lse[(size_t)r * a.n_q + h] = den == 0.0f ? -INFINITY : M + logf(den);
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
      const Seen s = seen_of(a, row_hi(a, r));
      if (t > s.hi || (t < s.lo && t >= s.ns)) continue;
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

}  // namespace

size_t attend_workspace_bytes(int n_q, int head_dim, int max_rows) {
  return (size_t)max_rows * n_q * (SPLITS * (head_dim + PART_HEAD) + 1) * sizeof(float);
}

cudaError_t launch_attend(const Launch& L, const AttendArgs& a) {
  const int G = a.kv_dim / a.head_dim;
  const long long cap = (long long)a.kv.max_blocks * a.kv.block_size;
  const int tiles = (int)((cap + TT - 1) / TT);
  const bool wide = a.head_dim == 128;
  cudaError_t e = launch_ex(L, dim3(a.rows, G, SPLITS), dim3(TT), 0,
                            wide ? attend_kernel<128> : attend_kernel<64>, a);
  if (e == cudaSuccess)
    e = launch_ex(L, dim3(a.rows, a.n_q), dim3(a.head_dim), 0,
                  wide ? attend_join_kernel<128> : attend_join_kernel<64>, a);
  if (e == cudaSuccess && a.weights)
    e = launch_ex(L, dim3(min(tiles, 1024), a.n_req), dim3(TT), 0,
                  wide ? attend_weights_kernel<128> : attend_weights_kernel<64>, a, tiles);
  return e;
}

}  // namespace mono
