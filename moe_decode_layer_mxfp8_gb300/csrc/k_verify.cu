// Verification of drafted tokens against the target's probabilities (rejection sampling).
//
// CTA = request.  The accept tests u q(x) < p(x) are exact (a product of two f32 in f64); the
// drawn token inverts the distribution function, with every sum in f64.
#include <cuda_fp16.h>

#include "cache_kernels.h"

namespace mono {
namespace {

constexpr int THREADS = 512;

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ double weight0(float v) { return v > 0.0f ? (double)v : 0.0; }

template <class T>
__global__ void __launch_bounds__(THREADS) verify_kernel(VerifyArgs a) {
  __shared__ double sums[THREADS];
  __shared__ float bv[THREADS];
  __shared__ int bi[THREADS];
  __shared__ int s_tok;
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x, V = a.vocab;
  const int r0 = min(max(a.row_start[b], 0), a.rows);
  const int r1 = min(max(a.row_start[b + 1], r0), a.rows);
  if (r1 == r0) {
    if (tid == 0) a.accepted[b] = 0;
    return;
  }
  const T* tp = reinterpret_cast<const T*>(a.target);
  const T* dp = reinterpret_cast<const T*>(a.draft);
  const bool greedy = a.greedy && a.greedy[b] != 0;
  int j = r0, tok = -1;
  for (;; ++j) {
    const T* p = tp + (long long)j * a.target_stride;
    const int x = a.draft_tokens[j];
    const bool valid = j < r1 - 1 && x >= 0 && x < V;
    if (greedy) {
      float best = -INFINITY;
      int idx = V;
      for (int v = tid; v < V; v += THREADS) {
        const float f = as_f32(p[v]);
        if (f > best || (idx == V && !(f != f))) best = f, idx = v;
      }
      bv[tid] = best;
      bi[tid] = idx;
      __syncthreads();
      for (int n = THREADS / 2; n > 0; n >>= 1) {
        if (tid < n && (bv[tid + n] > bv[tid] || (bv[tid + n] == bv[tid] && bi[tid + n] < bi[tid])))
          bv[tid] = bv[tid + n], bi[tid] = bi[tid + n];
        __syncthreads();
      }
      tok = bi[0] < V ? bi[0] : 0;
      __syncthreads();
      if (valid && tok == x) continue;
      break;
    }
    if (valid) {
      const double px = weight0(as_f32(p[x]));
      const double qx = dp ? weight0(as_f32(dp[(long long)j * a.draft_stride + x])) : 1.0;
      if ((double)a.u[j] * qx < px) continue;
    }
    // the drawn token
    const int per = (V + THREADS - 1) / THREADS, v0 = min(V, tid * per), v1 = min(V, v0 + per);
    const bool bonus = j == r1 - 1;
    for (int pass = bonus ? 1 : 0; pass < 2; ++pass) {  // 0: the residual, 1: the row itself
      const T* q = dp ? dp + (long long)j * a.draft_stride : nullptr;
      auto weight = [&](int v) {
        double w = weight0(as_f32(p[v]));
        if (pass == 0) w -= q ? weight0(as_f32(q[v])) : (v == x ? 1.0 : 0.0);
        return w > 0.0 ? w : 0.0;
      };
      double s = 0.0;
      for (int v = v0; v < v1; ++v) s += weight(v);
      sums[tid] = s;
      if (tid == 0) s_tok = -1;
      __syncthreads();
      double before = 0.0, total = 0.0;
      for (int i = 0; i < THREADS; ++i) {
        if (i < tid) before += sums[i];
        total += sums[i];
      }
      const double want = (double)a.r[b] * total;
      if (s > 0.0 && before <= want && want < before + s) {
        double c = before;
        for (int v = v0; v < v1; ++v) {
          const double w = weight(v);
          c += w;
          if (w > 0.0) s_tok = v;  // (the last one, should roundings leave c at want)
          if (c > want) break;
        }
      }
      __syncthreads();
      tok = s_tok;
      __syncthreads();
      if (total > 0.0) break;
    }
    break;
  }
  if (tid == 0) a.accepted[b] = j - r0;
  for (int i = r0 + tid; i < r1; i += THREADS)
    a.tokens[i] = i < j ? a.draft_tokens[i] : i == j ? tok : -1;
}

}  // namespace

cudaError_t launch_verify(const Launch& L, const VerifyArgs& a, int dtype) {
  const dim3 grid(a.n_req), block(THREADS);
  if (dtype == 0) return launch_ex(L, grid, block, 0, verify_kernel<float>, a);
  if (dtype == 1) return launch_ex(L, grid, block, 0, verify_kernel<__nv_bfloat16>, a);
  return launch_ex(L, grid, block, 0, verify_kernel<__half>, a);
}

}  // namespace mono
