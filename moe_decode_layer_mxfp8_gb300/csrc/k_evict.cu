// Eviction by accumulated attention weight: which tokens stay, and the move of their records.
//
// CTA = request.  The threshold weight is found by a radix selection over the order-preserving
// bit patterns of the weights, 8 bits a pass; tokens above it stay, and of those equal to it
// the lowest slots.  The kept tokens then move in slot order, a chunk at a time: a chunk is read
// whole before it is written, and every destination slot is at or below its source, so a write
// never reaches a record that a later chunk still has to read.
#include "cache_kernels.h"

namespace mono {
namespace {

constexpr int THREADS = 1024;
constexpr int CHUNK = 64;  // records per move

// Order-preserving key: larger weight, larger key; -0 as +0, NaN as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Exclusive prefix sum over the block; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  int base = 0, all = 0;
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < w) base += warp_sums[i];
    all += warp_sums[i];
  }
  *total = all;
  return base + x - v;
}

__global__ void __launch_bounds__(THREADS) evict_kernel(EvictArgs a) {
  __shared__ int hist[256], warp_sums[32];
  __shared__ uint32_t s_key;
  __shared__ int s_need;
  extern __shared__ __align__(16) uint8_t buf[];  // [CHUNK][copy_bytes]
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x;
  const float* w = a.weights + b * a.weights_stride;
  int* kept = a.kept + b * a.kept_stride;
  int len = max(0, a.lengths[b]);
  const long long cap = min((long long)a.src.max_blocks * a.src.block_size, a.weights_stride);
  if (len > cap) {
    len = (int)cap;
    if (tid == 0) atomicOr(a.status, ST_UNMAPPED_PAGE);
  }
  const int lo = a.sinks, hi = len - a.recent;  // candidates [lo, hi)
  int total = len;
  if (len > a.budget) {
    int need = a.budget - a.sinks - a.recent;
    uint32_t key = 0, mask = 0;
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
      for (int i = tid; i < 256; i += THREADS) hist[i] = 0;
      __syncthreads();
      for (int t = lo + tid; t < hi; t += THREADS) {
        const uint32_t k = weight_key(w[t]);
        if ((k & mask) == key) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255;
        for (; d > 0 && hist[d] < need; --d) need -= hist[d];
        s_key = key | ((uint32_t)d << shift);
        s_need = need;
      }
      __syncthreads();
      key = s_key;
      need = s_need;
      mask |= 255u << shift;
      __syncthreads();
    }
    const bool none = a.budget == a.sinks + a.recent;
    int out = 0, ties = 0;
    for (int t0 = 0; t0 < len; t0 += THREADS) {
      const int t = t0 + tid;
      int keep = 0, tie = 0;
      if (t < len) {
        if (t < lo || t >= hi) keep = 1;
        else if (!none) {
          const uint32_t k = weight_key(w[t]);
          keep = k > key;
          tie = k == key;
        }
      }
      int n;
      const int before = ties + block_scan(tie, warp_sums, &n);
      ties += n;
      if (tie && before < need) keep = 1;
      const int pos = out + block_scan(keep, warp_sums, &n);
      out += n;
      if (keep) kept[pos] = t;
    }
    total = out;
  } else {
    for (int t = tid; t < len; t += THREADS) kept[t] = t;
  }
  for (int i = total + tid; i < a.budget; i += THREADS) kept[i] = -1;
  if (tid == 0) a.new_lengths[b] = total;
  __syncthreads();
  float* wo = a.weights_out ? a.weights_out + b * a.weights_out_stride : nullptr;
  const long long wcap = a.weights_out_stride;
  if (wo)
    for (int i0 = 0; i0 < total; i0 += THREADS) {
      const int i = i0 + tid;
      const float v = i < total ? w[kept[i]] : 0.0f;
      __syncthreads();
      if (i < total && i < wcap) wo[i] = v;
      __syncthreads();
    }
  if (wo)
    for (int i = total + tid; i < len && i < wcap; i += THREADS) wo[i] = 0.0f;
  const int per = a.copy_bytes / 16;
  for (int c0 = 0; c0 < total; c0 += CHUNK) {
    const int n = min(CHUNK, total - c0);
    for (int j = tid; j < n * per; j += THREADS) {
      const int i = j / per, c = j - i * per;
      const long long so = record_offset(a.src, b, kept[c0 + i]);
      if (so >= 0)
        *reinterpret_cast<uint4*>(buf + 16 * j) =
            *reinterpret_cast<const uint4*>(a.src.base + so + 16 * c);
    }
    __syncthreads();
    for (int j = tid; j < n * per; j += THREADS) {
      const int i = j / per, c = j - i * per;
      const long long so = record_offset(a.src, b, kept[c0 + i]);
      const long long d = record_offset(a.dst, b, c0 + i);
      if (so < 0 || d < 0)
        atomicOr(a.status, ST_UNMAPPED_PAGE);
      else
        *reinterpret_cast<uint4*>(a.dst_base + d + 16 * c) =
            *reinterpret_cast<const uint4*>(buf + 16 * j);
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict(const Launch& L, const EvictArgs& a) {
  const int smem = CHUNK * a.copy_bytes;
  cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       CHUNK * 1040);
  if (e != cudaSuccess) return e;
  return launch_ex(L, dim3(a.n_req), dim3(THREADS), smem, evict_kernel, a);
}

}  // namespace mono
