// Eviction by accumulated attention weight: which tokens stay, and the move of their records.
//
// Selection (a cluster of up to 16 CTAs per request, each with a run of the slots): the smallest
// weight that stays is found by a radix selection over the order-preserving bit patterns of the
// weights, 8 bits a pass, the CTAs' histograms added through distributed shared memory; larger
// weights stay, of equal ones the lowest slots, and prefix sums over threads and CTAs give every
// kept slot its place.  Bound by its four exchanges' latencies: the weights are read once, into
// shared memory.
//
// Move (a CTA per 64 kept tokens, in order): the records go through registers, 16 bytes a lane,
// every load of a chunk in flight at once.  Within the same pages a chunk is written only after
// the chunks that read from its slots have loaded theirs: kept slots rise, so these are the one or
// two whose sources lie between its first slot and the next chunk's (the selection leaves those
// places behind).  Chunks are handed out in order, so a chunk waits only for chunks that have begun,
// and those publish their loads before they wait.  Weights move the same way.
// Bound by HBM and the chain of lookups ahead of a chunk's loads: each kept record is read once and
// written once.  Measured: 8 caches of 33K..64K tokens of 528 bytes cut to 32K on other pages, 63 us, of
// which the selection takes 14 and the move 47 (274 MB; copy: 40 us); in place, with the waits among
// chunks, 78 us.  3 of up to 5K tokens 12 us, latencies.
#include <algorithm>

#include "cache_kernels.h"

namespace mono {
namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int MAX_CS = 16;
constexpr int CACHED = 12288;  // weights of a CTA's run kept in shared memory (longer runs re-read)
constexpr int CHUNK = 64;      // kept tokens per move
constexpr int MOVE_THREADS = 256;
constexpr int PER_RECORD = 8;  // lanes of a record, 16 bytes each at a time
constexpr int ROUNDS = CHUNK * PER_RECORD / MOVE_THREADS;

// Order-preserving key: larger weight, larger key; -0 as +0, NaN as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ int ld_dsmem_i32(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}
// Exclusive prefix sum over the block (two counts in one 64-bit sum: no carry between them).
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* warp_sums, uint64_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  uint64_t base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    if (i < w) base += warp_sums[i];
    all += warp_sums[i];
  }
  *total = all;
  return base + x - v;
}

// The move's workspace: tickets; then per request, old lengths and the chunks' state.
struct Work {
  int* ticket;
  int* old_len;  // [n_req]
  int* loaded;   // [n_req][chunks]: the chunk's sources have been read
  int* from;     // [n_req][chunks]: kept tokens below the chunk's first slot
};

// (two CTAs an SM: with one, clusters of 16 wait for one another's places)
__global__ void __launch_bounds__(THREADS, 2) evict_select_kernel(EvictArgs a, Work ws, int cs, int chunks) {
  extern __shared__ float s_w[];  // the run's weights
  __shared__ int hist[4][256];
  __shared__ int s_tot[256], s_digit, s_need, s_last;
  __shared__ uint64_t warp_sums[WARPS], s_cnt;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x / cs, rank = blockIdx.x - b * cs, tid = threadIdx.x;
  const float* w = a.weights + b * a.weights_stride;
  int* kept = a.kept + b * a.kept_stride;
  int len = max(0, a.lengths[b]);
  const long long cap = min((long long)a.src.max_blocks * a.src.block_size, a.weights_cols);
  if (len > cap) {
    len = (int)cap;
    if (tid == 0 && rank == 0) atomicOr(a.status, ST_UNMAPPED_PAGE);
  }
  for (int i = rank * THREADS + tid; i < chunks; i += cs * THREADS) ws.loaded[(size_t)b * chunks + i] = 0;
  if (blockIdx.x == 0 && tid == 0) *ws.ticket = 0;
  const bool all = len <= a.budget;
  const int total = all ? len : a.budget;
  // this CTA's run, a contiguous share of it per thread
  const int per = ((len + cs * THREADS - 1) / (cs * THREADS)) | 1;  // (odd: no bank conflicts)
  const int t0 = min(len, rank * THREADS * per), t1 = min(len, t0 + THREADS * per);
  const bool cached = THREADS * per <= CACHED;
  const int lo = a.sinks, hi = len - a.recent;  // others: [lo, hi)
  uint32_t key = 0;
  int need = 0;
  if (!all) {
    for (int i = tid; i < 4 * 256; i += THREADS) (&hist[0][0])[i] = 0;
    if (cached)
      for (int t = t0 + tid; t < t1; t += THREADS) s_w[t - t0] = w[t];
    __syncthreads();
    need = a.budget - a.sinks - a.recent;
    uint32_t mask = 0;
#pragma unroll 1
    for (int pass = 0; pass < 4 && need > 0; ++pass) {
      const int shift = 24 - 8 * pass;
#pragma unroll 4
      for (int t = max(t0, lo) + tid; t < min(t1, hi); t += THREADS) {
        const uint32_t k = weight_key(cached ? s_w[t - t0] : w[t]);
        if ((k & mask) == key) atomicAdd(&hist[pass][(k >> shift) & 255], 1);
      }
      if (cs > 1) cluster_sync_all(); else __syncthreads();
      if (tid < 256) {
        const uint32_t at = smem_u32(&hist[pass][tid]);
        int v[MAX_CS], n = hist[pass][tid];
        if (cs > 1) {
#pragma unroll
          for (int k = 0; k < MAX_CS; ++k)  // (all on their way at once)
            v[k] = k < cs && k != rank ? ld_dsmem_i32(mapa_shared(at, k)) : 0;
#pragma unroll
          for (int k = 0; k < MAX_CS; ++k) n += v[k];
        }
        s_tot[tid] = n;
      }
      __syncthreads();
      if (tid < 32) {
        // the digit whose tokens, with those of the larger ones, first reach `need`: eight digits
        // a lane, from the largest down
        int n = 0, v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = s_tot[255 - 8 * tid - e], n += v[e];
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (tid >= o) incl += y;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, incl >= need);
        if (tid == __ffs(m) - 1) {
          int left = need - (incl - n), d = 255 - 8 * tid;
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (d == 255 - 8 * tid - e && v[e] < left) left -= v[e], --d;
          s_digit = d;
          s_need = left;
          s_last = s_tot[d] == left;  // all of the digit's stay: its lower bits need no look
        }
      }
      __syncthreads();
      key |= (uint32_t)s_digit << shift;
      need = s_need;
      mask |= 255u << shift;
      if (s_last) break;  // (alike in the cluster)
    }
  }
  // how many of this thread's slots stay for sure, and how many are equal to the threshold
  const bool none = !all && a.budget == a.sinks + a.recent;  // of the others nothing stays
  const int u0 = min(t1, t0 + tid * per), u1 = min(t1, u0 + per);
  auto state = [&](int t) {  // 1: stays, 2: equal
    if (all || t < lo || t >= hi) return 1;
    if (none) return 0;
    const uint32_t k = weight_key(cached ? s_w[t - t0] : w[t]);
    return k > key ? 1 : k == key ? 2 : 0;
  };
  uint64_t mine = 0;
#pragma unroll 4
  for (int t = u0; t < u1; ++t) {
    const int s = state(t);
    mine += s == 1 ? 1ull << 32 : s == 2 ? 1ull : 0ull;
  }
  uint64_t sum;
  uint64_t at = block_scan(mine, warp_sums, &sum);
  if (tid == 0) s_cnt = sum;
  if (cs > 1) {
    cluster_sync_all();
    uint64_t v = 0;  // a lane per CTA ahead of this one
    if ((tid & 31) < rank)
      asm volatile("ld.shared::cluster.u64 %0, [%1];"
                   : "=l"(v) : "r"(mapa_shared(smem_u32(&s_cnt), tid & 31)) : "memory");
#pragma unroll
    for (int o = MAX_CS / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    at += __shfl_sync(0xffffffffu, v, 0);
  }
  int sure = (int)(at >> 32), equal = (int)(at & 0xffffffffu);  // before this thread's slots
  for (int t = u0; t < u1; ++t) {
    const int s = state(t), pos = sure + min(equal, need);
    if (t % CHUNK == 0 && t / CHUNK < chunks) ws.from[(size_t)b * chunks + t / CHUNK] = pos;
    if (s == 1 || (s == 2 && equal < need)) kept[pos] = t;
    sure += s == 1;
    equal += s == 2;
  }
  for (long long i = total + rank * THREADS + tid; i < a.budget; i += cs * THREADS) kept[i] = -1;
  if (cs > 1) cluster_sync_all();  // every CTA has read the length, and its neighbours' counts
  if (rank == 0 && tid == 0) {
    ws.old_len[b] = len;
    a.new_lengths[b] = total;
  }
}

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(int* p, int v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Waits until the chunk's sources have been read (some 10^7 polls at most).
__device__ __forceinline__ void wait_loaded(const int* p, int* status) {
  for (uint32_t polls = 0; ld_acquire(p) == 0;)
    if (++polls == (1u << 22)) {
      atomicOr(status, ST_WAIT_TIMEOUT);
      return;
    }
}

// ordered: records or weights move within the storage that they are read from.  The grid's last
// n_req CTAs (by ticket) zero the weights behind the kept ones.  STEPS runs of 128 bytes hold a
// record: as few as do, since its registers bound the chunks in flight.
template <int STEPS>
__global__ void __launch_bounds__(MOVE_THREADS) evict_move_kernel(EvictArgs a, Work ws, int chunks,
                                                                  int ordered) {
  __shared__ int s_ticket, s_kept[CHUNK];
  __shared__ long long s_src[CHUNK], s_dst[CHUNK];
  pdl_wait();
  const int tid = threadIdx.x;
  if (tid == 0) s_ticket = atomicAdd(ws.ticket, 1);
  __syncthreads();
  const int chunk = s_ticket / a.n_req, b = s_ticket - chunk * a.n_req, i0 = chunk * CHUNK;
  // (all that a chunk looks up first, at once: kept is written up to the budget)
  const int* from = ws.from + (size_t)b * chunks + min(chunk, chunks - 1);
  const int n = a.new_lengths[b], len = ws.old_len[b], from0 = from[0], from1 = from[chunk + 1 < chunks ? 1 : 0];
  const int slot = tid < CHUNK && i0 + tid < a.budget ? a.kept[b * a.kept_stride + i0 + tid] : -1;
  const int* loaded = ws.loaded + (size_t)b * chunks;
  float* wo = a.weights_out + b * a.weights_out_stride;
  const long long wcap = a.weights_out_cols;
  if (chunk == chunks) {  // the tail of the weights
    if (ordered && n < len)
      for (int c = tid; c < (n + CHUNK - 1) / CHUNK; c += MOVE_THREADS) wait_loaded(loaded + c, a.status);
    __syncthreads();
    for (long long i = n + tid; i < min((long long)len, wcap); i += MOVE_THREADS) wo[i] = 0.0f;
    return;
  }
  const int count = min(CHUNK, n - i0);
  if (count <= 0) return;
  const bool still = a.in_place && n == len;  // everything stays where it is
  // the chunks ahead of this one that read from the slots that it writes
  int first = 0, end = 0;
  if (ordered && n < len) {
    first = from0 / CHUNK;
    end = min(chunk, (chunk + 1 < chunks && i0 + CHUNK < len ? from1 + CHUNK - 1 : n + CHUNK - 1) / CHUNK);
  }
  if (tid < count) {
    s_kept[tid] = slot;
    const long long so = record_offset(a.src, b, slot), d = record_offset(a.dst, b, i0 + tid);
    if (!still && (so < 0 || d < 0)) atomicOr(a.status, ST_UNMAPPED_PAGE);
    s_src[tid] = so < 0 || d < 0 || still ? -1 : so;
    s_dst[tid] = d;
  }
  __syncthreads();
  // every load of the chunk
  const int per = a.copy_bytes / 16, piece = tid % PER_RECORD;
  uint4 v[ROUNDS][STEPS];
#pragma unroll
  for (int h = 0; h < ROUNDS; ++h) {
    const int i = tid / PER_RECORD + h * (MOVE_THREADS / PER_RECORD);
    const long long so = i < count ? s_src[i] : -1;
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
      if (so >= 0 && piece + PER_RECORD * k < per)
        v[h][k] = *reinterpret_cast<const uint4*>(a.src.base + so + 16 * (piece + PER_RECORD * k));
  }
  const bool has_w = tid < count && i0 + tid < wcap;
  const float wv = has_w ? a.weights[b * a.weights_stride + s_kept[tid]] : 0.0f;
  if (ordered && n < len) {
    __threadfence();  // this thread's loads have been performed
    __syncthreads();
    if (tid == 0) st_release(const_cast<int*>(loaded) + chunk, 1);
    for (int c = first + tid; c < end; c += MOVE_THREADS) wait_loaded(loaded + c, a.status);
    __syncthreads();
  }
#pragma unroll
  for (int h = 0; h < ROUNDS; ++h) {
    const int i = tid / PER_RECORD + h * (MOVE_THREADS / PER_RECORD);
    const bool go = i < count && s_src[i] >= 0;
    const long long to = go ? s_dst[i] : 0;
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
      if (go && piece + PER_RECORD * k < per)
        *reinterpret_cast<uint4*>(a.dst_base + to + 16 * (piece + PER_RECORD * k)) = v[h][k];
  }
  if (has_w) wo[i0 + tid] = wv;
}

int chunks_of(int budget, long long cap) {
  return (int)((std::min((long long)budget, cap) + CHUNK - 1) / CHUNK);
}

}  // namespace

size_t evict_workspace_bytes(int max_req) {
  return 256 + ((size_t)max_req * 4 + 255) / 256 * 256 + 2 * (size_t)EVICT_MAX_CHUNKS * 4;
}

bool evict_fits(int n_req, int budget, long long cap) {
  return (long long)n_req * chunks_of(budget, cap) <= EVICT_MAX_CHUNKS;
}

cudaError_t evict_prepare() {
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CACHED * 4);
  return e;
}

cudaError_t launch_evict(const Launch& L, const EvictArgs& a, uint8_t* workspace, int max_req, int sms) {
  Work ws;
  ws.ticket = reinterpret_cast<int*>(workspace);
  ws.old_len = reinterpret_cast<int*>(workspace + 256);
  ws.loaded = ws.old_len + ((size_t)max_req * 4 + 255) / 256 * 64;
  ws.from = ws.loaded + EVICT_MAX_CHUNKS;
  const long long cap = std::min((long long)a.src.max_blocks * a.src.block_size, a.weights_cols);
  const int chunks = chunks_of(a.budget, cap);
  // as many CTAs a request as fit two an SM, eight slots a thread at least
  int cs = 1;
  while (cs < MAX_CS && (long long)a.n_req * cs * 2 <= 2 * sms && (long long)cs * 2 * THREADS * 8 <= cap) cs *= 2;
  const long long per = ((cap + cs * THREADS - 1) / (cs * THREADS)) | 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_req * cs);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)std::min<long long>(per * THREADS, CACHED) * 4;
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, ws, cs, chunks);
  if (e != cudaSuccess) return e;
  const int ordered = a.in_place || a.weights_out == a.weights;
  const auto move = a.copy_bytes <= 256 ? evict_move_kernel<2>
                    : a.copy_bytes <= 640 ? evict_move_kernel<5> : evict_move_kernel<9>;
  return launch_ex(L, dim3((chunks + 1) * a.n_req), dim3(MOVE_THREADS), 0, move, a, ws, chunks, ordered);
}

}  // namespace mono
