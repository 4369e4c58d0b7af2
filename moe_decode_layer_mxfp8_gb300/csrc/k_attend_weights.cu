// Gathering of attention weights: with the attention's lse known,
//
//   weights[b][t] += sum over b's rows that see t, and over heads, of 2^(s log2e - lse log2e)
//
// the score half of the attention alone, on m16n8k16 MMAs (f16, f32 accumulation): a warp takes 16
// tokens and all their chunks, widens the codes in registers (exact), and every row's heads of a
// slice, padded to 16, are the MMA's M.  Queries are f16 under a power of two per head (exact for
// every element down to 2^-24 of the head's largest).  Sums are f32, all of a token's in one warp,
// so their order is fixed and each has one writer.
#include "attend_plan.cuh"

namespace mono {
namespace {

using namespace attend;

constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int PASS_ROWS = 6;   // rows of a pass, while their queries fit the shared memory
constexpr int TILE = 128; // tokens of a unit: 16 a warp
constexpr int PLAN_BYTES = (3 * MAX_REQ + 4) * 4;
constexpr int SMEM_MAX = 110 * 1024;  // two CTAs an SM

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
// Eight elements from dimension d of a head as f16, times up, in the order in which lanes hold codes:
// dimension 64 p + 16 j + 4 u + e at K step 4 p + u, MMA column 2 j + e (e < 2) or 2 j + 6 + e.
__device__ __forceinline__ void store_query(__half* row, int d, const float (&v)[8], float up) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int dd = d + 4 * t, p = dd >> 6, j = (dd >> 4) & 3, u = (dd >> 2) & 3;
    uint32_t* at = reinterpret_cast<uint32_t*>(row + (4 * p + u) * 16 + 2 * j);
    at[0] = f16x2(v[4 * t] * up, v[4 * t + 1] * up);
    at[4] = f16x2(v[4 * t + 2] * up, v[4 * t + 3] * up);
  }
}
// The exponent that brings a largest magnitude m to [2^8, 2^9) (within f32's reach).
__device__ __forceinline__ int query_exponent(float m) {
  return m > 0.0f ? min(max((int)(__float_as_uint(m) >> 23) - 127 - 8, -100), 100) : 0;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// Bytes of a row's queries (rows of a slice's heads padded to 16, f16, 8 elements of padding each)
__host__ __device__ __forceinline__ int row_bytes(const AttendArgs& a) {
  return a.kv_dim / a.head_dim * 16 * (a.head_dim + 8) * 2;
}

template <int DH>
__global__ void __launch_bounds__(THREADS, 2) attend_weights_kernel(const AttendArgs a, const Shape sh,
                                                                    int* total, int rows_fit) {
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ Jobs s_start;
  __shared__ int s_row[PASS_ROWS], s_pos[PASS_ROWS], s_n;
  __shared__ float s_lse[PASS_ROWS * 256], s_qs[PASS_ROWS * 256];  // by (row, head), up to 256 heads
  Plan plan;
  plan.pre = reinterpret_cast<int*>(sm);
  plan.pmax = plan.pre + MAX_REQ + 4;
  plan.pmin = plan.pmax + MAX_REQ;
  plan.pos = nullptr;
  plan.req = nullptr;
  __half* sq = reinterpret_cast<__half*>(sm + PLAN_BYTES);
  constexpr int QLD = DH + 8, STEPS = DH / 16, PIECES = DH / 64;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i4 = lane >> 2, j4 = lane & 3;
  const int G = a.kv_dim / DH, hpg = a.n_q / G;
  derive_plan<THREADS>(a, sh, plan, blockIdx.x, true, &s_start, total);
  __syncthreads();
  Jobs items = s_start;
  Job im;
#pragma unroll 1
  while (next_job(a, sh, plan, items, im)) {
    // every row of the request in turn, rows_fit at a time
#pragma unroll 1
    for (int first = 0;; first += rows_fit) {
      __syncthreads();
      if (warp == 0) {
        int seen = 0, n = 0;
#pragma unroll 1
        for (int r0 = 0; r0 < a.rows && n < rows_fit; r0 += 32) {
          const int r = r0 + lane;
          const int qb = r < a.rows ? a.row_req[r] : -1, p0 = r < a.rows ? a.positions[r] : -1;
          const int p = qb == im.b ? p0 : -1;
          const uint32_t m = __ballot_sync(0xffffffffu, p >= 0);
          const int rank = seen + __popc(m & ((1u << lane) - 1)) - first;
          if (p >= 0 && rank >= 0 && rank < rows_fit) s_row[rank] = r, s_pos[rank] = p;
          seen += __popc(m);
          n = max(0, min(rows_fit, seen - first));
        }
        if (lane == 0) s_n = n;
      }
      __syncthreads();
      const int n = s_n;
      if (n == 0) break;
      // queries as f16 under a power of two per head
      constexpr int LN = DH / 8;  // lanes of a head
#pragma unroll 1
      for (int i0 = 0; i0 < n * G * 16 * LN; i0 += THREADS) {
        const int i = i0 + tid, c = i / LN, d = (i % LN) * 8;
        const int h16 = c % 16, g = (c / 16) % G, r = c / (16 * G);
        const bool in = r < n && h16 < hpg;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (in)
          x = *reinterpret_cast<const uint4*>(a.q + s_row[r] * a.q_stride + (g * hpg + h16) * DH + d);
        float v[8], m = 0.0f;
        bf16x8_to_f32(x, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (fabsf(v[e]) <= 3.4e38f) m = fmaxf(m, fabsf(v[e]));
#pragma unroll
        for (int o = 1; o < LN; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int ex = query_exponent(m);
        const float up = pow2(-ex);
        if (r >= n) continue;
        if (d == 0) {
          const int k = (r * G + g) * 16 + h16;
          s_qs[k] = pow2(ex) * a.scale * LOG2E;
          s_lse[k] = in ? a.lse[(long long)s_row[r] * a.n_q + g * hpg + h16] * LOG2E : INFINITY;
        }
        store_query(sq + (size_t)c * QLD, d, v, up);
      }
      __syncthreads();
#pragma unroll 1
      for (int k = 0; k < im.n; ++k) {
        // a warp's 16 tokens: lanes of a quad share tokens i4 and i4 + 8
        const int t0 = im.span.token(im.t0 + k) + 16 * warp;
        if (t0 > im.span.hi) continue;
        const uint8_t* rec[2];
        float sc[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = t0 + i4 + 8 * e;
          const long long off = t <= im.span.hi && (t >= im.span.lo || t < a.sinks)
                                    ? record_offset(a.kv, im.b, t) : -1;
          rec[e] = off >= 0 ? a.kv.base + off : nullptr;
        }
        float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // tokens 2j, 2j + 1, 2j + 8, 2j + 9
        float ct[4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          sc[e] = rec[e] ? *reinterpret_cast<const float*>(rec[e] + a.kv_dim) : 0.0f;
        const uint32_t there0 = __ballot_sync(0xffffffffu, rec[0] != nullptr);
        const uint32_t there1 = __ballot_sync(0xffffffffu, rec[1] != nullptr);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ct[e] = __shfl_sync(0xffffffffu, sc[e >> 1], 4 * (2 * j4 + (e & 1)));
        uint4 nx[2][PIECES];
        auto fetch = [&](int g) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int p = 0; p < PIECES; ++p)
              nx[e][p] = rec[e] ? __ldg(reinterpret_cast<const uint4*>(rec[e] + g * DH + 64 * p + 16 * j4))
                                : make_uint4(0, 0, 0, 0);
        };
        fetch(0);
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
          uint32_t b[2][STEPS][2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
              e4m3x4_to_f16x4(nx[e][p].x, b[e][4 * p]);
              e4m3x4_to_f16x4(nx[e][p].y, b[e][4 * p + 1]);
              e4m3x4_to_f16x4(nx[e][p].z, b[e][4 * p + 2]);
              e4m3x4_to_f16x4(nx[e][p].w, b[e][4 * p + 3]);
            }
          if (g + 1 < G) fetch(g + 1);
#pragma unroll 1
          for (int r = 0; r < n; ++r) {
            const int hi = a.causal ? s_pos[r] : im.span.hi;
            const int lo = a.window > 0 ? max(0, hi - a.window + 1) : 0;
            float c[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[0][e] = c[1][e] = 0.0f;
            const __half* src = sq + ((size_t)(r * G + g) * 16 + (lane & 15)) * QLD + (lane >> 4) * 8;
#pragma unroll
            for (int k16 = 0; k16 < STEPS; ++k16) {
              uint32_t qf[4];
              ldsm_x4(qf, src + 16 * k16);
              mma_f16_acc(c[0], qf, b[0][k16][0], b[0][k16][1]);
              mma_f16_acc(c[1], qf, b[1][k16][0], b[1][k16][1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int at = (r * G + g) * 16 + i4 + 8 * h;
              const float qs = s_qs[at], ls = s_lse[at];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int t = t0 + 2 * j4 + (e & 1) + 8 * (e >> 1);
                const bool see = t <= hi && (t >= lo || t < a.sinks) &&
                                 (((e >> 1 ? there1 : there0) >> (4 * (2 * j4 + (e & 1)))) & 1);
                const float p = ex2(fmaf(c[e >> 1][2 * h + (e & 1)] * ct[e], qs, -ls));
                if (see) w[e] += p;
              }
            }
          }
        }
        // the heads' sums, over the lanes that share tokens; in a fixed order
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] += __shfl_xor_sync(0xffffffffu, w[e], 4);
          w[e] += __shfl_xor_sync(0xffffffffu, w[e], 8);
          w[e] += __shfl_xor_sync(0xffffffffu, w[e], 16);
        }
        if (lane < 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = t0 + 2 * j4 + (e & 1) + 8 * (e >> 1);
            const bool there = ((e >> 1 ? there1 : there0) >> (4 * (2 * j4 + (e & 1)))) & 1;
            if (there && t < a.weights_stride) a.weights[im.b * a.weights_stride + t] += w[e];
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t attend_weights_prepare() {
  const cudaError_t e =
      cudaFuncSetAttribute(attend_weights_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(attend_weights_kernel<64>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
}

cudaError_t launch_attend_weights(const Launch& L, const AttendArgs& a, const attend::Pieces& ws, int sms) {
  Shape sh = shape_of(a, TILE, 16, 2 * sms);
  sh.rows_per = 1024;  // a unit is a tile with all its request's rows
  const int row = row_bytes(a);
  const int fit = std::max(1, std::min(PASS_ROWS, (SMEM_MAX - PLAN_BYTES) / row));
  const int smem = PLAN_BYTES + fit * row;
  return launch_ex(L, dim3(2 * sms), dim3(THREADS), smem,
                   a.head_dim == 128 ? attend_weights_kernel<128> : attend_weights_kernel<64>, a, sh,
                   ws.total, fit);
}

}  // namespace mono
