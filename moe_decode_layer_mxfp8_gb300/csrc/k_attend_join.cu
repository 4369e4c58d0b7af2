// The attention over the cache: its launches, and the join of its pieces.
#include <cudaTypedefs.h>

#include <algorithm>

#include "attend_plan.cuh"

namespace mono {
namespace attend {
namespace {

// Joins the pieces of a (row, head): a warp each, 4 dimensions a lane (64 wide: the half warps take
// every other piece).  Rows that one piece holds are done; pad rows and rows that see nothing get
// zeros.  Bound by latency (2 to 4.5 us): a lane per piece fetches m and l while the first pieces' O is
// on its way.  (Joined by the team that brings the last piece, 48 rows took 9 us longer.)
constexpr int JOIN_WARPS = 4, AHEAD = 4;
__global__ void __launch_bounds__(JOIN_WARPS * 32) attend_join_kernel(const AttendArgs a, const Shape sh,
                                                                      const Pieces ar) {
  const int r = blockIdx.x, h = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int chunk = h / sh.heads, hpg = a.n_q / (a.kv_dim / a.head_dim);
  const int cheads = hpg * (min(128, a.kv_dim - 128 * chunk) > a.head_dim ? 2 : 1);
  const int d = 4 * lane & (a.head_dim - 1), step = 128 / a.head_dim, first = lane * 4 / a.head_dim;
  __nv_bfloat16* o = a.o + r * a.o_stride + (long long)h * a.head_dim + d;
  const size_t team = (size_t)2 * sh.chunks * sh.cols * PART_LD;  // from a team's pieces to the next's
  pdl_trigger();
  pdl_wait();
  if (h >= a.n_q) return;
  const RowInfo info = ar.rows[r];
  if (info.k0 < 0) {
    *reinterpret_cast<uint2*>(o) = make_uint2(0u, 0u);
    if (lane == 0) a.lse[(long long)r * a.n_q + h] = -INFINITY;
    return;
  }
  if (info.k0 == info.k1) return;  // whole in one team
  const int c = info.place * cheads + (h - chunk * sh.heads), n = info.k1 - info.k0 + 1;
  // piece i: team k0 + i's first slot, but the first piece its second
  const float* base = ar.part + info.k0 * team + ((size_t)chunk * sh.cols + c) * PART_LD;
  auto piece = [&](int i) { return base + i * team + (i == 0 ? (size_t)sh.chunks * sh.cols * PART_LD : 0); };
  auto fetch = [&](int i) { return *reinterpret_cast<const float4*>(piece(i) + 4 + d); };
  float m = UNSET, den = 0.0f;
  float4 num = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int b = 0; b < n; b += 32) {
    const int in = min(32, n - b);
    float2 ml = {UNSET, 0.0f};
    if (lane < in) ml = *reinterpret_cast<const float2*>(piece(b + lane));
    float4 x[AHEAD];
#pragma unroll
    for (int e = 0; e < AHEAD; ++e)
      if (first + step * e < in) x[e] = fetch(b + first + step * e);
    const float to = fmaxf(m, warp_max(ml.x)), f = ex2(ml.x - to), old = ex2(m - to);
    m = to;
    den = fmaf(den, old, warp_sum(f * ml.y));
    num.x *= old, num.y *= old, num.z *= old, num.w *= old;
#pragma unroll 1
    for (int i = 0; i < in; i += step * AHEAD) {
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        const int at = i + first + step * e;
        const float g = __shfl_sync(0xffffffffu, f, at & 31);
        if (at < in) {
          num.x = fmaf(g, x[e].x, num.x), num.y = fmaf(g, x[e].y, num.y);
          num.z = fmaf(g, x[e].z, num.z), num.w = fmaf(g, x[e].w, num.w);
        }
        if (at + step * AHEAD < in) x[e] = fetch(b + at + step * AHEAD);
      }
    }
  }
  if (a.head_dim == 64) {
    num.x += __shfl_xor_sync(0xffffffffu, num.x, 16), num.y += __shfl_xor_sync(0xffffffffu, num.y, 16);
    num.z += __shfl_xor_sync(0xffffffffu, num.z, 16), num.w += __shfl_xor_sync(0xffffffffu, num.w, 16);
  }
  const float inv = den == 0.0f ? 0.0f : 1.0f / den;
  if (den == 0.0f) num = {0.0f, 0.0f, 0.0f, 0.0f};
  *reinterpret_cast<uint2*>(o) =
      make_uint2(pack_bf16x2(num.x * inv, num.y * inv), pack_bf16x2(num.z * inv, num.w * inv));
  if (lane == 0)
    a.lse[(long long)r * a.n_q + h] = den == 0.0f ? -INFINITY : (log2f(den) + m) * LN2;
}

}  // namespace

// The records as a 3D byte tensor [pages][tokens][width], boxes of run (128: swizzled, bytes beyond
// width read as 0) x box tokens; false where its strides are beyond a tensor map's.
static bool encode_cache_map(CUtensorMap* m, const PagedView& kv, int width, int run, int box) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      fn = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode || kv.num_blocks > INT32_MAX) return false;
  if (kv.stride_block >= (1ll << 40) || kv.stride_tok >= (1ll << 40)) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)kv.block_size, (cuuint64_t)kv.num_blocks};
  const cuuint64_t strides[2] = {(cuuint64_t)kv.stride_tok, (cuuint64_t)kv.stride_block};
  const cuuint32_t boxes[3] = {(cuuint32_t)run, (cuuint32_t)box, 1}, ones[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(kv.base), dims, strides,
                boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                run == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int encode_cache_maps(CUtensorMap* codes, CUtensorMap* scales, const AttendArgs& a) {
  const int bs = a.kv.block_size;
  if (bs % 8) return 0;
  const int box = std::min(bs & -bs, 128);
  return encode_cache_map(codes, a.kv, a.kv_dim, 128, box) &&
                 encode_cache_map(scales, a.kv, a.kv_dim + 16, 16, box)
             ? box
             : 0;
}

cudaError_t launch_join(const Launch& L, const AttendArgs& a, const Shape& sh, const Pieces& ws) {
  return launch_ex(L, dim3(a.rows, (a.n_q + JOIN_WARPS - 1) / JOIN_WARPS), dim3(JOIN_WARPS * 32), 0,
                   attend_join_kernel, a, sh, ws);
}

}  // namespace attend

namespace {
struct Layout {
  size_t rows, part, bytes;
};
Layout layout(int max_rows, int sms) {
  Layout l;
  l.rows = 0;
  l.part = l.rows + ((size_t)max_rows * sizeof(attend::RowInfo) + 255) / 256 * 256;
  // pieces: two per team and chunk, a team per `chunks` SMs
  l.bytes = l.part + (size_t)sms * 2 * attend::MAX_COLS * attend::PART_LD * sizeof(float);
  return l;
}
}  // namespace

size_t attend_workspace_bytes(int max_rows, int sms) { return layout(max_rows, sms).bytes; }

cudaError_t attend_prepare() {
  cudaError_t e = attend_tc_prepare();
  return e == cudaSuccess ? attend_weights_prepare() : e;
}

cudaError_t launch_attend(const Launch& L, const AttendArgs& a, uint8_t* base, int max_rows, int sms) {
  const Layout l = layout(max_rows, sms);
  const attend::Pieces ws = {reinterpret_cast<float*>(base + l.part),
                             reinterpret_cast<attend::RowInfo*>(base + l.rows)};
  cudaError_t e = launch_attend_tc(L, a, ws, sms);
  if (e == cudaSuccess && a.weights) e = launch_attend_weights(L, a, sms);
  return e;
}

}  // namespace mono
