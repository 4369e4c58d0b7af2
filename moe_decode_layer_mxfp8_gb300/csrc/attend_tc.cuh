// Parts that the tensor-core kernels over the cache share: queries as e4m3 terms, bounded waits, and
// the loading of a tile of tokens through the page table.
#pragma once

#include "attend_plan.cuh"
#include "f32x2.cuh"
#include "tc_common.cuh"

namespace mono {
namespace tc {

// Eight columns of the warp's lane quadrant, TMEM -> registers and back.  Loaded registers are
// to be used only behind tc_wait_ld and tc_loaded (which keeps the compiler from moving a use
// ahead of the wait).
__device__ __forceinline__ void tc_ld8(uint32_t taddr, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]),
                 "=f"(r[6]), "=f"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tc_loaded(float* r) {
  asm volatile(""
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]),
                 "+f"(r[7]));
}
__device__ __forceinline__ void tc_ld4(uint32_t taddr, float* r) {  // four columns
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tc_loaded4(float* r) {
  asm volatile("" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]));
}
__device__ __forceinline__ void tc_st8(uint32_t taddr, const float* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
               : "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
}  // namespace tc

namespace attend {

constexpr int TT = 128;        // tokens per tile
constexpr int GROUP = 16;      // rows of a group at most
constexpr int MAX_ROWS = 1024;
constexpr int K_TILE = TT * 128, IMG = 512;

// Instruction descriptor, M = 128; N, and the scale-byte selectors, are or-ed in.
// kind::mxf8f6f4: e4m3 x e4m3, E8M0 scales, K-major, or (TRANS) MN-major.
constexpr uint32_t IDESC = (1u << 23) | ((uint32_t)(TT >> 4) << 24);
constexpr uint32_t TRANS = (1u << 15) | (1u << 16);

// Two f32 as f16, the first in the low half.
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four values, as two pairs of f16, as a word of e4m3 codes and one of the codes of what is left.
__device__ __forceinline__ void hilo_x4(const float* v, uint32_t& hi, uint32_t& lo) {
  asm("{\n .reg .b16 h0, h1, l0, l1;\n .reg .b32 f0, f1;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 h0, %2;\n cvt.rn.satfinite.e4m3x2.f16x2 h1, %3;\n"
      " cvt.rn.f16x2.e4m3x2 f0, h0;\n cvt.rn.f16x2.e4m3x2 f1, h1;\n"
      " sub.rn.f16x2 f0, %2, f0;\n sub.rn.f16x2 f1, %3, f1;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 l0, f0;\n cvt.rn.satfinite.e4m3x2.f16x2 l1, f1;\n"
      " mov.b32 %0, {h0, h1};\n mov.b32 %1, {l0, l1};\n}"
      : "=r"(hi), "=r"(lo)
      : "r"(f16x2_of(v[0], v[1])), "r"(f16x2_of(v[2], v[3])));
}
template <int N>
__device__ __forceinline__ void bar_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}
// Barrier among 128 threads that also tells whether any of them brought a true value.
__device__ __forceinline__ bool bar_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// A wait for an mbarrier phase by a whole warp, in few instructions: some 10^6 polls (a second or
// two) at most, none once another wait has run out.  False if it ran out.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  uint32_t polls = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (*abort || ++polls == (1u << 20)) {
      atomicOr(status, ST_WAIT_TIMEOUT);
      *abort = 1;
      polls = ~0u;
      break;
    }
  }
  return __all_sync(0xffffffffu, polls != ~0u);
}
// The tiles [first, first + n) of an item that all its rows see whole (those of the sinks aside, where
// there is a window); by a whole warp.
struct Clear {
  int first, n;
  __device__ bool has(int i) const { return (uint32_t)(i - first) < (uint32_t)n; }
};
template <class M>
__device__ __forceinline__ Clear clear_tiles(const AttendArgs& a, const Job& im, const M& meta) {
  const int lane = threadIdx.x & 31, hi = a.causal ? meta.pos[lane < meta.nrows ? lane : 0] : im.span.hi;
  const int lo = __reduce_max_sync(0xffffffffu, a.window > 0 ? max(0, hi - a.window + 1) : 0);
  const int end = (__reduce_min_sync(0xffffffffu, hi) + 1) / TT;  // in tiles as tokens go
  if (lo == 0) return {-im.t0, max(0, end)};
  const int from = max((lo + TT - 1) / TT, im.span.body);
  return {from + im.span.head - im.span.body - im.t0, max(0, end - from)};
}

// Loads tiles, a warp each: TMA boxes through the page table, or cp.async where there are no maps
// (box 0).  A lane per box of the tile (of a token each without maps, four times): its page, looked up
// ahead of the load, and its first token's place in it.
struct TileLoader {
  int box, shift, boxes, t0;
  int page[4], row[4];
  __device__ explicit TileLoader(int b) {
    box = b ? b : 1;
    shift = __ffs(box) - 1;
    boxes = TT >> shift;
  }
  __device__ __forceinline__ void locate(const AttendArgs& a, const Job& im, int i) {
    const int lane = threadIdx.x & 31, bs = a.kv.block_size;
    t0 = im.span.token(im.t0 + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (32 * q >= boxes) break;
      const int t = t0 + ((32 * q + lane) << shift), lb = t / bs;
      page[q] = -1;
      row[q] = t - lb * bs;
      if (32 * q + lane < boxes && lb < a.kv.max_blocks && t <= im.span.hi &&
          (t + box > im.span.lo || t < a.sinks))
        page[q] = __ldg(a.kv.table + (size_t)im.b * a.kv.max_blocks + lb);
      else
        row[q] = -1;
    }
  }
  // The located tile's chunk into st (rows of 128 swizzled bytes) and the 16 bytes behind the codes
  // into sc; valid gets a bit per token that is there, full one arrival.
  __device__ __forceinline__ void load(const AttendArgs& a, const Job& im, const CUtensorMap& codes,
                                       const CUtensorMap& scales, int chunk, uint8_t* st, uint8_t* sc,
                                       uint32_t* valid, uint64_t* full, bool go) {
    const int lane = threadIdx.x & 31;
    if (box > 1) {
      // boxes with a token to see; their other tokens, and what the rest of the slot holds, are masked
      const bool m = page[0] >= 0 && page[0] < a.kv.num_blocks;
      if (row[0] >= 0 && !m) atomicOr(a.status, ST_UNMAPPED_PAGE);
      if (m && go) {
        tma_load_3d(st + ((lane * 128) << shift), &codes, 128 * chunk, row[0], page[0], full);
        tma_load_3d(sc + ((lane * 16) << shift), &scales, a.kv_dim, row[0], page[0], full);
      }
      const uint32_t have = __ballot_sync(0xffffffffu, m);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int t = t0 + 32 * q + lane;
        const bool see = ((have >> ((32 * q + lane) >> shift)) & 1) && t <= im.span.hi &&
                         (t >= im.span.lo || t < a.sinks);
        const uint32_t w = __ballot_sync(0xffffffffu, see);
        if (lane == q) valid[q] = w;
      }
      __syncwarp();
      // (bytes that land before they are expected wait for this arrival all the same)
      if (lane == 0) mbar_arrive_expect_tx(full, go ? __popc(have) * box * (128 + 16) : 0);
      __syncwarp();
    } else {
      const int piece = lane & 7;
      const uint32_t in_chunk = 16 * piece < min(128, a.kv_dim - 128 * chunk) ? 16 : 0;  // (rest: zeros)
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const int pg = q == 0 ? page[0] : q == 1 ? page[1] : q == 2 ? page[2] : page[3];
        const int rw = q == 0 ? row[0] : q == 1 ? row[1] : q == 2 ? row[2] : row[3];
        const bool m = pg >= 0 && pg < a.kv.num_blocks;
        if (rw >= 0 && !m) atomicOr(a.status, ST_UNMAPPED_PAGE);
        const long long off = m ? pg * a.kv.stride_block + rw * a.kv.stride_tok : 0;
        const uint32_t w = __ballot_sync(0xffffffffu, m);
        if (lane == 0) valid[q] = w;
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
          const int k = 4 * e + (lane >> 3), r = 32 * q + k;
          const long long ro = __shfl_sync(0xffffffffu, off, k);
          if (go && ((w >> k) & 1))
            cp_async16(st + r * 128 + ((piece ^ (r & 7)) << 4),
                       a.kv.base + ro + (in_chunk ? 128 * chunk + 16 * piece : 0), in_chunk);
        }
        if (go && m) cp_async16(sc + (32 * q + lane) * 16, a.kv.base + off + a.kv_dim, 16);
      }
      cp_async_wait_all();
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
  }
};

// Eight elements of a query (q: bf16) as two e4m3 terms under the power of two that four neighbouring
// lanes' 32 elements share: its code.  The largest element is in [2^7, 2^8) then, a code's least step
// 2^-9, and eight bits from 2^-2 up are the two terms' eight; smaller elements are off by up to 2^-10.
__device__ __forceinline__ uint32_t split_query(uint4 q, uint2& hi, uint2& lo) {
  float v[8];
  bf16x8_to_f32(q, v);
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (__builtin_expect(isinf(m), 0)) {  // (the codes have no infinity)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (isinf(v[e])) v[e] = __int_as_float(0x7FC00000);
  }
  const uint32_t code = e4m3_block_code(m);
  const float inv = e8m0_inverse(code);
#pragma unroll
  for (int e = 0; e < 8; e += 2) mul2(v[e], v[e + 1], inv);
  hilo_x4(v, hi.x, lo.x);
  hilo_x4(v + 4, hi.y, lo.y);
  return code;
}

}  // namespace attend
}  // namespace mono
