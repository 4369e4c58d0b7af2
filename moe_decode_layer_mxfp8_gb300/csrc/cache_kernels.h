// Internal launch interface between the host side of the cache operators (cache_ops.cu) and
// their kernels.
#pragma once

#include "kernels.h"

namespace mono {

// The paged cache as the kernels see it: record of (request, token) through the block table.
struct PagedView {
  const uint8_t* base;
  long long stride_block, stride_tok, num_blocks;
  const int* table;
  int max_blocks, block_size;
};
// Byte offset of token t's record of request b; negative where the page is unmapped.
__device__ __forceinline__ long long record_offset(const PagedView& v, int b, int t) {
  const int lb = t / v.block_size;
  if (lb >= v.max_blocks) return -1;
  const int pb = __ldg(v.table + (size_t)b * v.max_blocks + lb);
  if (pb < 0 || pb >= v.num_blocks) return -1;
  return (long long)pb * v.stride_block + (long long)(t - lb * v.block_size) * v.stride_tok;
}

struct AttendArgs {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  long long q_stride, o_stride;
  const int *positions, *row_req;
  PagedView kv;
  int rows, n_req;
  int n_q, head_dim, kv_dim;
  int window, sinks, causal;
  float scale;
  float* lse;  // [rows, n_q] (the caller's, or the workspace's when only weights are asked for)
  float* weights;
  long long weights_stride, weights_cols;
  int* status;
};

struct EvictArgs {
  const float* weights;
  float* weights_out;
  long long weights_stride, weights_out_stride, weights_cols, weights_out_cols;
  const int* lengths;
  int* new_lengths;
  int* kept;
  long long kept_stride;
  int budget, sinks, recent, n_req;
  PagedView src;
  PagedView dst;
  uint8_t* dst_base;
  int in_place;
  int copy_bytes;  // bytes of a record that move: kv_dim + 4 rounded up to 16
  int* status;
};

struct VerifyArgs {
  const void *target, *draft;
  long long target_stride, draft_stride;
  int vocab, rows, n_req;
  const int *row_start, *draft_tokens, *greedy;
  const float *u, *r;
  int *accepted, *tokens;
};

size_t attend_workspace_bytes(int max_rows, int sms);
cudaError_t attend_prepare();  // raises the dynamic shared-memory limit
cudaError_t launch_attend(const Launch&, const AttendArgs&, uint8_t* workspace, int max_rows,
                          int sms);
constexpr int EVICT_MAX_CHUNKS = 1 << 18;  // moves of 64 kept tokens that a call may have
size_t evict_workspace_bytes(int max_req);
bool evict_fits(int n_req, int budget, long long cap);
cudaError_t evict_prepare();
cudaError_t launch_evict(const Launch&, const EvictArgs&, uint8_t* workspace, int max_req, int sms);
cudaError_t launch_verify(const Launch&, const VerifyArgs&, int dtype, int sms);

}  // namespace mono
