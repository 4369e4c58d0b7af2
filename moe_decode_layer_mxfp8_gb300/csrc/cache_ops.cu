// Host side of the cache operators' C ABI (include/mono_cache.h): argument checks, the
// workspace, launches.
#include <algorithm>
#include <cmath>
#include <new>

#include "../../include/mono_cache.h"
#include "cache_kernels.h"

using namespace mono;

struct mono_cache {
  mono_cache_spec spec;
  int device = 0;
  uint8_t* arena = nullptr;
  float* lse = nullptr;
  // What a call's kernels leave to each other, whichever the operator: a handle's calls follow one another on the
  // GPU, every kernel waits for those before it ahead of its first access, and none reads what its call did not write.
  uint8_t* workspace = nullptr;
  int sms = 0;
  int* status = nullptr;
  cudaError_t shared_ready = cudaSuccess;  // (the others do without that kernel)
};

namespace {

int cuda_code(cudaError_t e) {
  if (e == cudaSuccess) return MONO_OK;
  (void)cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? MONO_ERR_OUT_OF_MEMORY : MONO_ERR_CUDA;
}

bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_layout(const mono_cache_spec& s) {
  if (s.head_dim != 64 && s.head_dim != 128) return MONO_ERR_UNSUPPORTED_DIMS;
  if (s.kv_dim <= 0 || s.kv_dim > 1024 || s.kv_dim % s.head_dim) return MONO_ERR_UNSUPPORTED_DIMS;
  const int G = s.kv_dim / s.head_dim;
  if (s.n_q_heads <= 0 || s.n_q_heads % G || s.n_q_heads / G > 16) return MONO_ERR_UNSUPPORTED_DIMS;
  if (s.block_size <= 0 || s.block_size > (1 << 20)) return MONO_ERR_UNSUPPORTED_DIMS;
  if (s.kv_record_bytes < s.kv_dim + 4 || s.kv_record_bytes % 16 || s.kv_record_bytes > (1 << 20))
    return MONO_ERR_UNSUPPORTED_DIMS;
  if (s.max_rows < 1 || s.max_rows > 1024 || s.max_req < 1 || s.max_req > 512)
    return MONO_ERR_TOO_MANY_ROWS;
  return MONO_OK;
}

// A cache view of the handle's layout: 16-byte aligned, records and pages not overlapping.
int check_view(const mono_cache_spec& s, const void* base, int64_t stride_block,
               int64_t stride_tok, int64_t num_blocks, int max_blocks) {
  if (num_blocks < 1 || max_blocks < 1) return MONO_ERR_INVALID_ARG;
  // token indices are 32-bit, also those of the rest of a tile and of a cluster's threads behind the last
  if ((int64_t)max_blocks * s.block_size > INT32_MAX - 65535) return MONO_ERR_INVALID_ARG;
  if (!aligned(base, 16) || stride_tok % 16 || stride_block % 16) return MONO_ERR_BAD_ALIGNMENT;
  if (stride_tok < s.kv_record_bytes || stride_tok > INT64_MAX / (1 << 20) ||
      stride_block < (int64_t)s.block_size * stride_tok)
    return MONO_ERR_BAD_KV_VIEW;
  return MONO_OK;
}

// Rows of `cols` elements (0: stride) that lie `stride` apart.
bool check_cols(int64_t stride, int64_t cols) { return stride >= 1 && cols >= 0 && cols <= stride; }

constexpr int MAX_ROTATED = 1 << 30;      // rows of a rotating call
constexpr int TYPE_BYTES[3] = {4, 2, 2};  // MONO_TYPE_*
bool check_dtype(int dtype) { return dtype >= MONO_TYPE_F32 && dtype <= MONO_TYPE_F16; }

// Rows of `width` elements that lie `stride` apart (0: packed), in whole 16 bytes.
int check_rows(const void* p, int64_t width, int64_t* stride, int bytes) {
  if (!*stride) *stride = width;
  if (*stride < width) return MONO_ERR_INVALID_ARG;
  return aligned(p, 16) && *stride * bytes % 16 == 0 ? MONO_OK : MONO_ERR_BAD_ALIGNMENT;
}

// A rotation of heads of head_dim elements.
int check_rope(const mono_rope& r, int head_dim, Rope* out) {
  if (!r.table) return MONO_ERR_INVALID_ARG;
  if (r.dim < 16 || r.dim % 16 || r.dim > head_dim || r.offset < 0 || r.offset % 8 ||
      r.offset > head_dim - r.dim)
    return MONO_ERR_UNSUPPORTED_DIMS;
  int64_t stride = r.stride;
  const int rc = check_rows(r.table, r.dim, &stride, 4);
  if (rc != MONO_OK) return rc;
  if (r.positions < 1 || r.positions > INT32_MAX || stride > INT64_MAX / 4 / r.positions)
    return MONO_ERR_INVALID_ARG;
  *out = {r.table, stride, (int)r.positions, r.dim, r.offset, r.interleaved != 0, r.inverse != 0};
  return MONO_OK;
}

int check_device(const mono_cache* h) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_code(e);
  return dev == h->device ? MONO_OK : MONO_ERR_UNSUPPORTED_DEVICE;
}

#define TRY(x)                      \
  do {                              \
    const int rc_ = (x);            \
    if (rc_ != MONO_OK) return rc_; \
  } while (0)

}  // namespace

extern "C" {

int mono_cache_build(const mono_cache_spec* spec, mono_cache_t** out) {
  if (!out) return MONO_ERR_INVALID_ARG;
  *out = nullptr;
  if (!spec) return MONO_ERR_INVALID_ARG;
  TRY(check_layout(*spec));
  int dev = 0;
  cudaDeviceProp prop;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaGetDeviceProperties(&prop, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return MONO_ERR_CUDA;
  }
  if (prop.major != 10 || prop.minor != 3) return MONO_ERR_UNSUPPORTED_DEVICE;
  mono_cache* h = new (std::nothrow) mono_cache();
  if (!h) return MONO_ERR_OUT_OF_MEMORY;
  h->spec = *spec;
  h->device = dev;
  const size_t lse = ((size_t)spec->max_rows * spec->n_q_heads * 4 + 255) / 256 * 256;
  const size_t bytes = 256 + lse +
                       std::max({attend_workspace_bytes(spec->max_rows, prop.multiProcessorCount),
                                 evict_workspace_bytes(spec->max_req),
                                 shared_workspace_bytes(spec->max_rows, spec->n_q_heads, spec->head_dim,
                                                        prop.multiProcessorCount)});
  cudaError_t e = cudaMalloc(&h->arena, bytes);
  if (e == cudaSuccess) e = cudaMemset(h->arena, 0, 256);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = attend_prepare();
  if (e == cudaSuccess) e = evict_prepare();
  if (e != cudaSuccess) {
    mono_cache_free(h);
    return cuda_code(e);
  }
  h->shared_ready = shared_prepare();
  if (h->shared_ready != cudaSuccess) (void)cudaGetLastError();
  h->status = reinterpret_cast<int*>(h->arena);
  h->lse = reinterpret_cast<float*>(h->arena + 256);
  h->workspace = h->arena + 256 + lse;
  h->sms = prop.multiProcessorCount;
  *out = h;
  return MONO_OK;
}

void mono_cache_free(mono_cache_t* h) {
  if (!h) return;
  if (h->arena) cudaFree(h->arena);
  delete h;
}

int mono_cache_status(mono_cache_t* h, int clear) {
  if (!h) return MONO_ERR_INVALID_ARG;
  int v = 0, dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev != h->device) e = cudaSetDevice(h->device);
  // (a copy on the default stream does not wait for streams that do not block with it)
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&v, h->status, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && clear) e = cudaMemset(h->status, 0, sizeof(int));
  if (e == cudaSuccess && clear) e = cudaDeviceSynchronize();
  if (dev >= 0 && dev != h->device) (void)cudaSetDevice(dev);
  return e == cudaSuccess ? v : cuda_code(e);
}

int mono_cache_attend(mono_cache_t* h, const mono_attend_args* a, void* stream) {
  if (!h || !a) return MONO_ERR_INVALID_ARG;
  const mono_cache_spec& s = h->spec;
  if (a->rows < 1 || a->n_req < 1) return MONO_ERR_INVALID_ARG;
  if (a->rows > s.max_rows || a->n_req > s.max_req) return MONO_ERR_TOO_MANY_ROWS;
  if (!a->q || !a->o || !a->positions || !a->row_req || !a->block_table || !a->kv_cache)
    return MONO_ERR_INVALID_ARG;
  if (a->window < 0 || a->sinks < 0 || !std::isfinite(a->scale) || a->scale < 0.0f)
    return MONO_ERR_INVALID_ARG;
  if (a->weights && !check_cols(a->weights_stride, a->weights_cols)) return MONO_ERR_INVALID_ARG;
  const int64_t width = (int64_t)s.n_q_heads * s.head_dim;
  const int64_t qs = a->q_stride ? a->q_stride : width, os = a->o_stride ? a->o_stride : width;
  if (qs < width || os < width) return MONO_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->o, 16) || qs % 8 || os % 8 || !aligned(a->positions, 4) ||
      !aligned(a->row_req, 4) || !aligned(a->block_table, 4) || !aligned(a->lse, 4) ||
      !aligned(a->weights, 4))
    return MONO_ERR_BAD_ALIGNMENT;
  TRY(check_view(s, a->kv_cache, a->kv_stride_block, a->kv_stride_tok, a->kv_num_blocks,
                 a->max_blocks));
  // (work is counted in 32 bits: tiles of 128 tokens, and some more, over all rows)
  if ((((int64_t)a->max_blocks * s.block_size + 127) / 128 + 16) * a->rows > INT32_MAX)
    return MONO_ERR_INVALID_ARG;
  TRY(check_device(h));
  AttendArgs k = {};
  k.q = static_cast<const __nv_bfloat16*>(a->q);
  k.o = static_cast<__nv_bfloat16*>(a->o);
  k.q_stride = qs;
  k.o_stride = os;
  k.positions = a->positions;
  k.row_req = a->row_req;
  k.kv = {a->kv_cache, a->kv_stride_block, a->kv_stride_tok, a->kv_num_blocks,
          a->block_table, a->max_blocks, s.block_size};
  k.rows = a->rows;
  k.n_req = a->n_req;
  k.n_q = s.n_q_heads;
  k.head_dim = s.head_dim;
  k.kv_dim = s.kv_dim;
  k.window = a->window;
  k.sinks = a->sinks;
  k.causal = a->causal != 0;
  k.scale = a->scale > 0.0f ? a->scale : 1.0f / sqrtf((float)s.head_dim);
  k.lse = a->lse ? a->lse : h->lse;
  k.weights = a->weights;
  k.weights_stride = a->weights_stride;
  k.weights_cols = a->weights_cols ? a->weights_cols : a->weights_stride;
  k.status = h->status;
  return cuda_code(launch_attend(Launch{reinterpret_cast<cudaStream_t>(stream), true}, k,
                                 h->workspace, s.max_rows, h->sms));
}

int mono_cache_attend_shared(mono_cache_t* h, const mono_shared_args* a, void* stream) {
  if (!h || !a) return MONO_ERR_INVALID_ARG;
  const mono_cache_spec& s = h->spec;
  if (a->rows < 1 || a->n_req < 1 || a->n_prefix < 1) return MONO_ERR_INVALID_ARG;
  if (a->rows > s.max_rows || a->n_req > s.max_req || a->n_prefix > MAX_PREFIX)
    return MONO_ERR_TOO_MANY_ROWS;
  if (!a->q || !a->o || !a->positions || !a->row_req || !a->block_table || !a->prefix_table ||
      !a->prefix_lengths || !a->kv_cache)
    return MONO_ERR_INVALID_ARG;
  // (the tokens' factors hold it, 2^64 times as large or 2^-64; a NaN is refused)
  if (a->scale != 0.0f && !(a->scale >= 0x1p-20f && a->scale <= 0x1p20f)) return MONO_ERR_INVALID_ARG;
  const int64_t width = (int64_t)s.n_q_heads * s.head_dim;
  int64_t qs = a->q_stride, os = a->o_stride;
  TRY(check_rows(a->q, width, &qs, 2));
  TRY(check_rows(a->o, width, &os, 2));
  if (!aligned(a->positions, 4) || !aligned(a->row_req, 4) || !aligned(a->block_table, 4) ||
      !aligned(a->prefix_table, 4) || !aligned(a->prefix_lengths, 4) || !aligned(a->prefix_of, 4) ||
      !aligned(a->lse, 4))
    return MONO_ERR_BAD_ALIGNMENT;
  TRY(check_view(s, a->kv_cache, a->kv_stride_block, a->kv_stride_tok, a->kv_num_blocks,
                 a->max_blocks));
  TRY(check_view(s, a->kv_cache, a->kv_stride_block, a->kv_stride_tok, a->kv_num_blocks,
                 a->prefix_max_blocks));
  if (!shared_fits(a->rows, s.kv_dim / s.head_dim,
                   (int64_t)std::max(a->max_blocks, a->prefix_max_blocks) * s.block_size))
    return MONO_ERR_INVALID_ARG;
  TRY(check_device(h));
  if (h->shared_ready != cudaSuccess) return cuda_code(h->shared_ready);
  SharedArgs k = {};
  k.q = static_cast<const __nv_bfloat16*>(a->q);
  k.o = static_cast<__nv_bfloat16*>(a->o);
  k.q_stride = qs;
  k.o_stride = os;
  k.positions = a->positions;
  k.row_req = a->row_req;
  k.kv = {a->kv_cache, a->kv_stride_block, a->kv_stride_tok, a->kv_num_blocks,
          a->block_table, a->max_blocks, s.block_size};
  k.pre = k.kv;
  k.pre.table = a->prefix_table;
  k.pre.max_blocks = a->prefix_max_blocks;
  k.prefix_lengths = a->prefix_lengths;
  k.prefix_of = a->prefix_of;
  k.rows = a->rows;
  k.n_req = a->n_req;
  k.n_prefix = a->n_prefix;
  k.n_q = s.n_q_heads;
  k.head_dim = s.head_dim;
  k.kv_dim = s.kv_dim;
  k.causal = a->causal != 0;
  k.scale = a->scale > 0.0f ? a->scale : 1.0f / sqrtf((float)s.head_dim);
  k.lse = a->lse;
  k.status = h->status;
  return cuda_code(launch_attend_shared(Launch{reinterpret_cast<cudaStream_t>(stream), true}, k,
                                        h->workspace, s.max_rows, h->sms));
}

int mono_cache_evict(mono_cache_t* h, const mono_evict_args* a, void* stream) {
  if (!h || !a) return MONO_ERR_INVALID_ARG;
  const mono_cache_spec& s = h->spec;
  if (a->n_req < 1) return MONO_ERR_INVALID_ARG;
  if (a->n_req > s.max_req) return MONO_ERR_TOO_MANY_ROWS;
  if (!a->weights || !a->lengths || !a->new_lengths || !a->kept || !a->block_table || !a->kv_cache)
    return MONO_ERR_INVALID_ARG;
  if (a->budget < 1 || a->sinks < 0 || a->recent < 0 ||
      (int64_t)a->sinks + a->recent > a->budget || a->kept_stride < a->budget)
    return MONO_ERR_INVALID_ARG;
  if (!check_cols(a->weights_stride, a->weights_cols) ||
      (a->weights_out && !check_cols(a->weights_out_stride, a->weights_out_cols)))
    return MONO_ERR_INVALID_ARG;
  const int64_t cols = a->weights_cols ? a->weights_cols : a->weights_stride;
  if (a->weights_out == a->weights && a->weights_out_stride != a->weights_stride)
    return MONO_ERR_INVALID_ARG;  // in place means row for row
  if (a->dst_cache && !a->dst_table) return MONO_ERR_INVALID_ARG;
  if (!aligned(a->weights, 4) || !aligned(a->weights_out, 4) || !aligned(a->lengths, 4) ||
      !aligned(a->new_lengths, 4) || !aligned(a->kept, 4) || !aligned(a->block_table, 4) ||
      !aligned(a->dst_table, 4))
    return MONO_ERR_BAD_ALIGNMENT;
  TRY(check_view(s, a->kv_cache, a->kv_stride_block, a->kv_stride_tok, a->kv_num_blocks,
                 a->max_blocks));
  EvictArgs k = {};
  k.src = {a->kv_cache, a->kv_stride_block, a->kv_stride_tok, a->kv_num_blocks,
           a->block_table, a->max_blocks, s.block_size};
  k.dst = k.src;
  k.dst_base = a->kv_cache;
  k.in_place = a->dst_table == nullptr;
  if (a->dst_table) {
    k.dst.table = a->dst_table;
    k.dst.max_blocks = a->dst_max_blocks;
    if (a->dst_cache) {
      k.dst_base = a->dst_cache;
      k.dst.base = a->dst_cache;
      k.dst.stride_block = a->dst_stride_block;
      k.dst.stride_tok = a->dst_stride_tok;
      k.dst.num_blocks = a->dst_num_blocks;
    }
    TRY(check_view(s, k.dst_base, k.dst.stride_block, k.dst.stride_tok, k.dst.num_blocks,
                   a->dst_max_blocks));
  }
  if (!evict_fits(a->n_req, a->budget,
                  std::min((int64_t)a->max_blocks * s.block_size, cols)))
    return MONO_ERR_TOO_MANY_ROWS;
  TRY(check_device(h));
  k.weights = a->weights;
  k.weights_out = a->weights_out ? a->weights_out : const_cast<float*>(a->weights);
  k.weights_stride = a->weights_stride;
  k.weights_out_stride = a->weights_out ? a->weights_out_stride : a->weights_stride;
  k.weights_cols = cols;
  k.weights_out_cols = !a->weights_out ? cols : a->weights_out_cols ? a->weights_out_cols : a->weights_out_stride;
  k.lengths = a->lengths;
  k.new_lengths = a->new_lengths;
  k.kept = a->kept;
  k.kept_stride = a->kept_stride;
  k.budget = a->budget;
  k.sinks = a->sinks;
  k.recent = a->recent;
  k.n_req = a->n_req;
  k.copy_bytes = (s.kv_dim + 4 + 15) / 16 * 16;
  k.status = h->status;
  return cuda_code(launch_evict(Launch{reinterpret_cast<cudaStream_t>(stream), true}, k,
                                h->workspace, s.max_req, h->sms));
}

int mono_cache_append(mono_cache_t* h, const mono_append_args* a, void* stream) {
  if (!h || !a) return MONO_ERR_INVALID_ARG;
  const mono_cache_spec& s = h->spec;
  if (a->rows < 1 || a->n_req < 1 || !check_dtype(a->dtype)) return MONO_ERR_INVALID_ARG;
  if (a->rows > MAX_ROTATED) return MONO_ERR_TOO_MANY_ROWS;
  if (!a->kv || !a->positions || !a->row_req || !a->block_table || !a->kv_cache)
    return MONO_ERR_INVALID_ARG;
  if (!a->q != !a->q_out || (a->q && !a->rope.table)) return MONO_ERR_INVALID_ARG;
  RotateArgs k = {};
  int64_t ks = a->kv_stride, qs = a->q_stride, os = a->q_out_stride;
  TRY(check_rows(a->kv, s.kv_dim, &ks, TYPE_BYTES[a->dtype]));
  if (a->q) {
    const int64_t width = (int64_t)s.n_q_heads * s.head_dim;
    TRY(check_rows(a->q, width, &qs, TYPE_BYTES[a->dtype]));
    TRY(check_rows(a->q_out, width, &os, TYPE_BYTES[a->dtype]));
    if (a->q == a->q_out && qs != os) return MONO_ERR_INVALID_ARG;  // in place means row for row
  }
  if (!aligned(a->positions, 4) || !aligned(a->rope_positions, 4) || !aligned(a->row_req, 4) ||
      !aligned(a->block_table, 4))
    return MONO_ERR_BAD_ALIGNMENT;
  if (a->rope.table) TRY(check_rope(a->rope, s.head_dim, &k.rope));
  TRY(check_view(s, a->kv_cache, a->kv_stride_block, a->kv_stride_tok, a->kv_num_blocks,
                 a->max_blocks));
  TRY(check_device(h));
  k.rows = a->rows;
  k.head_dim = s.head_dim;
  k.positions = a->positions;
  k.rope_positions = a->rope.table ? a->rope_positions : nullptr;
  k.x = a->q;
  k.out = a->q_out;
  k.x_stride = qs;
  k.out_stride = os;
  k.heads = s.n_q_heads;
  k.kv = a->kv;
  k.kv_stride = ks;
  k.kv_dim = s.kv_dim;
  k.n_req = a->n_req;
  k.row_req = a->row_req;
  k.cache = {a->kv_cache, a->kv_stride_block, a->kv_stride_tok, a->kv_num_blocks,
             a->block_table, a->max_blocks, s.block_size};
  k.status = h->status;
  return cuda_code(launch_rotate(Launch{reinterpret_cast<cudaStream_t>(stream), true}, k, a->dtype, h->sms));
}

int mono_cache_rotate(mono_cache_t* h, const mono_rotate_args* a, void* stream) {
  if (!h || !a) return MONO_ERR_INVALID_ARG;
  const mono_cache_spec& s = h->spec;
  if (a->rows < 1 || a->heads < 1 || !check_dtype(a->dtype)) return MONO_ERR_INVALID_ARG;
  if (a->rows > MAX_ROTATED) return MONO_ERR_TOO_MANY_ROWS;
  if (a->heads > (1 << 20)) return MONO_ERR_UNSUPPORTED_DIMS;
  if (!a->x || !a->out || !a->positions) return MONO_ERR_INVALID_ARG;
  RotateArgs k = {};
  int64_t xs = a->x_stride, os = a->out_stride;
  const int64_t width = (int64_t)a->heads * s.head_dim;
  TRY(check_rows(a->x, width, &xs, TYPE_BYTES[a->dtype]));
  TRY(check_rows(a->out, width, &os, TYPE_BYTES[a->dtype]));
  if (a->x == a->out && xs != os) return MONO_ERR_INVALID_ARG;
  if (!aligned(a->positions, 4)) return MONO_ERR_BAD_ALIGNMENT;
  TRY(check_rope(a->rope, s.head_dim, &k.rope));
  TRY(check_device(h));
  k.rows = a->rows;
  k.head_dim = s.head_dim;
  k.positions = a->positions;
  k.x = a->x;
  k.out = a->out;
  k.x_stride = xs;
  k.out_stride = os;
  k.heads = a->heads;
  k.status = h->status;
  return cuda_code(launch_rotate(Launch{reinterpret_cast<cudaStream_t>(stream), true}, k, a->dtype, h->sms));
}

int mono_verify_drafts(const mono_verify_args* a, void* stream) {
  if (!a) return MONO_ERR_INVALID_ARG;
  if (!a->target || !a->row_start || !a->draft_tokens || !a->u || !a->r || !a->accepted ||
      !a->tokens)
    return MONO_ERR_INVALID_ARG;
  if (a->vocab < 1 || a->rows < 1 || a->n_req < 1) return MONO_ERR_INVALID_ARG;
  if (a->vocab > INT32_MAX - 63) return MONO_ERR_INVALID_ARG;  // (indices run to the end of a vector)
  if (a->dtype < MONO_PROB_F32 || a->dtype > MONO_PROB_F16) return MONO_ERR_INVALID_ARG;
  if (a->target_stride < a->vocab || (a->draft && a->draft_stride < a->vocab))
    return MONO_ERR_INVALID_ARG;
  const int es = a->dtype == MONO_PROB_F32 ? 4 : 2;
  if (!aligned(a->target, es) || !aligned(a->draft, es) || !aligned(a->row_start, 4) ||
      !aligned(a->draft_tokens, 4) || !aligned(a->u, 4) || !aligned(a->r, 4) ||
      !aligned(a->greedy, 4) || !aligned(a->accepted, 4) || !aligned(a->tokens, 4))
    return MONO_ERR_BAD_ALIGNMENT;
  int dev = 0, major = 0, minor = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_code(e);
  if (major != 10 || minor != 3) return MONO_ERR_UNSUPPORTED_DEVICE;
  VerifyArgs k = {a->target, a->draft, a->target_stride, a->draft_stride, a->vocab, a->rows,
                  a->n_req, a->row_start, a->draft_tokens, a->greedy, a->u, a->r, a->accepted,
                  a->tokens};
  return cuda_code(
      launch_verify(Launch{reinterpret_cast<cudaStream_t>(stream), true}, k, a->dtype, sms));
}

}  // extern "C"
