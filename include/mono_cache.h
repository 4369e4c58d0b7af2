/*
 * mono_cache.h -- C ABI of the operators around the decode layer's paged KV cache, for one
 * GB300 (sm_103a): attention of a step's rows over their requests' whole cached context (or a
 * sliding window with first tokens that stay visible), eviction of the tokens that gathered
 * the least attention weight, and verification of drafted tokens.  They serve the layers
 * whose attention runs outside mono_layer_step (mono_ffn_step takes its output) and the
 * serving loop around a stack of layers; the same library and error codes (mono_layer.h).
 *
 * Conventions are those of mono_layer.h: device pointers borrowed from the caller, negative
 * MONO_ERR_* codes and no aborts, arguments checked on the host before anything is enqueued,
 * no allocation and no host synchronisation in a call (each can be captured in a CUDA graph),
 * work enqueued on the given stream of the handle's device, which must be current.
 */
#ifndef MONO_CACHE_H
#define MONO_CACHE_H

#include "mono_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mono_cache mono_cache_t; /* opaque handle: a cache layout and its workspace */

/*
 * The cache layout (the fields of mono_layer_spec of the same names, with the same
 * constraints: head_dim 64 or 128; kv_dim a multiple of head_dim, at most 1024; n_q_heads a
 * multiple of kv_dim/head_dim with at most 16 heads per latent slice; kv_record_bytes >=
 * kv_dim + 4 and a multiple of 16) and the largest step: 1..1024 rows of 1..512 requests.
 */
typedef struct {
  int32_t n_q_heads, head_dim, kv_dim;
  int32_t block_size, kv_record_bytes;
  int32_t max_rows, max_req;
} mono_cache_spec;

/* Validates the layout and allocates the workspace on the current device. */
int mono_cache_build(const mono_cache_spec *spec, mono_cache_t **out);
/* Releases it.  NULL is accepted. */
void mono_cache_free(mono_cache_t *h);
/* Waits for all work on the handle's device, whatever its stream, and reads the handle's status word
 * (MONO_STATUS_* bits, >= 0; or a negative error code); clears the word when `clear` is non-zero. */
int mono_cache_status(mono_cache_t *h, int clear);

/*
 * Attention over the cache.  Row r of request b = row_req[r] at position p = positions[r] sees
 * the cached tokens t <= hi with, when window > 0, t > hi - window or t < sinks; hi = p when
 * causal, else the largest position of b's rows in this call.  Its own token's record (and
 * those of the rows before it) must be in the cache already, as mono_layer_step's insert
 * leaves them.  Head h reads latent slice g = h / (n_q_heads / (kv_dim/head_dim)) as key and value:
 *   s[t] = scale * scale_t * (q_h . codes_t,g)     w = softmax(s)     o_h = sum_t w[t] scale_t codes_t,g
 * with every sum in f32.  o is rounded to bf16 once; before that w[t] scale_t is rounded to 8 bits (and
 * to 2^-17 of the largest of 32 tokens), or to 11 where rows / n_req, rounded up, times the heads of a
 * 128-byte run of the record is above 32 (lse is of weights as they are), and q's elements to 2^-17 of
 * the largest of their 32.  Rows with
 * positions[r] < 0 (pad rows) and rows that see no token give o = 0 and lse = -inf.  Tokens outside a
 * row's view never reach its result, whatever their records hold.  A NaN code of a token in view makes
 * NaN the heads whose slices lie in its 128-byte run of the record; a scale that is NaN or beyond 2^64 in
 * size, all heads.  A head whose largest scores (of all tokens, or of a run of them) are beyond 2^26 in
 * size is NaN.  Tokens of unmapped pages (table entries outside [0, kv_num_blocks), logical pages >=
 * max_blocks) and rows with row_req outside [0, n_req) are left out and raise
 * MONO_STATUS_UNMAPPED_PAGE.  A wait that runs out raises MONO_STATUS_WAIT_TIMEOUT; the step's outputs
 * are then undefined.
 *
 * n_req is the number of rows of block_table; those that no row of the step belongs to cost little, but
 * a table of the step's requests alone lets the kernels group rows best.
 *
 * weights, if given, gathers every cached token's attention weight: weights[b][t] += the sum
 * over b's rows and all heads of w[t], for t < weights_cols.  The order of that sum is fixed; it is added
 * a few of b's rows at a time (three at 16 heads a slice), each addition rounded to f32.
 *
 * Limits: max_blocks * block_size at most 2^31 - 2^16; its tiles of 128 tokens, and 16 more, times rows
 * below 2^31.
 *
 * One handle's calls share its workspace: they must be ordered on the GPU (one stream, or
 * events between streams; graphs captured from one handle must not run at the same time).
 */
typedef struct {
  const void *q;              /* bf16 [rows, n_q_heads * head_dim], 16-byte aligned */
  void *o;                    /* bf16 [rows, n_q_heads * head_dim], not overlapping q */
  int64_t q_stride, o_stride; /* elements between rows, multiples of 8; 0: rows packed */
  const int32_t *positions;   /* [rows], < 0 for a pad row */
  const int32_t *row_req;     /* [rows] request of each row, in any order */
  const int32_t *block_table; /* [n_req, max_blocks] physical page of each logical page */
  int32_t max_blocks, n_req;
  int32_t rows;               /* 1 <= rows <= max_rows */
  int32_t window, sinks;      /* window 0: the whole context */
  int32_t causal;
  float scale;                /* 0: 1/sqrt(head_dim) */
  const uint8_t *kv_cache;    /* [kv_num_blocks, block_size, record] view, as in mono_step_args */
  int64_t kv_stride_block, kv_stride_tok, kv_num_blocks;
  float *lse;                 /* optional [rows, n_q_heads]: ln sum_t exp(s[t]) */
  float *weights;             /* optional [n_req, weights_cols], added to */
  int64_t weights_stride;     /* elements between rows */
  int64_t weights_cols;       /* <= weights_stride; 0: the stride */
} mono_attend_args;

int mono_cache_attend(mono_cache_t *h, const mono_attend_args *args, void *stream);

/*
 * Eviction.  Request b holds lengths[b] tokens in slots 0, 1, ... of its pages.  If that is
 * more than `budget`, it keeps its first `sinks` slots, its last `recent` ones and, of the
 * others, those with the largest weights (of equal ones the lowest slots; a NaN counts as
 * -inf), `budget` in all; else it keeps everything.  The kept records move, in slot order, to slots
 * 0, 1, ... of the destination, their weights with them:
 *   kept[b][i] = old slot of the token now in slot i, -1 from new_lengths[b] up to budget
 *   weights_out[b][i] = weights[b][kept[b][i]], 0 from new_lengths[b] up to lengths[b]
 * (within weights_out's columns).  Positions of later steps continue at new_lengths[b].
 * Destination: dst_table NULL moves the records within the request's own pages; a dst_table
 * names other pages, of dst_cache or, where that is NULL, of kv_cache, none of them a page
 * that a request still holds tokens in.  weights_out NULL, or equal to weights with the same
 * stride, compacts them in place; any other overlap is undefined.  new_lengths may be lengths.
 * No two requests may share a page.  Slots and pages beyond the kept tokens are left as they
 * were.  Lengths beyond the pages of the table or the weights' rows are cut to them, records of
 * unmapped pages are not moved; both raise MONO_STATUS_UNMAPPED_PAGE.  A call keeps at most
 * 2^24 tokens over its requests, each counted with the budget (or what its table or weights
 * row hold, if less) rounded up to 64: MONO_ERR_TOO_MANY_ROWS.  Calls share the handle's workspace,
 * as mono_cache_attend's do.
 */
typedef struct {
  const float *weights;       /* [n_req, weights_cols] */
  float *weights_out;         /* optional [n_req, weights_out_cols] */
  int64_t weights_stride, weights_out_stride; /* elements between rows */
  const int32_t *lengths;     /* [n_req] */
  int32_t *new_lengths;       /* [n_req] */
  int32_t *kept;              /* [n_req, kept_stride] */
  int64_t kept_stride;        /* >= budget */
  int32_t budget, sinks, recent; /* budget >= 1, sinks + recent <= budget */
  int32_t n_req;              /* 1 <= n_req <= max_req */
  const int32_t *block_table; /* [n_req, max_blocks] */
  int32_t max_blocks;
  uint8_t *kv_cache;
  int64_t kv_stride_block, kv_stride_tok, kv_num_blocks;
  const int32_t *dst_table;   /* optional [n_req, dst_max_blocks] */
  int32_t dst_max_blocks;
  uint8_t *dst_cache;         /* optional; the strides below are read only when it is given */
  int64_t dst_stride_block, dst_stride_tok, dst_num_blocks;
  int64_t weights_cols, weights_out_cols; /* at most their strides; 0: the strides */
} mono_evict_args;

int mono_cache_evict(mono_cache_t *h, const mono_evict_args *args, void *stream);

/*
 * Verification of drafted tokens.  Request b's rows are [row_start[b], row_start[b + 1]): one
 * per drafted token and a last one behind them; target row j holds the target's probabilities
 * p_j for the token that draft_tokens[j] proposes, draft row j the draft model's q_j (NULL: the
 * drafts are certain, q_j(x_j) = 1 and 0 elsewhere).  In row order draft x_j is accepted while
 * u[j] * q_j(x_j) < p_j(x_j); at the first refusal the token is drawn from max(p_j - q_j, 0) (from
 * p_j where that is 0 everywhere), and from p_j in the last row if every draft stands, by
 * inversion: the smallest v with sum_{i <= v} w_i > r[b] * sum_i w_i.  The rows' tokens then
 * follow the target's distribution.  A request with greedy[b] != 0 accepts x_j while it is p_j's
 * first maximum, and takes p_j's first maximum where it stops (its target rows may then hold
 * logits; a NaN counts as -inf).
 *   accepted[b] = number of accepted drafts
 *   tokens[row] = accepted drafts, then the drawn token, then -1
 * Tests and sums are carried in enough bits (products exact, sums in two f32) that roundings
 * decide nothing in practice.  Rows need not be normalised; negative and NaN entries count as 0
 * where a token is drawn, and a draw from zeros yields -1.  An infinite target entry leaves nothing
 * to draw from (-1), an infinite draft entry takes all of the target's.  Drafted tokens outside
 * [0, vocab) are refused.  Requests without rows get accepted[b] = 0; rows outside every request
 * keep their tokens; row_start entries are cut to [0, rows].
 */
enum { MONO_PROB_F32 = 0, MONO_PROB_BF16 = 1, MONO_PROB_F16 = 2 };
typedef struct {
  const void *target;           /* [rows, vocab] */
  const void *draft;            /* optional [rows, vocab] */
  int64_t target_stride, draft_stride; /* elements between rows, >= vocab */
  int32_t dtype;                /* MONO_PROB_*, of both */
  int32_t vocab, rows, n_req;   /* vocab at most 2^31 - 64 */
  const int32_t *row_start;     /* [n_req + 1] */
  const int32_t *draft_tokens;  /* [rows] */
  const float *u;               /* [rows], uniform in [0, 1) */
  const float *r;               /* [n_req], uniform in [0, 1) */
  const int32_t *greedy;        /* optional [n_req] */
  int32_t *accepted;            /* [n_req] */
  int32_t *tokens;              /* [rows] */
} mono_verify_args;

int mono_verify_drafts(const mono_verify_args *args, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MONO_CACHE_H */
