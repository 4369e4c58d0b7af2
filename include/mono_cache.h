/*
 * mono_cache.h -- C ABI of the operators around the decode layer's paged KV cache, for one
 * GB300 (sm_103a): attention of a step's rows over their requests' whole cached context (or a
 * sliding window with first tokens that stay visible, or prefixes that requests share), eviction
 * of the tokens that gathered the least attention weight, appending rows' latents with their
 * rotary positions, and verification of drafted tokens.  They serve the layers whose attention
 * runs outside mono_layer_step (mono_ffn_step takes its output) and the serving loop around a
 * stack of layers; the same library and error codes (mono_layer.h).
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

/*
 * Validates the layout and allocates the workspace on the current device: that of the operator that needs
 * most, for the shared prefixes 8 * (head_dim + 8) bytes a row and head, and 1024 * (head_dim + 8) an SM
 * (25 MB at 48 rows of 64 heads of 128, 94 MB at 1024).
 */
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
 * Attention of requests that share prefixes.  As mono_cache_attend without a window, but the
 * first P = prefix_lengths[prefix_of[b]] tokens of request b are those of a prefix, at
 * prefix_table's row prefix_of[b], and read once for all rows of all its requests; its own tokens,
 * t >= P, are at block_table[b][t / block_size] as ever (entries that lie in the prefix alone are
 * not read), so that both tables may be those of whole contexts.  prefix_of[b] = -1: no prefix;
 * prefix_of NULL: prefix 0 for all.  Row r at position p sees t <= hi, hi as there; a row inside
 * its prefix sees that much of it.  Faster than mono_cache_attend over whole contexts from some 1000
 * shared tokens on, slower where little is shared and requests of a row or two hold many tokens of their own.
 *
 * Sums, refused and masked tokens, status bits, pad rows, lse and the handle's workspace are as in
 * mono_cache_attend; o is rounded to bf16 once, w[t] scale_t to 11 bits before that (and to 2^-30
 * of the largest of the 32 to 128 tokens that set a row's reference), q's elements to 2^-24 of a
 * head's largest; scale_t below 2^-64 in size lose bits of o.  A NaN code of a token in view makes
 * NaN the heads of its slice.  A head whose largest score, of all tokens that its row sees, is beyond
 * 2^27 ln 2 (2^26.5) in size is NaN; tokens that far below 0 weigh nothing beside others.  Rows of
 * requests whose prefix_of is outside [-1, n_prefix) are left out, o = 0, and raise
 * MONO_STATUS_UNMAPPED_PAGE.  A negative length counts as 0.
 *
 * Limits: n_prefix 1..128; 2 * rows * (kv_dim / head_dim) times the tiles (of 128 tokens) of the
 * longer table, and 4 more, below 2^31; both tables' max_blocks * block_size at most 2^31 - 2^16.
 */
typedef struct {
  const void *q;              /* bf16 [rows, n_q_heads * head_dim], 16-byte aligned */
  void *o;                    /* bf16 [rows, n_q_heads * head_dim], not overlapping q */
  int64_t q_stride, o_stride; /* elements between rows, multiples of 8; 0: rows packed */
  const int32_t *positions;   /* [rows], < 0 for a pad row */
  const int32_t *row_req;     /* [rows] request of each row, in any order */
  const int32_t *block_table; /* [n_req, max_blocks] */
  const int32_t *prefix_table; /* [n_prefix, prefix_max_blocks], pages of the same cache */
  const int32_t *prefix_lengths; /* [n_prefix] tokens */
  const int32_t *prefix_of;   /* optional [n_req] */
  int32_t max_blocks, n_req;
  int32_t prefix_max_blocks, n_prefix;
  int32_t rows;               /* 1 <= rows <= max_rows */
  int32_t causal;
  float scale;                /* 2^-20 .. 2^20; 0: 1/sqrt(head_dim) */
  const uint8_t *kv_cache;
  int64_t kv_stride_block, kv_stride_tok, kv_num_blocks;
  float *lse;                 /* optional [rows, n_q_heads] */
} mono_shared_args;

int mono_cache_attend_shared(mono_cache_t *h, const mono_shared_args *args, void *stream);

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
 * Rotary positions.  A row at rotary position t turns every head (or latent slice) x of head_dim
 * elements: of the pairs (x1, x2) of its dimensions [offset, offset + dim), which are neighbours
 * (interleaved != 0) or the halves' elements i and i + dim / 2, pair i becomes
 *   y1 = x1 cos_i - x2 sin_i     y2 = x2 cos_i + x1 sin_i
 * with cos_i = table[t][i], sin_i = table[t][dim / 2 + i] (inverse != 0: -sin_i), products and sums
 * rounded to f32 one by one, the result to its type.  dim is a multiple of 16 up to head_dim, offset
 * one of 8.  A row whose t is outside [0, positions) is skipped and raises MONO_STATUS_POSITION.
 */
typedef struct {
  const float *table;         /* [positions, dim], 16-byte aligned; NULL: no rotation */
  int64_t stride;             /* elements between rows, a multiple of 4; 0: dim */
  int64_t positions;          /* 1 .. 2^31 - 1 */
  int32_t dim, offset;
  int32_t interleaved, inverse;
} mono_rope;

/* Element types of the calls below. */
enum { MONO_TYPE_F32 = 0, MONO_TYPE_BF16 = 1, MONO_TYPE_F16 = 2 };

/*
 * Appending to the cache, with the rotation on the way.  Row r's latent kv[r], its slices turned
 * by rope_positions[r] (NULL: positions[r]; after an eviction the two differ), is stored as the
 * record of slot positions[r] of request row_req[r], as mono_layer_step stores one: s = amax / 448
 * (1 where that is 0), codes = e4m3 of latent / s, to nearest even and saturating, then s; bytes
 * behind them are left as they were.  The rotated latent is not rounded before.  q, if given, is
 * turned by the same positions into q_out (which may be q), every head of it.  Rows with
 * positions[r] < 0 (pad rows) write nothing.  Rows with row_req outside [0, n_req) and rows of
 * unmapped pages store no record (their queries are turned) and raise MONO_STATUS_UNMAPPED_PAGE.
 * A NaN of the latent is a NaN code and does not count in amax; a latent with an infinity gets an
 * infinite scale.  Rows that name the same slot leave an undefined record there.  Any number of
 * rows (at most 2^30) and requests: max_rows and max_req are no limits here, and no workspace is
 * used.
 */
typedef struct {
  const void *kv;             /* [rows, kv_dim], 16-byte aligned, not in the cache */
  const void *q;              /* optional [rows, n_q_heads * head_dim]; needs a table */
  void *q_out;                /* like q: q itself with its stride, or not overlapping it */
  int64_t kv_stride, q_stride, q_out_stride; /* elements between rows, whole 16 bytes; 0: packed */
  const int32_t *positions;   /* [rows], < 0 for a pad row */
  const int32_t *rope_positions; /* optional [rows]; not read without a table */
  const int32_t *row_req;     /* [rows] */
  const int32_t *block_table; /* [n_req, max_blocks] */
  uint8_t *kv_cache;          /* [kv_num_blocks, block_size, record] view, as in mono_step_args */
  int64_t kv_stride_block, kv_stride_tok, kv_num_blocks;
  mono_rope rope;
  int32_t dtype;              /* MONO_TYPE_*, of kv, q and q_out */
  int32_t rows, n_req, max_blocks;
} mono_append_args;

int mono_cache_append(mono_cache_t *h, const mono_append_args *args, void *stream);

/*
 * Rotation alone: heads of head_dim, x into out (which may be x).  The cached latents are values, too,
 * so where they are rotated an attention's output is a sum of values turned by their own positions:
 * turned back (inverse) by the row's position, it depends on the distances only.  Pad rows
 * (positions[r] < 0) are left as they were.  At most 2^30 rows and 2^20 heads.
 */
typedef struct {
  const void *x;              /* [rows, heads * head_dim], 16-byte aligned */
  void *out;                  /* like x: x itself with its stride, or not overlapping it */
  int64_t x_stride, out_stride; /* elements between rows, whole 16 bytes; 0: packed */
  const int32_t *positions;   /* [rows] rotary positions, < 0 for a pad row */
  mono_rope rope;
  int32_t dtype;              /* MONO_TYPE_*, of x and out */
  int32_t rows, heads;
} mono_rotate_args;

int mono_cache_rotate(mono_cache_t *h, const mono_rotate_args *args, void *stream);

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
