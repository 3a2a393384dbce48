/* tt_step.h -- the operators around the model in a serving step, on one gfx950 GPU.
 *
 * C ABI of libtt.so, beside tt_serve.h.  That one turns request lengths into
 * the slots of a paged cache and the model's logits into the ones a token is
 * chosen from; these calls put keys and values into the slots, let new tokens
 * attend to what the cache holds of their requests, and choose the token.
 *
 * Conventions are those of tt_serve.h: device pointers are the caller's, every
 * call only enqueues on the given stream, allocates nothing and can be captured
 * into a HIP graph; return values are 0 or a negative TT_E* code.  What a device
 * tensor names that is not there (a row, a block, a slot) is passed over.
 * Strides count elements; the elements of one head, and of one row of logits,
 * lie one behind the other; no alignment beyond that of the element is needed.
 * What is written must not overlap anything else that the call is given.
 * A workspace need not be initialised; calls that may run at the same time
 * (on two streams, or in two graphs that are replayed at once) need one each.
 */
#ifndef TT_STEP_H
#define TT_STEP_H

#include "tt_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of caches beside TT_F16 and TT_BF16: 8 bits, 1.4.3, no infinities, largest value 448. */
#define TT_E4M3 3

/* The keys and values of one layer: element d of head h at place p of block b is at
 * b * block_stride + p * place_stride + h * head_stride + d.  Slot s is place
 * s % block_size of block s / block_size, as tt_plan_blocks gives them.  An
 * element stands for its value times its head's scale. */
typedef struct tt_paged_cache {
  void* keys;
  int64_t key_block_stride, key_place_stride, key_head_stride;
  void* values;
  int64_t value_block_stride, value_place_stride, value_head_stride;
  const float* key_scale;    /* [heads]; NULL: 1 */
  const float* value_scale;  /* [heads]; NULL: 1 */
  int64_t blocks;            /* 0 .. 2^31 - 1 */
  int64_t block_size;        /* 1 .. 2^20 */
  int64_t heads;             /* 1 .. 4096 */
  int64_t dim;               /* a multiple of 8, 8 .. 256 */
  int64_t type;              /* TT_F16, TT_BF16, TT_E4M3 */
} tt_paged_cache;

typedef struct tt_write_args {
  const void* keys;          /* [tokens][heads][dim] of in_type */
  int64_t key_stride, key_head_stride;
  const void* values;
  int64_t value_stride, value_head_stride;
  const int64_t* slots;      /* [tokens] */
  int64_t tokens;            /* 0 .. 2^31 - 1 */
  int64_t in_type;           /* TT_F32, TT_F16, TT_BF16; the cache's type is in_type, TT_E4M3, or of 16 bits after TT_F32 */
  tt_paged_cache cache;
} tt_write_args;

/* tt_write_cache -- put the keys and values of new tokens into their slots.
 *
 * Each element is divided by its head's scale in 32 bits and rounded once to
 * the cache's type, with TT_E4M3 after being taken into -448 .. 448 (NaN stays).
 * Tokens whose slot is negative or past the cache are passed over, and nothing
 * else of the cache changes.  Of a slot named twice each element is one of
 * those given.  Returns TT_OK, TT_EINVAL, TT_ETOOBIG or TT_EHIP. */
int tt_write_cache(const tt_write_args* args, hipStream_t stream);

typedef struct tt_attend_args {
  const void* query;         /* [queries][heads][dim] of type */
  int64_t query_stride, query_head_stride;
  void* out;                 /* [queries][heads][dim] of type */
  int64_t out_stride, out_head_stride;
  float* lse;                /* [queries][heads]; NULL: not wanted */
  int64_t lse_stride;
  int64_t queries;           /* 0 .. 2^31 - 1; queries times heads at most 2^31 - 1 */
  int64_t heads;             /* a multiple of the cache's: heads / cache.heads one behind the other share a head of keys; at most 4096 */
  int64_t type;              /* TT_F16, TT_BF16 */
  tt_paged_cache cache;      /* its type is type or TT_E4M3 */
  const int32_t* table;      /* [table_rows][width] blocks of each request; a token in a block outside the cache is not seen */
  int64_t table_stride, table_rows, width;  /* width * cache.block_size <= 2^31 - 1 */
  const int32_t* lengths;    /* [queries] tokens that each query sees, from its request's first on; not above 0: none */
  /* [queries] row of the table that each goes by; NULL: row i.  No row of it: sees nothing.  Queries of a row read its tokens together where
   * queries are more than table_rows, 512 at most, and no more than 8 heads of them share a head of keys; else each by itself. */
  const int32_t* rows;
  double scale;              /* of the scores */
  double softcap;            /* 0, or 1e-6 .. 1e20: scores x become softcap * tanh(x / softcap) */
  int64_t window;            /* above 0: only the last `window` of the tokens are seen */
  void* workspace;           /* tt_attend_workspace bytes, at 16 bytes; may be NULL if that is 0 */
  int64_t workspace_bytes;
} tt_attend_args;

/* tt_attend_cache -- the attention of each query over the cached tokens of its request.
 *
 *   x_t = scale * key_scale * <query, key_t>, capped if softcap is above 0
 *   out = value_scale * sum_t e^x_t value_t / sum_t e^x_t        lse = ln sum_t e^x_t
 *
 * Scores, maxima and sums are held in 32 bits.  A weight goes into its product as two terms
 * of the query's type: off by 2^-16 of it at most with TT_BF16; with TT_F16 by 2^-22 of it, or of the
 * largest weight among the 32 tokens that it is taken together with (of less than 2^-64 of
 * the query's largest it has fewer bits).  out is rounded once.  A query that
 * sees nothing, or whose scores are all -infinity, gets zeros and -infinity; what the
 * cache holds elsewhere, NaN included, has no effect.  Values that are seen are
 * meant to be finite: an infinite one gives infinities or NaN to the queries that see it.
 * A query after tt_plan_blocks sees out_lengths[r] tokens of row r, or, of several new
 * tokens of a row, positions + 1 of row row_of; places without a token (-1) give zeros.
 * Made for single tokens and short runs of them: every query reads its tokens.
 * Returns TT_OK, TT_EINVAL, TT_ETOOBIG or TT_EHIP. */
int tt_attend_cache(const tt_attend_args* args, hipStream_t stream);

/* tt_attend_workspace -- bytes that a call of these sizes needs beside its tensors, or TT_EINVAL. */
int64_t tt_attend_workspace(int64_t queries, int64_t heads, int64_t cache_heads, int64_t dim);

typedef struct tt_sample_args {
  const void* logits;        /* [rows][vocab] of type */
  int64_t logits_stride;     /* rows may lie on each other (stride 0) */
  int64_t rows, vocab;       /* 0 .. 2^24 each, rows times vocab at most 2^35 */
  int64_t type;              /* TT_F32, TT_F16, TT_BF16 */
  const float* uniform;      /* [rows] random numbers from 0 to below 1; what is outside is taken as the nearest in it, NaN as 0 */
  const float* temperature;  /* [rows]; NULL: 1; not above 0: the likeliest token */
  const int32_t* top_k;      /* [rows]; NULL or not above 0: not limited */
  const float* top_p;        /* [rows]; NULL or not below 1: not limited */
  const float* min_p;        /* [rows]; NULL or not above 0: not limited */
  int32_t* tokens;           /* [rows] */
  float* logprobs;           /* [rows]; NULL: not wanted */
  void* workspace;           /* tt_sample_workspace bytes, at 16 bytes */
  int64_t workspace_bytes;
} tt_sample_args;

/* tt_sample_tokens -- draw each row's next token.
 *
 * Tokens go by falling logits, equal ones by rising ids, and weigh
 * w = e^((x - max) / temperature).  Kept are, of the row's tokens, the first top_k; of these
 * the fewest from the first on whose weights reach top_p times the sum of these; of those, the ones
 * that weigh min_p or more (all limits keep the first token).  The token drawn is the
 * first, by ids, at which the running sum of the kept weights is above uniform times their sum;
 * logprobs receives ln(w / sum of the kept weights).
 * Weights and sums are held in 64 bits; a weight below 2^-1000 is zero.  A logit that is NaN counts as -infinity; a
 * token of -infinity is never drawn, and a row without any other gets token -1 and
 * -infinity.  Where logits are +infinity the others weigh nothing.
 * Returns TT_OK, TT_EINVAL, TT_ETOOBIG or TT_EHIP. */
int tt_sample_tokens(const tt_sample_args* args, hipStream_t stream);

/* tt_sample_workspace -- bytes that a call of these sizes needs beside its tensors, or TT_EINVAL. */
int64_t tt_sample_workspace(int64_t rows, int64_t vocab);

#ifdef __cplusplus
}
#endif
#endif /* TT_STEP_H */
