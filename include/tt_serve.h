/* tt_serve.h -- what a serving step needs next to the tokenizer, on one gfx950 GPU.
 *
 * C ABI of libtt.so, beside tt.h.  Between two calls of the model a serving
 * program turns request lengths into block tables and slots of a paged cache,
 * and the model's logits into the ones a token is chosen from: repeated tokens
 * penalised, biases added, tokens that the answer's grammar forbids taken out.
 * These calls do that on the device, from the ids and offsets that
 * tt_encode_batch leaves there and from the byte strings of the tokens.
 *
 * Conventions
 *  - As in tt.h: device pointers are the caller's, every call only enqueues on
 *    the given stream, allocates nothing and can be captured into a HIP graph;
 *    return values are 0 or a negative TT_E* code for argument and launch
 *    errors, data errors are written on the device into the count the caller
 *    reads.  Except for tt_vocab_* no call needs a loaded tokenizer, and calls
 *    on different streams do not disturb each other.  tt_vocab_* are
 *    host-synchronous and may run beside a call that loads another tokenizer.
 *  - A token set is a row of 32-bit words: token id v is bit v & 31 of word
 *    v >> 5, and a vocabulary of V ids takes (V + 31) / 32 words.  A call
 *    takes at most 2^24 rows, and rows times words of at most 2^30.
 *  - Rows of matrices may be any number of elements apart (the *_stride
 *    arguments; in tt_shape_logits rows that are only read may share their
 *    memory: stride 0), and no alignment beyond that of the element is needed.
 */
#ifndef TT_SERVE_H
#define TT_SERVE_H

#include "tt.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TT_ENOBLOCKS -11 /* fewer free blocks than the requests need (device-side) */

/* Element types of logits. */
#define TT_F32  0
#define TT_F16  1
#define TT_BF16 2

/* States of a grammar that are not states of its automaton, and in
 * tt_shape_logits rows of `allowed` that are no rows of it. */
#define TT_STATE_DEAD -1 /* nothing may follow: an empty set */
#define TT_STATE_FREE -2 /* no grammar: every token may follow */

/* ------------------------------------------------------------ block tables
 *
 * A cache of keys and values is kept in blocks of block_size tokens.  Row r of
 * the table names the blocks of request r in order, so that token p of r lives
 * in slot  table[r][p / block_size] * block_size + p % block_size.  Blocks that
 * no request holds are the first n_free entries of the free list.
 */
typedef struct tt_plan_args {
  const int32_t* lengths;     /* [rows] tokens that each request has in the cache; negative: row not in use */
  const int64_t* offsets;     /* [rows + 1] new tokens of row r are offsets[r] .. offsets[r+1] (as tt_encode_batch
                                 gives them; offsets[0] == 0); NULL: one new token for every row in use */
  int64_t rows;               /* 0 .. 2^24 */
  int64_t places;             /* length of slots, positions, row_of; >= rows if offsets is NULL */
  int64_t block_size;         /* 1 .. 2^20 */
  int32_t* table;             /* [rows][width]; receives the new blocks, nothing else changes */
  int64_t table_stride;
  int64_t width;              /* blocks that a row has room for; width * block_size <= 2^31 - 1 */
  const int32_t* free_blocks; /* [free_cap] */
  int64_t free_cap;
  const int32_t* n_free;      /* [1] */
  int64_t* slots;             /* [places] */
  int32_t* positions;         /* [places] place of the token in its request; may be NULL */
  int32_t* row_of;            /* [places] its row; may be NULL */
  int32_t* out_lengths;       /* [rows]; may be lengths */
  int32_t* out_n_free;        /* [1]; may be n_free */
  int64_t* out_n;             /* [1] */
} tt_plan_args;

/* tt_plan_blocks -- give the requests the blocks that their new tokens need.
 *
 * The new tokens of row r follow its lengths[r] tokens.  A row not in use takes none if
 * offsets is NULL, and starts at 0 if offsets give it some.  Blocks are taken
 * from the end of the free list: the first new block of the first row is
 * free_blocks[n_free - 1].  Token i of row r is at place offsets[r] + i, or at
 * place r if offsets is NULL; places that hold no token receive -1 in slots, positions
 * and row_of, so that a launch of fixed size can skip them.  A slot whose block is negative is -1.
 * out_n receives the number of new tokens, out_lengths the new lengths,
 * out_n_free the blocks left.  On a data error nothing changes (out_lengths and
 * out_n_free are copies, every place is -1) and out_n receives TT_EOFFSETS
 * (offsets not from 0 or not in order), TT_ETOOBIG (a row beyond its width, or
 * more tokens than places), TT_EINVAL (n_free outside 0 .. free_cap) or
 * TT_ENOBLOCKS.
 * Buffers that are written must not overlap others, but for the two named.
 * Returns TT_OK, TT_EINVAL, TT_ETOOBIG or TT_EHIP. */
int tt_plan_blocks(const tt_plan_args* args, hipStream_t stream);

/* tt_release_blocks -- take back the blocks of the requests that ended.
 *
 * Rows r with done[r] != 0 that are in use give back their blocks, row by
 * row in the order of the table (whatever it holds, negative entries too), to free_blocks from entry n_free on;
 * out_lengths[r] = -1.  The other rows keep their lengths; the table itself is
 * not touched.  out_n receives the number of blocks, or, with nothing changed,
 * TT_ETOOBIG (a row beyond its width, or more blocks than free_cap has room for) or
 * TT_EINVAL (n_free outside 0 .. free_cap).  out_lengths may be lengths and
 * out_n_free n_free.  Returns TT_OK, TT_EINVAL, TT_ETOOBIG or TT_EHIP. */
int tt_release_blocks(const int32_t* lengths, const uint8_t* done, int64_t rows, int64_t block_size,
                      const int32_t* table, int64_t table_stride, int64_t width, int32_t* free_blocks,
                      int64_t free_cap, const int32_t* n_free, int32_t* out_lengths, int32_t* out_n_free,
                      int64_t* out_n, hipStream_t stream);

/* -------------------------------------------------------------- token sets */

/* tt_token_bits -- the set of the tokens of each text.
 *
 * ids          device int32[n]; ids outside 0 .. vocab-1 are passed over.
 * offsets      device int64[rows + 1]: text r is ids[offsets[r] .. offsets[r+1]);
 *              NULL: one text of n ids.  Bounds outside 0 .. n are taken as the nearest in it.
 * bits         device int32[rows][words], bits_stride words apart; with
 *              add != 0 the sets are joined to what is there, else written.
 * vocab        0 .. 2^24.
 * Returns TT_OK, TT_EINVAL, TT_ETOOBIG or TT_EHIP. */
int tt_token_bits(const int32_t* ids, int64_t n, const int64_t* offsets, int64_t rows, int64_t vocab,
                  int32_t* bits, int64_t bits_stride, int add, hipStream_t stream);

/* A grammar: an automaton over bytes, its bytes put into classes that it does
 * not tell apart.  Token strings: token v is bytes string_offsets[v] ..
 * string_offsets[v+1]; a token without bytes is never allowed. */
typedef struct tt_grammar {
  const uint8_t* classes;         /* device [256], each < n_classes */
  const int16_t* next;            /* device [n_states][n_classes]; an entry outside 0 .. n_states-1 is dead */
  const uint8_t* accept;          /* device [n_states] */
  int64_t n_states;               /* 1 .. 32767 */
  int64_t n_classes;              /* 1 .. 256 */
  int64_t end_id;                 /* token allowed where accept is set, and nowhere else; -1: none */
  const uint8_t* strings;         /* device [n_bytes] */
  int64_t n_bytes;                /* 0 .. 2^31 - 1 */
  const int32_t* string_offsets;  /* device [n_tokens + 1] */
  int64_t n_tokens;               /* 0 .. 2^24 */
} tt_grammar;

/* tt_grammar_bits -- the tokens that may follow each state.
 *
 * Bit v of row r is set where the bytes of token v can be read from
 * states[r] without a dead entry.  TT_STATE_FREE sets every bit below vocab;
 * any other value that is no state sets none.  Ids from n_tokens on are not
 * allowed, but for end_id. */
int tt_grammar_bits(const tt_grammar* grammar, const int32_t* states, int64_t rows, int32_t* bits,
                    int64_t bits_stride, int64_t vocab, hipStream_t stream);

/* tt_grammar_advance -- the states after one more token each.
 *
 * out_states[r] (may be states) is the state after the bytes of tokens[r]:
 * TT_STATE_DEAD after a token that is not allowed and after end_id,
 * TT_STATE_FREE stays.  A negative token leaves the state as it is. */
int tt_grammar_advance(const tt_grammar* grammar, const int32_t* states, const int32_t* tokens, int64_t rows,
                       int32_t* out_states, hipStream_t stream);

/* ------------------------------------------------------------------ logits */

typedef struct tt_shape_args {
  const void* logits;          /* [rows][vocab] of in_type */
  int64_t logits_stride;
  void* out;                   /* [rows][vocab] of out_type; may be logits if type and stride are the same */
  int64_t out_stride;
  int64_t rows, vocab;         /* vocab 0 .. 2^24 */
  int64_t in_type, out_type;   /* TT_F32, TT_F16, TT_BF16; out_type is in_type or TT_F32 */
  const int32_t* seen;         /* token sets [rows] of the prompts; NULL: none */
  int64_t seen_stride;
  const int32_t* generated;    /* [rows][generated_cap] tokens generated so far; NULL: none */
  int64_t generated_stride, generated_cap;  /* cap 0 .. 2^30 */
  const int32_t* n_generated;  /* [rows], taken into 0 .. generated_cap; NULL: generated_cap */
  const float* repetition;     /* [rows] rho; NULL: 1 */
  const float* frequency;      /* [rows] phi; NULL: 0 */
  const float* presence;       /* [rows] pi; NULL: 0 */
  const int64_t* bias_offsets; /* [rows + 1] biases of row r are entries bias_offsets[r] .. bias_offsets[r+1]; NULL: none */
  const int32_t* bias_ids;     /* [n_bias] */
  const float* bias_values;    /* [n_bias] */
  int64_t n_bias;              /* 0 .. 2^30 */
  const int32_t* allowed;      /* token sets [allowed_count]; NULL: every token is allowed */
  int64_t allowed_stride, allowed_count;
  const int32_t* allowed_rows; /* [rows] which set each row goes by, or TT_STATE_FREE; NULL: set r */
  const float* temperature;    /* [rows]; NULL or not above 0: not scaled */
} tt_shape_args;

/* tt_shape_logits -- the logits a token is chosen from.
 *
 * For row r and token v, with c the times v is in generated[r] and s whether c > 0 or v is in seen[r]:
 *   x = logits[r][v]
 *   s:   x = x > 0 ? x / rho : x * rho
 *        x = x - phi * c - pi * (c > 0)
 *        x = x + bias; of a token that a row's entries name twice the last entry counts
 *   v not in the row's allowed set (or allowed_rows[r] is no set and not TT_STATE_FREE): x = -infinity
 *   temperature > 0:  x = x / temperature
 * computed in 32 bits and rounded once to out_type.  A token that is not
 * allowed is -infinity whatever its logit, NaN included; a row with an empty
 * set is -infinity throughout.  Ids outside 0 .. vocab-1 are passed over.
 * Returns TT_OK, TT_EINVAL, TT_ETOOBIG or TT_EHIP. */
int tt_shape_logits(const tt_shape_args* args, hipStream_t stream);

/* -------------------------------------------------------------- vocabulary */

/* tt_vocab_size -- tokens of the loaded tokenizer (256 + merges) and the
 * length of their strings.  Reads the device, so it waits for it. */
int tt_vocab_size(int64_t* n_tokens, int64_t* n_bytes);

/* tt_vocab_strings -- the strings, to host buffers: bytes[n_bytes], offsets[n_tokens + 1], with the sizes that
 * tt_vocab_size gave.  TT_ESTALE, and nothing written, if the tokenizer that is loaded by now has others.
 * Returns TT_OK, TT_EINVAL, TT_ENOTLOADED, TT_ESTALE, TT_ENOMEM, TT_ETOOBIG (strings beyond 2^31 - 1 bytes) or TT_EHIP. */
int tt_vocab_strings(uint8_t* bytes, int32_t* offsets, int64_t n_tokens, int64_t n_bytes);

#ifdef __cplusplus
}
#endif
#endif /* TT_SERVE_H */
