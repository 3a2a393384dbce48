// tt_serve_api.cpp -- C ABI of the serving calls (include/tt_serve.h): argument
// checks, then one launch each.
#include "tt_serve_kernels.h"

namespace {

constexpr int64_t MAX_ROWS = (int64_t)1 << 24;
constexpr int64_t MAX_VOCAB = (int64_t)1 << 24;
constexpr int64_t MAX_INT32 = 0x7FFFFFFF;
constexpr int64_t MAX_BLOCK = (int64_t)1 << 20;
constexpr int64_t MAX_LIST = (int64_t)1 << 30;  // entries of a list that is counted in 32 bits
constexpr int64_t MAX_WORDS = (int64_t)1 << 30;  // words of all sets of a call, or that its logits' sets would have

int done(hipError_t e) { return e == hipSuccess ? TT_OK : TT_EHIP; }

// Arguments that plan and release share.
int check_blocks(int64_t rows, int64_t block_size, const void* table, int64_t stride, int64_t width,
                 const void* free_blocks, int64_t free_cap, const void* n_free, const void* lengths,
                 const void* out_lengths, const void* out_n_free, const void* out_n) {
  if (rows < 0 || block_size < 1 || width < 0 || free_cap < 0) return TT_EINVAL;
  if (!n_free || !out_n_free || !out_n || (rows > 0 && (!lengths || !out_lengths))) return TT_EINVAL;
  if ((free_cap > 0 && !free_blocks) || (rows > 0 && width > 0 && !table)) return TT_EINVAL;
  if (rows > 1 && stride < width) return TT_EINVAL;
  if (rows > MAX_ROWS || block_size > MAX_BLOCK || free_cap > MAX_INT32) return TT_ETOOBIG;
  if (width > MAX_INT32 / block_size) return TT_ETOOBIG;
  return TT_OK;
}

int check_grammar(const tt_grammar* g, const void* states, int64_t rows) {
  if (!g || rows < 0 || (rows > 0 && !states)) return TT_EINVAL;
  if (!g->classes || !g->next || !g->accept || g->n_states < 1 || g->n_classes < 1 || g->n_classes > 256)
    return TT_EINVAL;
  if (g->end_id < -1 || g->n_bytes < 0 || g->n_tokens < 0) return TT_EINVAL;
  if ((g->n_bytes > 0 && !g->strings) || (g->n_tokens > 0 && !g->string_offsets)) return TT_EINVAL;
  if (g->n_states > 32767 || g->n_bytes > MAX_INT32 || g->n_tokens > MAX_VOCAB || rows > MAX_ROWS) return TT_ETOOBIG;
  return TT_OK;
}

}  // namespace

extern "C" {

int tt_plan_blocks(const tt_plan_args* args, hipStream_t stream) {
  if (!args) return TT_EINVAL;
  const tt_plan_args& a = *args;
  const int rc = check_blocks(a.rows, a.block_size, a.table, a.table_stride, a.width, a.free_blocks, a.free_cap,
                              a.n_free, a.lengths, a.out_lengths, a.out_n_free, a.out_n);
  if (rc != TT_OK) return rc;
  if (a.places < 0 || (a.places > 0 && !a.slots) || (!a.offsets && a.places < a.rows)) return TT_EINVAL;
  if (a.places > MAX_INT32) return TT_ETOOBIG;
  return done(tt::launch_plan(a, stream));
}

int tt_release_blocks(const int32_t* lengths, const uint8_t* done_rows, int64_t rows, int64_t block_size,
                      const int32_t* table, int64_t table_stride, int64_t width, int32_t* free_blocks,
                      int64_t free_cap, const int32_t* n_free, int32_t* out_lengths, int32_t* out_n_free,
                      int64_t* out_n, hipStream_t stream) {
  const int rc = check_blocks(rows, block_size, table, table_stride, width, free_blocks, free_cap, n_free, lengths,
                              out_lengths, out_n_free, out_n);
  if (rc != TT_OK) return rc;
  if (rows > 0 && !done_rows) return TT_EINVAL;
  return done(tt::launch_release({lengths, done_rows, rows, block_size, table, table_stride, width, free_blocks,
                                  free_cap, n_free, out_lengths, out_n_free, out_n},
                                 stream));
}

int tt_token_bits(const int32_t* ids, int64_t n, const int64_t* offsets, int64_t rows, int64_t vocab, int32_t* bits,
                  int64_t bits_stride, int add, hipStream_t stream) {
  const int64_t words = (vocab + 31) / 32;
  if (n < 0 || rows < 0 || vocab < 0 || (!offsets && rows != 1) || (n > 0 && !ids)) return TT_EINVAL;
  if (vocab > MAX_VOCAB || rows > MAX_ROWS) return TT_ETOOBIG;
  if (rows == 0 || vocab == 0) return TT_OK;
  if (!bits || (rows > 1 && bits_stride < words)) return TT_EINVAL;
  if (rows * words > MAX_WORDS) return TT_ETOOBIG;
  return done(tt::launch_token_bits(ids, n, offsets, rows, vocab, bits, bits_stride, add != 0, stream));
}

int tt_grammar_bits(const tt_grammar* grammar, const int32_t* states, int64_t rows, int32_t* bits,
                    int64_t bits_stride, int64_t vocab, hipStream_t stream) {
  const int rc = check_grammar(grammar, states, rows);
  if (rc != TT_OK) return rc;
  if (vocab < 0) return TT_EINVAL;
  if (vocab > MAX_VOCAB) return TT_ETOOBIG;
  if (rows == 0 || vocab == 0) return TT_OK;
  const int64_t words = (vocab + 31) / 32;
  if (!bits || (rows > 1 && bits_stride < words)) return TT_EINVAL;
  if (rows * words > MAX_WORDS) return TT_ETOOBIG;
  return done(tt::launch_grammar_bits(*grammar, states, rows, bits, bits_stride, vocab, stream));
}

int tt_grammar_advance(const tt_grammar* grammar, const int32_t* states, const int32_t* tokens, int64_t rows,
                       int32_t* out_states, hipStream_t stream) {
  const int rc = check_grammar(grammar, states, rows);
  if (rc != TT_OK) return rc;
  if (rows == 0) return TT_OK;
  if (!tokens || !out_states) return TT_EINVAL;
  return done(tt::launch_grammar_advance(*grammar, states, tokens, rows, out_states, stream));
}

int tt_shape_logits(const tt_shape_args* args, hipStream_t stream) {
  if (!args) return TT_EINVAL;
  const tt_shape_args& a = *args;
  if (a.rows < 0 || a.vocab < 0) return TT_EINVAL;
  if (a.in_type < TT_F32 || a.in_type > TT_BF16 || (a.out_type != a.in_type && a.out_type != TT_F32)) return TT_EINVAL;
  if (a.rows > MAX_ROWS || a.vocab > MAX_VOCAB) return TT_ETOOBIG;
  if (a.rows == 0 || a.vocab == 0) return TT_OK;
  const int64_t words = (a.vocab + 31) / 32;
  if (!a.logits || !a.out) return TT_EINVAL;
  // rows that are only read may lie on each other (one row for all: stride 0)
  if (a.logits_stride < 0 || (a.rows > 1 && a.out_stride < a.vocab)) return TT_EINVAL;
  if (a.out == a.logits && (a.out_type != a.in_type || (a.rows > 1 && a.out_stride != a.logits_stride)))
    return TT_EINVAL;
  if (a.seen && a.seen_stride < 0) return TT_EINVAL;
  if (a.generated && (a.generated_cap < 0 || a.generated_stride < 0)) return TT_EINVAL;
  if (a.n_bias < 0 || (a.bias_offsets && a.n_bias > 0 && (!a.bias_ids || !a.bias_values))) return TT_EINVAL;
  if (a.allowed && (a.allowed_count < 0 || a.allowed_stride < 0)) return TT_EINVAL;
  if (a.generated_cap > MAX_LIST || a.n_bias > MAX_LIST) return TT_ETOOBIG;
  if (a.rows * words > MAX_WORDS) return TT_ETOOBIG;
  return done(tt::launch_shape(a, stream));
}

}  // extern "C"
