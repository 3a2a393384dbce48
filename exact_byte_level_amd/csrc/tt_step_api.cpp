// tt_step_api.cpp -- C ABI of the operators around the model (include/tt_step.h): argument checks, then the launches.
#include "tt_step_kernels.h"

namespace {

constexpr int64_t MAX_INT32 = 0x7FFFFFFF;
constexpr int64_t MAX_BLOCK = (int64_t)1 << 20;
constexpr int64_t MAX_HEADS = 4096;
constexpr int64_t MAX_ROWS = (int64_t)1 << 24;
constexpr int64_t MAX_VOCAB = (int64_t)1 << 24;
constexpr int64_t MAX_LOGITS = (int64_t)1 << 35;

int done(hipError_t e) { return e == hipSuccess ? TT_OK : TT_EHIP; }

int check_cache(const tt_paged_cache& c) {
  if (c.blocks < 0 || c.block_size < 1 || c.heads < 1 || c.dim < 8 || c.dim % 8) return TT_EINVAL;
  if (c.type != TT_F16 && c.type != TT_BF16 && c.type != TT_E4M3) return TT_EINVAL;
  if (c.blocks > 0 && (!c.keys || !c.values)) return TT_EINVAL;
  if (c.blocks > MAX_INT32 || c.block_size > MAX_BLOCK || c.heads > MAX_HEADS || c.dim > 256) return TT_ETOOBIG;
  return TT_OK;
}

}  // namespace

extern "C" {

int tt_write_cache(const tt_write_args* args, hipStream_t stream) {
  if (!args) return TT_EINVAL;
  const tt_write_args& a = *args;
  const int rc = check_cache(a.cache);
  if (rc != TT_OK) return rc;
  if (a.tokens < 0 || a.in_type < TT_F32 || a.in_type > TT_BF16) return TT_EINVAL;
  if (a.in_type != TT_F32 && a.cache.type != TT_E4M3 && a.cache.type != a.in_type) return TT_EINVAL;
  if (a.tokens > MAX_INT32) return TT_ETOOBIG;
  if (a.tokens == 0) return TT_OK;
  if (!a.keys || !a.values || !a.slots) return TT_EINVAL;
  if (a.cache.blocks == 0) return TT_OK;
  return done(tt::launch_write(a, stream));
}

int64_t tt_attend_workspace(int64_t queries, int64_t heads, int64_t cache_heads, int64_t dim) {
  if (queries < 0 || cache_heads < 1 || heads < cache_heads || heads % cache_heads || dim < 8 || dim % 8) return TT_EINVAL;
  if (heads > MAX_HEADS || dim > 256 || queries > MAX_INT32 / heads) return TT_ETOOBIG;
  return tt::attend_workspace(queries, heads, cache_heads, dim);
}

int tt_attend_cache(const tt_attend_args* args, hipStream_t stream) {
  if (!args) return TT_EINVAL;
  const tt_attend_args& a = *args;
  const int rc = check_cache(a.cache);
  if (rc != TT_OK) return rc;
  const int64_t bytes = tt_attend_workspace(a.queries, a.heads, a.cache.heads, a.cache.dim);
  if (bytes < 0) return (int)bytes;
  if ((a.type != TT_F16 && a.type != TT_BF16) || (a.cache.type != a.type && a.cache.type != TT_E4M3)) return TT_EINVAL;
  if (a.table_rows < 0 || a.width < 0 || a.window < 0 || !(a.softcap == 0 || (a.softcap >= 1e-6 && a.softcap <= 1e20))) return TT_EINVAL;
  if (a.table_rows > MAX_INT32 || a.width > MAX_INT32 / a.cache.block_size) return TT_ETOOBIG;
  if (a.queries == 0) return TT_OK;
  if (!a.query || !a.out || !a.lengths || (!a.table && a.table_rows > 0 && a.width > 0)) return TT_EINVAL;
  if (a.workspace_bytes < bytes || (bytes > 0 && (!a.workspace || reinterpret_cast<uintptr_t>(a.workspace) % 16))) return TT_EINVAL;
  return done(tt::launch_attend(a, stream));
}

int64_t tt_sample_workspace(int64_t rows, int64_t vocab) {
  if (rows < 0 || vocab < 0) return TT_EINVAL;
  if (rows > MAX_ROWS || vocab > MAX_VOCAB || rows * vocab > MAX_LOGITS) return TT_ETOOBIG;
  return tt::sample_workspace(rows, vocab);
}

int tt_sample_tokens(const tt_sample_args* args, hipStream_t stream) {
  if (!args) return TT_EINVAL;
  const tt_sample_args& a = *args;
  const int64_t bytes = tt_sample_workspace(a.rows, a.vocab);
  if (bytes < 0) return (int)bytes;
  if (a.type < TT_F32 || a.type > TT_BF16 || a.logits_stride < 0) return TT_EINVAL;
  if (a.rows == 0) return TT_OK;
  if (!a.uniform || !a.tokens || (a.vocab > 0 && !a.logits)) return TT_EINVAL;
  if (a.workspace_bytes < bytes || (bytes > 0 && (!a.workspace || reinterpret_cast<uintptr_t>(a.workspace) % 16))) return TT_EINVAL;
  return done(tt::launch_sample(a, stream));
}

}  // extern "C"
