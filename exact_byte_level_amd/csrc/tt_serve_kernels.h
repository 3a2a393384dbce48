// tt_serve_kernels.h -- launchers of the serving kernels (enqueue only, no host sync).
#pragma once
#include <hip/hip_runtime.h>

#include "tt_serve.h"

namespace tt {

struct ReleaseArgs {
  const int32_t* lengths;
  const uint8_t* done;
  int64_t rows, block_size;
  const int32_t* table;
  int64_t table_stride, width;
  int32_t* free_blocks;
  int64_t free_cap;
  const int32_t* n_free;
  int32_t* out_lengths;
  int32_t* out_n_free;
  int64_t* out_n;
};

hipError_t launch_plan(const tt_plan_args& a, hipStream_t st);
hipError_t launch_release(const ReleaseArgs& a, hipStream_t st);
hipError_t launch_token_bits(const int32_t* ids, int64_t n, const int64_t* offsets, int64_t rows, int64_t vocab,
                             int32_t* bits, int64_t stride, bool add, hipStream_t st);
hipError_t launch_grammar_bits(const tt_grammar& g, const int32_t* states, int64_t rows, int32_t* bits,
                               int64_t stride, int64_t vocab, hipStream_t st);
hipError_t launch_grammar_advance(const tt_grammar& g, const int32_t* states, const int32_t* tokens, int64_t rows,
                                  int32_t* out, hipStream_t st);
hipError_t launch_shape(const tt_shape_args& a, hipStream_t st);

}  // namespace tt
