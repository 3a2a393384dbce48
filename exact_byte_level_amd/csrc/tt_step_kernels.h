// tt_step_kernels.h -- launchers of the kernels around the model (enqueue only, no host sync).
#pragma once
#include <hip/hip_runtime.h>

#include "tt_step.h"

namespace tt {

hipError_t launch_write(const tt_write_args& a, hipStream_t st);
hipError_t launch_attend(const tt_attend_args& a, hipStream_t st);
int64_t attend_workspace(int64_t queries, int64_t heads, int64_t cache_heads, int64_t dim);
hipError_t launch_sample(const tt_sample_args& a, hipStream_t st);
int64_t sample_workspace(int64_t rows, int64_t vocab);

}  // namespace tt
