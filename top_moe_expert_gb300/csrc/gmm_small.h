// gmm_small.h -- the grouped product of a few rows (gmm_small.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_ffn.h"

namespace moe {

constexpr int kSmallRows = 4;

moe_status_t grouped_mm_small(const void *x, const void *w, int dt, const int32_t *off, int R, int E, int N, int K, void *y,
                              int ydt, int32_t *dev_status, cudaStream_t s);

}  // namespace moe
