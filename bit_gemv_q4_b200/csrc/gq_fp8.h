// gq_fp8.h -- the few-token product of 8-bit block-scaled matrices
// (gq_fp8_gemv.cu) as gq_gemm_fp8 sees it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gq.h"

namespace gq {

// Largest batch that takes it: two tiles of 8 tokens.
constexpr int64_t kFp8GemvMaxB = 16;

// Arguments as for gq_gemm_fp8, checked there; no workspace.
gq_status fp8_gemv(const void* W, const float* sw, int64_t M, int64_t K, const void* X, const float* sx,
                   int64_t B, void* Y, int yt, bool pdl, cudaStream_t s);

}  // namespace gq
