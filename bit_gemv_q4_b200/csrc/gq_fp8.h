// gq_fp8.h -- the few-token product of 8-bit block-scaled matrices
// (gq_fp8_gemv.cu) as gq_gemm_fp8 sees it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gq.h"

namespace gq {

// Whether a call takes it: up to 8 tokens, or up to 16 with few weights (16
// tokens x 4096 x 4096: 7.8 us against 9.3 on tcgen05; x 11008 x 4096: 19.8
// against 16.8).
inline bool fp8_gemv_takes(int64_t M, int64_t K, int64_t B) {
  return B <= 8 || (B <= 16 && M * K <= 3 * (int64_t{1} << 23));
}

// Arguments as for gq_gemm_fp8, checked there; no workspace.
gq_status fp8_gemv(const void* W, const float* sw, int64_t M, int64_t K, const void* X, const float* sx,
                   int64_t B, void* Y, int yt, cudaStream_t s);

}  // namespace gq
