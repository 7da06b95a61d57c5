// gq_fp8.h -- the few-token product of 8-bit block-scaled matrices
// (gq_fp8_gemv.cu) as gq_gemm_fp8 sees it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gq.h"

namespace gq {

// Whether a call takes it: up to 8 tokens, or up to 16 with few weights.
// Measured, weights cold, against tcgen05: 8 tokens x 4096 x 4096 5.9 and 9.1 us, x
// 11008 x 4096 13.9 and 16.2; 16 tokens x 1024 x 4096 4.5 and 7.6, x 4096 x 4096 9.2
// and 9.4, x 11008 x 4096 19.2 and 16.1, x 4096 x 11008 19.6 and 14.4.  At 2^24 to 3
// * 2^23 weights it depends on their shape: 16 tokens x 2304 x 8192 8.8 and 10.1, x
// 5120 x 4096 11.9 and 10.6 (its 320 CTAs of 16 rows are more than fit at once).
inline bool fp8_gemv_takes(int64_t M, int64_t K, int64_t B) {
  return B <= 8 || (B <= 16 && M * K <= 3 * (int64_t{1} << 23));
}

// Arguments as for gq_gemm_fp8, checked there; no workspace.
gq_status fp8_gemv(const void* W, const float* sw, int64_t M, int64_t K, const void* X, const float* sx,
                   int64_t B, void* Y, int yt, cudaStream_t s);

}  // namespace gq
