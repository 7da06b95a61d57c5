// gq_fp8.cu -- 8-bit floating-point (e4m3) codes with one fp32 scale for each
// block of 1 x 128 (activations) or 128 x 128 (weights) values.
//
// Rule, in the manner of this library's 4-bit quantizers: s = absmax / 448 (448
// is e4m3's largest value) and code = e4m3(x / s), both quotients IEEE fp32
// ones, the second rounded to nearest even and clamped to +-448; s == 0 gives
// codes 0.  Decoding: x_hat = s * code, one fp32 rounding.
//
// All three kernels are bound by memory: each value is read once, in 16-byte
// loads, eight values to a lane, and a block's values wait in registers for its
// largest one.  A row block is half a warp's; a 128 x 128 block is a CTA's.
// Measured: 11008 x 4096 fp32 values in 128 x 128 blocks, 36 us (6.3 TB/s); 7 x
// 4096 bf16 values in rows, 2.3 us, a launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gq.h"
#include "gq_device.cuh"
#include "gq_host.h"

namespace gq {
namespace {

constexpr int kBlk = 128;
constexpr float kTop = 448.0f;

template <int TYPE>
__device__ __forceinline__ void load8(const void* base, int64_t at, float v[8]) {
  if constexpr (TYPE == GQ_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldcs(p), b = __ldcs(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (TYPE == GQ_F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[q]));
        v[2 * q] = f.x, v[2 * q + 1] = f.y;
      } else {
        v[2 * q] = __uint_as_float(w[q] << 16);
        v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
      }
    }
  }
}

// The larger magnitude; NaN if there is one.
__device__ __forceinline__ float max_abs(float m, float v) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(m), "f"(fabsf(v)));
  return d;
}
__device__ __forceinline__ float absmax8(const float v[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_abs(m, v[i]);
  return m;
}

// A block's scale, and its reciprocal a little too small and too large (zeros
// where that would leave the normal numbers).
struct Scale {
  float s, lo, hi;
};
__device__ __forceinline__ Scale scale_of(float top) {
  Scale c;
  c.s = __fdiv_rn(top, kTop);
  const float r = c.s > 1e-37f && c.s < 1e37f ? __frcp_rn(c.s) : 0.f;
  c.lo = r * (1.0f - 0x1p-21f);
  c.hi = r * (1.0f + 0x1p-21f);
  return c;
}

__device__ __forceinline__ uint2 to_codes(const float q[8]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * h], q[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * h + 2], q[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
    w[h] = a | (b << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Eight codes.  The fp32 quotient lies between the products with the two
// reciprocals (each product and reciprocal is within 2^-23 of its exact value,
// the quotient within 2^-24, and they are 2^-21 apart from it), and rounding to
// codes is monotonic: where both products have the same code, so has the
// quotient.  Elsewhere (beside the middle between two codes, about 2^-16.5 of
// all values) it is divided: IEEE division of all values took most of the kernels'
// instructions, 93 against 37 us for 11008 x 4096 fp32 values.
__device__ __forceinline__ uint2 codes8(const float v[8], const Scale& c) {
  float q[8], p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = __fmul_rn(v[i], c.lo);
    p[i] = __fmul_rn(v[i], c.hi);
  }
  uint2 w = to_codes(q);
  const uint2 z = to_codes(p);
  if (w.x != z.x || w.y != z.y || c.lo == 0.f) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      float d = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) d = j == i ? v[j] : d;
      d = c.s > 0.f ? __fdiv_rn(d, c.s) : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = j == i ? d : q[j];
    }
    w = to_codes(q);
  }
  return w;
}

// Row blocks: half a warp each, eight values a lane.
template <int TYPE>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const void* x, int64_t R, int K, int kblocks,
                                                            uint8_t* q, float* scales, int* dev_status) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t block = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 4;
  const int lane = threadIdx.x & 15;
  const bool in = block < R * kblocks;
  const int64_t r = in ? block / kblocks : 0;
  const int kb = in ? static_cast<int>(block - r * kblocks) : 0;
  const int k = kb * kBlk + 8 * lane;
  float v[8] = {};
  const bool mine = in && k < K;
  if (mine) load8<TYPE>(x, r * K + k, v);
  float m = absmax8(v);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const Scale c = scale_of(m);
  if (!mine) return;
  *reinterpret_cast<uint2*>(q + r * K + k) = codes8(v, c);
  if (lane == 0) {
    scales[block] = c.s;
    if (!isfinite(m)) report(dev_status, GQ_DEV_NONFINITE);
  }
}

// 128 x 128 blocks: one CTA each, 16 lanes to a row, 32 rows at a time.
constexpr int kTileThreads = 512;
template <int TYPE>
__global__ void __launch_bounds__(kTileThreads, 2) quantize_tiles_kernel(const void* x, int64_t R, int K, int kblocks,
                                                                      uint8_t* q, float* scales, int* dev_status) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kRowsAtOnce = kTileThreads / 16, kPasses = kBlk / kRowsAtOnce;
  __shared__ unsigned top[kTileThreads / 32];  // bits: magnitudes and NaN are ordered as integers
  const int64_t rb = blockIdx.x / kblocks;
  const int kb = static_cast<int>(blockIdx.x - rb * kblocks);
  const int k = kb * kBlk + 8 * (threadIdx.x & 15);
  const int64_t r0 = rb * kBlk + (threadIdx.x >> 4);
  float v[kPasses][8];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    if (r0 + kRowsAtOnce * i < R && k < K) load8<TYPE>(x, (r0 + kRowsAtOnce * i) * K + k, v[i]);
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    if (r0 + kRowsAtOnce * i < R && k < K) m = max_abs(m, absmax8(v[i]));
  const unsigned mw = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = mw;
  __syncthreads();
  m = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, top[threadIdx.x & (kTileThreads / 32 - 1)]));
  const Scale c = scale_of(m);
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    if (r0 + kRowsAtOnce * i < R && k < K)
      *reinterpret_cast<uint2*>(q + (r0 + kRowsAtOnce * i) * K + k) = codes8(v[i], c);
  if (threadIdx.x == 0) {
    scales[blockIdx.x] = c.s;
    if (!isfinite(m)) report(dev_status, GQ_DEV_NONFINITE);
  }
}

// Sixteen codes a thread.
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t* q, const float* scales, int64_t R,
                                                         int K, int kblocks, int shift, void* out, int type) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 16;
  if (i >= R * K) return;
  const int64_t r = i / K;
  const int k = static_cast<int>(i - r * K);
  const float s = scales[(r >> shift) * kblocks + k / kBlk];
  const uint4 u = __ldcs(reinterpret_cast<const uint4*>(q + i));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float v[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));  // exact
    v[2 * j] = __fmul_rn(s, f.x);
    v[2 * j + 1] = __fmul_rn(s, f.y);
  }
  if (type == GQ_F32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(out) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) __stcs(d + j, make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
  } else {
    uint32_t p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (type == GQ_F16) {
        const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        p[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        p[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + i);
    __stcs(d, make_uint4(p[0], p[1], p[2], p[3]));
    __stcs(d + 1, make_uint4(p[4], p[5], p[6], p[7]));
  }
}

gq_status check_matrix(int64_t R, int64_t K, int64_t rows) {
  if (R < 0 || K < 0 || (rows != 1 && rows != kBlk)) return GQ_ERR_INVALID_ARG;
  if (K % 16 || K > (1LL << 24) || R > 0x7FFFFFFFLL) return GQ_ERR_SHAPE;
  return GQ_OK;
}

}  // namespace
}  // namespace gq

extern "C" {

GQ_API size_t gq_fp8_scales(int64_t R, int64_t K, int64_t rows) {
  if (gq::check_matrix(R, K, rows) != GQ_OK) return 0;
  return static_cast<size_t>((R + rows - 1) / rows) * static_cast<size_t>((K + gq::kBlk - 1) / gq::kBlk);
}

GQ_API gq_status gq_quantize_fp8(const void* x, int x_dtype, int64_t R, int64_t K, int64_t rows,
                                 void* q, float* scales, int* dev_status, void* stream) {
  using namespace gq;
  if (!valid_act_dtype(x_dtype)) return GQ_ERR_DTYPE;
  const gq_status st = check_matrix(R, K, rows);
  if (st != GQ_OK) return st;
  if (dev_status && (reinterpret_cast<uintptr_t>(dev_status) & 3u)) return GQ_ERR_ALIGNMENT;
  if (R == 0 || K == 0) return GQ_OK;
  if (!x || !q || !scales) return GQ_ERR_INVALID_ARG;
  if (misaligned16(x) || misaligned16(q) || misaligned16(scales)) return GQ_ERR_ALIGNMENT;
  const int kblocks = static_cast<int>((K + kBlk - 1) / kBlk);
  const int64_t blocks = static_cast<int64_t>(gq_fp8_scales(R, K, rows));
  const int64_t grid = rows == 1 ? (blocks + 15) / 16 : blocks;
  if (grid > 0x7FFFFFFFLL) return GQ_ERR_SHAPE;
  auto run = [&](auto kern) {
    return launch(kern, dim3(static_cast<unsigned>(grid)), dim3(rows == 1 ? 256 : kTileThreads), 0, as_stream(stream), true, x, R,
                  static_cast<int>(K), kblocks, static_cast<uint8_t*>(q), scales, dev_status);
  };
  if (rows == 1)
    return x_dtype == GQ_F32   ? run(quantize_rows_kernel<GQ_F32>)
           : x_dtype == GQ_F16 ? run(quantize_rows_kernel<GQ_F16>)
                               : run(quantize_rows_kernel<GQ_BF16>);
  return x_dtype == GQ_F32   ? run(quantize_tiles_kernel<GQ_F32>)
         : x_dtype == GQ_F16 ? run(quantize_tiles_kernel<GQ_F16>)
                             : run(quantize_tiles_kernel<GQ_BF16>);
}

GQ_API gq_status gq_dequantize_fp8(const void* q, const float* scales, int64_t R, int64_t K,
                                   int64_t rows, void* out, int out_dtype, void* stream) {
  using namespace gq;
  if (!valid_act_dtype(out_dtype)) return GQ_ERR_DTYPE;
  const gq_status st = check_matrix(R, K, rows);
  if (st != GQ_OK) return st;
  if (R == 0 || K == 0) return GQ_OK;
  if (!q || !scales || !out) return GQ_ERR_INVALID_ARG;
  if (misaligned16(q) || misaligned16(scales) || misaligned16(out)) return GQ_ERR_ALIGNMENT;
  const int64_t grid = (R * K / 16 + 255) / 256;
  if (grid > 0x7FFFFFFFLL) return GQ_ERR_SHAPE;
  return launch(dequantize_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, as_stream(stream), true,
                static_cast<const uint8_t*>(q), scales, R, static_cast<int>(K),
                static_cast<int>((K + kBlk - 1) / kBlk), rows == 1 ? 0 : 7, out, out_dtype);
}

}  // extern "C"
