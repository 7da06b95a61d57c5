// gq_fp8_gemv.cu -- the product of 8-bit block-scaled matrices for few tokens,
// where reading the weights once sets the time.
//
// Operation: that of gq_fp8_gemm.cu,
//   Y[b][m] = sum_g sx[b][g] * sw[m / 128][g] * sum_{k in group g} X[b][k] * W[m][k].
//
// Warp MMAs m16n8k32 on e4m3 codes as they are stored: 16 weight rows by 8
// tokens, 4.9 cycles a scheduler each, so that decode batches stay bound by
// memory (tcgen05 tiles would have 128 tokens, and splitting K over SMs costs an
// exchange through memory).  K indexes of a group are dealt to the lanes 16 at
// a time, the same for both operands, so that a lane reads 16 bytes of a row and
// four lanes a whole 64-byte piece.  A group's sums come out of four MMAs and
// are added, times its two scales, in fp32.
//
// A CTA takes 16 weight rows and all of K, which its eight warps share
// group by group; their sums are added in warp order through shared memory.  A
// warp reads several groups of weights at once: what is in flight, not
// arithmetic, sets the rate.
//
// Measured, weights cold: one token x 4096 x 4096, 6.4 us (2.6 TB/s; 4.4 us with
// the weights in L2); four tokens x 11008 x 4096, 13.4 us (3.4 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gq.h"
#include "gq_device.cuh"
#include "gq_fp8.h"
#include "gq_host.h"

namespace gq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

struct Args {
  const uint8_t* W;
  const float* sw;
  const uint8_t* X;
  const float* sx;
  void* Y;
  int64_t M, K;
  int B, groups, ytype;
};

__device__ __forceinline__ void mma_e4m3(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (Volatile, and not through the read-only path: the weights may be the preceding kernel's.)
__device__ __forceinline__ uint4 read_once(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p));
  return v;
}

// NT tiles of 8 tokens; AHEAD groups of K read at once (four, at two CTAs to an
// SM: fewer at three or four CTAs were slower, and so were CTAs that go through
// several row groups, reading the next one's weights before joining).
template <int NT, int AHEAD>
__global__ void __launch_bounds__(kThreads) fp8_gemv_kernel(const Args a) {
  __shared__ float part[kWarps][16][8 * NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16;
  pdl_wait();
  pdl_launch_dependents();
  const uint8_t* w[2];  // rows g8 and g8 + 8 (the last row stands in for those past it)
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = a.W + i64min(m0 + 8 * i + g8, a.M - 1) * a.K + 16 * t;
  const uint8_t* x[NT];
  const float* sx[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    x[j] = a.X + static_cast<int64_t>(min(8 * j + g8, a.B - 1)) * a.K + 16 * t;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      sx[j][i] = a.sx + static_cast<int64_t>(min(8 * j + 2 * t + i, a.B - 1)) * a.groups;
  }
  const float* sw = a.sw + m0 / 128 * a.groups;
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;

  for (int g0 = warp; g0 < a.groups; g0 += kWarps * AHEAD) {
    uint4 wv[AHEAD][2][2];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int g = g0 + kWarps * u;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t k = static_cast<int64_t>(g) * 128 + 64 * h;
          wv[u][i][h] = (g < a.groups && k + 16 * t < a.K) ? read_once(w[i] + k) : make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int g = g0 + kWarps * u;
      if (g >= a.groups) break;
      const float s = sw[g];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint4 xv[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t k = static_cast<int64_t>(g) * 128 + 64 * h;
          xv[h] = k + 16 * t < a.K ? *reinterpret_cast<const uint4*>(x[j] + k) : make_uint4(0, 0, 0, 0);
        }
        const float f0 = s * sx[j][0][g], f1 = s * sx[j][1][g];
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 lo = wv[u][0][h], hi = wv[u][1][h];
          mma_e4m3(c, lo.x, hi.x, lo.y, hi.y, xv[h].x, xv[h].y);
          mma_e4m3(c, lo.z, hi.z, lo.w, hi.w, xv[h].z, xv[h].w);
        }
        acc[j][0] = fmaf(f0, c[0], acc[j][0]);
        acc[j][1] = fmaf(f1, c[1], acc[j][1]);
        acc[j][2] = fmaf(f0, c[2], acc[j][2]);
        acc[j][3] = fmaf(f1, c[3], acc[j][3]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][g8 + 8 * (i >> 1)][8 * j + 2 * t + (i & 1)] = acc[j][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * 8 * NT; i += kThreads) {
    const int row = i % 16, c = i / 16;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) v += part[q][row][c];
    if (m0 + row < a.M && c < a.B) store_elem(a.Y, static_cast<int64_t>(c) * a.M + m0 + row, v, a.ytype);
  }
}

template <int NT, int AHEAD>
gq_status run(const Args& a, cudaStream_t s) {
  return launch(fp8_gemv_kernel<NT, AHEAD>, dim3(static_cast<unsigned>((a.M + 15) / 16)), dim3(kThreads), 0, s, true, a);
}

}  // namespace

gq_status fp8_gemv(const void* W, const float* sw, int64_t M, int64_t K, const void* X, const float* sx,
                   int64_t B, void* Y, int yt, cudaStream_t s) {
  Args a{static_cast<const uint8_t*>(W), sw, static_cast<const uint8_t*>(X), sx, Y, M, K, static_cast<int>(B),
         static_cast<int>((K + 127) / 128), yt};
  if (B <= 8) return run<1, 4>(a, s);
  return run<2, 4>(a, s);
}

}  // namespace gq
