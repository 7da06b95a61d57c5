// gq_route.cu -- the router of a mixture-of-experts layer: scores of every
// expert for every token, the k best of each token, and their weights.
//
// Operation: z[t][e] = sum_h x[t][h] * Wr[e][h]; s = z (softmax) or
// sigmoid(z); a token takes the k experts of largest s + bias, the lowest
// index among equals; their weights are softmax(z) or sigmoid(z), optionally
// divided by their sum.
//
// Which experts are taken hangs on values next to each other, so products and
// sums are fp64: the choice does not depend on the order of a sum.  The fp64
// warp MMA (m8n8k4) takes eight experts by eight tokens; a lane converts one
// value of each operand for eight multiply-adds, which matters because
// conversions to fp64 are slower than the arithmetic.  K indexes of a chunk
// are dealt to the lanes eight at a time (the same for both operands), so that
// a lane's values come from one 16- or 32-byte piece of a row.
//
// A CTA takes eight experts and eight tokens, its warps sharing H; their sums
// are added in warp order.  The CTA that completes a group of eight tokens
// picks their experts, one warp for each token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gq.h"
#include "gq_device.cuh"
#include "gq_host.h"

namespace gq {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 8;  // experts and tokens of a CTA
constexpr int kMaxE = 1024, kMaxTopK = 16;
constexpr int64_t kMaxTokens = 65536;
// the counts' part of a workspace has one size for every call, so that calls of any sizes may follow
constexpr size_t kCountBytes = kMaxTokens / kTile * sizeof(int);

struct RouteArgs {
  const void* x;
  const void* w;
  const float* bias;
  double* scores;  // [T][E]
  int* counts;     // [groups of 8 tokens] CTAs done, zero between calls
  int32_t* ids;
  float* weights;
  int* dev_status;
  int64_t T;
  int H, E, k, xtype, wtype, sigmoid, norm;
  float scale;
};

// Values h .. h+7 of a row (zeros past H).
__device__ __forceinline__ void load8(const void* base, int64_t row, int h, int H, int type, bool ok,
                                      float v[8]) {
  if (!ok || h >= H) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    return;
  }
  const int64_t at = row * H + h;
  if (type == GQ_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (type == GQ_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[q]));
      v[2 * q] = f.x, v[2 * q + 1] = f.y;
    } else {
      v[2 * q] = __uint_as_float(w[q] << 16);
      v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ void mma_f64(double c[2], double a, double b) {
  asm("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
      : "+d"(c[0]), "+d"(c[1])
      : "d"(a), "d"(b));
}

// A double's bits in an order that unsigned integers have.
__device__ __forceinline__ uint64_t sortable(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// One warp: the experts of token t from its scores (shared memory).
__device__ void pick(const RouteArgs& a, int64_t t, const double* s) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int e = lane; e < a.E; e += 32) bad |= !isfinite(s[e]);
  if (__any_sync(0xFFFFFFFFu, bad)) {  // no experts: the token's outputs are zeros
    if (lane < a.k) {
      a.ids[t * a.k + lane] = -1;
      a.weights[t * a.k + lane] = 0.f;
    }
    if (lane == 0) report(a.dev_status, GQ_DEV_NONFINITE);
    return;
  }
  unsigned taken = 0;  // this lane's experts lane + 32 i that are taken
  uint64_t best = 0;   // largest key among the others (0: none left) and its index
  int at = 0;
  auto scan = [&]() {
    best = 0;
    for (int i = 0, e = lane; e < a.E; ++i, e += 32) {
      if ((taken >> i) & 1u) continue;
      // -0 and +0 are equal keys
      const double v = (a.bias ? s[e] + static_cast<double>(__ldg(a.bias + e)) : s[e]) + 0.0;
      const uint64_t key = sortable(v);
      if (key > best) {
        best = key;
        at = e;
      }
    }
  };
  scan();
  int mine = 0;  // lane j: the j-th expert
  for (int j = 0; j < a.k; ++j) {
    const unsigned hi = static_cast<unsigned>(best >> 32);
    const unsigned top = __reduce_max_sync(0xFFFFFFFFu, hi);
    const unsigned lo = hi == top ? static_cast<unsigned>(best) : 0u;
    const unsigned low = __reduce_max_sync(0xFFFFFFFFu, lo);
    const bool is = best != 0 && hi == top && lo == low;
    const unsigned e = __reduce_min_sync(0xFFFFFFFFu, is ? static_cast<unsigned>(at) : 0xFFFFFFFFu);
    if (lane == j) mine = static_cast<int>(e);
    if (is && static_cast<unsigned>(at) == e) {
      taken |= 1u << (e >> 5);
      scan();
    }
  }
  float w = 0.f, sum = 0.f;
  if (a.sigmoid) {
    if (lane < a.k) w = static_cast<float>(s[mine]);
  } else {
    double m = s[lane < a.E ? lane : 0];
    for (int e = lane; e < a.E; e += 32) m = fmax(m, s[e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane < a.k) w = expf(static_cast<float>(s[mine] - m));
    if (!a.norm)
      for (int e = lane; e < a.E; e += 32) sum += expf(static_cast<float>(s[e] - m));
  }
  if (a.norm) sum = w;
  if (a.norm || !a.sigmoid) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    w = sum > 0.f ? w / sum : 0.f;  // sigmoids that all round to zero: no weight
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = mine;
    a.weights[t * a.k + lane] = w * a.scale;
  }
}

__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a) {
  extern __shared__ __align__(16) double keys[];  // [8][E] of the picking CTA
  __shared__ double part[kWarps][64];
  __shared__ int last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 2, t4 = lane & 3;
  const int e0 = blockIdx.x * kTile;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kTile;
  pdl_wait();
  pdl_launch_dependents();
  double c[2] = {0.0, 0.0};
  const bool eok = e0 + row < a.E, tok = t0 + row < a.T;
#pragma unroll 2
  for (int h = 32 * warp; h < a.H; h += 32 * kWarps) {
    float w[8], x[8];
    load8(a.w, e0 + row, h + 8 * t4, a.H, a.wtype, eok, w);
    load8(a.x, t0 + row, h + 8 * t4, a.H, a.xtype, tok, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) mma_f64(c, static_cast<double>(w[i]), static_cast<double>(x[i]));
  }
  part[warp][row * 8 + 2 * t4] = c[0];
  part[warp][row * 8 + 2 * t4 + 1] = c[1];
  __syncthreads();
  if (threadIdx.x < 64) {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) z += part[i][threadIdx.x];
    if (a.sigmoid) z = 1.0 / (1.0 + exp(-z));  // NaN stays NaN
    const int e = e0 + (threadIdx.x >> 3);
    const int64_t t = t0 + (threadIdx.x & 7);
    if (e < a.E && t < a.T) a.scores[t * a.E + e] = z;
    __threadfence();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.counts + blockIdx.y, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  const int nt = static_cast<int>(i64min(kTile, a.T - t0));
  for (int i = threadIdx.x; i < nt * a.E; i += kThreads) keys[i] = __ldcg(a.scores + t0 * a.E + i);
  if (threadIdx.x == 0) a.counts[blockIdx.y] = 0;
  __syncthreads();
  if (warp < nt) pick(a, t0 + warp, keys + warp * a.E);
}

}  // namespace
}  // namespace gq

extern "C" {

GQ_API size_t gq_moe_route_workspace_bytes(int64_t T, int64_t E) {
  if (T <= 0 || E <= 0 || T > gq::kMaxTokens || E > gq::kMaxE) return 0;
  return gq::kCountBytes + static_cast<size_t>(T * E) * sizeof(double);
}

GQ_API gq_status gq_moe_route(const void* x, int x_dtype, int64_t T, int64_t H, const void* Wr,
                              int w_dtype, int64_t E, const float* bias, int64_t k, float scale,
                              int32_t* ids, float* weights, void* workspace, size_t ws_bytes,
                              unsigned flags, int* dev_status, void* stream) {
  using namespace gq;
  if (T < 0 || H < 0 || E < 0 || k < 0) return GQ_ERR_INVALID_ARG;
  if (!valid_act_dtype(x_dtype) || !valid_act_dtype(w_dtype)) return GQ_ERR_DTYPE;
  if (flags & ~(GQ_GEMV_PDL | GQ_ROUTE_NORM | GQ_ROUTE_SIGMOID)) return GQ_ERR_INVALID_ARG;
  const bool sigmoid = (flags & GQ_ROUTE_SIGMOID) != 0;
  if (bias && !sigmoid) return GQ_ERR_INVALID_ARG;
  if (T > kMaxTokens || E > kMaxE || k > kMaxTopK || k > E || H % 8 || H > (1LL << 24)) return GQ_ERR_SHAPE;
  if (dev_status && (reinterpret_cast<uintptr_t>(dev_status) & 3u)) return GQ_ERR_ALIGNMENT;
  if (T == 0 || k == 0) return GQ_OK;
  if (!ids || !weights || (H > 0 && (!x || !Wr))) return GQ_ERR_INVALID_ARG;
  if (misaligned16(x) || misaligned16(Wr) || misaligned16(ids) || misaligned16(weights) ||
      misaligned16(bias))
    return GQ_ERR_ALIGNMENT;
  if (!workspace || ws_bytes < gq_moe_route_workspace_bytes(T, E)) return GQ_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GQ_ERR_ALIGNMENT;
  RouteArgs a{};
  a.x = x;
  a.w = Wr;
  a.bias = bias;
  a.counts = static_cast<int*>(workspace);
  a.scores = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + kCountBytes);
  a.ids = ids;
  a.weights = weights;
  a.dev_status = dev_status;
  a.T = T;
  a.H = static_cast<int>(H);
  a.E = static_cast<int>(E);
  a.k = static_cast<int>(k);
  a.xtype = x_dtype;
  a.wtype = w_dtype;
  a.sigmoid = sigmoid;
  a.norm = (flags & GQ_ROUTE_NORM) != 0;
  a.scale = scale;
  thread_local unsigned long long configured_ctx = 0;  // per host thread and context
  const unsigned long long ctx = context_id();
  if (ctx == 0 || ctx != configured_ctx) {
    if (cudaFuncSetAttribute(route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kTile * kMaxE * static_cast<int>(sizeof(double))) != cudaSuccess)
      return GQ_ERR_CUDA;
    configured_ctx = ctx;
  }
  const dim3 grid(static_cast<unsigned>((E + kTile - 1) / kTile), static_cast<unsigned>((T + kTile - 1) / kTile));
  return launch(route_kernel, grid, dim3(kThreads), static_cast<size_t>(kTile * E) * sizeof(double),
                as_stream(stream), (flags & GQ_GEMV_PDL) != 0, a);
}

}  // extern "C"
