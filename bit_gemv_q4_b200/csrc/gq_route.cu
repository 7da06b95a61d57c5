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
//
// Measured: one token, 64 experts, H = 2048, 4.9 us; 48 tokens, 256 experts, H =
// 4096, 12.5 us.  Bound by latency: a load, a chain of MMAs, an atomic on the
// count, and k rounds of a maximum over the warp.
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
  int H, E, k, sigmoid, norm;
  float scale;
};

// Eight consecutive values as they are stored.
template <int TYPE>
struct Raw {
  uint4 v[TYPE == GQ_F32 ? 2 : 1];
};
template <int TYPE>
__device__ __forceinline__ void load8(Raw<TYPE>& r, const void* base, int64_t at, bool ok) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + at * (TYPE == GQ_F32 ? 4 : 2));
  r.v[0] = ok ? p[0] : uint4{};
  if constexpr (TYPE == GQ_F32) r.v[1] = ok ? p[1] : uint4{};
}
// Value i of them (i a constant).
template <int TYPE>
__device__ __forceinline__ double value(const Raw<TYPE>& r, int i) {
  const uint4 u = r.v[TYPE == GQ_F32 ? i >> 2 : 0];
  const int j = TYPE == GQ_F32 ? i & 3 : i >> 1;
  const uint32_t w = j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w;
  if constexpr (TYPE == GQ_F32) return static_cast<double>(__uint_as_float(w));
  if constexpr (TYPE == GQ_BF16) return static_cast<double>(__uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16));
  return static_cast<double>(__half2float(__ushort_as_half(static_cast<unsigned short>((i & 1) ? w >> 16 : w))));
}

__device__ __forceinline__ void mma_f64(double c[2], double a, double b) {
  asm("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
      : "+d"(c[0]), "+d"(c[1])
      : "d"(a), "d"(b));
}

// A double's bits in an order that unsigned integers have, and back.
__device__ __forceinline__ uint64_t sortable(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double unsorted(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? k & 0x7FFFFFFFFFFFFFFFull : ~k));
}

// One warp: the experts of token t; lane l has the keys of experts l + 32 i, N
// at most, in registers.
template <int N>
__device__ __forceinline__ void pick(const RouteArgs& a, int64_t t) {
  const int lane = threadIdx.x & 31;
  const double* s = a.scores + t * a.E;
  uint64_t key[N];  // 0: no expert, or taken
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    double v = e < a.E ? __ldcg(s + e) : 0.0;
    bad |= !isfinite(v);
    if (a.bias && e < a.E) v += static_cast<double>(a.bias[e]);
    bad |= isnan(v);
    key[i] = e < a.E ? sortable(v + 0.0) : 0;  // (-0 and +0 are equal keys)
  }
  if (__any_sync(0xFFFFFFFFu, bad)) {  // no experts: the token's outputs are zeros
    if (lane < a.k) {
      a.ids[t * a.k + lane] = -1;
      a.weights[t * a.k + lane] = 0.f;
    }
    if (lane == 0) report(a.dev_status, GQ_DEV_NONFINITE);
    return;
  }
  float sum = 0.f;  // of exp(z - max) over this lane's experts (softmax)
  double top = 0.0;
  int mine = 0;         // lane j: the j-th expert
  uint64_t mykey = 0;   // and its key
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    }
    const unsigned hi = static_cast<unsigned>(best >> 32);
    const unsigned thi = __reduce_max_sync(0xFFFFFFFFu, hi);
    const unsigned tlo = __reduce_max_sync(0xFFFFFFFFu, hi == thi ? static_cast<unsigned>(best) : 0u);
    const bool is = hi == thi && static_cast<unsigned>(best) == tlo && best != 0;
    const unsigned e = __reduce_min_sync(0xFFFFFFFFu, is ? static_cast<unsigned>(lane + 32 * at) : 0xFFFFFFFFu);
    const uint64_t win = static_cast<uint64_t>(thi) << 32 | tlo;
    if (j == 0 && !a.sigmoid) {  // the largest z is known: the softmax's sum, before any key goes
      top = unsorted(win);
      if (!a.norm) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (key[i]) sum += expf(static_cast<float>(unsorted(key[i]) - top));
      }
    }
    if (lane == j) {
      mine = static_cast<int>(e);
      mykey = win;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (static_cast<unsigned>(lane + 32 * i) == e) key[i] = 0;
  }
  float w = 0.f;
  if (lane < a.k) {
    if (!a.sigmoid) w = expf(static_cast<float>(unsorted(mykey) - top));
    else w = static_cast<float>(a.bias ? __ldcg(s + mine) : unsorted(mykey));
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

template <int XT, int WT>
__global__ void __launch_bounds__(kThreads, 2) route_kernel(const __grid_constant__ RouteArgs a) {
  constexpr int kBatch = XT == GQ_F32 || WT == GQ_F32 ? 2 : 4;  // pieces of a row read at once
  __shared__ double part[kWarps][64];
  __shared__ int last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 2, t4 = lane & 3;
  const int e0 = blockIdx.x * kTile;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kTile;
  pdl_wait();
  pdl_launch_dependents();
  double c[2][2] = {};
  const bool eok = e0 + row < a.E, tok = t0 + row < a.T;
  const int64_t we = static_cast<int64_t>(e0 + row) * a.H + 8 * t4, xe = (t0 + row) * a.H + 8 * t4;
  for (int h0 = 32 * warp; h0 < a.H; h0 += 32 * kWarps * kBatch) {
    Raw<WT> w[kBatch];
    Raw<XT> x[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = h0 + 32 * kWarps * b;
      const bool in = h + 8 * t4 < a.H;
      load8(w[b], a.w, we + h, eok && in);
      load8(x[b], a.x, xe + h, tok && in);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (h0 + 32 * kWarps * b >= a.H) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) mma_f64(c[i & 1], value(w[b], i), value(x[b], i));
    }
  }
  part[warp][row * 8 + 2 * t4] = c[0][0] + c[1][0];
  part[warp][row * 8 + 2 * t4 + 1] = c[0][1] + c[1][1];
  __syncthreads();
  if (threadIdx.x < 64) {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) z += part[i][threadIdx.x];
    if (a.sigmoid) z = 1.0 / (1.0 + exp(-z));  // NaN stays NaN
    const int e = e0 + (threadIdx.x >> 3);
    const int64_t t = t0 + (threadIdx.x & 7);
    if (e < a.E && t < a.T) __stcg(a.scores + t * a.E + e, z);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.counts + blockIdx.y, 1) == static_cast<int>(gridDim.x) - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  if (threadIdx.x == 0) a.counts[blockIdx.y] = 0;
  const int64_t t = t0 + warp;
  if (warp >= kTile || t >= a.T) return;
  if (a.E <= 64) pick<2>(a, t);
  else if (a.E <= 128) pick<4>(a, t);
  else if (a.E <= 256) pick<8>(a, t);
  else if (a.E <= 512) pick<16>(a, t);
  else pick<32>(a, t);
}

template <int XT>
gq_status launch_route(const RouteArgs& a, int wtype, dim3 grid, cudaStream_t s) {
  switch (wtype) {
    case GQ_F32: return launch(route_kernel<XT, GQ_F32>, grid, dim3(kThreads), 0, s, true, a);
    case GQ_F16: return launch(route_kernel<XT, GQ_F16>, grid, dim3(kThreads), 0, s, true, a);
    default: return launch(route_kernel<XT, GQ_BF16>, grid, dim3(kThreads), 0, s, true, a);
  }
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
  a.sigmoid = sigmoid;
  a.norm = (flags & GQ_ROUTE_NORM) != 0;
  a.scale = scale;
  const dim3 grid(static_cast<unsigned>((E + kTile - 1) / kTile), static_cast<unsigned>((T + kTile - 1) / kTile));
  cudaStream_t s = as_stream(stream);
  return x_dtype == GQ_F32   ? launch_route<GQ_F32>(a, w_dtype, grid, s)
         : x_dtype == GQ_F16 ? launch_route<GQ_F16>(a, w_dtype, grid, s)
                             : launch_route<GQ_BF16>(a, w_dtype, grid, s);
}

}  // extern "C"
