// gq_moe.cu -- a mixture-of-experts layer for a few tokens on 4-bit experts in
// tiled storage.
//
// Operation: y[t] = sum_j w[t][j] * D_e (silu(G_e x_t) * (U_e x_t)), e =
// ids[t][j], with G, U, D decoded from Q4_0 blocks ("GGUF 量化内幕 第4章" 4.3:
// d * (code - 8)) or super-blocks ("GGUF K-quants" 套娃, step 5).  The taken
// experts' weights set the time (the decode setting of the TurboQuant W4A8
// post, section 2.3): every byte of them is read once, and nothing else is
// large.
//
// One cooperative launch of one CTA per SM in three phases with a grid barrier
// between them: gate and up with the activation (h, fp32, in the workspace),
// down (one fp32 row of outputs for each token and slot), and the weighted sum
// over a token's slots.  The first copies of down's weights are under way while
// a CTA waits for the others.  (As three launches joined by programmatic
// dependent launch the phases cost 8 us between the weight streams of the first
// two: a CTA's shared memory keeps the next launch out of its SM.)
//
// Plan.  Every CTA reads the ids and builds the same plan in shared memory:
// the (token, slot) pairs sorted by expert (stable), and segments of an expert
// with at most `cap` of its pairs.  The work of all segments, 16 weight rows
// at a time, is cut into even runs, one for each CTA; a run's row groups form
// one string of stages (8 blocks of 32 weights x 16 rows, 2.3 KB), which its 16
// warps share evenly, so that the split is even whatever the sizes are.  Each
// warp copies its own stages to its own ring in shared memory (cp.async), a
// few ahead: tiled storage is ordered by the lanes that multiply it, so the
// copies are whole lines and a lane reads back its own codes, and warps wait
// for nothing but their own copies.  (Reading units straight into registers,
// eight ahead, ran at 1.5 TB/s: loads that share a scoreboard are waited for
// together.)  Sums of a row group that several warps share meet in a shared
// table and are added in warp order: results do not depend on scheduling.
//
// Arithmetic.  Codes become the fp16 values code - 8, exactly: the nibble goes
// to the low mantissa bits of 1024, from which 1032 is subtracted, or stays in
// the high nibble (1024 + 16 code, times 1/16, minus 72).  The warp MMA's eight
// columns are the expert's tokens.  Activations are scaled by a power of two
// for each token so that the largest lies in [2^14, 2^15); 16-bit inputs then
// enter as one fp16 column, exact down to 2^-39 of the largest.  fp32 inputs,
// and h when y is fp32, enter as two columns (the fp16 value and the fp16
// remainder: 22 bits); for a 16-bit y, h enters as one column, rounded to 11
// bits, which is below the rounding of y.  Products are exact, sums are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gq.h"
#include "gq_device.cuh"
#include "gq_host.h"

namespace gq {
namespace {

constexpr int kWarps = 24;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxT = 64, kMaxTopK = 16, kMaxE = 1024;
constexpr int kMaxPairs = kMaxT * kMaxTopK;
constexpr int kMaxK = 16384;
constexpr int kMaxCols = 16;                // columns of a segment: two n8 tiles
constexpr size_t kSmemBudget = 227 * 1024;

// A stage: 8 blocks of 32 weights x 16 rows, what a warp copies at a time.  At
// the end of a Q4_0 row group it may hold fewer (whole units of two blocks).
constexpr int kStageCodes = 2048;
constexpr int kStageBytes = 2304;   // codes, then scales
constexpr int kDepth = 2;           // stages of a warp's ring
constexpr size_t kRingBytes = static_cast<size_t>(kWarps) * kDepth * kStageBytes;

// One of the two products: gate and up, or down.
struct Phase {
  const uint8_t* w0;        // gate, or down
  const uint8_t* w1;        // up
  int K;                    // columns of the weights
  int groups;               // row groups (16 rows) of one expert
  int64_t group_bytes;
  int two;                  // two columns for each token
  int cap;                  // tokens of a segment at most
};

struct MoeArgs {
  Phase ph[2];
  const void* x;            // [T][H]
  const int32_t* ids;       // [T][k]
  const float* weights;     // [T][k]
  void* y;                  // [T][H]
  float* h;                 // [pairs][I], by slot
  float* out;               // [pairs][H], by pair
  unsigned* hmax;           // [pairs] largest |h| of a slot as bits, zero between calls
  unsigned long long* arrivals;  // at the grid barriers, a multiple of the grid between calls
  int* dev_status;
  long long budget;
  int T, k, E, H;
  int xtype, ytype;
  int tabslots;             // parts that one table holds
  int tabfloats;            // floats of one table
  uint32_t b_off, tab_off, plan_off;  // dynamic shared memory, after the rings
};

struct Seg {
  short e, slot0;
  int n;
};

struct Plan {
  int nseg[2];
  int go;                   // the grid barrier was passed
  float inv[2][kMaxCols];   // 1 / scale of a segment's tokens
  unsigned xmax[kMaxT];     // largest |x| of a token as bits
  unsigned hmax[kMaxCols];  // of a string's tokens
  // in dynamic shared memory
  Seg* seg[2];              // [pairs] of each phase
  short* order;             // [pairs] slot -> pair
  short* first;             // [E] pairs of an expert, then its first slot
  short* rank;              // [pairs] only while planning (in the rings' place)
};

extern __shared__ __align__(1024) uint8_t msm[];

// 16 bytes, global to shared, past L1.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the newest N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------- plan
// Eight consecutive values of an element type as floats.
__device__ __forceinline__ void load8(const void* base, int64_t i, int type, float v[8]) {
  if (type == GQ_F32) {
    const float4 a = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i));
    const float4 b = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i + 4));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 u = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i));
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
}

// Pairs sorted by expert (stable), and the segments of both phases (warp 0);
// the tokens' largest |x| (the other warps).  ids outside [0, E) are left out.
__device__ void make_plan(Plan& pl, const MoeArgs& a) {
  const int P = a.T * a.k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.E; e += kThreads) pl.first[e] = 0;
  if (threadIdx.x < kMaxT) pl.xmax[threadIdx.x] = 0u;
  const int id0 = warp == 0 && lane < P ? __ldcg(a.ids + lane) : -1;
  __syncthreads();
  if (warp == 0) {
    // rank of each pair among its expert's, 32 pairs at a time
    for (int p0 = 0; p0 < P; p0 += 32) {
      const int p = p0 + lane;
      const int id = p0 == 0 ? id0 : p < P ? __ldcg(a.ids + p) : -1;
      const bool ok = id >= 0 && id < a.E;
      if (blockIdx.x == 0 && (id < -1 || id >= a.E)) report(a.dev_status, GQ_DEV_RANGE);
      const unsigned peers = __match_any_sync(0xFFFFFFFFu, ok ? id : -1 - lane);
      const int before = __popc(peers & ((1u << lane) - 1u));
      const int base = ok ? pl.first[id] : 0;
      __syncwarp();
      if (ok && before == 0) pl.first[id] = static_cast<short>(base + __popc(peers));
      if (p < P) pl.rank[p] = static_cast<short>(ok ? base + before : -1);
      __syncwarp();
    }
    // counts -> first slots, and segments, in the order of the experts
    int slots = 0, segs[2] = {0, 0};
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < a.E ? pl.first[e] : 0;
      if (!__any_sync(0xFFFFFFFFu, n)) continue;
      int sn = n;  // inclusive sums over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, sn, o);
        if (lane >= o) sn += u;
      }
      const int first = slots + sn - n;
      if (e < a.E) pl.first[e] = static_cast<short>(first);
      slots += __shfl_sync(0xFFFFFFFFu, sn, 31);
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int cap = a.ph[f].cap, ns = (n + cap - 1) / cap;
        int ss = ns;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xFFFFFFFFu, ss, o);
          if (lane >= o) ss += u;
        }
        for (int i = 0; i < ns; ++i)
          pl.seg[f][segs[f] + ss - ns + i] =
              Seg{static_cast<short>(e), static_cast<short>(first + i * cap), min(cap, n - i * cap)};
        segs[f] += __shfl_sync(0xFFFFFFFFu, ss, 31);
      }
    }
    if (lane < 2) pl.nseg[lane] = lane ? segs[1] : segs[0];
  } else {
    const int share = max(1, (kWarps - 1) / a.T), vecs = a.H / 8;  // warps for each token
    for (int i = warp - 1; i < a.T * share; i += kWarps - 1) {
      const int t = i / share;
      unsigned m = 0;
#pragma unroll 4
      for (int r = (i - t * share) * 32 + lane; r < vecs; r += 32 * share) {
        float v[8];
        load8(a.x, static_cast<int64_t>(t) * a.H + 8 * r, a.xtype, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(v[q]) & 0x7FFFFFFFu);
      }
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      if (lane == 0) atomicMax(&pl.xmax[t], m);
    }
  }
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += kThreads) {
    const int r = pl.rank[p];
    if (r >= 0) pl.order[pl.first[__ldcg(a.ids + p)] + r] = static_cast<short>(p);
  }
  __syncthreads();
}

// ------------------------------------------------------------- activations
// The power of two that brings the largest |value| (its bits) into [2^14,
// 2^15); 1 for infinities and NaN, which stay what they are.
__device__ __forceinline__ float scale_of(unsigned maxbits) {
  const int e = static_cast<int>(maxbits >> 23) - 127;
  if (e > 127) return 1.0f;
  return __uint_as_float(static_cast<unsigned>(127 + 14 - max(e, -100)) << 23);
}

// Columns that the B fragments of a segment have room for: a power of two, so
// that every offset in the inner loop is a constant.
__device__ __forceinline__ int col_pitch(int ncol) {
  return ncol <= 2 ? ncol : ncol <= 4 ? 4 : ncol <= 8 ? 8 : 16;
}

// B fragments of a segment's tokens.  Column c of block b and lane group t: 16
// bytes at ((b * pitch + c) * 4 + t) * 16, the values 4t, 4t+2, 4t+1, 4t+3 of the
// block and the same at +16.
template <bool GATE_UP>
__device__ void load_b(const MoeArgs& a, const Phase& ph, Plan& pl, const Seg& sg, int buf) {
  const int pitch = col_pitch(ph.two ? 2 * sg.n : sg.n);
  const int vecs = ph.K / 8;
  auto row_of = [&](int c) { return GATE_UP ? pl.order[sg.slot0 + c] / a.k : sg.slot0 + c; };
  auto max_of = [&](int c) { return GATE_UP ? pl.xmax[row_of(c)] : __ldcg(a.hmax + sg.slot0 + c); };
  const int type = GATE_UP ? a.xtype : GQ_F32;
  const void* src = GATE_UP ? a.x : a.h;
  if (threadIdx.x < sg.n)  // scale_of() is a power of two: the reciprocal is exact
    pl.inv[buf][threadIdx.x] = 1.0f / scale_of(max_of(threadIdx.x));
  const int nvec = sg.n * vecs;
  for (int i = threadIdx.x; i < nvec; i += kThreads) {
    const int c = i / vecs, r = i - c * vecs;
    const int b = r >> 2, q = r & 3;
    float v[8];
    load8(src, static_cast<int64_t>(row_of(c)) * ph.K + 8 * r, type, v);
    const float s = scale_of(max_of(c));
    const int col = ph.two ? 2 * c : c;
    const int t0 = 2 * (q & 1);
    for (int part = 0; part <= ph.two; ++part) {
      __half hv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = part ? v[j] : v[j] * s;  // the second pass holds remainders
        hv[j] = __float2half_rn(f);
        v[j] = f - __half2float(hv[j]);
      }
      uint8_t* d = msm + a.b_off + (static_cast<uint32_t>(b * pitch + col + part) * 4 + t0) * 16 + (q >> 1) * 8;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const __half2 lo = __halves2half2(hv[4 * u], hv[4 * u + 2]);
        const __half2 hi = __halves2half2(hv[4 * u + 1], hv[4 * u + 3]);
        *reinterpret_cast<uint2*>(d + 16 * u) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                           *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------------ stages
__device__ __forceinline__ uint32_t ld32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint4 ld128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ float2 halves(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// INT8 in byte h of q (its sign bit flipped beforehand) as a float, exact.
__device__ __forceinline__ float flipped_byte(uint32_t q, int h) {
  return __uint_as_float(__byte_perm(q, 0x4B000000u, 0x7540u + h)) - 8388736.0f;  // 2^23 + 128
}

// Two codes of a word as fp16 values code - 8: the low nibbles of bytes 0 and 2,
// or their high nibbles.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {
  const uint32_t u = lop3_and_or(w, 0x000F000Fu, 0x64006400u);  // 1024 + code
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6408)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) {
  const uint32_t u = lop3_and_or(w, 0x00F000F0u, 0x64006400u);  // 1024 + 16 code
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x2C00)),
                            __half2half2(__ushort_as_half(0xD480)));  // / 16 - 72
  return *reinterpret_cast<const uint32_t*>(&r);
}

// acc += one block of 32 weights: wa, wb this lane's code words of rows g and
// g+8, da, db the rows' scales, xb this lane's B fragment of column tile 0.
// With one column a lane keeps one sum for each row.
template <int CP>
__device__ __forceinline__ void block_math(uint32_t wa, uint32_t wb, float da, float db, float (*acc)[4],
                                           const uint8_t* xb) {
  const uint32_t wa8 = wa >> 8, wb8 = wb >> 8;
  const uint32_t l0 = low_codes(wa), l1 = low_codes(wb), l2 = low_codes(wa8), l3 = low_codes(wb8);
  const uint32_t h0 = high_codes(wa), h1 = high_codes(wb), h2 = high_codes(wa8), h3 = high_codes(wb8);
#pragma unroll
  for (int j = 0; j < (CP + 7) / 8; ++j) {
    const uint4 xv = ld128(xb + 512 * j);
    float c[4];
    mma_f16_z(c, l0, l1, l2, l3, xv.x, xv.y);
    mma_f16(c, h0, h1, h2, h3, xv.z, xv.w);
    acc[j][0] = fmaf(da, c[0], acc[j][0]);
    if (CP > 1) acc[j][1] = fmaf(da, c[1], acc[j][1]);
    acc[j][2] = fmaf(db, c[2], acc[j][2]);
    if (CP > 1) acc[j][3] = fmaf(db, c[3], acc[j][3]);
  }
}

// A stage from its ring slot: n units of two blocks (Q4_0) or one super-block.
template <int FMT, int CP, bool FULL>
__device__ __forceinline__ void stage_math(const uint8_t* st, int n, int lane, float (*acc)[4],
                                           const uint8_t* xb) {
  const uint8_t* code = st + (FMT == GQ_FMT_Q4_0 ? 16 : 32) * lane;
  const uint8_t* sc = st + kStageCodes + 4 * (lane >> 2);
  if constexpr (FMT == GQ_FMT_Q4_0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (FULL || i < n) {
        const uint4 v = ld128(code + 512 * i);
        const float2 da = halves(ld32(sc + 64 * i));
        const float2 db = halves(ld32(sc + 64 * i + 32));
        block_math<CP>(v.x, v.y, da.x, db.x, acc, xb + (2 * i) * (64 * CP));
        block_math<CP>(v.z, v.w, da.y, db.y, acc, xb + (2 * i + 1) * (64 * CP));
      }
    }
  } else {
    const uint8_t* ss = st + kStageCodes + 128 + 2 * (lane >> 2);
    const float sa = __half2float(*reinterpret_cast<const __half*>(ss));
    const float sb = __half2float(*reinterpret_cast<const __half*>(ss + 16));
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // half a super-block: lane-ordered 32 bytes of codes
      const uint32_t qa = ld32(sc + 64 * i) ^ 0x80808080u, qb = ld32(sc + 64 * i + 32) ^ 0x80808080u;
      const uint4 v = ld128(code + 1024 * i), w = ld128(code + 1024 * i + 16);
      const uint8_t* x = xb + (4 * i) * (64 * CP);
      block_math<CP>(v.x, v.y, sa * flipped_byte(qa, 0), sb * flipped_byte(qb, 0), acc, x);
      block_math<CP>(v.z, v.w, sa * flipped_byte(qa, 1), sb * flipped_byte(qb, 1), acc, x + 64 * CP);
      block_math<CP>(w.x, w.y, sa * flipped_byte(qa, 2), sb * flipped_byte(qb, 2), acc, x + 128 * CP);
      block_math<CP>(w.z, w.w, sa * flipped_byte(qa, 3), sb * flipped_byte(qb, 3), acc, x + 192 * CP);
    }
  }
}

// A string of row groups [i0, i0 + n) of one expert (gate and up: row group i
// is one of gate's, then the same of up's).
template <bool GATE_UP>
__device__ __forceinline__ const uint8_t* group_at(const Phase& a, int e, int i) {
  const uint8_t* w = (GATE_UP && (i & 1)) ? a.w1 : a.w0;
  const int g = GATE_UP ? i >> 1 : i;
  return w + (static_cast<int64_t>(e) * a.groups + g) * a.group_bytes;
}

// A warp's next copy: stage k of row group q of the string, `left` stages in
// all; this lane's sources in it.
template <int FMT, bool GATE_UP>
struct Feed {
  const uint8_t* code;
  const uint8_t* scale;
  int e, q, k, left;

  // Sources of stage k of a row group.
  __device__ __forceinline__ void seek(const Phase& a, int i0, int lane) {
    const uint8_t* group = group_at<GATE_UP>(a, e, i0 + q);
    const int c = k >> 3, j = k & 7;
    if constexpr (FMT == GQ_FMT_Q4_0) {
      // tiles of 32 units (512 bytes of codes, 64 of scales); a stage is four
      const int nu = min(32, (a.K >> 6) - 32 * c);
      const uint8_t* tile = group + static_cast<int64_t>(c) * 18432;
      code = tile + 2048 * j + 16 * lane;
      scale = tile + 512 * nu + 256 * j + 16 * lane;
    } else {
      // tiles of 8 super-blocks (2048 bytes of codes, 128 of sub-scales, 32 of S); a stage is one
      const int ns = min(8, (a.K >> 8) - 8 * c);
      const uint8_t* tile = group + static_cast<int64_t>(c) * 17664;
      code = tile + 2048 * j + 16 * lane;
      scale = lane < 8 ? tile + 2048 * ns + 128 * j + 16 * lane : tile + 2176 * ns + 32 * j + 16 * (lane - 8);
    }
  }
  __device__ __forceinline__ void step(const Phase& a, int i0, int stages, uint32_t dst, int lane) {
    if (left > 0) {
      dst += 16 * lane;
      const int n = FMT == GQ_FMT_Q4_0 && k == stages - 1 ? (a.K >> 6) - 4 * k : 4;  // units
      if (n == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) copy16(dst + 512 * i, code + 512 * i);
      } else {
        for (int i = 0; i < n; ++i) copy16(dst + 512 * i, code + 512 * i);
      }
      if (lane < (FMT == GQ_FMT_Q4_0 ? 4 * n : 10)) copy16(dst + kStageCodes, scale);
      --left;
      ++k;
      if (k == stages || (k & 7) == 0) {  // another tile
        if (k == stages) {
          k = 0;
          ++q;
        }
        if (left > 0) seek(a, i0, lane);
      } else {
        code += 2048;
        scale += FMT == GQ_FMT_Q4_0 ? 256 : (lane < 8 ? 128 : 32);
      }
    }
    copies_commit();  // also an empty group: groups count stages
  }
};

// This warp's stages [u, u1) of the string, the first kDepth of them under way:
// partial sums to the table, part (row group + warp) for each row group that
// the warp has stages of.
template <int FMT, int CP, bool GATE_UP>
__device__ __forceinline__ void stream(const Phase& a, uint32_t b_off, Feed<FMT, GATE_UP>& feed, int i0, int stages, int u,
                                       int u1, uint32_t ring, float* tab) {
  constexpr int NT = (CP + 7) / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;
  // columns past the last repeat existing ones (or hold what was there); their sums are not used
  const uint8_t* xb = msm + b_off + (g8 & (CP - 1)) * 64 + t * 16;
  const uint32_t sbase = smem_addr(msm);
  const int last_n = FMT == GQ_FMT_Q4_0 ? (a.K >> 6) - 4 * (stages - 1) : 4;  // units of a row's last stage
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  int q = u / stages, k = u - q * stages;
  uint32_t st = ring;
  const uint8_t* x = xb + k * (8 * 64 * CP);
  for (; u < u1; ++u) {
    copies_wait<kDepth - 1>();
    __syncwarp();  // every lane's copies of the stage
    const bool end = ++k == stages;
    if (FMT == GQ_FMT_KSB || !end || last_n == 4)
      stage_math<FMT, CP, true>(msm + st, 4, lane, acc, x);
    else
      stage_math<FMT, CP, false>(msm + st, last_n, lane, acc, x);
    x += 8 * 64 * CP;
    __syncwarp();  // every lane has read the stage
    feed.step(a, i0, stages, sbase + st, lane);
    st = st == ring + (kDepth - 1) * kStageBytes ? ring : st + kStageBytes;
    if (end || u + 1 == u1) {
      float* d = tab + (q + warp) * (16 * CP);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int c = 8 * j + 2 * t;
        if (CP == 1) {
          if (t == 0) {
            d[g8] = acc[j][0];
            d[g8 + 8] = acc[j][2];
          }
        } else if (c < CP) {
          *reinterpret_cast<float2*>(d + g8 * CP + c) = make_float2(acc[j][0], acc[j][1]);
          *reinterpret_cast<float2*>(d + (g8 + 8) * CP + c) = make_float2(acc[j][2], acc[j][3]);
        }
        acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
      }
      k = 0;
      ++q;
      x = xb;
    }
  }
}

// The run of this CTA: row groups (pairs of them for gate and up) [r0, r1) of
// all segments', cut into strings of one segment that the table holds.
struct String {
  int seg, i0, n;  // segment, first row group (of the string's kind), how many
};
template <int FMT, bool GATE_UP>
struct Work {
  int r, r1;    // row groups left (pairs of them for gate and up)
  int stages;   // of a row group
  bool more;
  String st;
  Feed<FMT, GATE_UP> feed;

  __device__ __forceinline__ void next(const Phase& ph, int most) {
    more = r < r1;
    if (!more) return;
    st.seg = r / ph.groups;
    const int g = r - st.seg * ph.groups;
    const int left = min(r1 - r, ph.groups - g);
    const int strings = (left + most - 1) / most;
    const int n = (left + strings - 1) / strings;  // even strings
    st.i0 = GATE_UP ? 2 * g : g;
    st.n = GATE_UP ? 2 * n : n;
    r += n;
  }
  // The first copies of this warp's share of the string.
  __device__ __forceinline__ void fetch(const Phase& ph, const Plan& pl, uint32_t ring) {
    if (!more) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tu = st.n * stages;
    const int u0 = tu * warp / kWarps;
    feed.e = pl.seg[!GATE_UP][st.seg].e;
    feed.q = u0 / stages;
    feed.k = u0 - feed.q * stages;
    feed.left = tu * (warp + 1) / kWarps - u0;
    if (feed.left > 0) feed.seek(ph, st.i0, lane);
    for (int i = 0; i < kDepth; ++i) feed.step(ph, st.i0, stages, smem_addr(msm) + ring + i * kStageBytes, lane);
  }
  __device__ __forceinline__ void start(const MoeArgs& a, const Plan& pl, uint32_t ring) {
    const Phase& ph = a.ph[!GATE_UP];
    const unsigned total = static_cast<unsigned>(pl.nseg[!GATE_UP]) * ph.groups;  // at most 2^20
    r = static_cast<int>(total * blockIdx.x / gridDim.x);
    r1 = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
    stages = FMT == GQ_FMT_Q4_0 ? (ph.K + 255) / 256 : ph.K / 256;
    next(ph, (a.tabslots - kWarps) / (GATE_UP ? 2 : 1));
    fetch(ph, pl, ring);
  }
};

// All strings of a phase.
template <int FMT, bool GATE_UP>
__device__ __forceinline__ void run_phase(const MoeArgs& a, Plan& pl, Work<FMT, GATE_UP>& wk, uint32_t ring) {
  const Phase& ph = a.ph[!GATE_UP];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = wk.stages;
  int buf = 0, loaded = -1;
  while (wk.more) {
    const String st = wk.st;
    const Seg sg = pl.seg[!GATE_UP][st.seg];
    const int pitch = col_pitch(ph.two ? 2 * sg.n : sg.n);
    if (loaded != st.seg) {
      load_b<GATE_UP>(a, ph, pl, sg, st.seg & 1);
      loaded = st.seg;
    }
    float* tab = reinterpret_cast<float*>(msm + a.tab_off) + buf * a.tabfloats;
    const int tu = st.n * stages;
    const int u0 = tu * warp / kWarps, u1 = tu * (warp + 1) / kWarps;
    switch (pitch) {
      case 1: stream<FMT, 1, GATE_UP>(ph, a.b_off, wk.feed, st.i0, stages, u0, u1, ring, tab); break;
      case 2: stream<FMT, 2, GATE_UP>(ph, a.b_off, wk.feed, st.i0, stages, u0, u1, ring, tab); break;
      case 4: stream<FMT, 4, GATE_UP>(ph, a.b_off, wk.feed, st.i0, stages, u0, u1, ring, tab); break;
      case 8: stream<FMT, 8, GATE_UP>(ph, a.b_off, wk.feed, st.i0, stages, u0, u1, ring, tab); break;
      default: stream<FMT, 16, GATE_UP>(ph, a.b_off, wk.feed, st.i0, stages, u0, u1, ring, tab);
    }
    wk.next(ph, (a.tabslots - kWarps) / (GATE_UP ? 2 : 1));
    wk.fetch(ph, pl, ring);
    if (GATE_UP && threadIdx.x < kMaxCols) pl.hmax[threadIdx.x] = 0u;
    __syncthreads();  // the table is complete; B and the other table are free
    // A warp takes two row groups (gate and up of the same rows, or two of
    // down's), 16 lanes each, and adds their parts in warp order.
    const float* inv = pl.inv[st.seg & 1];
    const int row = lane & 15, half = lane >> 4;
    for (int p = warp; p < (st.n + 1) / 2; p += kWarps) {
      const int q = min(2 * p + half, st.n - 1);
      const int lo = q * stages, hi = lo + stages - 1;
      const int w0 = (kWarps * (lo + 1) - 1) / tu, w1 = (kWarps * (hi + 1) - 1) / tu;
      for (int c = 0; c < sg.n; ++c) {
        const int col = ph.two ? 2 * c : c;
        float v = 0.f;
        for (int w = w0; w <= w1; ++w) {
          if (tu * w / kWarps == tu * (w + 1) / kWarps) continue;  // no stages
          const float* t = tab + ((q + w) * 16 + row) * pitch + col;
          v += ph.two ? t[0] + t[1] : t[0];
        }
        v *= inv[c];
        if constexpr (GATE_UP) {
          const float up = __shfl_down_sync(0xFFFFFFFFu, v, 16);
          const float h = v / (1.0f + expf(-v)) * up;
          unsigned m = 0;
          if (half == 0) {
            __stcg(a.h + static_cast<int64_t>(sg.slot0 + c) * (ph.groups * 16) + (st.i0 / 2 + p) * 16 + row, h);
            m = __float_as_uint(h) & 0x7FFFFFFFu;
          }
          m = __reduce_max_sync(0xFFFFFFFFu, m);
          if (lane == 0) atomicMax(&pl.hmax[c], m);
        } else if (2 * p + half < st.n) {
          const int pair = pl.order[sg.slot0 + c];
          __stcg(a.out + static_cast<int64_t>(pair) * (ph.groups * 16) + (st.i0 + q) * 16 + row, v);
        }
      }
    }
    if (GATE_UP) {
      __syncthreads();
      if (threadIdx.x < sg.n) atomicMax(a.hmax + sg.slot0 + threadIdx.x, pl.hmax[threadIdx.x]);
    }
    buf ^= 1;
  }
}

// All CTAs of the grid arrive, and what each wrote before is seen by all after;
// false once the budget has passed.  The arrivals only ever count up (in 64
// bits), so nothing has to be cleared.
__device__ __forceinline__ bool grid_barrier(const MoeArgs& a, Plan& pl) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned long long n = atomicAdd(a.arrivals, 1ull);
    const unsigned long long target = (n / gridDim.x + 1) * gridDim.x;
    const long long t0 = clock64();
    int go = 1;
    for (;;) {
      unsigned long long v;
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(a.arrivals) : "memory");
      if (v >= target) break;
      if (clock64() - t0 > a.budget) {
        go = 0;
        break;
      }
    }
    __threadfence();
    pl.go = go;
  }
  __syncthreads();
  return pl.go != 0;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const __grid_constant__ MoeArgs a) {
  __shared__ Plan pl;
  if (threadIdx.x == 0) {
    const int pairs = a.T * a.k;
    pl.seg[0] = reinterpret_cast<Seg*>(msm + a.plan_off);
    pl.seg[1] = pl.seg[0] + pairs;
    pl.order = reinterpret_cast<short*>(pl.seg[1] + pairs);
    pl.first = pl.order + pairs;
    pl.rank = reinterpret_cast<short*>(msm);
  }
  pdl_wait();  // ids and x are final
  pdl_launch_dependents();
  __syncthreads();
  make_plan(pl, a);
  const uint32_t ring = static_cast<uint32_t>((threadIdx.x >> 5) * kDepth * kStageBytes);
  Work<FMT, true> gate_up;
  gate_up.start(a, pl, ring);
  run_phase<FMT, true>(a, pl, gate_up, ring);
  Work<FMT, false> down;
  down.start(a, pl, ring);  // the first copies are under way while this CTA waits
  bool ok = grid_barrier(a, pl);
  if (ok) {
    run_phase<FMT, false>(a, pl, down, ring);
    ok = grid_barrier(a, pl);
  }
  if (!ok) {
    copies_wait<0>();
    if (threadIdx.x == 0) report(a.dev_status, GQ_DEV_TIMEOUT);
    return;
  }
  // y[t] = sum_j w[t][j] * out[t][j] over the slots that name an expert; the
  // slots' largest values are cleared for the next call
  const int n = a.T * a.H;
  const int i0 = static_cast<int>(blockIdx.x * kThreads + threadIdx.x);
  if (i0 < a.T * a.k) a.hmax[i0] = 0u;
  for (int i = i0; i < n; i += static_cast<int>(gridDim.x) * kThreads) {
    const int t = i / a.H, c = i - t * a.H;
    float v = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int id = __ldcg(a.ids + t * a.k + j);
      if (id >= 0 && id < a.E)
        v = fmaf(__ldcg(a.weights + t * a.k + j), __ldcg(a.out + static_cast<int64_t>(t * a.k + j) * a.H + c), v);
    }
    store_elem(a.y, i, v, a.ytype);
  }
}

// ------------------------------------------------------------------- host
size_t round256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

struct Ws {
  size_t arrivals, hmax, h, out, total;
};
Ws ws_layout(int64_t T, int64_t k, int64_t H, int64_t I) {
  Ws w;
  w.arrivals = 0;
  w.hmax = 256;
  w.h = w.hmax + kMaxPairs * 4;  // one size for every call, so that calls of any sizes may follow
  w.out = w.h + round256(static_cast<size_t>(T * k * I) * 4);
  w.total = w.out + round256(static_cast<size_t>(T * k * H) * 4);
  return w;
}

bool moe_dims(int64_t T, int64_t k, int64_t E) {
  return T <= kMaxT && k <= kMaxTopK && E <= kMaxE;
}
bool moe_width(int fmt, int64_t K) { return K % (fmt == GQ_FMT_Q4_0 ? 64 : 256) == 0 && K <= kMaxK; }

// Tokens of a segment and the layout of shared memory after the rings: the B
// fragments (2 bytes for each value of a column), two tables of parts, and the
// plan.  A table holds at least a string of 16 row groups.
constexpr int kMinSlots = kWarps + 16, kMaxSlots = kWarps + 64;
static_assert(sizeof(Plan) <= 1024, "the static part, up to the dynamic one's alignment");
constexpr size_t kDynSmem = kSmemBudget - 1024;
size_t shape_smem(MoeArgs& a) {
  const int pairs = a.T * a.k;
  const size_t plan = (static_cast<size_t>(pairs) * (2 * sizeof(Seg) + 2) + static_cast<size_t>(a.E) * 2 + 15) & ~size_t(15);
  const size_t left = kDynSmem - kRingBytes - plan;
  const size_t part = 2 * 16 * sizeof(float);  // of both tables, for each column
  size_t b = 0, cols = 2;
  for (Phase& ph : a.ph) {
    const size_t most = left / (static_cast<size_t>(ph.K) * 2 + kMinSlots * part);
    const size_t need = static_cast<size_t>(pairs) * (ph.two ? 2 : 1);
    size_t c = 2;  // powers of two
    while (c < kMaxCols && 2 * c <= most && c < need) c *= 2;
    ph.cap = static_cast<int>(ph.two ? c / 2 : c);
    b = c * ph.K * 2 > b ? c * ph.K * 2 : b;
    cols = c > cols ? c : cols;
  }
  // each phase alone leaves room for kMinSlots parts of its own columns
  size_t slots = (left - b) / (part * cols);
  while (slots < static_cast<size_t>(kMinSlots)) {
    cols /= 2;
    for (Phase& ph : a.ph)
      if (static_cast<size_t>(ph.cap) * (ph.two ? 2 : 1) > cols) ph.cap = static_cast<int>(cols) / (ph.two ? 2 : 1);
    slots = (left - b) / (part * cols);
  }
  a.tabslots = static_cast<int>(slots < static_cast<size_t>(kMaxSlots) ? slots : kMaxSlots);
  a.tabfloats = a.tabslots * 16 * static_cast<int>(cols);
  a.b_off = kRingBytes;
  a.tab_off = a.b_off + static_cast<uint32_t>(b);
  a.plan_off = a.tab_off + 2 * a.tabfloats * 4;
  return a.plan_off + plan;
}

template <int FMT>
gq_status launch_moe(MoeArgs& a, bool pdl, cudaStream_t s) {
  auto kern = moe_kernel<FMT>;
  thread_local unsigned long long configured_ctx = 0;  // per host thread and context
  const unsigned long long ctx = context_id();
  if (ctx == 0 || ctx != configured_ctx) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kDynSmem)) != cudaSuccess)
      return GQ_ERR_CUDA;
    configured_ctx = ctx;
  }
  const size_t smem = shape_smem(a);
  return launch_cooperative(kern, dim3(sm_count()), dim3(kThreads), smem, s, pdl, a);
}

template <int FMT>
gq_status moe_entry(const void* gate, const void* up, const void* down, int64_t E, int64_t H,
                    int64_t I, const void* x, int x_dtype, int64_t T, const int32_t* ids,
                    const float* weights, int64_t k, void* y, int y_dtype, void* workspace,
                    size_t ws_bytes, unsigned flags, int* dev_status, void* stream) {
  if (E < 0 || H < 0 || I < 0 || T < 0 || k < 0) return GQ_ERR_INVALID_ARG;
  if (!valid_act_dtype(x_dtype) || !valid_act_dtype(y_dtype)) return GQ_ERR_DTYPE;
  if (flags & ~GQ_GEMV_PDL) return GQ_ERR_INVALID_ARG;
  if (!moe_dims(T, k, E) || !moe_width(FMT, H) || !moe_width(FMT, I)) return GQ_ERR_SHAPE;
  if (dev_status && (reinterpret_cast<uintptr_t>(dev_status) & 3u)) return GQ_ERR_ALIGNMENT;
  if (T == 0 || H == 0) return GQ_OK;
  if (!y) return GQ_ERR_INVALID_ARG;
  if (misaligned16(y)) return GQ_ERR_ALIGNMENT;
  cudaStream_t s = as_stream(stream);
  if (I == 0 || E == 0 || k == 0)
    return cudaMemsetAsync(y, 0, static_cast<size_t>(T * H * dtype_size(y_dtype)), s) == cudaSuccess
               ? GQ_OK
               : GQ_ERR_CUDA;
  if (!gate || !up || !down || !x || !ids || !weights) return GQ_ERR_INVALID_ARG;
  if (misaligned16(gate) || misaligned16(up) || misaligned16(down) || misaligned16(x) ||
      misaligned16(ids) || misaligned16(weights))
    return GQ_ERR_ALIGNMENT;
  const Ws l = ws_layout(T, k, H, I);
  if (!workspace || ws_bytes < l.total) return GQ_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GQ_ERR_ALIGNMENT;
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  const auto row_bytes = [](int64_t K) { return FMT == GQ_FMT_Q4_0 ? K / 32 * 18 : K / 256 * 138; };
  MoeArgs a{};
  a.ph[0] = Phase{static_cast<const uint8_t*>(gate), static_cast<const uint8_t*>(up), static_cast<int>(H),
                  static_cast<int>(I / 16), 16 * row_bytes(H), x_dtype == GQ_F32, 0};
  a.ph[1] = Phase{static_cast<const uint8_t*>(down), nullptr, static_cast<int>(I), static_cast<int>(H / 16),
                  16 * row_bytes(I), y_dtype == GQ_F32, 0};
  a.x = x;
  a.ids = ids;
  a.weights = weights;
  a.y = y;
  a.h = reinterpret_cast<float*>(ws + l.h);
  a.out = reinterpret_cast<float*>(ws + l.out);
  a.hmax = reinterpret_cast<unsigned*>(ws + l.hmax);
  a.arrivals = reinterpret_cast<unsigned long long*>(ws + l.arrivals);
  a.dev_status = dev_status;
  a.budget = kWaitBudget;
  a.T = static_cast<int>(T);
  a.k = static_cast<int>(k);
  a.E = static_cast<int>(E);
  a.H = static_cast<int>(H);
  a.xtype = x_dtype;
  a.ytype = y_dtype;
  return launch_moe<FMT>(a, (flags & GQ_GEMV_PDL) != 0, s);
}

}  // namespace
}  // namespace gq

extern "C" {

GQ_API size_t gq_moe_workspace_bytes(int fmt, int64_t H, int64_t I, int64_t T, int64_t k) {
  if ((fmt != GQ_FMT_Q4_0 && fmt != GQ_FMT_KSB) || H <= 0 || I <= 0 || T <= 0 || k <= 0) return 0;
  if (!gq::moe_dims(T, k, 0) || !gq::moe_width(fmt, H) || !gq::moe_width(fmt, I)) return 0;
  return gq::ws_layout(T, k, H, I).total;
}

GQ_API gq_status gq_moe_q4_0_tiled(const void* gate, const void* up, const void* down, int64_t E,
                                   int64_t H, int64_t I, const void* x, int x_dtype, int64_t T,
                                   const int32_t* ids, const float* weights, int64_t k, void* y,
                                   int y_dtype, void* workspace, size_t ws_bytes, unsigned flags,
                                   int* dev_status, void* stream) {
  return gq::moe_entry<GQ_FMT_Q4_0>(gate, up, down, E, H, I, x, x_dtype, T, ids, weights, k, y, y_dtype,
                                    workspace, ws_bytes, flags, dev_status, stream);
}

GQ_API gq_status gq_moe_ksb_tiled(const void* gate, const void* up, const void* down, int64_t E,
                                  int64_t H, int64_t I, const void* x, int x_dtype, int64_t T,
                                  const int32_t* ids, const float* weights, int64_t k, void* y,
                                  int y_dtype, void* workspace, size_t ws_bytes, unsigned flags,
                                  int* dev_status, void* stream) {
  return gq::moe_entry<GQ_FMT_KSB>(gate, up, down, E, H, I, x, x_dtype, T, ids, weights, k, y, y_dtype,
                                   workspace, ws_bytes, flags, dev_status, stream);
}

}  // extern "C"
