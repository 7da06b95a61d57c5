// gq_moe.cu -- a mixture-of-experts layer for a few tokens on 4-bit experts in
// tiled storage.
//
// Operation: y[t] = sum_j w[t][j] * D_e (silu(G_e x_t) * (U_e x_t)), e =
// ids[t][j], with G, U, D decoded from Q4_0 blocks ("GGUF 量化内幕 第4章" 4.3:
// d * (code - 8)) or super-blocks ("GGUF K-quants" 套娃, step 5).  The taken
// experts' weights set the time (the decode setting of the TurboQuant W4A8
// post, section 2.3): every byte of them is read once for each segment of the
// expert's tokens (below), and nothing else is large.
//
// One cooperative launch of one CTA per SM in three phases with a grid barrier
// between them: gate and up with the activation (h, fp32, in the workspace),
// down (one fp32 row of outputs for each token and slot), and the weighted sum
// over a token's slots.  For a single token whose slots' h all fit in shared
// memory, down's rows run over all slots, with the weights folded into h, and y
// is stored at once: no third phase.  The first copies of down's weights are
// under way while a CTA waits for the others.  (As three launches joined by
// programmatic dependent launch the phases cost 8 us between the weight streams
// of the first two: a CTA's shared memory keeps the next launch out of its SM.)
//
// Plan.  Every CTA reads the ids and builds the same plan in shared memory:
// the (token, slot) pairs sorted by expert (stable), and segments of an expert
// with at most `cap` of its pairs.  The work of all segments, one item for 16
// weight rows (of gate and of up, or of down), is cut into even runs, one for
// each CTA.  A run is a string of stages (8 blocks of 32 weights x 16 rows, 2.3
// KB) that its 20 warps share evenly, so that the split is even whatever the
// sizes are.  Each warp copies its own stages to its own ring in shared memory
// (cp.async): tiled storage is ordered by the lanes that multiply it, so the
// copies are whole lines and a lane reads back its own codes, and warps wait
// for nothing but their own copies.  (Reading stages straight into registers,
// one or two ahead, ran at half the rate: loads that share a scoreboard are
// waited for together.)  A warp finishes the items that it has all of in its
// registers; the parts of an item that several warps share meet in a table and
// are added in warp order: results do not depend on scheduling.
//
// Arithmetic.  Codes become the fp16 values code - 8, exactly: the nibble goes
// to the low mantissa bits of 1024, from which 1032 is subtracted, or stays in
// the high nibble (1024 + 16 code, times 1/16, minus 72).  The warp MMA's eight
// columns are the expert's tokens.  Activations are scaled by a power of two
// for each token so that the largest lies in [2^14, 2^15).  fp16 x needs no scale
// and enters as one exact column.  bf16 x enters as one column, too: exact above
// 2^-31 of the largest, and to half of fp16's smallest step, 2^-39 of the largest,
// below.  fp32 x, and h always, enter as two columns (the fp16 value and the fp16
// remainder: 22 bits, and the same 2^-39).  (h as one column, 11 bits, let 40 % of
// the fp16 and 10 % of the bf16 outputs be rounded to another value than 64 bits
// give; it took 24.5 us for 25.0 with one token on six of 64 experts, 56.2 for 57.5
// on two of eight 4096 x 11008 ones, and 87.2 for 91.5 at 32 tokens, where twice as
// many fit a segment, all with the router.)  A scale is 2^114 at most, so values
// are cut to 2^-138 at the least.  Products are exact, sums are fp32.
//
// Measured, weights cold: one token on two of eight 4096 x 11008 experts, 152 MB
// in 49 us: about 16 and 10 are the two streams (6.2 and 5.1 TB/s), 5 the plan
// and x, 6 h, 12 joins, barriers, the sum and the launch.  32 tokens on 64
// experts of 2048 x 1408, 299 MB in 85 us; one token on six of them, 29 MB in
// 18.9 us.  Bound by memory while weights stream, by the latency of the steps
// between elsewhere (where warps wait longest for instructions, all of them new).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gq.h"
#include "gq_device.cuh"
#include "gq_host.h"

namespace gq {
namespace {

constexpr int kWarps = 20;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxT = 64, kMaxTopK = 16, kMaxE = 1024;
constexpr int kMaxPairs = kMaxT * kMaxTopK;
constexpr int kMaxK = 16384;
constexpr int kMaxCols = 8;   // columns of a segment: the MMA's n
constexpr int kMaxSegs = 16;  // segments of a string
constexpr size_t kSmemBudget = 227 * 1024;

// A stage: 8 blocks of 32 weights x 16 rows, what a warp copies at a time.  At
// the end of a Q4_0 row group it may hold fewer (whole units of two blocks).
constexpr int kStageCodes = 2048;
constexpr int kStageBytes = 2304;   // codes, then scales
constexpr int kDepth = 2;           // stages of a warp's ring
constexpr size_t kRingBytes = static_cast<size_t>(kWarps) * kDepth * kStageBytes;

// n / d for n * d < 2^32, d known to the host.  (Every warp divides a few times
// at each phase; as the compiler's division these cost 1 us a phase.)
struct Div {
  unsigned d, m;
  __device__ __forceinline__ int operator()(int n) const {
    return m ? static_cast<int>(__umulhi(static_cast<unsigned>(n), m)) : n;
  }
};
Div make_div(unsigned d) { return Div{d, d > 1 ? static_cast<unsigned>((1ull << 32) / d + 1) : 0u}; }

// One of the two products: gate and up, or down.
struct Phase {
  const uint8_t* w0;        // gate, or down
  const uint8_t* w1;        // up
  int K;                    // columns of the weights
  int groups;               // row groups (16 rows) of one expert
  int stages;               // of a row group
  Div by_groups, by_item, by_vecs;  // row groups, stages of an item, 8-value pieces of a padded row
  int64_t group_bytes;
  int two;                  // two columns for each token (always so for down)
  int cap;                  // tokens of a segment at most, a power of two
  int part;                 // floats of a part in the table
};

// Down's activations are two terms each, whatever the types; x's are where x is fp32.
template <bool GATE_UP>
__device__ __forceinline__ bool two_terms(const Phase& ph) {
  return !GATE_UP || ph.two;
}

struct MoeArgs {
  Phase ph[2];
  const void* x;            // [T][H]
  const int32_t* ids;       // [T][k]
  const float* weights;     // [T][k]
  void* y;                  // [T][H]
  float* h;                 // [pairs][I], by slot
  float* out;               // [pairs][H], by pair
  unsigned long long* hmax; // [pairs] largest |h| of a slot, under the call's number; see note_hmax()
  unsigned long long* arrivals;  // at the grid barriers, a multiple of the grid between calls
  int* dev_status;
  long long budget;
  int missing;              // arrivals that a grid barrier waits for in vain (the self-test), or 0
  int T, k, E, H;
  Div by_grid;
  int single;               // one token: down's rows run over its slots
  Div by_slots[kMaxTopK];   // stages of such a row, by slots
  int xtype, ytype;
  int bbytes;               // room for B fragments
  uint32_t b_off, tab_off, plan_off;  // dynamic shared memory, after the rings
};

struct Seg {
  short e, slot0;
  int n;
};

struct Col {
  int row;           // of x, or of h
  float mul;         // a single token's slot weight
  int dst, pitch;    // of its B fragments: shared offset, columns
};

struct Plan {
  int nseg[2];
  int go;                              // the grid barrier was passed
  unsigned long long call;             // this call's number; see note_hmax()
  unsigned common;                     // a single token's largest |weight * h|
  // of a string's segments
  int ncols;                           // tokens of all segments
  Col col[kMaxSegs * kMaxCols];
  unsigned top[kMaxSegs * kMaxCols];   // their largest magnitude as bits
  int boff[kMaxSegs];                  // their B fragments
  float inv[kMaxSegs][kMaxCols];       // 1 / scale of their tokens
  unsigned hmax[kMaxSegs][kMaxCols];   // largest |h|
  // in dynamic shared memory
  Seg* seg[2];                         // [pairs] of each phase
  short* order;                        // [pairs] slot -> pair
  float* weight;                       // [pairs]; used only where the id names an expert
  int* id;                             // [pairs, rounded up to 4] the expert, or kNobody
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
// Eight consecutive values of an element type, as they are stored and as floats.
struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ Raw read8(const void* base, int64_t i, int type) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * (type == GQ_F32 ? 4 : 2));
  Raw r;
  r.a = __ldcg(p);
  r.b = type == GQ_F32 ? __ldcg(p + 1) : uint4{};
  return r;
}
__device__ __forceinline__ void values(const Raw& r, int type, float v[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  if (type == GQ_F32) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(w[q]);
    return;
  }
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

constexpr int kNobody = kMaxE;  // sorts behind every expert

// Pairs sorted by expert (stable), and the segments of both phases; ids outside
// [0, E) are left out.  A pair's slot is the number of smaller keys (expert,
// pair), counted by one or more lanes of its own.
__device__ void make_plan(Plan& pl, const MoeArgs& a) {
  const int P = a.T * a.k, P4 = (P + 3) & ~3;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* key = reinterpret_cast<int*>(msm);  // in the rings' place, until the first copies
  short* expert = reinterpret_cast<short*>(key + P4);  // by slot
  for (int p = threadIdx.x; p < P4; p += kThreads) {
    const int id = p < P ? __ldcg(a.ids + p) : -1;
    const float w = p < P ? __ldcg(a.weights + p) : 0.f;
    const bool ok = id >= 0 && id < a.E;
    if (blockIdx.x == 0 && (id < -1 || id >= a.E)) report(a.dev_status, GQ_DEV_RANGE);
    pl.id[p] = ok ? id : kNobody;
    if (p < P) pl.weight[p] = w;
    key[p] = (ok ? id : kNobody) * kMaxPairs + p;
  }
  __syncthreads();
  int share_log = 0;  // 2^share_log lanes for each pair
  while (share_log < 5 && (P << (share_log + 1)) <= kThreads) ++share_log;
  const int lanes = 1 << share_log, sub = lane & (lanes - 1);
  int slots = 0;  // pairs that name an expert
  for (int p0 = 0; p0 < P; p0 += kThreads >> share_log) {
    const int p = p0 + (threadIdx.x >> share_log);
    const int mine = p < P ? key[p] : 0x7FFFFFFF;
    int less = 0;
    for (int q = 4 * sub; q < P4; q += 4 * lanes) {
      const int4 v = *reinterpret_cast<const int4*>(key + q);
      less += (v.x < mine) + (v.y < mine) + (v.z < mine) + (v.w < mine);
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) less += __shfl_xor_sync(0xFFFFFFFFu, less, o);
    const bool ok = sub == 0 && mine < kNobody * kMaxPairs;
    if (ok) {
      pl.order[less] = static_cast<short>(p);
      expert[less] = static_cast<short>(pl.id[p]);
    }
    slots += __syncthreads_count(ok);
  }
  if (warp < 2) {  // a segment begins with an expert and after every cap of its pairs
    const int cap = a.ph[warp].cap;
    Seg* seg = pl.seg[warp];
    int n = 0, first = 0;  // segments; the current expert's first slot
    for (int s0 = 0; s0 < slots; s0 += 32) {
      const int s = s0 + lane;
      const bool head = s < slots && (s == 0 || expert[s] != expert[s - 1]);
      const unsigned heads = __ballot_sync(0xFFFFFFFFu, head), upto = heads & (0xFFFFFFFFu >> (31 - lane));
      const int run = upto ? s0 + 31 - __clz(upto) : first;
      const bool begins = s < slots && ((s - run) & (cap - 1)) == 0;
      const unsigned b = __ballot_sync(0xFFFFFFFFu, begins);
      if (begins) seg[n + __popc(b & ((1u << lane) - 1u))] = Seg{expert[s], static_cast<short>(s), 0};
      n += __popc(b);
      if (heads) first = s0 + 31 - __clz(heads);
    }
    __syncwarp();
    for (int i = lane; i < n; i += 32) seg[i].n = (i + 1 < n ? seg[i + 1].slot0 : slots) - seg[i].slot0;
    if (lane == 0) pl.nseg[warp] = n;
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

// The largest |h| of a slot is agreed on through the workspace, by all CTAs that
// have rows of it.  An entry is the number of the call that wrote it (48 bits)
// over the upper 16 bits of the value's (its exponent, which sets the scale, and
// seven bits more): entries of other calls are smaller and count as zero, so none
// has to be cleared, and what a call leaves that gave up at a barrier does no harm.
// The number is one more than the barriers that the grid has passed: no CTA of
// this call can have changed it before this CTA arrives, and it grows with every
// call, also with one that gives up (all its CTAs arrive at its barriers).
__device__ __forceinline__ unsigned long long call_number(const MoeArgs& a) {
  return __ldcg(a.arrivals) / gridDim.x + 1;
}
__device__ __forceinline__ void note_hmax(const MoeArgs& a, const Plan& pl, int slot, unsigned bits) {
  atomicMax(a.hmax + slot, pl.call << 16 | bits >> 15);
}
__device__ __forceinline__ unsigned read_hmax(const MoeArgs& a, const Plan& pl, int slot) {
  const unsigned long long v = __ldcg(a.hmax + slot);
  return v >> 16 == pl.call ? static_cast<unsigned>(v & 0xFFFFu) << 15 : 0u;
}

// Columns that the B fragments of a segment have room for: a power of two, so
// that every offset in the inner loop is a constant.
__device__ __forceinline__ int col_pitch(int ncol) {
  return ncol <= 2 ? ncol : ncol <= 4 ? 4 : 8;
}

__host__ __device__ __forceinline__ int padded(int K) { return (K + 255) & ~255; }

// B fragments of the tokens of a string's segments (all threads call it).
// Column c of block b and lane group t: 16 bytes at ((b * pitch + c) * 4 + t) * 16
// of its segment, the values 4t, 4t+2, 4t+1, 4t+3 of the block and the same at
// +16; zeros up to whole stages.  fp16 x goes in as it is; otherwise a token's
// largest magnitude sets its scale: of h it is known, of x it is taken here, from
// the values of this CTA's tokens as they pass (reading all tokens for it in every
// CTA cost 5 us at 32 tokens).  A
// single token's h is multiplied by its slot's weight and scaled by the largest
// product of all slots.
template <bool GATE_UP>
__device__ __forceinline__ void load_b(const MoeArgs& a, const Phase& ph, Plan& pl, int seg0, int segs) {
  const bool single = !GATE_UP && a.single, two = two_terms<GATE_UP>(ph);
  const int type = GATE_UP ? a.xtype : GQ_F32;
  const bool find = GATE_UP && type != GQ_F16;
  const int i = threadIdx.x / kMaxCols, c = threadIdx.x % kMaxCols;
  int before = 0;  // columns of the segments before this thread's
  Seg sg{0, 0, 0};
  if (i < segs) sg = pl.seg[!GATE_UP][seg0 + i];
  if (c < sg.n) {
    const int row = GATE_UP ? pl.order[sg.slot0 + c] / a.k : sg.slot0 + c;
    unsigned top = find ? 0u : GATE_UP ? 0x46800000u : read_hmax(a, pl, row);  // (2^14: a scale of 1)
    float mul = 1.0f;
    if (single) {
      mul = pl.weight[pl.order[row]];
      top = __float_as_uint(fabsf(__uint_as_float(top) * mul));
      atomicMax(&pl.common, top);
    }
    int off = a.b_off;
    for (int j = 0; j < i; ++j) {
      const int n = pl.seg[!GATE_UP][seg0 + j].n;
      before += n;
      off += col_pitch(two ? 2 * n : n) * padded(ph.K) * 2;
    }
    pl.col[before + c] = Col{row, mul, off + (two ? 2 * c : c) * 64, col_pitch(two ? 2 * sg.n : sg.n)};
    pl.top[before + c] = top;
    pl.hmax[i][c] = 0u;
    if (c == 0) pl.boff[i] = off;
    if (i == segs - 1 && c == 0) pl.ncols = before + sg.n;
  }
  __syncthreads();
  const int vecs = padded(ph.K) / 8, real = ph.K / 8, nvec = pl.ncols * vecs;
  const void* src = GATE_UP ? a.x : a.h;
  auto fetch = [&](int i) -> Raw {  // piece i of the columns
    const int cc = ph.by_vecs(i), r = i - cc * vecs;
    if (i >= nvec || r >= real) return Raw{};
    return read8(src, static_cast<int64_t>(pl.col[cc].row) * ph.K + 8 * r, type);
  };
  const Raw first = fetch(threadIdx.x);  // (keeping more than one between the passes made longer code, and slower)
  if (find) {
    auto note = [&](const Raw& r, int i) {
      float v[8];
      values(r, type, v);
      unsigned m = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(v[q]) & 0x7FFFFFFFu);
      // (whole warps are of one column but where a column ends inside a warp)
      const int cc = i < nvec ? ph.by_vecs(i) : -1;
      if (__match_any_sync(0xFFFFFFFFu, cc) == 0xFFFFFFFFu) {
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if ((threadIdx.x & 31) == 0 && cc >= 0) atomicMax(&pl.top[cc], m);
      } else if (cc >= 0) {
        atomicMax(&pl.top[cc], m);
      }
    };
    note(first, threadIdx.x);
    for (int i0 = kThreads; i0 < nvec; i0 += kThreads) note(fetch(i0 + threadIdx.x), i0 + threadIdx.x);
    __syncthreads();
  }
  if (c < sg.n)  // scale_of() is a power of two: the reciprocal is exact
    pl.inv[i][c] = 1.0f / scale_of(single ? pl.common : pl.top[before + c]);
  auto put8 = [&](const Raw& raw, int i) {
    if (i >= nvec) return;
    const int cc = ph.by_vecs(i), r = i - cc * vecs;
    const Col col = pl.col[cc];
    const float f = scale_of(single ? pl.common : pl.top[cc]) * col.mul;
    float v[8];
    values(raw, type, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f;
    uint8_t* d = msm + col.dst + (r >> 2) * col.pitch * 64 + (r & 1) * 32 + (r & 2) * 4;
    auto store = [&](uint8_t* d) {  // and leaves what fp16 leaves out
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const __half2 lo = __floats2half2_rn(v[4 * w], v[4 * w + 2]), hi = __floats2half2_rn(v[4 * w + 1], v[4 * w + 3]);
        *reinterpret_cast<uint2*>(d + 16 * w) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                           *reinterpret_cast<const uint32_t*>(&hi));
        const float2 l = __half22float2(lo), h = __half22float2(hi);
        v[4 * w] -= l.x, v[4 * w + 2] -= l.y, v[4 * w + 1] -= h.x, v[4 * w + 3] -= h.y;
      }
    };
    store(d);
    if (two) store(d + 64);
  };
  put8(first, threadIdx.x);
  for (int i0 = kThreads; i0 < nvec; i0 += kThreads) put8(fetch(i0 + threadIdx.x), i0 + threadIdx.x);
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
// g+8, da, db the rows' scales, xb this lane's B fragment.  With one column a
// lane keeps one sum for each row.
template <int CP>
__device__ __forceinline__ void block_math(uint32_t wa, uint32_t wb, float da, float db, float acc[4],
                                           const uint8_t* xb) {
  const uint32_t wa8 = wa >> 8, wb8 = wb >> 8;
  const uint4 xv = ld128(xb);
  float c[4];
  mma_f16_z(c, low_codes(wa), low_codes(wb), low_codes(wa8), low_codes(wb8), xv.x, xv.y);
  mma_f16(c, high_codes(wa), high_codes(wb), high_codes(wa8), high_codes(wb8), xv.z, xv.w);
  acc[0] = fmaf(da, c[0], acc[0]);
  if (CP > 1) acc[1] = fmaf(da, c[1], acc[1]);
  acc[2] = fmaf(db, c[2], acc[2]);
  if (CP > 1) acc[3] = fmaf(db, c[3], acc[3]);
}

// acc += the stage in ring slot st: four units of two blocks (Q4_0) or one super-block.
template <int FMT, int CP>
__device__ __forceinline__ void stage_math(const uint8_t* st, int lane, float acc[4], const uint8_t* xb) {
  const uint8_t* code = st + (FMT == GQ_FMT_Q4_0 ? 16 : 32) * lane;
  const uint8_t* sc = st + kStageCodes + 4 * (lane >> 2);
  if constexpr (FMT == GQ_FMT_Q4_0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = ld128(code + 512 * i);
      const float2 da = halves(ld32(sc + 64 * i));
      const float2 db = halves(ld32(sc + 64 * i + 32));
      block_math<CP>(v.x, v.y, da.x, db.x, acc, xb + (2 * i) * (64 * CP));
      block_math<CP>(v.z, v.w, da.y, db.y, acc, xb + (2 * i + 1) * (64 * CP));
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

// Items [ra, rb) of all segments' (item r is row group r % groups of segment r /
// groups) whose B fragments are in shared memory together.
struct String {
  int ra, rb, seg0, segs;
};

// A warp's next copy: stage k of row group g of segment s (gate's stages, then
// up's), `left` stages in all; this lane's sources in it.
template <int FMT, bool GATE_UP>
struct Feed {
  const uint8_t* code;
  const uint8_t* scale;
  int s, g, k, left;
  int segs;  // a single token's down: segments of a row (0: one)

  __device__ __forceinline__ void seek(const Phase& ph, const Plan& pl, int stages, int lane) {
    const bool up = GATE_UP && k >= stages;
    const int kk = up ? k - stages : k;
    const uint8_t* group = (up ? ph.w1 : ph.w0) +
                           (static_cast<int64_t>(pl.seg[!GATE_UP][s].e) * ph.groups + g) * ph.group_bytes;
    const int c = kk >> 3, j = kk & 7;
    if constexpr (FMT == GQ_FMT_Q4_0) {
      // tiles of 32 units (512 bytes of codes, 64 of scales); a stage is four
      const int nu = min(32, (ph.K >> 6) - 32 * c);
      const uint8_t* tile = group + static_cast<int64_t>(c) * 18432;
      code = tile + 2048 * j + 16 * lane;
      scale = tile + 512 * nu + 256 * j + 16 * lane;
    } else {
      // tiles of 8 super-blocks (2048 bytes of codes, 128 of sub-scales, 32 of S); a stage is one
      const int ns = min(8, (ph.K >> 8) - 8 * c);
      const uint8_t* tile = group + static_cast<int64_t>(c) * 17664;
      code = tile + 2048 * j + 16 * lane;
      scale = lane < 8 ? tile + 2048 * ns + 128 * j + 16 * lane : tile + 2176 * ns + 32 * j + 16 * (lane - 8);
    }
  }
  // Copies it to ring slot `slot` (a byte offset); always a group, so that groups count stages.
  __device__ __forceinline__ void step(const Phase& ph, const Plan& pl, int stages, uint32_t slot, int lane) {
    if (left > 0) {
      const uint32_t dst = smem_addr(msm) + slot + 16 * lane;
      const int kk = GATE_UP && k >= stages ? k - stages : k;
      const bool end = kk == stages - 1;
      const int n = FMT == GQ_FMT_Q4_0 && end ? (ph.K >> 6) - 4 * kk : 4;  // units
      if (n == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) copy16(dst + 512 * i, code + 512 * i);
      } else {
        for (int i = 0; i < n; ++i) copy16(dst + 512 * i, code + 512 * i);
        // units that are not there: scales of zero (and their activations are zeros)
        if (lane >= 4 * n && lane < 16) *reinterpret_cast<uint4*>(msm + slot + kStageCodes + 16 * lane) = uint4{};
      }
      if (lane < (FMT == GQ_FMT_Q4_0 ? 4 * n : 10)) copy16(dst + kStageCodes, scale);
      --left;
      ++k;
      if (end || ((kk + 1) & 7) == 0) {  // another tile
        if (k == (GATE_UP ? 2 * stages : stages)) {
          k = 0;
          if (!GATE_UP && segs) {
            if (++s == segs) {
              s = 0;
              ++g;
            }
          } else if (++g == ph.groups) {
            g = 0;
            ++s;
          }
        }
        if (left > 0) seek(ph, pl, stages, lane);
      } else {
        code += 2048;
        scale += FMT == GQ_FMT_Q4_0 ? 256 : (lane < 8 ? 128 : 32);
      }
    }
    copies_commit();
  }
};

// The parts of items that warps share, of both matrices for gate and up.  The
// later warps' parts of an item are in a table, one for each warp; the part of
// the warp that began it, which adds the others to it, is in the last slot of
// its own ring, which is empty from the end of its stages until the next
// string's activations are there.
__device__ __forceinline__ float* later_part(const MoeArgs& a, const Phase& ph, int warp) {
  return reinterpret_cast<float*>(msm + a.tab_off) + warp * ph.part;
}
__device__ __forceinline__ float* first_part() {
  return reinterpret_cast<float*>(msm + ((threadIdx.x >> 5) * kDepth + kDepth - 1) * kStageBytes);
}
static_assert(kDepth > 1 && 2 * 16 * kMaxCols * sizeof(float) <= kStageBytes, "a part of both matrices");
template <int CP>
__device__ __forceinline__ void store_part(float* d, const float acc[4], int lane) {
  const int g8 = lane >> 2, t = lane & 3;
  if (CP == 1) {
    if (t == 0) {
      d[g8] = acc[0];
      d[g8 + 8] = acc[2];
    }
  } else if (2 * t < CP) {
    *reinterpret_cast<float2*>(d + g8 * CP + 2 * t) = make_float2(acc[0], acc[1]);
    *reinterpret_cast<float2*>(d + (g8 + 8) * CP + 2 * t) = make_float2(acc[2], acc[3]);
  }
}

// Token c's row of a finished item: h (whose size it returns, as bits), or the
// pair's output.
template <bool GATE_UP>
__device__ __forceinline__ unsigned put(const MoeArgs& a, const Phase& ph, const Plan& pl, const Seg& sg, int c,
                                        int row, float v, float up) {
  if constexpr (GATE_UP) {
    // within 2 steps; a quotient by 2^126 or more is zero (silu of less than -87)
    const float h = __fdividef(v, 1.0f + expf(-v)) * up;
    __stcg(a.h + static_cast<int64_t>(sg.slot0 + c) * (ph.groups * 16) + row, h);
    return __float_as_uint(h) & 0x7FFFFFFFu;
  } else if (a.single) {
    store_elem(a.y, row, v, a.ytype);
    return 0u;
  } else {
    __stcg(a.out + static_cast<int64_t>(pl.order[sg.slot0 + c]) * (ph.groups * 16) + row, v);
    return 0u;
  }
}

// Row group g of an item, whose sums a warp has: rows g8 and g8 + 8, columns 2t
// and 2t+1 in each lane (two tokens, or one in two columns); top: the largest
// |h| of the lane's tokens.
template <bool GATE_UP>
__device__ __forceinline__ void finish(const MoeArgs& a, const Phase& ph, const Plan& pl, const Seg& sg, int local,
                                       int g, const float acc[4], const float gate[4], unsigned top[2]) {
  const int lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;
  const bool two = two_terms<GATE_UP>(ph);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = two ? t : 2 * t + i;
    if (c < sg.n && !(two && i)) {
      const float f = pl.inv[local][c];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float v = two ? acc[2 * half] + acc[2 * half + 1] : acc[2 * half + i];
        const float w = two ? gate[2 * half] + gate[2 * half + 1] : gate[2 * half + i];
        const unsigned m = put<GATE_UP>(a, ph, pl, sg, c, 16 * g + g8 + 8 * half, (GATE_UP ? w : v) * f, v * f);
        top[i] = max(top[i], m);
      }
    }
  }
}
// The segment's largest |h|, from those of the lanes.
__device__ __forceinline__ void note_tops(const Phase& ph, Plan& pl, const Seg& sg, int local, const unsigned top[2]) {
  const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    unsigned m = top[i];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const int c = ph.two ? t : 2 * t + i;
    if (lane < 4 && c < sg.n && !(ph.two && i) && m) atomicMax(&pl.hmax[local][c], m);
  }
}

template <int FMT, bool GATE_UP>
struct Work {
  int r, r1;      // items left to this CTA
  bool more;
  String st;
  int u0, u1;     // this warp's stages of the string
  int s0, g0, k0; // where they begin
  Div item;       // stages of an item
  Feed<FMT, GATE_UP> feed;

  __device__ __forceinline__ static uint32_t ring() { return (threadIdx.x >> 5) * (kDepth * kStageBytes); }
  // The next string, and the first copy of this warp's share of it.
  __device__ __forceinline__ void next(const MoeArgs& a, const Phase& ph, const Plan& pl) {
    more = r < r1;
    if (!more) return;
    st.ra = r;
    if (!GATE_UP && a.single) {  // one string: all slots' h are in shared memory
      st.seg0 = 0;
      st.segs = pl.nseg[1];
      r = r1;
    } else {
      st.seg0 = ph.by_groups(r);
      st.segs = 0;
    }
    int bytes = 0;
    while (r < r1 && st.segs < kMaxSegs) {
      const int s = st.seg0 + st.segs;
      bytes += col_pitch(two_terms<GATE_UP>(ph) ? 2 * pl.seg[!GATE_UP][s].n : pl.seg[!GATE_UP][s].n) * padded(ph.K) * 2;
      if (bytes > a.bbytes && st.segs) break;  // (one segment always fits)
      r = min(r1, (s + 1) * ph.groups);
      ++st.segs;
    }
    st.rb = r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned tu = (st.rb - st.ra) * item.d;
    u0 = static_cast<int>(tu * warp / kWarps);
    u1 = static_cast<int>(tu * (warp + 1) / kWarps);
    const int i = item(u0);
    feed.k = k0 = u0 - i * item.d;
    feed.segs = 0;
    if (!GATE_UP && a.single) {
      s0 = 0;
      g0 = st.ra + i;
      feed.segs = st.segs;
      feed.s = ph.by_item(k0);
      feed.k = k0 - feed.s * ph.stages;
    } else {
      feed.s = s0 = ph.by_groups(st.ra + i);
      g0 = st.ra + i - s0 * ph.groups;
    }
    feed.g = g0;
    feed.left = u1 - u0;
    if (feed.left > 0) feed.seek(ph, pl, ph.stages, lane);
    feed.step(ph, pl, ph.stages, ring(), lane);
  }
  __device__ __forceinline__ void start(const MoeArgs& a, const Plan& pl) {
    const Phase& ph = a.ph[!GATE_UP];
    const bool single = !GATE_UP && a.single;
    const int nseg = pl.nseg[!GATE_UP];
    const int total = single ? (nseg ? ph.groups : 0) : nseg * ph.groups;  // at most 2^20
    item = single && nseg ? a.by_slots[nseg - 1] : ph.by_item;
    const int each = a.by_grid(total), rest = total - each * static_cast<int>(gridDim.x);
    const int b = static_cast<int>(blockIdx.x);
    r = each * b + a.by_grid(rest * b);
    r1 = each * (b + 1) + a.by_grid(rest * (b + 1));
    next(a, ph, pl);
  }
};

// This warp's stages [u, ue) of the string, all of one segment, from stage k of
// row group g on.  `whole`: the warp has its item from the first stage on.
template <int FMT, int CP, bool GATE_UP>
__device__ __forceinline__ void stream(const MoeArgs& a, const Phase& ph, Plan& pl, Work<FMT, GATE_UP>& wk,
                                       const Seg& sg, int local, int u, int ue, int g, int k, bool& whole,
                                       uint32_t& slot) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;
  // columns past the last repeat existing ones (or hold what was there); their sums are not used
  const uint8_t* xb = msm + pl.boff[local] + (g8 & (CP - 1)) * 64 + t * 16;
  const int all = wk.item.d, stages = GATE_UP ? ph.stages : all;  // of an item, and of a row of it
  float acc[4] = {}, gate[4] = {};
  unsigned top[2] = {0u, 0u};  // largest |h| of this lane's tokens
  int kk = GATE_UP && k >= stages ? k - stages : k;
  const uint8_t* x = xb + kk * (8 * 64 * CP);
  // the row group ends: the gate's sums wait for up's, or the item is done
  auto row_end = [&]() {
    kk = 0;
    x = xb;
    if (GATE_UP && k == stages) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gate[i] = acc[i];
        acc[i] = 0.f;
      }
      return;
    }
    if (whole) {
      finish<GATE_UP>(a, ph, pl, sg, local, g, acc, gate, top);
    } else {
      float* d = later_part(a, ph, warp);
      if (GATE_UP) store_part<CP>(d, gate, lane);
      store_part<CP>(d + (GATE_UP ? 16 * CP : 0), acc, lane);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = gate[i] = 0.f;
    whole = true;
    k = 0;
    ++g;
  };
  for (; u < ue; ++u) {
    copies_wait<kDepth - 1>();
    __syncwarp();  // every lane's copies of the stage
    stage_math<FMT, CP>(msm + slot, lane, acc, x);
    x += 8 * 64 * CP;
    __syncwarp();  // every lane has read the stage
    wk.feed.step(ph, pl, ph.stages, slot, lane);
    slot = slot == wk.ring() + (kDepth - 1) * kStageBytes ? wk.ring() : slot + kStageBytes;
    ++k;
    if (++kk == stages) row_end();
  }
  if (k > 0 && k < all && u == wk.u1 && wk.u1 > wk.u0) {  // the run ends inside an item
    float* d = whole ? first_part() : later_part(a, ph, warp);
    if (GATE_UP) {
      store_part<CP>(d, k < stages ? acc : gate, lane);
      if (k < stages) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = 0.f;
      }
    }
    store_part<CP>(d + (GATE_UP ? 16 * CP : 0), acc, lane);
  }
  if (GATE_UP) note_tops(ph, pl, sg, local, top);
}

// After the last stage of a string (stage `u1` of the string would follow): the
// item that this warp began and did not end (`cut`: row group g of segment sg,
// `end` its last stage + 1) takes the later warps' parts in order.
template <int FMT, bool GATE_UP>
__device__ __forceinline__ void join_parts(const MoeArgs& a, const Phase& ph, Plan& pl, const String& st,
                                           unsigned tu, bool cut, const Seg& sg, int local, int g, unsigned u1,
                                           unsigned end) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool two = two_terms<GATE_UP>(ph);
  __syncthreads();  // the parts are there; nobody reads B any more
  if (cut) {
    const int pitch = col_pitch(two ? 2 * sg.n : sg.n);
    const int row = lane & 15, half = lane >> 4;
    unsigned tops = 0;  // lane c: token c's largest
    // two tokens at a time, a lane for each row
#pragma unroll 1  // (run through once, so that each instruction has to be fetched: short code is faster)
    for (int c0 = 0; c0 < sg.n; c0 += 2) {
      const int c = min(c0 + half, sg.n - 1), at = row * pitch + (two ? 2 * c : c), up = 16 * pitch;
      const float* d = first_part() + at;
      float v = two ? d[0] + d[1] : d[0], u = 0.f;
      if (GATE_UP) u = two ? d[up] + d[up + 1] : d[up];
      d = later_part(a, ph, warp + 1) + at;
      unsigned begin = u1;
      for (unsigned w = warp + 1; begin < end; ++w) {
        const unsigned next = tu * (w + 1) / kWarps;
        if (next > begin) {  // (a warp without stages has no part)
          v += two ? d[0] + d[1] : d[0];
          if (GATE_UP) u += two ? d[up] + d[up + 1] : d[up];
        }
        begin = next;
        d += ph.part;
      }
      const float f = pl.inv[local][c];
      unsigned m = 0;
      if (c0 + half < sg.n) m = put<GATE_UP>(a, ph, pl, sg, c, 16 * g + row, v * f, u * f);
      if (GATE_UP) {
        const unsigned m0 = __reduce_max_sync(0xFFFFFFFFu, half ? 0u : m), m1 = __reduce_max_sync(0xFFFFFFFFu, half ? m : 0u);
        if (lane == c0) tops = m0;
        if (lane == c0 + 1) tops = m1;
      }
    }
    if (GATE_UP && lane < sg.n) atomicMax(&pl.hmax[local][lane], tops);
  }
  if (GATE_UP) {
    __syncthreads();
    if (threadIdx.x < st.segs * kMaxCols) {
      const int i = threadIdx.x / kMaxCols, c = threadIdx.x % kMaxCols;
      const Seg sh = pl.seg[0][st.seg0 + i];
      if (c < sh.n) note_hmax(a, pl, sh.slot0 + c, pl.hmax[i][c]);
    }
  }
}

// All strings of a phase.
template <int FMT, bool GATE_UP>
__device__ __forceinline__ void run_phase(const MoeArgs& a, Plan& pl, Work<FMT, GATE_UP>& wk) {
  const Phase& ph = a.ph[!GATE_UP];
  const int all = wk.item.d;
  while (wk.more) {
    const String st = wk.st;
    load_b<GATE_UP>(a, ph, pl, st.seg0, st.segs);
    // the rest of the ring (the first copies went ahead of B: a full ring of them would hold it up)
    for (int d = 1; d < kDepth; ++d)
      wk.feed.step(ph, pl, ph.stages, wk.ring() + d * kStageBytes, threadIdx.x & 31);
    __syncthreads();
    int u = wk.u0, s = wk.s0, g = wk.g0, k = wk.k0;
    const int u1 = wk.u1;
    int base = u - k - g * all;  // the stage of the string that segment s begins with
    bool whole = k == 0;
    uint32_t slot = wk.ring();
    Seg sg{0, 0, 0};
    int last_base = 0, last_s = 0;
    while (u < u1) {
      sg = pl.seg[!GATE_UP][s];
      const int ue = min(u1, base + ph.groups * all);
      switch (col_pitch(two_terms<GATE_UP>(ph) ? 2 * sg.n : sg.n)) {
        case 1:
          if constexpr (GATE_UP) stream<FMT, 1, GATE_UP>(a, ph, pl, wk, sg, s - st.seg0, u, ue, g, k, whole, slot);
          break;  // (down has two columns at least)
        case 2: stream<FMT, 2, GATE_UP>(a, ph, pl, wk, sg, s - st.seg0, u, ue, g, k, whole, slot); break;
        case 4: stream<FMT, 4, GATE_UP>(a, ph, pl, wk, sg, s - st.seg0, u, ue, g, k, whole, slot); break;
        default: stream<FMT, 8, GATE_UP>(a, ph, pl, wk, sg, s - st.seg0, u, ue, g, k, whole, slot);
      }
      u = ue;
      last_base = base;
      last_s = s;
      base += ph.groups * all;
      ++s;
      g = k = 0;
    }
    // the item that the warp's last stage is of
    const int li = wk.item(max(u1 - 1 - last_base, 0)), begin = last_base + li * all;
    const bool cut = u1 > wk.u0 && begin >= wk.u0 && u1 < begin + all;
    const unsigned tu = (st.rb - st.ra) * all;
    wk.next(a, ph, pl);
    join_parts<FMT, GATE_UP>(a, ph, pl, st, tu, cut, sg, last_s - st.seg0, li, u1, begin + all);
    if (wk.more) __syncthreads();  // before the next string's values
  }
}

// A barrier of the grid in two halves: what each CTA wrote before it arrives is
// seen by all after the wait, which gives up (false) once the budget has passed.
// The arrivals only ever count up (in 64 bits), so nothing has to be cleared.
// arrive() returns the count to wait for, in thread 0.
__device__ __forceinline__ unsigned long long grid_arrive(const MoeArgs& a) {
  __syncthreads();
  if (threadIdx.x) return 0;
  unsigned long long before;
  asm volatile("atom.add.release.gpu.global.u64 %0, [%1], 1;" : "=l"(before) : "l"(a.arrivals) : "memory");
  return (before / gridDim.x + 1) * gridDim.x;
}
__device__ __forceinline__ bool grid_wait(const MoeArgs& a, Plan& pl, unsigned long long target) {
  if (threadIdx.x == 0) {
    const long long t0 = clock64();
    int go = 1;
    for (;;) {
      unsigned long long v;
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(a.arrivals) : "memory");
      if (v >= target + a.missing) break;
      if (clock64() - t0 > a.budget) {
        go = 0;
        break;
      }
    }
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
    pl.id = reinterpret_cast<int*>(pl.seg[1] + pairs);
    pl.weight = reinterpret_cast<float*>(pl.id + ((pairs + 3) & ~3));
    pl.order = reinterpret_cast<short*>(pl.weight + pairs);
  }
  if (threadIdx.x == 0) pl.common = 0u;
  __syncthreads();
  pdl_wait();  // ids and x are final
  pdl_launch_dependents();
  if (threadIdx.x == 0) pl.call = call_number(a);
  make_plan(pl, a);
  {
    Work<FMT, true> gate_up;
    gate_up.start(a, pl);
    run_phase<FMT, true>(a, pl, gate_up);
  }
  unsigned long long target = grid_arrive(a);
  Work<FMT, false> down;
  down.start(a, pl);  // its first copies are under way while this CTA waits for the others
  bool ok = grid_wait(a, pl, target);
  if (ok) {
    run_phase<FMT, false>(a, pl, down);
    if (a.single) {
      if (pl.nseg[1] == 0)  // no slot names an expert
        for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.H; i += static_cast<int>(gridDim.x) * kThreads)
          store_elem(a.y, i, 0.f, a.ytype);
      return;
    }
  }
  if (!a.single) {  // (arrived at even after a wait that gave up: the count stays a multiple of the grid)
    target = grid_arrive(a);
    ok = ok && grid_wait(a, pl, target);
  }
  if (!ok) {
    copies_wait<0>();
    if (threadIdx.x == 0) report(a.dev_status, GQ_DEV_TIMEOUT);
    return;
  }
  // y[t] = sum_j w[t][j] * out[t][j] over the slots that name an expert
  const int n = a.T * a.H;
  const int i0 = static_cast<int>(blockIdx.x * kThreads + threadIdx.x);
  for (int i = i0; i < n; i += static_cast<int>(gridDim.x) * kThreads) {
    const int t = i / a.H, c = i - t * a.H;
    float v = 0.f;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
      const int p = t * a.k + j;
      if (pl.id[p] != kNobody) v = fmaf(pl.weight[p], __ldcg(a.out + static_cast<int64_t>(p) * a.H + c), v);
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
  w.h = w.hmax + kMaxPairs * 8;  // one size for every call, so that calls of any sizes may follow
  w.out = w.h + round256(static_cast<size_t>(T * k * I) * 4);
  w.total = w.out + round256(static_cast<size_t>(T * k * H) * 4);
  return w;
}

bool moe_dims(int64_t T, int64_t k, int64_t E) {
  return T <= kMaxT && k <= kMaxTopK && E <= kMaxE;
}
bool moe_width(int fmt, int64_t K) { return K % (fmt == GQ_FMT_Q4_0 ? 64 : 256) == 0 && K <= kMaxK; }

// Tokens of a segment and the layout of shared memory after the rings: the B
// fragments (2 bytes for each value of a column), the table of parts, and the
// plan.  Segments are as wide as both phases' columns and parts fit; what is
// left takes more segments of a string.
static_assert(sizeof(Plan) <= 5120, "the static part");
constexpr size_t kDynSmem = kSmemBudget - 5120;
size_t shape_smem(MoeArgs& a) {
  const int pairs = a.T * a.k;
  const size_t plan = (static_cast<size_t>(pairs) * (2 * sizeof(Seg) + 2 + 8) + 12 + 15) & ~size_t(15);
  const size_t left = kDynSmem - kRingBytes - plan;
  size_t tab = 0, b = 0;
  // one token: two columns for each slot, if all of them fit beside the parts
  const size_t slots = static_cast<size_t>(a.k) * padded(a.ph[1].K) * 2 * 2;
  // and if they are few enough for every CTA to read them all.  It saves a barrier
  // and costs the most where there are few rows.  Against a third phase, in us with
  // the router: 6 x 1408 values on 2048 rows 25.3 and 27.4; 8 x 2048 on 4096 rows
  // 48.4 and 49.8; 16 x 1024 on 1024 rows 26.8 and 26.8, on 512 24.6 and 23.5; 2 x
  // 11008 on 4096 rows 55.9 and 56.8, on 512 25.2 and 23.5; 16 x 1408 on 512 27.4 and
  // 24.3.
  a.single = a.T == 1 && a.k * padded(a.ph[1].K) <= 16384 &&
             slots + kWarps * 2 * 16 * 2 * sizeof(float) <= left;
  for (int f = 0; f < 2; ++f) {
    Phase& ph = a.ph[f];
    const size_t part = kWarps * (f == 0 ? 2 : 1) * 16 * sizeof(float);  // for each column
    const size_t need = (f == 1 && a.single ? 1 : static_cast<size_t>(pairs)) * (ph.two ? 2 : 1);
    size_t c = ph.two ? 2 : 1;  // powers of two
    while (c < kMaxCols && c < need && 2 * c * (static_cast<size_t>(padded(ph.K)) * 2 + part) <= left) c *= 2;
    ph.cap = static_cast<int>(ph.two ? c / 2 : c);
    tab = c * part > tab ? c * part : tab;
    b = c * padded(ph.K) * 2 > b ? c * padded(ph.K) * 2 : b;
  }
  if (a.single) b = slots > b ? slots : b;
  // the phases use the same room one after the other: narrower segments if both do not fit
  while (b + tab > left) {
    const size_t c0 = static_cast<size_t>(a.ph[0].cap) * (a.ph[0].two ? 2 : 1);
    const size_t c1 = static_cast<size_t>(a.ph[1].cap) * (a.ph[1].two ? 2 : 1);
    const size_t t0 = c0 * 2 * kWarps * 16 * sizeof(float), t1 = c1 * kWarps * 16 * sizeof(float);
    const size_t b0 = c0 * padded(a.ph[0].K) * 2, b1 = c1 * padded(a.ph[1].K) * 2;
    tab = t0 > t1 ? t0 : t1;
    b = b0 > b1 ? b0 : b1;
    if (a.single && slots > b) b = slots;
    if (b + tab <= left) break;
    Phase& ph = t0 >= t1 && a.ph[0].cap > 1 ? a.ph[0] : a.ph[1].cap > 1 ? a.ph[1] : a.ph[0];
    ph.cap /= 2;
  }
  for (Phase& ph : a.ph) {
    ph.by_groups = make_div(ph.groups);
    ph.by_item = make_div((&ph == a.ph ? 2 : 1) * ph.stages);
    ph.by_vecs = make_div(padded(ph.K) / 8);
  }
  for (int f = 0; f < 2; ++f) a.ph[f].part = (f == 0 ? 2 : 1) * 16 * a.ph[f].cap * (a.ph[f].two ? 2 : 1);
  for (int n = 0; n < kMaxTopK; ++n) a.by_slots[n] = make_div((n + 1) * a.ph[1].stages);
  a.b_off = kRingBytes;
  a.bbytes = static_cast<int>((left - tab) & ~size_t(15));
  a.tab_off = a.b_off + a.bbytes;
  a.plan_off = a.tab_off + static_cast<uint32_t>(tab);
  return a.plan_off + plan;
}

template <int FMT>
gq_status launch_moe(MoeArgs& a, cudaStream_t s) {
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
  return launch_cooperative(kern, dim3(sm_count()), dim3(kThreads), smem, s, a);
}

template <int FMT>
gq_status moe_entry(const void* gate, const void* up, const void* down, int64_t E, int64_t H,
                    int64_t I, const void* x, int x_dtype, int64_t T, const int32_t* ids,
                    const float* weights, int64_t k, void* y, int y_dtype, void* workspace,
                    size_t ws_bytes, unsigned flags, int* dev_status, void* stream,
                    long long budget = kWaitBudget, int missing = 0) {
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

  MoeArgs a{};
  auto phase = [](const void* w0, const void* w1, int64_t rows, int64_t K, bool two) {
    Phase ph{};
    ph.w0 = static_cast<const uint8_t*>(w0);
    ph.w1 = static_cast<const uint8_t*>(w1);
    ph.K = static_cast<int>(K);
    ph.groups = static_cast<int>(rows / 16);
    ph.stages = static_cast<int>((K + 255) / 256);
    ph.group_bytes = 16 * (FMT == GQ_FMT_Q4_0 ? K / 32 * 18 : K / 256 * 138);
    ph.two = two;
    return ph;
  };
  a.ph[0] = phase(gate, up, I, H, x_dtype == GQ_F32);
  a.ph[1] = phase(down, nullptr, H, I, true);
  a.by_grid = make_div(static_cast<unsigned>(sm_count()));
  a.x = x;
  a.ids = ids;
  a.weights = weights;
  a.y = y;
  a.h = reinterpret_cast<float*>(ws + l.h);
  a.out = reinterpret_cast<float*>(ws + l.out);
  a.hmax = reinterpret_cast<unsigned long long*>(ws + l.hmax);
  a.arrivals = reinterpret_cast<unsigned long long*>(ws + l.arrivals);
  a.dev_status = dev_status;
  a.budget = budget;
  a.missing = missing;
  a.T = static_cast<int>(T);
  a.k = static_cast<int>(k);
  a.E = static_cast<int>(E);
  a.H = static_cast<int>(H);
  a.xtype = x_dtype;
  a.ytype = y_dtype;
  return launch_moe<FMT>(a, s);
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

GQ_API gq_status gq_selftest_moe_timeout(const void* gate, const void* up, const void* down, int64_t E,
                                         int64_t H, int64_t I, const void* x, int64_t T,
                                         const int32_t* ids, const float* weights, int64_t k, void* y,
                                         void* workspace, size_t ws_bytes, int* dev_status,
                                         void* stream) {
  if (!dev_status) return GQ_ERR_INVALID_ARG;
  return gq::moe_entry<GQ_FMT_Q4_0>(gate, up, down, E, H, I, x, GQ_F16, T, ids, weights, k, y, GQ_F16,
                                    workspace, ws_bytes, 0u, dev_status, stream, 2000000LL, 1);
}

}  // extern "C"
