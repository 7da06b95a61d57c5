// gq_fp8_gemm.cu -- product of 8-bit block-scaled matrices on the tcgen05
// tensor cores,
//   Y[b][m] = sum_g sx[b][g] * sw[m / 128][g] * sum_{k in group g} X[b][k] * W[m][k],
// groups of 128 along K, e4m3 codes, fp32 scales.
//
// The scales change every 128 values of K, so the tensor core sums one group
// at a time and the groups are added in registers.  Tokens are the rows of the
// accumulator (the lanes of tensor memory) and weight rows its columns, which
// makes the factor of a group one number for a thread: its token's scale times
// the weight block's.
//
// One CTA per SM, over tiles of 128 tokens x BN weight rows and k-steps of one
// group:
//  * warp 8 (producer): both operands' 128-byte rows by TMA, 128-byte swizzle;
//  * warp 9 (MMA): four tcgen05.mma (K = 32) to a k-step, into one of the
//    accumulator buffers in tensor memory (512 columns in all);
//  * warp 10 (scales): the factors of four k-steps at a time, ahead of their
//    use, into shared memory;
//  * warps 0..7: read the buffer back and add it, times the factor, to sums in
//    registers (a thread holds one token and half of the columns); at the
//    end of a tile they round once and store, through shared memory and TMA
//    where Y's rows allow it (from registers the stores of a 180 MB output cost
//    48 us: the tile's sums have to leave before the next one's begin).
// While the warps add one group the MMAs fill other buffers.
//
// With many tiles two CTAs of a cluster share one of 256 tokens x 256 weight
// rows (cta_group::2): each holds its 128 tokens and half of the weight rows, so
// that a k-step takes 64 KB of shared-memory traffic in each instead of 96 KB
// (writes and the MMAs' reads at 128 bytes a cycle, beside 512 cycles of MMA).
// The leader's MMA warp issues for both; loads of both count on its barriers,
// commits arrive at both CTAs', and both epilogues release its buffers.
//
// When tiles are few, each is cut along K into the same number of pieces, which
// leave fp32 sums in the workspace; a second launch adds them in order.  (Cutting
// the k-steps of all tiles evenly and joining in the CTA that came last cost 10
// us more at 37 tokens.)
// For fewer than 128 tokens only the rows that exist are loaded; the other
// lanes hold garbage that nothing reads.
//
// Measured: 4096 tokens x 11008 x 4096 (fp32 out), 209 us, 1.77 PFLOP/s, in short
// runs and 238 us in a long loop, at 1610 MHz under the power limit.  Loads and
// MMAs alone take 113 us; with sixteen promoting warps the whole took 212, without
// the reads of tensor memory 197, without the MMAs 186, without either and without
// loads 172: the handshakes and sums of each k-step bound it.  So they do 500
// tokens x 4096 x 11008, 35 us (39 in a long loop), and 37 x 11000 x 4096, 16.3 us:
// 0.38 us a k-step, 0.37 without loads, MMAs and reads.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gq.h"
#include "gq_device.cuh"
#include "gq_fp8.h"
#include "gq_host.h"
#include "gq_tc.cuh"

namespace gq {
namespace {

constexpr int kBM = 128;                 // tokens of a tile
constexpr int kBK = 128;                 // bytes of K in a step: one group of scales
constexpr int kEpiWarps = 8;              // (sixteen: the largest case 210 us instead of 204, others the same)
constexpr int kThreads = 32 * (kEpiWarps + 3);
constexpr int kStoreBytes = 2048;        // 32 rows x 64 bytes of outputs, for each epilogue warp
constexpr int kFactorSteps = 4;          // k-steps of a slot of factors
constexpr int kFactorSlots = 3;
constexpr int kFactorBytes = kFactorSlots * kFactorSteps * 2 * kBM * 4;  // for each half of the columns
constexpr int kTileX = kBM * kBK;

// Tile t covers tokens rows * (t / tm) .. and weight rows BN * (t % tm) ..; it is
// cut into `cuts` pieces along its S k-steps.  CTA (or pair) i of P takes pieces
// i, i + P, ...
struct Split {
  int S, T, P, tm, cuts;
};

struct Args {
  const float* sx;
  const float* sw;
  void* Y;
  int* dev_status;
  long long budget;
  int64_t M;
  int B, kblocks, ytype, xrows;  // xrows: rows of an X box
  int skip;                      // k-steps of each CTA that are never loaded (the self-test: the first), or 0
  int tma_y;                     // Y's rows are whole 16-byte pieces, so that TMA can store them
  Split sp;
  float* parts;  // [pieces][rows][BN] of cut tiles
};

extern __shared__ __align__(1024) uint8_t fsm[];

__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Instruction descriptor, kind::f8f6f4: e4m3 A and B (both K-major), fp32 D.
constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack2(float a, float b, int type) {
  if (type == GQ_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// N consecutive outputs of one token from weight row m on.
template <int N>
__device__ __forceinline__ void store_row(const Args& a, int64_t row, int64_t m, const float* v) {
  const int64_t at = row * a.M + m;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (m + i < a.M) store_elem(a.Y, at + i, v[i], a.ytype);
}

// This thread's bulk stores have read their shared memory (READ), or are done.
template <bool READ>
__device__ __forceinline__ void bulk_stores_wait() {
  if constexpr (READ) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  else asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// A warp's 32 tokens x N columns (lane: token) from column m, token row on: 64
// bytes of each row at a time through `buf` (64-byte swizzle, so that lanes
// write without bank conflicts).  Rows and columns past Y's end are not stored.
template <int N>
__device__ __forceinline__ void store_tile(const CUtensorMap* map, uint8_t* buf, const float* v, int m, int row,
                                           int64_t M, int type) {
  const int lane = threadIdx.x & 31, turn = (lane >> 1) & 3;
  auto send = [&](int col) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && col < M) {
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(col),
                   "r"(row), "r"(smem_addr(buf))
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      bulk_stores_wait<true>();
    }
    __syncwarp();
  };
  if (type == GQ_F32) {
#pragma unroll
    for (int c = 0; c < N; c += 16) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4*>(buf + lane * 64 + ((q ^ turn) << 4)) =
            make_float4(v[c + 4 * q], v[c + 4 * q + 1], v[c + 4 * q + 2], v[c + 4 * q + 3]);
      send(m + c);
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 32) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(buf + lane * 64 + ((q ^ turn) << 4)) =
            make_uint4(pack2(v[c + 8 * q], v[c + 8 * q + 1], type), pack2(v[c + 8 * q + 2], v[c + 8 * q + 3], type),
                       pack2(v[c + 8 * q + 4], v[c + 8 * q + 5], type), pack2(v[c + 8 * q + 6], v[c + 8 * q + 7], type));
      send(m + c);
    }
  }
}

// The pieces of a CTA (or pair).
struct Run {
  int first;
  const Split& sp;
  __device__ __forceinline__ int count() const { return (sp.T * sp.cuts - first + sp.P - 1) / sp.P; }
  __device__ __forceinline__ void get(int k, int& t, int& k0, int& k1) const {
    const int p = first + k * sp.P, c = p % sp.cuts;
    t = p / sp.cuts;
    k0 = static_cast<int>(static_cast<int64_t>(sp.S) * c / sp.cuts);
    k1 = static_cast<int>(static_cast<int64_t>(sp.S) * (c + 1) / sp.cuts);
  }
  __device__ __forceinline__ int64_t steps() const {
    int64_t n = 0;
    for (int k = 0; k < count(); ++k) {
      int t, k0, k1;
      get(k, t, k0, k1);
      n += k1 - k0;
    }
    return n;
  }
};

template <int BN, bool PAIR>
struct Cfg {
  static constexpr int kRowsW = PAIR ? BN / 2 : BN;  // weight rows in this CTA's shared memory
  static constexpr int kStageBytes = kTileX + kRowsW * kBK;
  static constexpr int kStages = 5;
  static constexpr int kBufs = 512 / BN;  // accumulator buffers
  static constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kStoreBytes + kFactorBytes + 1024 + 256;
};

// ------------------------------------------------------------ pairs of CTAs
// The pair's forms of the tensor-core and TMA operations (no multicast loads).
template <bool PAIR>
__device__ __forceinline__ void acc_alloc(uint32_t* dst, uint32_t ncols) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, ncols);
    tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void acc_dealloc(uint32_t taddr, uint32_t ncols) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
  else
    tmem_dealloc(taddr, ncols);
}
template <bool PAIR>
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    umma_e4m3(d, a, b, idesc, accumulate);
}
// Arrives at `bar` (of both CTAs) when the MMAs issued so far have finished.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    umma_commit(bar);
}
// Loads a box into this CTA's shared memory, counted on the leader's barrier.
template <bool PAIR>
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(cluster_map(smem_addr(bar), 0))
        : "memory");
  else
    tma_load_2d(dst, map, x, y, bar);
}

// Arrives on the leader's barrier.  Only tensor-memory reads are ordered by it
// (tcgen05 fences on both sides), so the release stays at CTA scope: at cluster
// scope it waited for the warp's stores, 1000 cycles a k-step.
__device__ __forceinline__ void leader_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_map(smem_addr(bar), 0)) : "memory");
}

template <int BN, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                    const __grid_constant__ CUtensorMap ymap, const __grid_constant__ Args a) {
  using C = Cfg<BN, PAIR>;
  constexpr int kStages = C::kStages, kBufs = C::kBufs, kCols = BN / (kEpiWarps / 4);  // columns of an epilogue warp
  const uint32_t base = smem_addr(fsm);
  const uint32_t ring = ((base + 1023u) & ~1023u) - base;
  uint8_t* staging = fsm + ring + kStages * C::kStageBytes;
  float* factors = reinterpret_cast<float*>(staging + kEpiWarps * kStoreBytes);  // [slot][step][half][token]
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kStoreBytes + kFactorBytes);
  uint64_t* empty = full + kStages;
  uint64_t* d_full = empty + kStages;  // [buffers] a group's sums are in the buffer
  uint64_t* d_empty = d_full + kBufs;  // [buffers] they have been read
  uint64_t* done = d_empty + kBufs;        // every MMA of the CTA has finished
  uint64_t* f_full = done + 1;         // [slots] factors
  uint64_t* f_empty = f_full + kFactorSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(f_empty + kFactorSlots);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const Run run{PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x), a.sp};
  constexpr int kRows = PAIR ? 2 * kBM : kBM;  // tokens of a tile
  const int nrun = run.count();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    for (int i = 0; i < kFactorSlots; ++i) {
      mbar_init(&f_full[i], 1);
      mbar_init(&f_empty[i], kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kEpiWarps + 1) {
    acc_alloc<PAIR>(tmem_slot, kBufs * BN);
  }
  tc_fence_before();
  if (PAIR) cluster_sync_all();  // both CTAs' barriers are there
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(abort_flag) != 0; };
  auto fail = [&]() {
    report(a.dev_status, GQ_DEV_TIMEOUT);
    *reinterpret_cast<volatile int*>(abort_flag) = 1;
  };
  pdl_wait();
  pdl_launch_dependents();  // only now: a dependent may rely on what ran before this call

  if (warp == kEpiWarps) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      bool ok = true;
      int g = 0;
      const uint32_t bytes = static_cast<uint32_t>(a.xrows * kBK + C::kRowsW * kBK) * (PAIR ? 2 : 1);
      for (int k = 0; k < nrun && ok; ++k) {
        int t, k0, k1;
        run.get(k, t, k0, k1);
        const int row0 = (t / a.sp.tm) * kRows + rank * kBM, m0 = (t % a.sp.tm) * BN + rank * C::kRowsW;
        for (int ks = k0; ks < k1; ++ks, ++g) {
          const int s = g % kStages;
          if (!mbar_wait(&empty[s], ((g / kStages) & 1u) ^ 1u, a.budget) || aborted()) {
            ok = false;
            break;
          }
          if (g < a.skip) continue;
          uint8_t* st = fsm + ring + s * C::kStageBytes;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          load_box<PAIR>(st, &xmap, ks * kBK, row0, &full[s]);
          load_box<PAIR>(st + kTileX, &wmap, ks * kBK, m0, &full[s]);
        }
      }
      if (!ok) fail();
      // every issued copy lands before shared memory is released (a pair's count in the leader)
      for (int i = max(a.skip, g - kStages); i < g && rank == 0; ++i)
        if (!mbar_wait(&full[i % kStages], (i / kStages) & 1u, kWaitBudget)) report(a.dev_status, GQ_DEV_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    // --------------------------------------------------------------- MMA
    // The whole warp runs the loop and one elected lane issues: the
    // descriptors are then warp-uniform for the compiler, too.  (In a branch of
    // one lane each MMA took about 160 cycles to issue.)
    constexpr uint32_t idesc = idesc_e4m3(kRows, BN);
    bool ok = true;
    const int64_t steps = rank == 0 ? run.steps() : 0;
    int s = 0;
    uint32_t phase = 0;
    for (int64_t g = 0; g < steps; ++g) {
      const int buf = static_cast<int>(g % kBufs);
      const uint32_t dphase = (static_cast<uint32_t>(g / kBufs) & 1u) ^ 1u;
      ok = mbar_wait(&full[s], phase, a.budget) && mbar_wait(&d_empty[buf], dphase, a.budget);
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint64_t xd = umma_desc_sw128(base + ring + s * C::kStageBytes);
      const uint64_t wd = umma_desc_sw128(base + ring + s * C::kStageBytes + kTileX);
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < kBK / 32; ++i) mma_step<PAIR>(tmem + buf * BN, xd + 2 * i, wd + 2 * i, idesc, i != 0);
        mma_commit<PAIR>(&empty[s]);
        mma_commit<PAIR>(&d_full[buf]);
      }
      __syncwarp();
      if (++s == kStages) {
        s = 0;
        phase ^= 1u;
      }
    }
    if (rank == 0 && elect_one()) {
      if (!ok) fail();
      mma_commit<PAIR>(done);  // also on the abort path: tensor memory is quiet before exit
    }
    __syncwarp();
  } else if (warp == kEpiWarps + 2) {
    // ------------------------------------------------------------- scales
    // Four k-steps of a tile at a time; a lane has four tokens.
    bool ok = true;
    int q = 0;  // slots filled
    for (int k = 0; k < nrun && ok; ++k) {
      int t, k0, k1;
      run.get(k, t, k0, k1);
      const int row0 = (t / a.sp.tm) * kRows + rank * kBM;
      const int64_t m0 = static_cast<int64_t>(t % a.sp.tm) * BN, last = (a.M - 1) / 128;
      const float* swl = a.sw + min(m0 / 128, last) * a.kblocks;
      const float* swh = a.sw + min((m0 + BN / 2) / 128, last) * a.kblocks;
      for (int ks = k0; ks < k1; ks += kFactorSteps, ++q) {
        float x[4][kFactorSteps], lo[kFactorSteps], hi[kFactorSteps];
#pragma unroll
        for (int j = 0; j < kFactorSteps; ++j) {
          const int kj = min(ks + j, k1 - 1);
          lo[j] = swl[kj];
          hi[j] = swh[kj];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = min(row0 + lane + 32 * i, a.B - 1);
            x[i][j] = a.sx[static_cast<int64_t>(row) * a.kblocks + kj];
          }
        }
        const int slot = q % kFactorSlots;
        ok = mbar_wait(&f_empty[slot], ((q / kFactorSlots) & 1u) ^ 1u, a.budget) && !aborted();
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        float* f = factors + slot * (kFactorSteps * 2 * kBM) + lane;
#pragma unroll
        for (int j = 0; j < kFactorSteps; ++j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[(2 * j) * kBM + 32 * i] = x[i][j] * lo[j];
            f[(2 * j + 1) * kBM + 32 * i] = x[i][j] * hi[j];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&f_full[slot]);
      }
    }
    if (!ok && lane == 0) fail();
  } else {
    // ---------------------------------------------------------- epilogue
    const int quarter = warp & 3, half = (warp >> 2) * kCols / (BN / 2);  // rows; which factors
    const uint32_t lane_base = static_cast<uint32_t>(32 * quarter) << 16;
    const int cols0 = (warp >> 2) * kCols;
    const int prows = min(kBM, a.B);  // rows of a part
    auto release = [&](int buf) {  // the buffer may be filled again
      if (PAIR) leader_arrive(&d_empty[buf]);
      else mbar_arrive(&d_empty[buf]);
    };
    bool ok = true;
    uint32_t g = 0, fq = 0;  // k-steps and slots of factors done
    for (int k = 0; k < nrun && ok; ++k) {
      int t, k0, k1;
      run.get(k, t, k0, k1);
      const int row0 = (t / a.sp.tm) * kRows + rank * kBM;
      const int64_t m0 = static_cast<int64_t>(t % a.sp.tm) * BN;
      const int row = row0 + 32 * quarter + lane;
      const bool row_ok = row < a.B;
      const bool any = row0 + 32 * quarter < a.B;  // some lane of the warp has a token
      float2 acc2[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc2[i] = make_float2(0.f, 0.f);
      float* acc = reinterpret_cast<float*>(acc2);
      for (int ks = k0; ks < k1; ++ks, ++g) {
        const int buf = g % kBufs;
        const int fs = fq % kFactorSlots, fj = (ks - k0) % kFactorSteps;
        bool got = fj != 0 || mbar_wait(&f_full[fs], (fq / kFactorSlots) & 1u, a.budget);
        const float fac = factors[((fs * kFactorSteps + fj) * 2 + half) * kBM + 32 * quarter + lane];
        got = got && mbar_wait(&d_full[buf], (g / kBufs) & 1u, a.budget);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (any) {
          // 16 columns at a time; two warps on each scheduler take turns
          const float2 f = make_float2(fac, fac);
          const uint32_t src = tmem + lane_base + static_cast<uint32_t>(buf * BN + cols0);
#pragma unroll
          for (int c = 0; c < kCols / 16; ++c) {
            uint32_t v[16];
            tmem_ld16(src + 16 * c, v);
            tmem_wait_ld();
            if (c + 1 == kCols / 16) {  // the buffer is free
              tc_fence_before();
              __syncwarp();
              if (lane == 0) release(buf);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              acc2[8 * c + i] = __ffma2_rn(f, make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])),
                                           acc2[8 * c + i]);
          }
        } else if (lane == 0) {
          release(buf);
        }
        if (fj == kFactorSteps - 1 || ks + 1 == k1) {
          __syncwarp();  // every lane has its factor
          if (lane == 0) mbar_arrive(&f_empty[fs]);
          ++fq;
        }
      }
      if (!ok) break;
      if (a.sp.cuts > 1) {  // a piece: its sums go to the workspace
        const int prow = 32 * quarter + lane;
        if (row_ok) {
          float4* d = reinterpret_cast<float4*>(
              a.parts + (static_cast<int64_t>(run.first + k * a.sp.P) * prows + prow) * BN + cols0);
#pragma unroll
          for (int i = 0; i < kCols / 4; ++i)
            __stcg(d + i, make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]));
        }
      } else if (a.tma_y) {
        if (any) store_tile<kCols>(&ymap, staging + warp * kStoreBytes, acc, static_cast<int>(m0) + cols0,
                                   row0 + 32 * quarter, a.M, a.ytype);
      } else if (row_ok) {
        store_row<kCols>(a, row, m0 + cols0, acc);
      }
    }
    bulk_stores_wait<false>();
    if (!ok && lane == 0) fail();
  }

  // teardown: every MMA has finished before tensor memory is freed, and a
  // pair's CTAs leave together
  tc_fence_before();
  __syncthreads();
  if (warp == kEpiWarps + 1) {
    if (lane == 0 && !mbar_wait(done, 0, kWaitBudget)) report(a.dev_status, GQ_DEV_TIMEOUT);
    __syncwarp();
    tc_fence_after();
  }
  if (PAIR) cluster_sync_all();
  if (warp == kEpiWarps + 1) acc_dealloc<PAIR>(tmem, kBufs * BN);
}

// Y of a call whose tiles (of BN weight rows) were cut: the pieces' sums in
// order, four weight rows of a token to a thread.
template <int BN>
__global__ void __launch_bounds__(256) fp8_sum_kernel(const float* parts, void* Y, int64_t M, int B, int rows, int tm,
                                                      int cuts, int ytype) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t quads = static_cast<int64_t>(tm) * (BN / 4);
  const int64_t b = i / quads, q = i - b * quads;
  if (b >= B) return;
  const int64_t m = q * 4;
  const int tile = static_cast<int>(b / kBM) * tm + static_cast<int>(m / BN);
  const float4* p = reinterpret_cast<const float4*>(
      parts + (static_cast<int64_t>(tile) * cuts * rows + b % kBM) * BN + m % BN);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 0; c < cuts; ++c) {
    const float4 u = __ldcg(p + static_cast<int64_t>(c) * rows * (BN / 4));
    v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
  }
  const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (m + j < M) store_elem(Y, b * M + m + j, o[j], ytype);
}

// ------------------------------------------------------------------- host
// Tiles of 128 x 128 take one unit of time for a k-step (0.38 us) and about
// three more for a tile or piece; a second launch to add pieces up takes five,
// and writing and reading them an eighth for each of 128 rows.  A pair's 256 x
// 256 tile takes 1.55 units a k-step, on half as many SM pairs.  The plan with
// the shortest longest CTA is taken.
// Measured, 128 x 128 (uncut) against pairs: 500 tokens x 4096 x 4096, 16.2 and
// 21.0 us; 1000 tokens, 29.0 and 22.0; 200 tokens x 11008 x 4096, 28.8 and 22.0;
// 500 tokens, 45 and 42 (where the rule takes the former); 2048 tokens, 143 and
// 100.  Whole tiles against pieces: 128 tokens x 4096 x 11008, 37 and 18.2 (four);
// 300 tokens, 36.4 and 34.3 (three; the rule takes whole ones); 256 tokens x 2048 x
// 2048, 9.6 and 10.8 (two); 64 tokens x 4096 x 4096, 15.2 and 10.6 (four); 37
// tokens x 11000 x 4096, 16.3 and 17.0 (three).
struct Choice {
  int bn;
  bool pair;
  Split sp;
};
Choice choose(int64_t M, int64_t K, int64_t B) {
  const int64_t sms = sm_count();
  const int64_t S = (K + kBK - 1) / kBK;
  auto split = [&](int rows, int bn, int64_t ctas, int64_t cuts) {
    Split s;
    s.S = static_cast<int>(S);
    s.tm = static_cast<int>((M + bn - 1) / bn);
    s.T = static_cast<int>((B + rows - 1) / rows * s.tm);
    s.cuts = static_cast<int>(cuts);
    s.P = static_cast<int>(i64min(ctas, s.T * cuts));
    return s;
  };
  const int64_t tpair = (B + 255) / 256 * ((M + 255) / 256), t128 = (B + 127) / 128 * ((M + 127) / 128);
  const int64_t whole = (t128 + sms - 1) / sms * (S + 3);
  const int64_t pairs = (tpair + sms / 2 - 1) / (sms / 2) * (S + 3) * 14 / 9;
  int64_t best = 1, least = whole;
  for (int64_t c = 2; c <= 16 && c <= S && t128 < 2 * sms; ++c) {
    const int64_t steps =
        (t128 * c + sms - 1) / sms * ((S + c - 1) / c + 3) + 5 + t128 * c * i64min(B, 128) / 1024;
    if (steps < least) {
      least = steps;
      best = c;
    }
  }
  if (B > 128 && pairs < least) return Choice{256, true, split(256, 256, sms / 2, 1)};
  return Choice{128, false, split(128, 128, sms, best)};
}

size_t ws_bytes_of(const Choice& c, int64_t M, int64_t K, int64_t B) {
  if (fp8_gemv_takes(M, K, B) || c.sp.cuts == 1) return 0;
  const int64_t rows = B < kBM ? B : kBM;
  return static_cast<size_t>(c.sp.T) * c.sp.cuts * static_cast<size_t>(rows) * c.bn * sizeof(float);
}

bool gemm_dims(int64_t M, int64_t K, int64_t B) {
  if (K % 16 || K > (1LL << 24) || M > 0x7FFFFFFFLL - 256 || B > 0x7FFFFFFFLL - 256) return false;
  const int64_t t = ((B + kBM - 1) / kBM) * ((M + 127) / 128);
  return t <= 0x7FFFFFFFLL;
}

gq_status encode(CUtensorMap* map, CUtensorMapDataType type, int esize, const void* p, int64_t rows, int64_t cols,
                 int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
  EncodeTiled enc = tensor_map_encoder();
  if (!enc) return GQ_ERR_CUDA;
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(cols) * esize};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t es[2] = {1, 1};
  return enc(map, type, 2, const_cast<void*>(p), dim, stride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? GQ_OK
             : GQ_ERR_CUDA;
}

template <int BN, bool PAIR>
gq_status launch_fp8(const CUtensorMap& xmap, const CUtensorMap& wmap, const CUtensorMap& ymap, const Args& a,
                     cudaStream_t s) {
  auto kern = fp8_gemm_kernel<BN, PAIR>;
  constexpr int smem = Cfg<BN, PAIR>::kSmem;
  thread_local unsigned long long configured_ctx = 0;  // per host thread and context
  const unsigned long long ctx = context_id();
  if (ctx == 0 || ctx != configured_ctx) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return GQ_ERR_CUDA;
    configured_ctx = ctx;
  }
  if (PAIR)
    return launch_cluster(kern, dim3(static_cast<unsigned>(2 * a.sp.P)), dim3(kThreads), smem, s, true, 2u, xmap,
                          wmap, ymap, a);
  return launch(kern, dim3(static_cast<unsigned>(a.sp.P)), dim3(kThreads), smem, s, true, xmap, wmap, ymap,
                a);
}

// gq_gemm_fp8 with a wait budget; `skip` k-steps of each CTA are never loaded.
gq_status gemm_fp8(const void* W, const float* w_scales, int64_t M, int64_t K, const void* X, const float* x_scales,
                   int64_t B, void* Y, int y_dtype, void* workspace, size_t ws_bytes, unsigned flags, int* dev_status,
                   void* stream, long long budget, int skip) {
  if (M < 0 || K < 0 || B < 0) return GQ_ERR_INVALID_ARG;
  if (!valid_act_dtype(y_dtype)) return GQ_ERR_DTYPE;
  if (flags & ~GQ_GEMV_PDL) return GQ_ERR_INVALID_ARG;
  if (!gemm_dims(M, K, B)) return GQ_ERR_SHAPE;
  if (dev_status && (reinterpret_cast<uintptr_t>(dev_status) & 3u)) return GQ_ERR_ALIGNMENT;
  if (M == 0 || B == 0) return GQ_OK;
  if (!Y) return GQ_ERR_INVALID_ARG;
  if (misaligned16(Y)) return GQ_ERR_ALIGNMENT;
  cudaStream_t s = as_stream(stream);
  if (K == 0)
    return cudaMemsetAsync(Y, 0, static_cast<size_t>(B) * M * dtype_size(y_dtype), s) == cudaSuccess
               ? GQ_OK
               : GQ_ERR_CUDA;
  if (!W || !w_scales || !X || !x_scales) return GQ_ERR_INVALID_ARG;
  if (misaligned16(W) || misaligned16(X) || misaligned16(w_scales) || misaligned16(x_scales))
    return GQ_ERR_ALIGNMENT;
  const Choice c = choose(M, K, B);
  const size_t need = ws_bytes_of(c, M, K, B);
  if (need && (!workspace || ws_bytes < need)) return GQ_ERR_WORKSPACE;
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u)) return GQ_ERR_ALIGNMENT;
  if (fp8_gemv_takes(M, K, B)) return fp8_gemv(W, w_scales, M, K, X, x_scales, B, Y, y_dtype, s);

  Args a{};
  a.sx = x_scales;
  a.sw = w_scales;
  a.Y = Y;
  a.dev_status = dev_status;
  a.budget = budget;
  a.skip = skip;
  a.M = M;
  a.B = static_cast<int>(B);
  a.kblocks = static_cast<int>((K + kBK - 1) / kBK);
  a.ytype = y_dtype;
  a.xrows = static_cast<int>(B < kBM ? (B + 7) / 8 * 8 : kBM);
  const int esize = dtype_size(y_dtype);
  a.tma_y = M * esize % 16 == 0;
  a.sp = c.sp;
  a.parts = static_cast<float*>(workspace);
  CUtensorMap xmap, wmap, ymap = {};
  gq_status st = encode(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, X, B, K, kBK, a.xrows, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st == GQ_OK) st = encode(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, W, M, K, kBK, c.pair ? c.bn / 2 : c.bn,
                                 CU_TENSOR_MAP_SWIZZLE_128B);
  if (st == GQ_OK && a.tma_y)
    st = encode(&ymap,
                y_dtype == GQ_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                : y_dtype == GQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                esize, Y, B, M, 64 / esize, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (st != GQ_OK) return st;
  if (c.pair) return launch_fp8<256, true>(xmap, wmap, ymap, a, s);
  st = launch_fp8<128, false>(xmap, wmap, ymap, a, s);
  if (st != GQ_OK || c.sp.cuts == 1) return st;
  const int64_t threads = B * c.sp.tm * (128 / 4);
  return launch(fp8_sum_kernel<128>, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, s, true,
                a.parts, Y, M, a.B, static_cast<int>(B < kBM ? B : kBM), c.sp.tm, c.sp.cuts, y_dtype);
}

}  // namespace
}  // namespace gq

extern "C" {

GQ_API size_t gq_gemm_fp8_workspace_bytes(int64_t M, int64_t K, int64_t B) {
  if (M <= 0 || K <= 0 || B <= 0 || !gq::gemm_dims(M, K, B)) return 0;
  return gq::ws_bytes_of(gq::choose(M, K, B), M, K, B);
}

GQ_API gq_status gq_gemm_fp8(const void* W, const float* w_scales, int64_t M, int64_t K, const void* X,
                             const float* x_scales, int64_t B, void* Y, int y_dtype, void* workspace,
                             size_t ws_bytes, unsigned flags, int* dev_status, void* stream) {
  return gq::gemm_fp8(W, w_scales, M, K, X, x_scales, B, Y, y_dtype, workspace, ws_bytes, flags, dev_status, stream,
                      gq::kWaitBudget, 0);
}

GQ_API gq_status gq_selftest_gemm_fp8_timeout(const void* W, const float* w_scales, int64_t M, int64_t K,
                                              const void* X, const float* x_scales, int64_t B, void* Y,
                                              void* workspace, size_t ws_bytes, int* dev_status, void* stream) {
  if (!dev_status) return GQ_ERR_INVALID_ARG;
  if (M > 0 && K > 0 && B > 0 && gq::fp8_gemv_takes(M, K, B)) return GQ_ERR_SHAPE;  // (a kernel without waits)
  return gq::gemm_fp8(W, w_scales, M, K, X, x_scales, B, Y, GQ_F32, workspace, ws_bytes, 0u, dev_status, stream,
                      2000000LL, 1);
}

}  // extern "C"
