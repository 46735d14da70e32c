// blockwise_gemm.cu - FP8 GEMMs whose operands carry one FP32 scale for each block of 128
// along the reduction.
//
// The recipe that "End-to-End MXFP8 RL on Blackwell" (verl blog post) contrasts with MXFP8
// (section "A different grid, and drift"): E4M3 weights with 128 x 128 blocks, activations
// and gradients with 1 x 128 blocks, FP32 or power-of-two scales.
//   C[r][c] = sum_b sr(b, r) sc(b, c) P_b[r][c],  P_b = sum over the 128 k of block b of
//   a[r][k] w[c][k]
// The tensor cores apply no FP32 scale, so each 128-deep product P_b is a separate FP32
// accumulation in TMEM (tcgen05.mma kind::f8f6f4, four K = 32 steps) and the epilogue warps
// fold it into FP32 registers: acc += (sr sc) P_b. Two TMEM accumulators alternate, so the
// tensor cores work on block b + 1 while the warps fold block b.
//
// What bounds it: the tensor cores take 512 cycles for a 128 x 256 x 128 block per SM, the
// fold 256 (one FMA per element, 128 lanes; 512 with a scale for every column), TMEM reads
// 256. All overlap.
//
// Roles of a CTA's 320 threads: warp 0 TMA producer, warp 1 MMA issuer (and TMEM
// allocation), warps 2-9 fold and store, two per TMEM lane quarter, each half the columns.
//
// Modes, by which operand lies along the 128 TMEM lanes ("rows") and the columns:
//   kFprop    rows = A (a scale per row and block), columns = B (128 x 128 blocks)
//   kWgrad    both with a scale per row / column and block
//   kSwapped  rows = B, columns = A, C stored transposed: for few rows of A, where a
//             128-row tile of A would be mostly empty
// and by size: pairs of CTAs (cta_group::2, 256 x 256 tiles, each SM stages half of the
// column operand), or single CTAs (128 x BN tiles) whose reduction may be split over a
// cluster, the parts joined through distributed shared memory in rank order.
//
// Every wait is bounded as in gemm.cu: past the limit the CTA latches MXFP8_ERR_TIMEOUT,
// every role leaves its loop, outstanding copies and MMAs are waited for, TMEM is freed.

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "device.cuh"
#include "internal.h"
#include "mxfp8.h"

namespace mxfp8 {
namespace {

constexpr int BM = 128;        // tile rows per CTA = TMEM lanes
constexpr int BK = 128;        // K per block and pipeline stage
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;

enum Mode : int { kFprop = 0, kWgrad = 1, kSwapped = 2 };

template <int BN, bool kPair>
struct Cfg {
  static constexpr int kBRows = kPair ? BN / 2 : BN;   // column-operand rows staged per CTA
  static constexpr int kABytes = BM * BK;
  static constexpr int kBBytes = kBRows * BK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // narrow tiles leave room for two or three CTAs on an SM
  static constexpr int kStages = BN >= 128 ? 6 : 4;
  static constexpr int kNC = BN / 2;                   // columns per epilogue warp
  static constexpr int kOffA = 0;
  static constexpr int kOffB = kOffA + kStages * kABytes;
  static constexpr int kOffScale = kOffB + kStages * kBBytes;  // column scales, per warp
  static constexpr int kOffBar = kOffScale + kEpiWarps * kNC * 4;
  static constexpr int kNumBars = 2 * kStages + 5;     // full, empty, acc_full, acc_empty, done
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;  // + slack for 1024-byte alignment
  static constexpr int kTmemCols = 2 * BN;             // two accumulators
  static constexpr int kMinCtas = BN <= 64 ? 2 : 1;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512, "TMEM columns");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory overflow");
  static_assert(BN * BM * 4 <= kStages * kStageBytes, "split-K partial overflow");
};

struct Params {
  const float* sr;      // scales of the row operand: [nkb][ldr], or [row blocks][nkb] (kSwapped)
  const float* sc;      // scales of the column operand: [nkb][ldc], or [column blocks][nkb] (kFprop)
  int64_t ldr, ldc;
  void* C;
  int64_t ldo;          // output row pitch in elements
  int64_t nr, nc;       // valid rows and columns
  int nkb;              // blocks of 128 along K
  int out_fp32;
  int vec32;            // output rows take 32-byte stores
  int split;            // CTAs that share a tile's reduction (a cluster)
  uint32_t tiles, row_tiles, col_tiles;  // pairs: row tiles are of 256 rows
  uint32_t band;        // row tiles per raster band
  int* status;
  uint64_t wait_ns, drain_ns;
};

// Tile `id` of a banded raster: bands of `band` row tiles sweep across the columns, rows
// fastest, so that concurrent CTAs share operand tiles in L2.
__device__ __forceinline__ void tile_at(const Params& p, uint32_t id, int64_t& rt, int64_t& ct) {
  const uint32_t per = p.band * p.col_tiles;
  const uint32_t b = id / per, r = id - b * per;
  const uint32_t first = b * p.band;
  const uint32_t h = p.row_tiles - first < p.band ? p.row_tiles - first : p.band;
  const uint32_t c = r / h;
  ct = c;
  rt = first + (r - c * h);
}

// TMEM loads of G columns of the warp's lanes, and the wait for them. The wait carries the
// registers, so that no use of them moves ahead of it.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7])
               :: "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :: "memory");
}

__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
  return pack2(__uint_as_float(lo), __uint_as_float(hi));
}

// Scales of extreme magnitude. |P_b| <= 448^2 * 128 < 2^25, so P_b times a factor within
// 2^-100 .. 2^100 stays inside FP32's normal range; beyond it the factor sr is split into
// two of half its exponent, and the column's scale is applied between them.
__device__ __forceinline__ bool extreme(float s) { return s < 0x1p-100f || s > 0x1p100f; }

__device__ __forceinline__ void halves_of(float s, float& s1, float& s2) {
  const int e = static_cast<int>((__float_as_uint(s) >> 23) & 0xFFu) - 127;
  s1 = __uint_as_float(static_cast<uint32_t>(e / 2 + 127) << 23);
  s2 = s * __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23);
}

// acc[i] += s1 sc_i s2 P_i for the warp's kNC columns of one block: P from TMEM, read one
// group ahead of its use.
//   kColVec  the column scales sc_i come from shared memory; else all are `sc`
//   kSplit   the row scale is s1 s2, applied on both sides of the column's; else it is s1
//            (kColVec), or s1 is the product of both scales and nothing else applies
template <int kNC, bool kColVec, bool kSplit>
__device__ __forceinline__ void fold(uint64_t (&acc)[kNC / 2], uint32_t taddr, float s1, float s2,
                                     float sc, const float* col_scale) {
  constexpr int G = kNC < 16 ? kNC : 16;
  constexpr int kGroups = kNC / G;
  uint32_t r[2][G];
  tmem_ld(taddr, r[0]);
  const uint64_t f1 = pack2(s1, s1), f2 = pack2(s2, s2), fc = pack2(sc, sc);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    tmem_wait(r[g & 1]);
    if (g + 1 < kGroups) tmem_ld(taddr + G * (g + 1), r[(g + 1) & 1]);
#pragma unroll
    for (int i = 0; i < G / 2; ++i) {
      const uint64_t v = pair_of(r[g & 1][2 * i], r[g & 1][2 * i + 1]);
      uint64_t& a = acc[g * (G / 2) + i];
      uint64_t c2 = fc;
      if constexpr (kColVec) {
        const float2 cs = *reinterpret_cast<const float2*>(col_scale + g * G + 2 * i);
        c2 = pack2(cs.x, cs.y);
      }
      if constexpr (kSplit) a = fma2(mul2(mul2(v, f1), c2), f2, a);
      else if constexpr (kColVec) a = fma2(mul2(v, f1), c2, a);
      else a = fma2(v, f1, a);
    }
  }
}

__device__ __forceinline__ void store_one(const Params& p, int64_t at, float v) {
  if (p.out_fp32)
    static_cast<float*>(p.C)[at] = v;
  else
    static_cast<uint16_t*>(p.C)[at] = static_cast<uint16_t>(cvt_bf16x2(0.f, v));
}

// One thread's row of kNC columns, from column c0, in 32- or 16-byte stores (the number of
// columns is a multiple of 8).
template <int kNC>
__device__ __forceinline__ void store_row(const Params& p, const uint64_t (&acc)[kNC / 2],
                                          int64_t row, int64_t c0) {
#pragma unroll
  for (int g = 0; g < kNC / 8; ++g) {
    const int64_t c = c0 + 8 * g;
    if (c >= p.nc) return;
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(acc[4 * g + i], f[2 * i], f[2 * i + 1]);
    if (p.out_fp32) {
      float* o = static_cast<float*>(p.C) + row * p.ldo + c;
      if (p.vec32) {
        st_global_cg_v8(o, __float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                        __float_as_uint(f[3]), __float_as_uint(f[4]), __float_as_uint(f[5]),
                        __float_as_uint(f[6]), __float_as_uint(f[7]));
      } else {
        reinterpret_cast<float4*>(o)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
    } else {
      uint16_t* o = static_cast<uint16_t*>(p.C) + row * p.ldo + c;
      const uint4 w = make_uint4(cvt_bf16x2(f[1], f[0]), cvt_bf16x2(f[3], f[2]),
                                 cvt_bf16x2(f[5], f[4]), cvt_bf16x2(f[7], f[6]));
      *reinterpret_cast<uint4*>(o) = w;
    }
  }
}

template <int BN, int kMode, bool kPair>
__global__ void __launch_bounds__(kThreads, Cfg<BN, kPair>::kMinCtas)
blockwise_gemm_kernel(const __grid_constant__ CUtensorMap map_r,
                      const __grid_constant__ CUtensorMap map_c, const Params p) {
  using C = Cfg<BN, kPair>;
  constexpr int kStages = C::kStages, kNC = C::kNC;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // pair: the leader's
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2]; pair: the leader's
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  // drain records: [0] / [1] stage uses issued by the producer of CTA 0 / 1 of the pair (a
  // single CTA writes both), [2] stage uses consumed by the MMA issuer (one accumulator
  // commit each), [3] this CTA's producer tail completed
  volatile uint32_t* rec = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = kPair ? cluster_ctarank() : 0;
  const bool leader = crank == 0;
  const uint32_t group = kPair ? 2u : static_cast<uint32_t>(p.split);  // CTAs on one tile
  const uint32_t first_id = blockIdx.x / group, id_step = gridDim.x / group;
  // this CTA's part of the reduction
  const uint32_t part = kPair ? 0u : blockIdx.x - first_id * group;
  const int kb0 = kPair ? 0 : static_cast<int>(static_cast<int64_t>(p.nkb) * part / p.split);
  const int kb1 = kPair ? p.nkb
                        : static_cast<int>(static_cast<int64_t>(p.nkb) * (part + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kPair ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) rec[i] = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map_r);
    tma_prefetch_desc(&map_c);
  }
  if (warp == 1) {
    if constexpr (kPair) tmem_alloc_2sm(tmem_slot, C::kTmemCols);
    else tmem_alloc(tmem_slot, C::kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // both CTAs' barriers exist before any cross-CTA arrive
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer
    const bool issuer = elect_one();
    const uint32_t full0 = kPair ? cluster_map(&full[0], 0) : smem_u32(&full[0]);
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t id = first_id; ok && id < p.tiles; id += id_step) {
      int64_t rt, ct;
      tile_at(p, id, rt, ct);
      const int32_t r0 = static_cast<int32_t>(kPair ? (2 * rt + crank) * BM : rt * BM);
      const int32_t c0 = static_cast<int32_t>(ct * BN + crank * C::kBRows);
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1;
        if (!warp_wait(&empty[s], ph ^ 1, abort_flag, p.wait_ns)) { ok = false; break; }
        if (issuer) {
          uint8_t* as = smem + C::kOffA + s * C::kABytes;
          uint8_t* bs = smem + C::kOffB + s * C::kBBytes;
          if constexpr (kPair) {
            if (leader) mbar_arrive_expect_tx(&full[s], 2 * C::kStageBytes);
            tma_load_2d_2sm(as, &map_r, kb * BK, r0, full0 + 8 * s);
            tma_load_2d_2sm(bs, &map_c, kb * BK, c0, full0 + 8 * s);
          } else {
            mbar_arrive_expect_tx(&full[s], C::kStageBytes);
            tma_load_2d(as, &map_r, kb * BK, r0, &full[s]);
            tma_load_2d(bs, &map_c, kb * BK, c0, &full[s]);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && issuer) {
      *abort_flag = 1;
      latch_error(p.status, MXFP8_ERR_TIMEOUT);
    }
    if (issuer) {
      if constexpr (kPair) {
        for (uint32_t r = 0; r < 2; ++r)
          st_cluster_u32(cluster_map(const_cast<uint32_t*>(&rec[crank]), r), it);
      } else {
        rec[0] = rec[1] = it;
      }
    }
    // the MMA issuer's release of the last stage uses must have arrived before the CTA exits
    bool tail_ok = ok;
    for (uint32_t i = it > kStages ? it - kStages : 0; tail_ok && i < it; ++i)
      tail_ok = warp_wait(&empty[i % kStages], (i / kStages) & 1, abort_flag, p.wait_ns);
    if (issuer) rec[3] = tail_ok ? 1u : 0u;
    __syncwarp();
  } else if (warp == 1 && leader) {
    // ------------------------------------------------------------- MMA issuer
    const bool issuer = elect_one();
    uint32_t it = 0;
    bool ok = true;
    const uint64_t a_desc0 = smem_desc(smem_u32(smem + C::kOffA), 16, 1024, 2);
    const uint64_t b_desc0 = smem_desc(smem_u32(smem + C::kOffB), 16, 1024, 2);
    constexpr uint32_t kId = f8_idesc(kPair ? 2 * BM : BM, BN);
    for (uint32_t id = first_id; ok && id < p.tiles; id += id_step) {
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1;
        const uint32_t b = it & 1, aph = (it >> 1) & 1;
        if (!warp_wait(&acc_empty[b], aph ^ 1, abort_flag, p.wait_ns) ||
            !warp_wait(&full[s], ph, abort_flag, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t ad = a_desc0 + s * (C::kABytes / 16);
        const uint64_t bd = b_desc0 + s * (C::kBBytes / 16);
        const uint32_t d = tmem + b * BN;
        if (issuer) {  // a K step of 32 starts 32 bytes further; past K the tiles are zero
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kPair) mma_f8_2sm(d, ad + 2 * k, bd + 2 * k, kId, k > 0);
            else mma_f8(d, ad + 2 * k, bd + 2 * k, kId, k > 0);
          }
          if constexpr (kPair) {
            mma_commit_2sm_mc(&empty[s], 3);
            mma_commit_2sm_mc(&acc_full[b], 3);
          } else {
            mma_commit(&empty[s]);
            mma_commit(&acc_full[b]);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && issuer) {
      *abort_flag = 1;
      latch_error(p.status, MXFP8_ERR_TIMEOUT);
    }
    if (issuer) {
      if constexpr (kPair) {
        for (uint32_t r = 0; r < 2; ++r)
          st_cluster_u32(cluster_map(const_cast<uint32_t*>(&rec[2]), r), it);
        mma_commit_2sm_mc(mma_done, 1);
      } else {
        rec[2] = it;
        mma_commit(mma_done);
      }
      mbar_wait_timed(mma_done, 0, p.drain_ns);
    }
    __syncwarp();
  } else if (warp >= 2) {
    // ------------------------------------------------------------- fold and store
    const int q = warp & 3;            // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;  // which half of the columns
    float* cs = reinterpret_cast<float*>(smem + C::kOffScale) + (warp - 2) * kNC;
    const uint32_t acc_empty0 = kPair ? cluster_map(&acc_empty[0], 0) : smem_u32(&acc_empty[0]);
    constexpr bool kColVec = kMode != kFprop;
    constexpr int kPre = (kNC + 31) / 32;  // column scales prefetched per lane
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t id = first_id; ok && id < p.tiles; id += id_step) {
      int64_t rt, ct;
      tile_at(p, id, rt, ct);
      const int64_t row0 = (kPair ? 2 * rt + crank : rt) * BM;
      const int64_t row = row0 + 32 * q + lane;
      const int64_t col = ct * BN + half * kNC;  // this warp's first column
      uint64_t acc[kNC / 2];
#pragma unroll
      for (int i = 0; i < kNC / 2; ++i) acc[i] = 0;
      // scales one block ahead: of this thread's row (or the row tile's block), and of the
      // warp's columns (or their block)
      const bool row_ok = row < p.nr;
      const float* srp = kMode == kSwapped ? p.sr + rt * p.nkb : p.sr + (row_ok ? row : 0);
      const int64_t srs = kMode == kSwapped ? 1 : p.ldr;
      const float* scp = kColVec ? p.sc
                                 : p.sc + ((col < p.nc ? col : p.nc - 1) / 128) * p.nkb;
      float sr = 0.f, sc[kPre] = {};
      auto prefetch = [&](int kb) {
        sr = row_ok || kMode == kSwapped ? __ldg(srp + kb * srs) : 1.f;
        if constexpr (kColVec) {
#pragma unroll
          for (int i = 0; i < kPre; ++i) {
            const int64_t c = col + 32 * i + lane;
            sc[i] = c < p.nc && 32 * i + lane < kNC ? __ldg(scp + kb * p.ldc + c) : 0.f;
          }
        } else {
          sc[0] = __ldg(scp + kb);
        }
      };
      if (kb0 < kb1) prefetch(kb0);
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t b = it & 1, ph = (it >> 1) & 1;
        const float s = sr, s2 = sc[0];
        if constexpr (kColVec) {
#pragma unroll
          for (int i = 0; i < kPre; ++i)
            if (32 * i + lane < kNC) cs[32 * i + lane] = sc[i];
          __syncwarp();
        }
        if (kb + 1 < kb1) prefetch(kb + 1);
        int got = 0;  // one lane waits, the warp follows its verdict
        if (lane == 0) got = mbar_wait_bounded(&acc_full[b], ph, abort_flag, p.wait_ns);
        got = __shfl_sync(0xFFFFFFFFu, got, 0);
        if (!got) { ok = false; break; }
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + b * BN + half * kNC;
        const float both = kColVec ? s : s * s2;
        if (__any_sync(0xFFFFFFFFu, extreme(both))) {
          float h1, h2;
          halves_of(s, h1, h2);
          fold<kNC, kColVec, true>(acc, taddr, h1, h2, s2, cs);
        } else {
          fold<kNC, kColVec, false>(acc, taddr, both, 0.f, 0.f, cs);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair) mbar_arrive_cluster_relaxed(acc_empty0 + 8 * b);
          else mbar_arrive_relaxed(&acc_empty[b]);
        }
      }
      if (!ok) break;
      if (!kPair && p.split > 1) {
        // partial sums into the (now idle) stages, [column][row]
        float* part_sum = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int i = 0; i < kNC / 2; ++i) {
          float a, b2;
          unpack2(acc[i], a, b2);
          part_sum[(half * kNC + 2 * i) * BM + 32 * q + lane] = a;
          part_sum[(half * kNC + 2 * i + 1) * BM + 32 * q + lane] = b2;
        }
      } else if constexpr (kMode == kSwapped) {
        if (row_ok) {
#pragma unroll
          for (int i = 0; i < kNC / 2; ++i) {
            float a, b2;
            unpack2(acc[i], a, b2);
            if (col + 2 * i < p.nc) store_one(p, (col + 2 * i) * p.ldo + row, a);
            if (col + 2 * i + 1 < p.nc) store_one(p, (col + 2 * i + 1) * p.ldo + row, b2);
          }
        }
      } else {
        if (row_ok) store_row<kNC>(p, acc, row, col);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      latch_error(p.status, MXFP8_ERR_TIMEOUT);
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // both CTAs have stopped issuing; records in place
  // Drain, after an abort: nothing that this CTA (or its pair) started may still be landing
  // when it exits. In a pair the leader completes the stage uses that only one CTA issued:
  // the missing half of the bytes by hand, or the missing arm by an arrive that expects the
  // peer's half alone. Without an abort every use was consumed and released already.
  const uint32_t i0 = rec[0], i1 = rec[1], consumed = rec[2];
  const uint32_t issued = i0 > i1 ? i0 : i1;
  if (threadIdx.x == 0 && !(rec[3] && !*abort_flag && issued == consumed)) {
    if (leader) {
      for (uint32_t i = consumed; kPair && i < issued; ++i) {
        uint64_t* bar = &full[i % kStages];
        if (i < i0 && i >= i1) mbar_complete_tx(bar, C::kStageBytes);
        else if (i >= i0 && i < i1) mbar_arrive_expect_tx(bar, C::kStageBytes);
      }
      for (uint32_t i = consumed; i < issued; ++i)
        mbar_wait_timed(&full[i % kStages], (i / kStages) & 1, p.drain_ns);
    }
    for (uint32_t i = consumed > kStages ? consumed - kStages : 0; i < consumed; ++i)
      mbar_wait_timed(&empty[i % kStages], (i / kStages) & 1, p.drain_ns);
    for (uint32_t i = consumed > 2 ? consumed - 2 : 0; i < consumed; ++i)
      mbar_wait_timed(&acc_full[i & 1], (i >> 1) & 1, p.drain_ns);
  }
  __syncthreads();
  if constexpr (kPair) {
    if (issued > consumed) cluster_sync();  // the leader's drain covered the peer's copies too
  } else if (p.split > 1) {
    // Join the parts: CTA `part` adds its share of the tile's columns over all parts, in
    // rank order, and stores them. One tile per cluster.
    cluster_sync();
    int64_t rt, ct;
    tile_at(p, first_id, rt, ct);
    const int c_lo = BN * static_cast<int>(part) / p.split;
    const int c_hi = BN * static_cast<int>(part + 1) / p.split;
    const uint32_t base = smem_u32(smem);
    for (int i = c_lo * BM + static_cast<int>(threadIdx.x); i < c_hi * BM; i += kThreads) {
      const int64_t row = rt * BM + i % BM, col = ct * BN + i / BM;
      if (row >= p.nr || col >= p.nc) continue;
      float sum = 0.f;
      for (int r = 0; r < p.split; ++r) {
        uint32_t from;
        float v;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(base + 4 * i), "r"(r));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from) : "memory");
        sum += v;
      }
      store_one(p, kMode == kSwapped ? col * p.ldo + row : row * p.ldo + col, sum);
    }
    cluster_sync();  // no CTA leaves while its shared memory is being read
  }
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (kPair) tmem_dealloc_2sm(tmem, C::kTmemCols);
    else tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------------- host side

template <int BN, int kMode, bool kPair>
int launch(const CUtensorMap& mr, const CUtensorMap& mc, const Params& p, int64_t grid,
           int cluster, cudaStream_t stream) {
  auto k = blockwise_gemm_kernel<BN, kMode, kPair>;
  constexpr int kSmem = Cfg<BN, kPair>::kSmemBytes;
  static std::atomic<bool> attr_set[64] = {};  // per device; setting it twice is harmless
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MXFP8_ERR_CUDA;
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
        cudaSuccess)
      return MXFP8_ERR_CUDA;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = pdl_attr(&attr[0]);
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, k, mr, mc, p) == cudaSuccess ? MXFP8_OK : MXFP8_ERR_CUDA;
}

// 256 x 256 tiles on CTA pairs. `a` is the row operand.
template <int kMode>
int launch_pairs(const BlockwiseGemmArgs& a, Params p, cudaStream_t stream) {
  using C = Cfg<256, true>;
  CUtensorMap mr, mc;
  if (!make_operand_map(&mr, a.A, a.K, a.M, BM) || !make_operand_map(&mc, a.B, a.K, a.N, C::kBRows))
    return MXFP8_ERR_CUDA;
  p.row_tiles = static_cast<uint32_t>((a.M + 255) / 256);
  p.col_tiles = static_cast<uint32_t>((a.N + 255) / 256);
  const int64_t tiles = static_cast<int64_t>(p.row_tiles) * p.col_tiles;
  if (tiles > 0x7FFFFFFF / 2) return MXFP8_ERR_INVALID_ARG;
  p.tiles = static_cast<uint32_t>(tiles);
  p.band = p.row_tiles < 8 ? p.row_tiles : 8;
  p.split = 1;
  const int64_t pairs = num_sms() / 2;
  return launch<256, kMode, true>(mr, mc, p, 2 * (tiles < pairs ? tiles : pairs), 2, stream);
}

// 128 x BN tiles on single CTAs, the reduction split over clusters of `split`.
template <int BN, int kMode>
int launch_single(const void* R, int64_t nr, const void* Cop, int64_t nc, int64_t K, Params p,
                  int split, cudaStream_t stream) {
  CUtensorMap mr, mc;
  if (!make_operand_map(&mr, R, K, nr, BM) || !make_operand_map(&mc, Cop, K, nc, BN))
    return MXFP8_ERR_CUDA;
  p.row_tiles = static_cast<uint32_t>((nr + BM - 1) / BM);
  p.col_tiles = static_cast<uint32_t>((nc + BN - 1) / BN);
  const int64_t tiles = static_cast<int64_t>(p.row_tiles) * p.col_tiles;
  if (tiles > 0x7FFFFFFF / 8) return MXFP8_ERR_INVALID_ARG;
  p.tiles = static_cast<uint32_t>(tiles);
  p.band = kMode == kSwapped ? 1 : (p.row_tiles < 8 ? p.row_tiles : 8);
  p.split = split;
  int64_t grid = tiles * split;
  const int64_t fit = static_cast<int64_t>(num_sms()) * Cfg<BN, false>::kMinCtas;
  if (split == 1 && grid > fit) grid = fit;  // persistent
  return launch<BN, kMode, false>(mr, mc, p, grid, split, stream);
}

// Parts of the reduction: enough to give every SM a CTA, at least 4 blocks each.
int split_for(int64_t tiles, int64_t nkb) {
  int s = 1;
  while (s < 8 && tiles * s * 2 <= num_sms() && nkb >= 8 * s) s *= 2;
  return s;
}

}  // namespace

int launch_blockwise_gemm(const BlockwiseGemmArgs& a, cudaStream_t stream) {
  Params p{};
  p.C = a.C;
  p.ldo = a.N;
  p.nkb = static_cast<int>((a.K + BK - 1) / BK);
  p.out_fp32 = a.out_fp32 ? 1 : 0;
  p.vec32 = (reinterpret_cast<uintptr_t>(a.C) & 31u) == 0 && (a.N * 4) % 32 == 0;
  p.status = a.status;
  p.wait_ns = pipeline_wait_ns();
  p.drain_ns = pipeline_drain_ns();
  if (!a.wgrad && a.M <= 128) {
    p.sr = a.sB;
    p.sc = a.sA;
    p.ldc = a.M;
    p.nr = a.N;
    p.nc = a.M;
    const int64_t rt = (a.N + BM - 1) / BM;
    const int split = split_for(rt, p.nkb);
    if (a.M <= 16) return launch_single<16, kSwapped>(a.B, a.N, a.A, a.M, a.K, p, split, stream);
    if (a.M <= 32) return launch_single<32, kSwapped>(a.B, a.N, a.A, a.M, a.K, p, split, stream);
    if (a.M <= 64) return launch_single<64, kSwapped>(a.B, a.N, a.A, a.M, a.K, p, split, stream);
    return launch_single<128, kSwapped>(a.B, a.N, a.A, a.M, a.K, p, split, stream);
  }
  p.sr = a.sA;
  p.sc = a.sB;
  p.ldr = a.M;
  p.ldc = a.N;
  p.nr = a.M;
  p.nc = a.N;
  const int64_t pair_tiles = ((a.M + 255) / 256) * ((a.N + 255) / 256);
  if (pair_tiles >= num_sms() / 4)
    return a.wgrad ? launch_pairs<kWgrad>(a, p, stream) : launch_pairs<kFprop>(a, p, stream);
  const int split = split_for(((a.M + 127) / 128) * ((a.N + 127) / 128), p.nkb);
  return a.wgrad ? launch_single<128, kWgrad>(a.A, a.M, a.B, a.N, a.K, p, split, stream)
                 : launch_single<128, kFprop>(a.A, a.M, a.B, a.N, a.K, p, split, stream);
}

}  // namespace mxfp8
