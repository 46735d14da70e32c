// blockwise_gemm.cu - FP8 GEMMs whose operands carry one FP32 scale for each block of 128
// along the reduction.
//
// The recipe that "End-to-End MXFP8 RL on Blackwell" (verl blog post) contrasts with MXFP8
// (section "A different grid, and drift"): E4M3 weights with 128 x 128 blocks, activations
// and gradients with 1 x 128 blocks, FP32 or power-of-two scales.
//   C[r][c] = sum_b sr(b, r) sc(b, c) P_b[r][c],  P_b = sum over the 128 k of block b of
//   a[r][k] w[c][k]
// The tensor cores apply no FP32 scale, so each 128-deep product P_b is a separate FP32
// accumulation in TMEM (tcgen05.mma kind::f8f6f4, four K = 32 steps) and the fold warps add it
// into FP32 registers: acc += (sr sc) P_b, the product of the two scales rounded to FP32 once.
// Two TMEM accumulators alternate, so the tensor cores work on the next block while the warps
// fold this one. (Scales that are powers of two take another way, see the conversion
// kernel below.)
//
// What bounds it: not the tensor cores (512 cycles for a 256 x 256 x 128 block of a CTA pair) nor
// the FMAs (256), but the chain of one block: barrier wait, TMEM read, fold, barrier arrival,
// the next block's MMA. Each hand-over through shared memory answers in 150 to 180 cycles
// beside the TMA and MMA traffic, and a pair's block takes about 800 cycles in all. What can
// leave the chain does: the producer copies the scales (with each fold warp fetching its own:
// 4096 x 24576 x 4096 317 us, 299 now; weight gradient 6144 x 4096 x 4096 132 and 112), and
// one barrier a block says that both its product and its scales are there.
// Measured on GB300, BF16 results, kernels back to back: 4096 x 24576 x 4096 300 us (2.75
// PFLOP/s; up to 325 once the GPU is at its power limit), 4096^3 58 us (2.37); weight gradient
// 6144 x 4096 x 4096 115 us (1.79), 119 with FP32 results, 121 at K = 4016. One row is bound by the
// weights' bytes: 1 x 24576 x 4096 13 us (7.8 TB/s, part of it from L2); 1 x 4096 x 4096 takes 6.1
// us, mostly launch and latency. 37 x 24576 x 4096 takes 21 us, bound by 192 tiles on 152 SMs, 40
// of which run two (152 tiles take 14.3).
//
// Roles: warp 0 TMA producer and scales, warp 1 MMA issuer (and TMEM allocation), the last 8 or
// 12 warps fold and store: one per TMEM lane quarter and group of columns.
//
// Modes, by which operand lies along the 128 TMEM lanes ("rows") and the columns:
//   kFprop    rows = A (a scale per row and block), columns = B (128 x 128 blocks)
//   kWgrad    both with a scale per row / column and block
//   kSwapped  rows = B, columns = A, C stored transposed: for up to 64 rows of A, where a
//             128-row tile of A would be mostly empty: 64 x 4096 x 4096 7.8 us, 8.8 in 128-row
//             tiles of A (128 x 4096 x 4096: 10.4 swapped, 8.8 in those)
//   kMx       both with power-of-two scales, as E8M0 scales of the block-scaled MMA: FP32 results
//             of those (see the conversion kernel). TMEM adds up four blocks, the fold warps
//             those sums. 6144 x 4096 x 4096 78 us, 119 with the scales folded in
// and by size: pairs of CTAs (cta_group::2, 256 x 256 tiles, 256 x 192 of the weight gradient and
// kMx, each SM stages half of the column operand), or single CTAs (128 x BN tiles) whose reduction
// may be split over a cluster, the parts joined through distributed shared memory in rank
// order. Which of them, and how many parts, is chosen by estimated time (see Cost).
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
// Blocks whose scales have a place in shared memory, in groups that the fold warps hand back
// together (one block at a time: weight gradient 6144 x 4096 x 4096 114.5 us, 112.4 by fours).
constexpr int kScaleRing = 16, kScaleGroup = 4, kScaleGroups = kScaleRing / kScaleGroup;

enum Mode : int { kFprop = 0, kWgrad = 1, kSwapped = 2, kMx = 3 };

template <int BN, int kMode, bool kPair>
struct Cfg {
  static constexpr int kBRows = kPair ? BN / 2 : BN;  // column-operand rows staged per CTA
  static constexpr int kABytes = BM * BK;
  static constexpr int kBBytes = kBRows * BK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // kMx: E8M0 scale tiles of 128 rows, one of A and two of B (192 rows start within the first)
  static constexpr int kSfBytes = kMode == kMx ? 3 * 512 : 0;
  static constexpr int kTxBytes = kStageBytes + kSfBytes;
  static constexpr int kChunk = kMode == kMx ? 4 : 1;  // blocks that TMEM adds up before the fold
  // narrow tiles leave room for two CTAs on an SM
  static constexpr int kStages = kMode == kMx ? 7 : BN < 128 ? 4 : 5;
  // four folding warps (a TMEM lane quarter each) for each group of columns. The weight
  // gradient's pairs take 192 columns so that a warp's 64 stay in registers with their scales:
  // 256 spilled (6144 x 4096 x 4016 FP32: 208 us; 159 with 192, both before other steps)
  static constexpr int kColGroups = BN == 192 && kMode == kWgrad ? 3 : 2;
  static constexpr int kNC = BN / kColGroups;         // columns per folding warp
  static constexpr int kFoldWarps = 4 * kColGroups;
  // warps 0 and 1 copy and issue; a pair has two idle ones after them, because registers move
  // between whole warpgroups
  static constexpr int kFoldFirst = kPair ? 4 : 2;
  static constexpr int kThreads = 32 * (kFoldFirst + kFoldWarps);
  static constexpr int kOffA = 0;
  static constexpr int kOffB = kOffA + kStages * kABytes;
  // store staging: two 32-row x 64-byte boxes per folding warp, 1024-byte aligned
  static constexpr int kBoxBytes = 32 * 64;
  static constexpr int kBoxes = kMode == kMx ? 1 : 2;  // (kMx needs the room for its stages)
  static constexpr int kOffBox = kOffB + kStages * kBBytes;
  static constexpr int kOffScale =
      kOffBox + (kMode == kSwapped ? 0 : kBoxes * kFoldWarps * kBoxBytes);
  static constexpr int kRowScales = kMode == kSwapped ? 4 : BM;  // (kSwapped: one)
  static constexpr int kColScales = kMode == kFprop ? 4 : BN;    // (kFprop: one for 128 columns)
  static constexpr int kScaleFloats = kRowScales + kColScales;   // a tile's scales of a block
  static constexpr int kOffBar =
      kOffScale + (kMode == kMx ? kStages * kSfBytes : kScaleRing * kScaleFloats * 4);
  // TMEM: two accumulators; kMx: then the scales of the stages, 4 columns of A and 8 of B
  static constexpr int kSfaCol = 2 * BN, kSfbCol = kSfaCol + 4 * kStages;
  static constexpr int kNumBars = 2 * kStages + kScaleRing + kScaleGroups + 3;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;  // + slack for 1024-byte alignment
  static constexpr int kTmemCols = BN == 192 ? 512 : 2 * BN;  // two accumulators
  static constexpr int kMinCtas = BN <= 64 ? 2 : 1;
  static_assert(kMode != kMx || kSfbCol + 8 * kStages <= kTmemCols, "TMEM columns");
  static_assert(kTmemCols >= 32 && kTmemCols <= 512, "TMEM columns");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory overflow");
  // split-K partial sums: [row][column], or (kSwapped) [column][row]; the padding keeps the
  // rows of a 16-byte access on different banks
  static constexpr int kPartPitch = (kMode == kSwapped ? BM : BN) + 4;
  static_assert((kMode == kSwapped ? BN : BM) * kPartPitch * 4 <= kStages * kStageBytes,
                "split-K partial overflow");
};

// Pairs need more registers for their sums than an even share: the folding warpgroups take
// some over from the first one (12 warps x 168 = 8 x 224 + 4 x 56; 16 x 128 = 12 x 152 + 4 x 56).
template <int kFoldWarps>
constexpr int kFoldRegs = kFoldWarps == 12 ? 152 : 224;
constexpr int kOtherRegs = 56;

// How a wait is limited, in nanoseconds. The clock is read, and the abort flag looked at, only
// after failed polls whose number has no bit of `mask`: the hand-overs of the fold are on the
// critical path. The time counts from the first such reading, or from `t0` if that is not zero.
struct WaitLimit {
  uint64_t ns, t0;
  uint32_t mask;
};

struct Params {
  const float* sr;      // scales of the row operand: [nkb][ldr], or [row blocks][nkb] (kSwapped)
  const float* sc;      // of the column operand: [nkb][ldc], or [column blocks][nkb] (kFprop)
  int64_t ldr, ldc;
  void* C;
  int64_t ldo;          // output row pitch in elements
  int64_t nr, nc;       // valid rows and columns
  int nkb;              // blocks of 128 along K
  int out_fp32;
  int split;            // CTAs that share a tile's reduction (a cluster)
  uint32_t tiles, row_tiles, col_tiles;  // pairs: row tiles are of 256 rows
  uint32_t band;        // row tiles per raster band
  int* status;
  WaitLimit wait;
  uint64_t drain_ns;
  // the kernel returns at once unless one of these words is set (nullptr: it runs)
  const uint32_t* only_if;
  int num_only_if;
  const uint32_t* unless;  // and at once if one of these is
  int num_unless;
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
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31,"
      " %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47,"
      " %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]),
        "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]),
        "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
        "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]),
        "=r"(r[62]), "=r"(r[63])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) {
  tmem_ld_32x32b_x32(taddr, r);
}
template <int G>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[G]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < G; ++i) asm volatile("" : "+r"(r[i]) :: "memory");
}

// 4 bytes global -> shared.
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
// This thread's arrival on a barrier, once its copies so far are in.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// One poll; within a brief limit (mask 0) one that does not suspend the thread, which could
// outlast the limit.
__device__ __forceinline__ bool poll_brief(uint64_t* bar, uint32_t parity, uint32_t mask) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, patient;\n\t"
      "setp.ne.u32 patient, %3, 0;\n\t"
      "@patient mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@!patient mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(mask)
      : "memory");
  return ok != 0;
}

// Waits for a phase, within a limit. kTail: the producer's last waits, the place where a brief
// limit is sure to run out (the abort then ends the other roles' waits). With such polls in every
// role 4096 x 4096 x 4096 took 60.2 us instead of 58.0, and in all of the producer's 300 x 4096 x
// 4096 13.2 instead of 12.5.
template <bool kTail = false>
__device__ __forceinline__ bool poll_phase(uint64_t* bar, uint32_t parity, volatile int* abort,
                                           const WaitLimit& limit) {
  auto poll = [&] {
    return kTail ? poll_brief(bar, parity, limit.mask) : mbar_try_wait(bar, parity);
  };
  bool ok = poll();
  if (!ok) {
    uint64_t t0 = limit.t0;
    for (uint32_t i = 1;; ++i) {
      if ((i & limit.mask) == 0) {
        if (*abort) break;
        const uint64_t t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        else if (t - t0 > limit.ns) break;
      }
      ok = poll();
      if (ok) break;
    }
  }
  return ok;
}

// A whole warp waits, every lane for itself (one lane and a shuffle or vote took longer); true
// for all lanes or for none, and the warp is converged again.
template <bool kTail = false>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort,
                                           const WaitLimit& limit) {
  const bool ok = __all_sync(0xFFFFFFFFu, poll_phase<kTail>(bar, parity, abort, limit));
  __syncwarp();  // a vote does not reconverge the warp, as the .aligned instructions need it
  return ok;
}

// An arrival by one lane of the warp, as a predicated instruction instead of a branch.
__device__ __forceinline__ void arrive_if(bool one, uint32_t cluster_addr) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}"
      ::"r"(cluster_addr), "r"(one ? 1 : 0)
      : "memory");
}

__device__ __forceinline__ void arrive_if(bool one, uint64_t* bar) {  // of this CTA
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(one ? 1 : 0)
      : "memory");
}

// Moves registers between the warpgroups of a CTA; executed by every warp of a warpgroup.
template <int kRegs>
__device__ __forceinline__ void set_max_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void set_max_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// acc[0], acc[1] += s (two packed) times v0, v1
__device__ __forceinline__ void add_scaled(float* acc, uint32_t v0, uint32_t v1, uint64_t s) {
  const uint64_t a =
      fma2(pack2(__uint_as_float(v0), __uint_as_float(v1)), s, pack2(acc[0], acc[1]));
  unpack2(a, acc[0], acc[1]);
}

// acc[i] += s v[i] for G columns of one block, or += s c[i] v[i] with a scale for each column
// (kColVec), which all lanes read from the same place in shared memory.
template <int G, bool kColVec>
__device__ __forceinline__ void fold(float* acc, const uint32_t (&v)[G], float s,
                                     const float* c) {
#pragma unroll
  for (int i = 0; i < G; i += 4) {
    if constexpr (kColVec) {
      const float4 c4 = *reinterpret_cast<const float4*>(c + i);
      add_scaled(acc + i, v[i], v[i + 1], mul2(pack2(s, s), pack2(c4.x, c4.y)));
      add_scaled(acc + i + 2, v[i + 2], v[i + 3], mul2(pack2(s, s), pack2(c4.z, c4.w)));
    } else {
      add_scaled(acc + i, v[i], v[i + 1], pack2(s, s));
      add_scaled(acc + i + 2, v[i + 2], v[i + 3], pack2(s, s));
    }
  }
}

// The weight gradient's fold: a scale for every row and every column. A scale that each lane
// needs for every column costs one shared-memory cycle a warp and column, 1024 for a 256-wide
// block (measured 837 cycles a block in the fold alone). So TMEM is read in the 16x256b shape,
// which gives a lane few columns of several rows: of columns 8 j + 2 (lane % 4) and the next,
// rows lane / 4 (r[4 j], r[4 j + 1]) and lane / 4 + 8 (r[4 j + 2], r[4 j + 3]), of 16 rows and
// 32 columns a read; column scales are read two at a time and serve four rows.
__device__ __forceinline__ void tmem_ld_quads(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void fold_quads(float (*acc)[4], const uint32_t (&r)[16], float s0,
                                           float s1, const float2 (&c)[4]) {
  const uint64_t p0 = pack2(s0, s0), p1 = pack2(s1, s1);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t cc = pack2(c[j].x, c[j].y);
    const uint64_t a = fma2(pack2(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])),
                            mul2(p0, cc), pack2(acc[j][0], acc[j][1]));
    const uint64_t b = fma2(pack2(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])),
                            mul2(p1, cc), pack2(acc[j][2], acc[j][3]));
    unpack2(a, acc[j][0], acc[j][1]);
    unpack2(b, acc[j][2], acc[j][3]);
  }
}

__device__ __forceinline__ void store_one(const Params& p, int64_t at, float v) {
  if (p.out_fp32)
    static_cast<float*>(p.C)[at] = v;
  else
    static_cast<uint16_t*>(p.C)[at] = static_cast<uint16_t>(cvt_bf16x2(0.f, v));
}

// A warp's 32 rows x kNC columns of the tile leave through kBoxes staging boxes in turn: each
// 64-byte column group is written into a box (16-byte chunks XOR-swizzled as the tensor map's
// 64-byte swizzle expects) and sent with one TMA store, clipped at the matrix edge. Stores of
// one row per lane touch 32 cache lines an instruction: with those, a tile's stores took 2.5
// us, a sixth of the tile at K = 4096.
template <int kBoxes>
struct BoxStore {
  const CUtensorMap* map;
  uint8_t* boxes;
  int turn;

  // the box to write into, free again
  __device__ __forceinline__ uint8_t* open(int lane) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kBoxes - 1) : "memory");
    __syncwarp();
    return boxes + turn % kBoxes * (32 * 64);
  }
  // its first column and row
  __device__ __forceinline__ void send(int64_t col, int64_t row, int lane) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(map, boxes + turn % kBoxes * (32 * 64), static_cast<int32_t>(col),
                   static_cast<int32_t>(row));
      bulk_commit_group();
    }
    ++turn;
  }
};

// Sums held one row per lane (acc[i]: column i).
template <int kNC, int kBoxes>
__device__ __forceinline__ void store_rows(BoxStore<kBoxes>& out, const Params& p,
                                           const float (&acc)[kNC],
                                           int64_t row0, int64_t c0, int lane) {
  if (row0 >= p.nr) return;
#pragma unroll
  for (int u = 0; u < kNC; u += 16) {
    if (!p.out_fp32 && (u & 16)) continue;  // BF16: 32 columns a box
    if (c0 + u >= p.nc) continue;
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p.out_fp32) {
        const float* a = &acc[u + 4 * j];
        w[j] = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]),
                          __float_as_uint(a[3]));
      } else {
        const float* a = &acc[(u & ~31) + 8 * j];
        w[j] = make_uint4(cvt_bf16x2(a[1], a[0]), cvt_bf16x2(a[3], a[2]),
                          cvt_bf16x2(a[5], a[4]), cvt_bf16x2(a[7], a[6]));
      }
    }
    uint8_t* box = out.open(lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint4*>(box + lane * 64 + 16 * (j ^ ((lane >> 1) & 3))) = w[j];
    out.send(c0 + u, row0, lane);
  }
}

// Sums held in quads (see fold_quads).
__device__ __forceinline__ void store_quads(BoxStore<2>& out, const Params& p,
                                            const float (&acc)[2][8][4], int64_t row0, int64_t c0,
                                            int lane) {
  if (row0 >= p.nr) return;
  const int t4 = lane & 3;
#pragma unroll
  for (int u = 0; u < 64; u += 16) {
    if (!p.out_fp32 && (u & 16)) continue;  // BF16: 32 columns a box
    if (c0 + u >= p.nc) continue;
    uint8_t* box = out.open(lane);
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // rows lane / 4 + 8 h
      const int row = (lane >> 2) + 8 * h, x = (row >> 1) & 3;
      if (p.out_fp32) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float* a = &acc[h >> 1][u / 8 + j][2 * (h & 1)];
          *reinterpret_cast<float2*>(box + row * 64 + 16 * ((2 * j + (t4 >> 1)) ^ x) +
                                     8 * (t4 & 1)) = make_float2(a[0], a[1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float* a = &acc[h >> 1][(u & ~31) / 8 + j][2 * (h & 1)];
          *reinterpret_cast<uint32_t*>(box + row * 64 + 16 * (j ^ x) + 4 * t4) =
              cvt_bf16x2(a[1], a[0]);
        }
      }
    }
    out.send(c0 + u, row0, lane);
  }
}

// Adds CTA `part`'s share of a tile over the kSplit CTAs of the cluster, in rank order, and
// stores it: four neighbours of an output row at a time, the loads of several of them (eight
// in all) under way together, because a load from another SM takes about a microsecond.
template <typename C, int kMode, int kSplit>
__device__ __forceinline__ void join_parts(const Params& p, uint32_t sums, int64_t row0,
                                           int64_t col0, uint32_t part) {
  constexpr bool kT = kMode == kSwapped;
  constexpr int kLines = kT ? 2 * C::kNC : BM;        // output rows in the tile
  constexpr int kFours = (kT ? BM : 2 * C::kNC) / 4;  // groups of four in each
  constexpr int kAhead = 8 / kSplit;
  constexpr int kShare = kLines * kFours / kSplit;
  const int lo = kShare * static_cast<int>(part);
  for (int i0 = threadIdx.x; i0 < kShare; i0 += kAhead * C::kThreads) {
    float4 v[kAhead][kSplit];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = lo + i0 + u * C::kThreads;
      const uint32_t at = sums + 4 * (i / kFours * C::kPartPitch + i % kFours * 4);
#pragma unroll
      for (int k = 0; k < kSplit; ++k) {
        if (i0 + u * C::kThreads >= kShare) continue;
        uint32_t from;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(k));
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[u][k].x), "=f"(v[u][k].y), "=f"(v[u][k].z), "=f"(v[u][k].w)
                     : "r"(from) : "memory");
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i0 + u * C::kThreads >= kShare) continue;
      const int i = lo + i0 + u * C::kThreads;
      float4 s = v[u][0];
#pragma unroll
      for (int k = 1; k < kSplit; ++k) {
        s.x += v[u][k].x;
        s.y += v[u][k].y;
        s.z += v[u][k].z;
        s.w += v[u][k].w;
      }
      // the output's row, and the first of four places in it (rows of N values, N % 8 == 0)
      const int64_t line = (kT ? col0 : row0) + i / kFours;
      const int64_t place = (kT ? row0 : col0) + i % kFours * 4;
      if (line >= (kT ? p.nc : p.nr) || place >= (kT ? p.nr : p.nc)) continue;
      if (p.out_fp32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.C) + line * p.ldo + place) = s;
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.C) + line * p.ldo + place) =
            make_uint2(cvt_bf16x2(s.y, s.x), cvt_bf16x2(s.w, s.z));
    }
  }
}

template <int BN, int kMode, bool kPair>
__global__ void __launch_bounds__(Cfg<BN, kMode, kPair>::kThreads, Cfg<BN, kMode, kPair>::kMinCtas)
blockwise_gemm_kernel(const __grid_constant__ CUtensorMap map_r,
                      const __grid_constant__ CUtensorMap map_c,
                      const __grid_constant__ CUtensorMap map_o,
                      const __grid_constant__ CUtensorMap map_sr,  // kMx: the scales' tiles
                      const __grid_constant__ CUtensorMap map_sc, const Params p) {
  using C = Cfg<BN, kMode, kPair>;
  constexpr int kStages = C::kStages, kNC = C::kNC;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // pair: the leader's
  uint64_t* empty = full + kStages;
  uint64_t* ready = empty + kStages;            // [kScaleRing]: a block's product and scales
  uint64_t* scale_empty = ready + kScaleRing;   // [kScaleGroups]
  uint64_t* acc_empty = scale_empty + kScaleGroups;  // [2]; pair: the leader's
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  // drain records: [0] / [1] stage uses issued by the producer of CTA 0 / 1 of the pair (a
  // single CTA writes both), [2] stage uses consumed by the MMA issuer (one accumulator
  // commit each), [3] this CTA's producer tail completed, [4] accumulators committed
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

  if (p.only_if && !any_word_set(p.only_if, p.num_only_if)) return;  // the whole cluster does
  if (kMode == kMx && p.unless && any_word_set(p.unless, p.num_unless)) return;
  if (warp == 0) {
    for (int i = lane; i < C::kNumBars; i += 32) {
      uint64_t* bar = full + i;
      mbar_init(bar, bar < ready         ? 1
                     // the MMA's commit, the scales' copies
                     : bar < scale_empty ? (kMode == kMx ? 1 : 1 + 32)
                     : bar < acc_empty   ? C::kFoldWarps
                     : bar < mma_done    ? (kPair ? 2 : 1) * C::kFoldWarps
                                         : 1);
    }
    if (lane == 0) {
      *abort_flag = 0;
      for (int i = 0; i < 5; ++i) rec[i] = 0;
      if constexpr (kMode == kMx) {
        tma_prefetch_desc(&map_sr);
        tma_prefetch_desc(&map_sc);
      }
      tma_prefetch_desc(&map_r);
      tma_prefetch_desc(&map_c);
      tma_prefetch_desc(&map_o);
    }
    fence_barrier_init();
    __syncwarp();
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

  // each role sets its own register limit, inside its branch
  if (warp == 0) {
    if constexpr (kPair) set_max_regs_dec<kOtherRegs>();
    // ------------------------------------------------------------- TMA producer, scales
    const bool issuer = elect_one();
    const uint32_t full0 = kPair ? cluster_map(&full[0], 0) : smem_u32(&full[0]);
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t id = first_id; ok && id < p.tiles; id += id_step) {
      int64_t rt, ct;
      tile_at(p, id, rt, ct);
      const int32_t r0 = static_cast<int32_t>(kPair ? (2 * rt + crank) * BM : rt * BM);
      const int32_t c0 = static_cast<int32_t>(ct * BN);
      const int64_t rows_here = p.nr - r0, cols_here = p.nc - c0;
      const float* srp =
          kMode == kSwapped ? p.sr + rt * p.nkb + kb0 : p.sr + kb0 * p.ldr + r0 + lane;
      const float* scp = kMode == kFprop
                             ? p.sc + (c0 / 128 + lane) * static_cast<int64_t>(p.nkb) + kb0
                             : p.sc + kb0 * p.ldc + c0 + lane;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1;
        const uint32_t sl = it % kScaleRing;
        ok = wait_phase(&empty[s], ph ^ 1, abort_flag, p.wait) &&
             (kMode == kMx || it % kScaleGroup != 0 ||
              wait_phase(&scale_empty[sl / kScaleGroup], ((it / kScaleRing) & 1) ^ 1, abort_flag,
                         p.wait));
        if (!ok) break;
        if (issuer) {
          uint8_t* as = smem + C::kOffA + s * C::kABytes;
          uint8_t* bs = smem + C::kOffB + s * C::kBBytes;
          if constexpr (kPair) {
            if (leader) mbar_arrive_expect_tx(&full[s], 2 * C::kTxBytes);
            tma_load_2d_2sm(as, &map_r, kb * BK, r0, full0 + 8 * s);
            tma_load_2d_2sm(bs, &map_c, kb * BK, c0 + crank * (BN / 2), full0 + 8 * s);
            if constexpr (kMode == kMx) {
              uint8_t* sf = smem + C::kOffScale + s * C::kSfBytes;
              tma_load_3d_2sm(sf, &map_sr, 0, kb, r0 / BM, full0 + 8 * s);
              tma_load_3d_2sm(sf + 512, &map_sc, 0, kb, c0 / BM, full0 + 8 * s);
            }
          } else {
            mbar_arrive_expect_tx(&full[s], C::kStageBytes);
            tma_load_2d(as, &map_r, kb * BK, r0, &full[s]);
            tma_load_2d(bs, &map_c, kb * BK, c0, &full[s]);
          }
        }
        __syncwarp();
        // the block's scales; what lies past the matrix is not read: it meets zero products,
        // unstored
        if constexpr (kMode == kMx) continue;
        float* slot = reinterpret_cast<float*>(smem + C::kOffScale) + sl * C::kScaleFloats;
        if constexpr (kMode == kSwapped) {
          if (lane == 0) cp_async4(slot, srp);
        } else {
#pragma unroll
          for (int i = 0; i < BM; i += 32)
            if (i + lane < rows_here) cp_async4(slot + i + lane, srp + i);
        }
        if constexpr (kMode == kFprop) {
          if (lane < BN / 128 && 128 * lane < cols_here)
            cp_async4(slot + C::kRowScales + lane, scp);
        } else {
#pragma unroll
          for (int i = 0; i < BN; i += 32)
            if (i + lane < cols_here) cp_async4(slot + C::kRowScales + i + lane, scp + i);
        }
        srp += kMode == kSwapped ? 1 : p.ldr;
        scp += kMode == kFprop ? 1 : p.ldc;
        cp_async_arrive(&ready[sl]);
      }
    }
    cp_async_wait_all();
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
      tail_ok = wait_phase<true>(&empty[i % kStages], (i / kStages) & 1, abort_flag, p.wait);
    if (!tail_ok && issuer) {
      *abort_flag = 1;
      latch_error(p.status, MXFP8_ERR_TIMEOUT);
    }
    if (issuer) rec[3] = tail_ok ? 1u : 0u;
    __syncwarp();
  } else if (warp < C::kFoldFirst && !(warp == 1 && leader)) {
    if constexpr (kPair) set_max_regs_dec<kOtherRegs>();
  } else if (warp == 1) {
    if constexpr (kPair) set_max_regs_dec<kOtherRegs>();
    // ------------------------------------------------------------- MMA issuer
    const bool issuer = elect_one();
    uint32_t it = 0;
    bool ok = true;
    const uint64_t a_desc0 = smem_desc(smem_u32(smem + C::kOffA), 16, 1024, 2);
    const uint64_t b_desc0 = smem_desc(smem_u32(smem + C::kOffB), 16, 1024, 2);
    const uint64_t sf_desc0 = smem_desc(smem_u32(smem + C::kOffScale), 0, 128, 0);
    constexpr uint32_t kId = f8_idesc(kPair ? 2 * BM : BM, BN);
    // A single CTA's blocks take half as long as a pair's, and the vote after each wait of a whole
    // warp would be a tenth of one: there the issuing thread goes alone (512 x 4096 x 12288: 29.5
    // us, 35.8 as a warp), and in kMx, where the MMAs are the chain (80 us, 100 as a warp and
    // with the tile's place worked out at every block). Other pairs lose 2% that way.
    constexpr bool kWarpIssues = kPair && kMode != kMx;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return kWarpIssues ? wait_phase(bar, parity, abort_flag, p.wait)
                         : poll_phase(bar, parity, abort_flag, p.wait);
    };
    uint32_t acc_it = 0;
    for (uint32_t id = first_id; (kWarpIssues || issuer) && ok && id < p.tiles; id += id_step) {
      uint32_t sfb_shift = 0;
      if constexpr (kMode == kMx) {
        int64_t rt, ct;
        tile_at(p, id, rt, ct);
        sfb_shift = static_cast<uint32_t>(ct * BN % BM / 32);
      }
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1;
        const uint32_t b = acc_it & 1, aph = (acc_it >> 1) & 1;
        const bool starts = C::kChunk == 1 || (kb - kb0) % C::kChunk == 0;
        const bool ends =
            C::kChunk == 1 || (kb - kb0) % C::kChunk == C::kChunk - 1 || kb == kb1 - 1;
        ok = wait(&full[s], ph) && (!starts || wait(&acc_empty[b], aph ^ 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = a_desc0 + s * (C::kABytes / 16);
        const uint64_t bd = b_desc0 + s * (C::kBBytes / 16);
        const uint32_t d = tmem + b * BN;
        if (issuer) {  // a K step of 32 starts 32 bytes further; past K the tiles are zero
          if constexpr (kMode == kMx) {
            // the stage's scales into TMEM; 192 columns start on or 64 rows into a tile of B's
            const uint32_t sfa = tmem + C::kSfaCol + 4 * s, sfb = tmem + C::kSfbCol + 8 * s;
            const uint64_t sd = sf_desc0 + s * (C::kSfBytes / 16);
            tmem_cp_32x128b_x4_2sm(sfa, sd);
            tmem_cp_32x128b_x4_2sm(sfb, sd + 512 / 16);
            tmem_cp_32x128b_x4_2sm(sfb + 4, sd + 1024 / 16);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_mxf8_2sm(d, ad + 2 * k, bd + 2 * k, mxf8_idesc(2 * BM, BN, k, k), sfa,
                           sfb + sfb_shift, !starts || k > 0);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (kPair) mma_f8_2sm(d, ad + 2 * k, bd + 2 * k, kId, k > 0);
              else mma_f8(d, ad + 2 * k, bd + 2 * k, kId, k > 0);
            }
          }
          if constexpr (kPair) {
            if (ends) mma_commit_2sm_mc(&ready[acc_it % kScaleRing], 3);
            mma_commit_2sm_mc(&empty[s], 3);
          } else {
            mma_commit(&ready[acc_it % kScaleRing]);
            mma_commit(&empty[s]);
          }
        }
        if (ends) ++acc_it;
        if constexpr (kWarpIssues) __syncwarp();
      }
    }
    __syncwarp();
    if (!ok && issuer) {
      *abort_flag = 1;
      latch_error(p.status, MXFP8_ERR_TIMEOUT);
    }
    if (issuer) {
      if constexpr (kPair) {
        for (uint32_t r = 0; r < 2; ++r)
          st_cluster_u32(cluster_map(const_cast<uint32_t*>(&rec[2]), r), it);
        for (uint32_t r = 0; r < 2; ++r)
          st_cluster_u32(cluster_map(const_cast<uint32_t*>(&rec[4]), r), acc_it);
        mma_commit_2sm_mc(mma_done, 1);
      } else {
        rec[2] = it;
        rec[4] = acc_it;
        mma_commit(mma_done);
      }
      mbar_wait_timed(mma_done, 0, p.drain_ns);
    }
    __syncwarp();
  } else {
    if constexpr (kPair) set_max_regs_inc<kFoldRegs<C::kFoldWarps>>();
    // ------------------------------------------------------------- fold and store
    const int q = warp & 3;                   // TMEM lane quarter this warp may access
    const int half = (warp - C::kFoldFirst) >> 2;  // which group of the columns
    BoxStore<C::kBoxes> out{
        &map_o, smem + C::kOffBox + (warp - C::kFoldFirst) * C::kBoxes * C::kBoxBytes, 0};
    const uint32_t acc_empty0 = kPair ? cluster_map(&acc_empty[0], 0) : smem_u32(&acc_empty[0]);
    constexpr bool kColVec = kMode == kWgrad || kMode == kSwapped;
    constexpr bool kQuads = kMode == kWgrad;
    static_assert(!kQuads || kNC == 64, "a warp of the weight gradient folds 64 columns");
    // columns a TMEM read: as many as the registers allow
    constexpr int G = kMode == kSwapped ? (kNC < 32 ? kNC : kNC / 2) : kMode == kMx ? 32 : 64;
    const uint32_t tbase = tmem + (static_cast<uint32_t>(32 * q) << 16) + half * kNC;
    const float* ring = reinterpret_cast<const float*>(smem + C::kOffScale);
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t id = first_id; ok && id < p.tiles; id += id_step) {
      int64_t rt, ct;
      tile_at(p, id, rt, ct);
      const int64_t row0 = (kPair ? 2 * rt + crank : rt) * BM + 32 * q;
      const int64_t col = ct * BN + half * kNC;  // this warp's first column
      const bool row_ok = row0 + lane < p.nr;
      float acc[kQuads ? 1 : kNC], quads[2][8][4];
#pragma unroll
      for (int i = 0; i < (kQuads ? 1 : kNC); ++i) acc[i] = 0.f;
#pragma unroll
      for (int i = 0; i < 64; ++i) (&quads[0][0][0])[i] = 0.f;
#pragma unroll 1
      for (int kb = kb0; kb < kb1; kb += C::kChunk, ++it) {  // `it` counts accumulators
        const uint32_t b = it & 1;
        const float* rows = ring + (it % kScaleRing) * C::kScaleFloats;
        const float* cols =
            rows + C::kRowScales + (kMode == kFprop ? half * kNC / 128 : half * kNC);
        float rq[4];
        float2 cq[4];  // the scales of 32 of the columns
        auto load_cq = [&](int u) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            cq[j] = *reinterpret_cast<const float2*>(cols + 32 * u + 8 * j + 2 * (lane & 3));
        };
        const uint32_t sl = it % kScaleRing;
        ok = wait_phase(&ready[sl], (it / kScaleRing) & 1, abort_flag, p.wait);
        if (!ok) break;
        tc_fence_after();
        if constexpr (kQuads) {
          // four reads of 16 rows and 32 columns; the next one is under way during the fold
          uint32_t r[2][16];
          auto read = [&](int i) {
            const uint32_t row = static_cast<uint32_t>(16 * (i & 1)) << 16;
            tmem_ld_quads(tbase + b * BN + row + 16 * (i & 2), r[i & 1]);
          };
          read(0);
#pragma unroll
          for (int h = 0; h < 4; ++h) rq[h] = rows[32 * q + (lane >> 2) + 8 * h];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i == 0) load_cq(0);
            if (i == 2) load_cq(1);
            tmem_wait(r[i & 1]);
            if (i < 3) {
              read(i + 1);
            } else {  // the block has left TMEM
              tc_fence_before();
              arrive_if(lane == 0, acc_empty0 + 8 * b);
            }
            fold_quads(&quads[i & 1][2 * (i & 2)], r[i & 1], rq[2 * (i & 1)],
                       rq[2 * (i & 1) + 1], cq);
          }
        } else {
          float s = 0.f;
#pragma unroll
          for (int g = 0; g < kNC; g += G) {
            uint32_t r[G];
            tmem_ld(tbase + b * BN + g, r);
            if (g == 0 && kMode != kMx)
              s = kMode == kSwapped ? rows[0] : rows[32 * q + lane] * cols[0];
            tmem_wait(r);
            if (g + G == kNC) {  // the block has left TMEM
              tc_fence_before();
              arrive_if(lane == 0, acc_empty0 + 8 * b);
            }
            if constexpr (kMode == kMx) {
#pragma unroll
              for (int i = 0; i < G; i += 2)
                unpack2(add2(pack2(acc[g + i], acc[g + i + 1]),
                             pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]))),
                        acc[g + i], acc[g + i + 1]);
            } else {
              fold<G, kColVec>(acc + g, r, s, cols + g);
            }
          }
        }
        if constexpr (kMode == kMx) continue;
        __syncwarp();  // every lane has read the block's scales
        arrive_if(lane == 0 && it % kScaleGroup == kScaleGroup - 1, &scale_empty[sl / kScaleGroup]);
      }
      if (!ok) break;
      if (!kPair && p.split > 1) {
        // partial sums into the (now idle) stages
        float* part_sum = reinterpret_cast<float*>(smem);
        if constexpr (kMode == kSwapped) {
#pragma unroll
          for (int i = 0; i < kNC; ++i)
            part_sum[(half * kNC + i) * C::kPartPitch + 32 * q + lane] = acc[i];
        } else if constexpr (kQuads) {
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float2*>(
                  part_sum + (32 * q + (lane >> 2) + 8 * h) * C::kPartPitch + half * kNC + 8 * j +
                  2 * (lane & 3)) =
                  make_float2(quads[h >> 1][j][2 * (h & 1)], quads[h >> 1][j][2 * (h & 1) + 1]);
        } else {
#pragma unroll
          for (int i = 0; i < kNC; i += 4)
            *reinterpret_cast<float4*>(part_sum + (32 * q + lane) * C::kPartPitch + half * kNC +
                                       i) =
                make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        }
      } else if constexpr (kMode == kSwapped) {
        if (row_ok) {
#pragma unroll
          for (int i = 0; i < kNC; ++i)
            if (col + i < p.nc) store_one(p, (col + i) * p.ldo + row0 + lane, acc[i]);
        }
      } else {
        if constexpr (kQuads) store_quads(out, p, quads, row0, col, lane);
        else store_rows<kNC>(out, p, acc, row0, col, lane);
      }
    }
    // its stores must have finished reading shared memory before the CTA exits
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
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
        if (i < i0 && i >= i1) mbar_complete_tx(bar, C::kTxBytes);
        else if (i >= i0 && i < i1) mbar_arrive_expect_tx(bar, C::kTxBytes);
      }
      for (uint32_t i = consumed; i < issued; ++i)
        mbar_wait_timed(&full[i % kStages], (i / kStages) & 1, p.drain_ns);
    }
    for (uint32_t i = consumed > kStages ? consumed - kStages : 0; i < consumed; ++i)
      mbar_wait_timed(&empty[i % kStages], (i / kStages) & 1, p.drain_ns);
    for (uint32_t i = rec[4] > 2 ? rec[4] - 2 : 0; i < rec[4]; ++i)
      mbar_wait_timed(&ready[i % kScaleRing], (i / kScaleRing) & 1, p.drain_ns);
  }
  __syncthreads();
  if constexpr (kPair) {
    if (issued > consumed) cluster_sync();  // the leader's drain covered the peer's copies too
  } else if (p.split > 1) {
    // Join the parts: CTA `part` adds its share of the tile over all parts, in rank order, and
    // stores it. One tile per cluster.
    cluster_sync();
    int64_t rt, ct;
    tile_at(p, first_id, rt, ct);
    const uint32_t sums = smem_u32(smem);
    if (p.split == 2) join_parts<C, kMode, 2>(p, sums, rt * BM, ct * BN, part);
    else if (p.split == 4) join_parts<C, kMode, 4>(p, sums, rt * BM, ct * BN, part);
    else join_parts<C, kMode, 8>(p, sums, rt * BM, ct * BN, part);
    cluster_sync();  // no CTA leaves while its shared memory is being read
  }
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (kPair) tmem_dealloc_2sm(tmem, C::kTmemCols);
    else tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------- power-of-two scales (MXFP8 form)
//
// A power-of-two scale on a block of 128 is the same E8M0 scale on each of its four blocks of
// 32, so operands quantized with power-of-two scales can run on the block-scaled MMA
// (mxfp8_gemm), where the tensor cores apply the scales and nothing is folded. Whether all
// scales are powers of two is known on the device only: this kernel writes the scales in the
// MMA's 128 x 4 tile layout and, for each CTA, a word that says whether it met another one.
// The block-scaled kernel then returns at once if any word is set, the folding one if none
// is. BF16 results come from mxfp8_gemm, where the tensor cores sum over all of K (see kMxMaxK); for
// FP32 results kMx takes only 512 products at a time from them and adds those up in FP32
// registers (products of one sign, K = 4096 to 32768: 1.2e-6 off, 7e-7 folded; of both, 1e-7 and
// 6e-8). Measured back to back, BF16: 4096 x 24576 x 4096 228 to 246 us (3.6 to 3.4 PFLOP/s, by
// power; a single call with cold caches 256), 300 to 325 folded; weight gradient 6144 x 4096 x 4096
// 66 and 115; FP32: 78 and 119, 4096 x 12288 x 8192 274 and 438. Scales that turn out not to be
// powers of two pay the two other launches: 65 us instead of 58 at 4096^3.
constexpr int kConvertCtas = 608;  // four on each SM
constexpr int kConvertThreads = 256;

struct ConvertArgs {
  const float* s[2];       // A's and B's scales
  uint32_t* tiles[2];      // their tiles, 512 bytes each
  int64_t rows[2];
  int row_tiles[2];
  bool two_d[2];           // [row tiles][nkb] instead of [nkb][rows]
  int nkb;
  uint32_t* other;         // [kConvertCtas]
};

__global__ void __launch_bounds__(kConvertThreads) convert_scales_kernel(const ConvertArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  bool other = false;
  const int t = threadIdx.x & 127;  // row within a tile; two tiles at a time
  constexpr int kUnroll = 4;
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const uint32_t row_tiles = static_cast<uint32_t>(a.row_tiles[o]);
    const uint32_t tiles = row_tiles * static_cast<uint32_t>(a.nkb);
    const uint32_t step = 2 * gridDim.x;
    for (uint32_t i0 = 2 * blockIdx.x + (threadIdx.x >> 7); i0 < tiles; i0 += kUnroll * step) {
      uint32_t bits[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint32_t i = i0 + u * step, kb = i / row_tiles, rt = i - kb * row_tiles;
        const int64_t row = static_cast<int64_t>(rt) * BM + t;
        bits[u] = i < tiles && row < a.rows[o]
                      ? __float_as_uint(a.two_d[o] ? a.s[o][static_cast<int64_t>(rt) * a.nkb + kb]
                                                   : a.s[o][kb * a.rows[o] + row])
                      : 0x3F800000u;
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint32_t i = i0 + u * step, kb = i / row_tiles, rt = i - kb * row_tiles;
        if (i >= tiles) continue;
        const uint32_t e = bits[u] >> 23;  // the sign too: a negative scale is another one
        uint32_t byte = e & 0xFFu;
        if ((bits[u] & 0x7FFFFFFFu) > 0x7F800000u) byte = 0xFFu;                 // NaN
        else if (bits[u] != 0x00400000u /* 2^-127 */ &&
                 ((bits[u] & 0x7FFFFFu) != 0 || e == 0 || e > 254)) other = true;
        // scale (r, k) of a tile at byte (r % 32) * 16 + (r / 32) * 4 + k
        a.tiles[o][(static_cast<int64_t>(rt) * a.nkb + kb) * 128 + (t & 31) * 4 + (t >> 5)] =
            byte * 0x01010101u;
      }
    }
  }
  const int any = __syncthreads_or(other);
  if (threadIdx.x == 0) a.other[blockIdx.x] = any ? 1u : 0u;
}

// ------------------------------------------------------------------------- host side

// The kernel, allowed its shared memory; nullptr after a CUDA error.
template <int BN, int kMode, bool kPair>
auto ready_kernel() -> decltype(&blockwise_gemm_kernel<BN, kMode, kPair>) {
  auto k = blockwise_gemm_kernel<BN, kMode, kPair>;
  static std::atomic<bool> attr_set[64] = {};  // per device; setting it twice is harmless
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<BN, kMode, kPair>::kSmemBytes) != cudaSuccess)
      return nullptr;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  return k;
}

template <int BN, int kMode, bool kPair>
int launch(const CUtensorMap& mr, const CUtensorMap& mc, const CUtensorMap& mo,
           const CUtensorMap& msr, const CUtensorMap& msc, const Params& p, int64_t grid,
           int cluster, cudaStream_t stream) {
  auto k = ready_kernel<BN, kMode, kPair>();
  if (!k) return MXFP8_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(Cfg<BN, kMode, kPair>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<BN, kMode, kPair>::kSmemBytes;
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
  return cudaLaunchKernelEx(&cfg, k, mr, mc, mo, msr, msc, p) == cudaSuccess ? MXFP8_OK
                                                                             : MXFP8_ERR_CUDA;
}

// 256 x BN tiles on CTA pairs. `a` is the row operand.
template <int BN, int kMode>
int launch_pairs(const BlockwiseGemmArgs& a, Params p, cudaStream_t stream) {
  using C = Cfg<BN, kMode, true>;
  CUtensorMap mr, mc, mo;
  if (!make_operand_map(&mr, a.A, a.K, a.M, BM) ||
      !make_operand_map(&mc, a.B, a.K, a.N, C::kBRows) ||
      !make_store_map(&mo, a.C, a.M, a.N, a.out_fp32))
    return MXFP8_ERR_CUDA;
  p.row_tiles = static_cast<uint32_t>((a.M + 255) / 256);
  p.col_tiles = static_cast<uint32_t>((a.N + BN - 1) / BN);
  const int64_t tiles = static_cast<int64_t>(p.row_tiles) * p.col_tiles;
  if (tiles > 0x7FFFFFFF / 2) return MXFP8_ERR_INVALID_ARG;
  p.tiles = static_cast<uint32_t>(tiles);
  p.band = p.row_tiles < 8 ? p.row_tiles : 8;
  p.split = 1;
  const int64_t pairs = num_sms() / 2;
  CUtensorMap msr = mr, msc = mc;  // unused but for kMx
  if (kMode == kMx &&
      (!make_scale_map(&msr, p.sr, (a.M + 127) / 128, p.nkb, 1) ||
       !make_scale_map(&msc, p.sc, (a.N + 127) / 128, p.nkb, 2)))
    return MXFP8_ERR_CUDA;
  return launch<BN, kMode, true>(mr, mc, mo, msr, msc, p, 2 * (tiles < pairs ? tiles : pairs), 2,
                                 stream);
}

// 128 x BN tiles on single CTAs, the reduction split over clusters of `split`.
template <int BN, int kMode>
int launch_single(const void* R, int64_t nr, const void* Cop, int64_t nc, int64_t K, Params p,
                  int split, cudaStream_t stream) {
  CUtensorMap mr, mc, mo;
  if (!make_operand_map(&mr, R, K, nr, BM) || !make_operand_map(&mc, Cop, K, nc, BN))
    return MXFP8_ERR_CUDA;
  // swapped tiles are stored transposed, without a map
  if (kMode == kSwapped) mo = mr;
  else if (!make_store_map(&mo, p.C, nr, nc, p.out_fp32 != 0)) return MXFP8_ERR_CUDA;
  p.row_tiles = static_cast<uint32_t>((nr + BM - 1) / BM);
  p.col_tiles = static_cast<uint32_t>((nc + BN - 1) / BN);
  const int64_t tiles = static_cast<int64_t>(p.row_tiles) * p.col_tiles;
  if (tiles > 0x7FFFFFFF / 8) return MXFP8_ERR_INVALID_ARG;
  p.tiles = static_cast<uint32_t>(tiles);
  p.band = kMode == kSwapped ? 1 : (p.row_tiles < 8 ? p.row_tiles : 8);
  p.split = split;
  int64_t grid = tiles * split;
  const int64_t fit = static_cast<int64_t>(num_sms()) * Cfg<BN, kMode, false>::kMinCtas;
  if (split == 1 && grid > fit) grid = fit;  // persistent
  return launch<BN, kMode, false>(mr, mc, mo, mr, mc, p, grid, split, stream);
}

// Clusters of `split` single CTAs that the device runs at a time. Fewer than its SMs would hold,
// because a cluster lies within a group of SMs whose size is no multiple of it: 76, 36 and 15
// of 2, 4 and 8 on 152 SMs. The query counts one CTA an SM; narrow tiles have two.
template <int BN, int kMode>
int64_t clusters_at_once(int split) {
  using C = Cfg<BN, kMode, false>;
  if (split == 1) return static_cast<int64_t>(num_sms()) * C::kMinCtas;
  static std::atomic<int> known[64][9] = {};  // per device and split; 0: not asked yet
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev >= 0 && dev < 64 && (n = known[dev][split].load(std::memory_order_relaxed)) > 0) return n;
  auto k = ready_kernel<BN, kMode, false>();
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(split), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!k || cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) return 1;
  n *= C::kMinCtas;
  if (dev >= 0 && dev < 64) known[dev][split].store(n, std::memory_order_relaxed);
  return n;
}

// Estimated microseconds, from which shapes and splits are chosen. Measured on GB300 (16 to 96
// blocks of K, splits of 1 to 8, 16 to 192 row tiles): what a block takes, a tile's first
// operands and store, and the join of two or four parts, or of eight.
struct Cost {
  double block, tile, join, join8;
};
template <int BN, int kMode>
constexpr Cost kCost = BN == 16   ? Cost{0.24, 2.7, 1.2, 3.0}
                       : BN == 32 ? Cost{0.265, 3.1, 1.1, 3.9}
                       : BN == 64 ? Cost{0.29, 4.0, 1.9, 5.8}
                       : kMode == kFprop ? Cost{0.265, 3.3, 3.0, 6.0}
                                         : Cost{0.365, 3.6, 2.8, 6.0};
struct Plan {
  double us;
  int split;
};

template <int BN, int kMode>
Plan single_plan(int64_t tiles, int64_t nkb) {
  constexpr Cost c = kCost<BN, kMode>;
  Plan best{1e30, 1};
  for (int s = 1; s <= 8 && (s == 1 || nkb >= 4 * s); s *= 2) {
    const int64_t at_once = clusters_at_once<BN, kMode>(s);
    const double waves = static_cast<double>((tiles + at_once - 1) / at_once);
    const double us = waves * (static_cast<double>((nkb + s - 1) / s) * c.block + c.tile +
                               (s == 8 ? c.join8 : s > 1 ? c.join : 0.0));
    if (us < best.us) best = Plan{us, s};
  }
  return best;
}

// A block takes a 256 x 256 pair tile 0.42 us, a 256 x 192 one of the weight gradient 0.47.
double pair_us(int64_t tiles, int64_t nkb, bool wgrad) {
  const int64_t pairs = num_sms() / 2;
  return static_cast<double>((tiles + pairs - 1) / pairs) *
             (static_cast<double>(nkb) * (wgrad ? 0.47 : 0.42) + 1.2) + 2.0;
}

template <int BN>
int launch_swapped(const BlockwiseGemmArgs& a, const Params& p, cudaStream_t stream) {
  const Plan plan = single_plan<BN, kSwapped>((a.N + BM - 1) / BM, p.nkb);
  return launch_single<BN, kSwapped>(a.B, a.N, a.A, a.M, a.K, p, plan.split, stream);
}

// How a product of more than 64 rows (or a weight gradient) is folded, and its estimated time.
struct FoldPlan {
  bool pairs;
  int split;
  double us;
};

FoldPlan fold_plan(int64_t M, int64_t N, int64_t nkb, bool wgrad) {
  const int bn = wgrad ? 192 : 256;  // columns of a pair tile
  const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
  const Plan single =
      wgrad ? single_plan<128, kWgrad>(tiles, nkb) : single_plan<128, kFprop>(tiles, nkb);
  const double pairs = pair_us(((M + 255) / 256) * ((N + bn - 1) / bn), nkb, wgrad);
  return pairs < single.us ? FoldPlan{true, 1, pairs} : FoldPlan{false, single.split, single.us};
}

// The block-scaled MMA for power-of-two scales, with the conversion before and the folding
// kernel's empty launch behind it: estimated microseconds. A block takes a 256-wide pair tile of
// mxfp8_gemm 0.307 us, a 256 x 192 one of kMx 0.215; neither splits the reduction.
double block_scaled_us(int64_t M, int64_t N, int64_t nkb, bool out_fp32) {
  const int64_t pairs = num_sms() / 2, tiles = ((M + 255) / 256) * ((N + 191) / 192);
  const double k = static_cast<double>(nkb);
  return out_fp32 ? 9.6 + static_cast<double>((tiles + pairs - 1) / pairs) * (0.215 * k + 1.9)
                  : 9.1 + dense_gemm_waves(M, N, false) * (0.307 * k + 1.3);
}

// What the conversion, the check and an empty launch cost a product whose scales turn out not to
// be powers of two: the block-scaled MMA is tried where it saves others as much. Measured with both
// kinds of scale at 112 sizes of 8 to 825 GFLOP, a third of them drawn at random, forward and weight
// gradient, BF16 and FP32 results: the rule decides as the measured times would at 102 of them; what
// it misses is mostly K of 512 or 1024, where stores count for more than estimated. Saved / paid,
// us: forward BF16 4096 x 6144 x 4096 21 / 8, 4096^3 9 / 7, 2048 x 6144 x 4096 5 / 7, 512 x 512 x
// 200000 -282 / 12; weight gradient FP32 6144 x 4096 x 2048 18 / 7, 1024 x 4096 x 4096 3 / 6, 1024
// x 1024 x 65536 -18 / 9.
constexpr double kCheckUs = 7;
// The longest reduction that a BF16 result leaves to the tensor cores' own sum. They drop what lies
// below the sum's last bit at each step of 32 products: up to 2^-23 of it, so K 2^-28 in all where
// the products have one sign (measured, same sign, of sum |a b|: 0.002 at K = 2^20, 0.015 at 2^23;
// the folding kernel 2e-6). Up to here that is 2^-11, an eighth of BF16's own rounding.
constexpr int64_t kMxMaxK = int64_t{1} << 17;

bool block_scaled_pays(int64_t M, int64_t N, int64_t K, bool wgrad, bool out_fp32) {
  if (M <= 128 || N <= 128 || (!out_fp32 && K > kMxMaxK)) return false;
  const int64_t nkb = (K + BK - 1) / BK;
  return fold_plan(M, N, nkb, wgrad).us - block_scaled_us(M, N, nkb, out_fp32) >= kCheckUs;
}

int64_t workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t nkb = (K + BK - 1) / BK;
  return ((M + 127) / 128 + (N + 127) / 128) * nkb * 512 + kConvertCtas * 4;
}

}  // namespace

int64_t blockwise_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, bool out_fp32) {
  return block_scaled_pays(M, N, K, false, out_fp32) || block_scaled_pays(M, N, K, true, out_fp32)
             ? workspace_bytes(M, N, K)
             : 0;
}

int launch_blockwise_gemm(const BlockwiseGemmArgs& a, cudaStream_t stream) {
  Params p{};
  p.C = a.C;
  p.ldo = a.N;
  p.nkb = static_cast<int>((a.K + BK - 1) / BK);
  p.out_fp32 = a.out_fp32 ? 1 : 0;
  p.status = a.status;
  p.wait.ns = pipeline_wait_ns();
  p.drain_ns = pipeline_drain_ns();
  // A limit of about a poll's own time or less runs out at the first failed poll. (Under the rule
  // for others it never did: no wait of a sound pipeline takes 64 polls.)
  const bool brief = p.wait.ns < 10000;
  p.wait.t0 = brief ? 1 : 0;
  p.wait.mask = brief ? 0 : 63;
  if (!a.wgrad && a.M <= 64) {
    p.sr = a.sB;
    p.sc = a.sA;
    p.ldc = a.M;
    p.nr = a.N;
    p.nc = a.M;
    if (a.M <= 16) return launch_swapped<16>(a, p, stream);
    if (a.M <= 32) return launch_swapped<32>(a, p, stream);
    return launch_swapped<64>(a, p, stream);
  }
  p.sr = a.sA;
  p.sc = a.sB;
  p.ldr = a.M;
  p.ldc = a.N;
  p.nr = a.M;
  p.nc = a.N;
  if (a.workspace && a.workspace_bytes >= static_cast<size_t>(workspace_bytes(a.M, a.N, a.K)) &&
      block_scaled_pays(a.M, a.N, a.K, a.wgrad, a.out_fp32)) {
    const int64_t rta = (a.M + 127) / 128, rtb = (a.N + 127) / 128;
    if ((rta + rtb) * p.nkb > 0x7FFFFFFF) return MXFP8_ERR_INVALID_ARG;  // 32-bit tile index
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    ConvertArgs c{};
    c.s[0] = a.sA;
    c.s[1] = a.sB;
    c.tiles[0] = reinterpret_cast<uint32_t*>(ws);
    c.tiles[1] = c.tiles[0] + rta * p.nkb * 128;
    c.rows[0] = a.M;
    c.rows[1] = a.N;
    c.row_tiles[0] = static_cast<int>(rta);
    c.row_tiles[1] = static_cast<int>(rtb);
    c.two_d[1] = !a.wgrad;
    c.nkb = p.nkb;
    c.other = c.tiles[1] + rtb * p.nkb * 128;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kConvertCtas, 1, 1);
    cfg.blockDim = dim3(kConvertThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    cfg.numAttrs = pdl_attr(&attr[0]);
    if (cudaLaunchKernelEx(&cfg, convert_scales_kernel, c) != cudaSuccess) return MXFP8_ERR_CUDA;
    if (a.out_fp32) {
      Params x = p;
      x.sr = reinterpret_cast<const float*>(c.tiles[0]);
      x.sc = reinterpret_cast<const float*>(c.tiles[1]);
      x.unless = c.other;
      x.num_unless = kConvertCtas;
      const int st = launch_pairs<192, kMx>(a, x, stream);
      if (st != MXFP8_OK) return st;
    } else {
      GemmArgs g{a.A, c.tiles[0], a.B, c.tiles[1], a.C, a.M, a.N, a.K, MXFP8_OP_FPROP,
                 MXFP8_OUT_BF16, nullptr, 0, 0, a.status};
      g.unless = c.other;
      g.num_unless = kConvertCtas;
      const int st = launch_gemm(g, stream);
      if (st != MXFP8_OK) return st;
    }
    p.only_if = c.other;
    p.num_only_if = kConvertCtas;
  }
  const FoldPlan plan = fold_plan(a.M, a.N, p.nkb, a.wgrad);
  if (plan.pairs)
    return a.wgrad ? launch_pairs<192, kWgrad>(a, p, stream)
                   : launch_pairs<256, kFprop>(a, p, stream);
  return a.wgrad ? launch_single<128, kWgrad>(a.A, a.M, a.B, a.N, a.K, p, plan.split, stream)
                 : launch_single<128, kFprop>(a.A, a.M, a.B, a.N, a.K, p, plan.split, stream);
}

}  // namespace mxfp8
