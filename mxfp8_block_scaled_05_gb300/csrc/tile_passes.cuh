// tile_passes.cuh - the row-wise and the column-wise MXFP8 copy of a 128 x 128 BF16 tile in shared
// memory, by the 256 threads of a CTA (format and layouts: quantize.cu).
#pragma once

#include <cstdint>

#include "convert.cuh"
#include "device.cuh"
#include "mxfp8.h"

namespace mxfp8 {

constexpr int kTile = 128;        // rows and columns of a CTA tile
constexpr int kThreads = 256;
constexpr int kTilePitch = kTile + 8;  // BF16 row pitch of the shared tile: 272 bytes

// 16 bytes global -> shared, bypassing L1; `valid` false writes 16 zero bytes instead.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 16u : 0u) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

struct QOut {
  uint8_t* codes;
  uint8_t* scales;
  int64_t scale_item_bytes;  // bytes of one batch item's scale block
};

// Row-wise copy of a 128 x 128 tile staged in shared memory: one thread per 32-block (8
// consecutive rows per 8 lanes, conflict-free with the padded pitch), 32 code bytes per
// thread; the scale bytes go to the 512-byte tile stile_r (swizzled) or straight out.
template <bool kSwizzled>
__device__ __forceinline__ void row_pass_smem(const uint16_t (*tile)[kTilePitch],
                                              uint8_t* stile_r, const QOut& ro, int64_t cols,
                                              int64_t row0, int rows_valid, int64_t col0,
                                              int cols_valid, int rule) {
  const int t = threadIdx.x;
  const int64_t s_cols = cols / 32;
  const int w = t >> 5, l = t & 31;
  const int b = l >> 3;
  const bool block_ok = 32 * b < cols_valid;
  const bool wide = (reinterpret_cast<uintptr_t>(ro.codes) & 31) == 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 8 * w + (l & 7) + 64 * i;
    const uint4* rp = reinterpret_cast<const uint4*>(&tile[r][32 * b]);
    const uint4 x0 = rp[0], x1 = rp[1], x2 = rp[2], x3 = rp[3];
    uint32_t m2 = max_abs_bf16x2(
        max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(x0.x, x0.y), max_abs_bf16x2(x0.z, x0.w)),
                       max_abs_bf16x2(max_abs_bf16x2(x1.x, x1.y), max_abs_bf16x2(x1.z, x1.w))),
        max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(x2.x, x2.y), max_abs_bf16x2(x2.z, x2.w)),
                       max_abs_bf16x2(max_abs_bf16x2(x3.x, x3.y), max_abs_bf16x2(x3.z, x3.w))));
    m2 &= kAbs2;
    const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    const bool valid = block_ok && r < rows_valid;
    const uint32_t s = scale_byte(m, rule);
    if (valid) {
      uint32_t o[8];
      if (__builtin_expect(s != 0xFFu, 1)) {
        const uint32_t mul2 = inv_scale_bf16(s) * 0x10001u;
        o[0] = e4m3x4_pow2(x0.x, x0.y, mul2); o[1] = e4m3x4_pow2(x0.z, x0.w, mul2);
        o[2] = e4m3x4_pow2(x1.x, x1.y, mul2); o[3] = e4m3x4_pow2(x1.z, x1.w, mul2);
        o[4] = e4m3x4_pow2(x2.x, x2.y, mul2); o[5] = e4m3x4_pow2(x2.z, x2.w, mul2);
        o[6] = e4m3x4_pow2(x3.x, x3.y, mul2); o[7] = e4m3x4_pow2(x3.z, x3.w, mul2);
      } else {
        o[0] = nan4(x0.x, x0.y); o[1] = nan4(x0.z, x0.w);
        o[2] = nan4(x1.x, x1.y); o[3] = nan4(x1.z, x1.w);
        o[4] = nan4(x2.x, x2.y); o[5] = nan4(x2.z, x2.w);
        o[6] = nan4(x3.x, x3.y); o[7] = nan4(x3.z, x3.w);
      }
      uint8_t* dst = ro.codes + (row0 + r) * cols + col0 + 32 * b;
      if (wide) {
        st_global_v8(dst, o);
      } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
    if (kSwizzled)
      stile_r[(r & 31) * 16 + (r >> 5) * 4 + b] = valid ? static_cast<uint8_t>(s) : 0;
    else if (valid)
      ro.scales[(row0 + r) * s_cols + col0 / 32 + b] = static_cast<uint8_t>(s);
  }
}

// Column-wise copy (transpose) of a 128 x 128 tile staged in shared memory; the tile
// buffer is reused to stage the transposed codes, so it is dead once this returns.
template <bool kSwizzled>
__device__ __forceinline__ void col_pass_smem(uint16_t (*tile)[kTilePitch], uint8_t* stile_c,
                                              const QOut& co, int64_t rows, int64_t row0,
                                              int rows_valid, int64_t col0, int cols_valid,
                                              int rule) {
  const int t = threadIdx.x;
  // thread = column pair (2cp, 2cp+1) x token block j (32 rows); each word read holds
  // both columns of one row (column c in the low half)
  const int w = t >> 5, lane = t & 31;
  const int cp = (w & 1) * 32 + lane;
  const int j = w >> 1;
  const int c = 2 * cp;
  const bool valid = c < cols_valid && 32 * j < rows_valid;
  const uint32_t* colw = reinterpret_cast<const uint32_t*>(&tile[32 * j][c]);
  constexpr int kRowWords = kTilePitch / 2;
  uint32_t m01 = 0;  // both columns' block maxima, one per half
#pragma unroll
  for (int i = 0; i < 32; ++i) m01 = max_abs_bf16x2(m01, colw[i * kRowWords]);
  m01 &= kAbs2;
  const uint32_t s0 = scale_byte(m01 & 0xFFFFu, rule), s1 = scale_byte(m01 >> 16, rule);
  uint4 stage_o0[2], stage_o1[2];
  if (valid) {
    uint32_t o0[8], o1[8];
    if (__builtin_expect(s0 != 0xFFu && s1 != 0xFFu, 1)) {
      // each row word holds column c (low half) and c + 1 (high half): one packed product
      // scales both by their own block's 2^-e
      const uint32_t mulp = inv_scale_bf16(s0) | (inv_scale_bf16(s1) << 16);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t b0 = mul_bf16x2(colw[(4 * q) * kRowWords], mulp);
        const uint32_t b1 = mul_bf16x2(colw[(4 * q + 1) * kRowWords], mulp);
        const uint32_t b2 = mul_bf16x2(colw[(4 * q + 2) * kRowWords], mulp);
        const uint32_t b3 = mul_bf16x2(colw[(4 * q + 3) * kRowWords], mulp);
        o0[q] = e4m3x2_of(b0 << 16, b1 << 16) | (e4m3x2_of(b2 << 16, b3 << 16) << 16);
        o1[q] = e4m3x2_of(b0 & 0xFFFF0000u, b1 & 0xFFFF0000u) |
                (e4m3x2_of(b2 & 0xFFFF0000u, b3 & 0xFFFF0000u) << 16);
      }
    } else {  // a NaN/Inf block in either column (rare)
      const float mul0 = inv_scale(s0), mul1 = inv_scale(s1);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t a0 = colw[(4 * q) * kRowWords], a1 = colw[(4 * q + 1) * kRowWords];
        const uint32_t a2 = colw[(4 * q + 2) * kRowWords], a3 = colw[(4 * q + 3) * kRowWords];
        const uint32_t c0a = __byte_perm(a0, a1, 0x5410), c0b = __byte_perm(a2, a3, 0x5410);
        const uint32_t c1a = __byte_perm(a0, a1, 0x7632), c1b = __byte_perm(a2, a3, 0x7632);
        o0[q] = s0 == 0xFFu ? nan4(c0a, c0b) : e4m3x4(c0a, c0b, mul0);
        o1[q] = s1 == 0xFFu ? nan4(c1a, c1b) : e4m3x4(c1a, c1b, mul1);
      }
    }
    stage_o0[0] = make_uint4(o0[0], o0[1], o0[2], o0[3]);
    stage_o0[1] = make_uint4(o0[4], o0[5], o0[6], o0[7]);
    stage_o1[0] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
    stage_o1[1] = make_uint4(o1[4], o1[5], o1[6], o1[7]);
  }
  if (kSwizzled) {
    stile_c[(c & 31) * 16 + (c >> 5) * 4 + j] = valid ? static_cast<uint8_t>(s0) : 0;
    stile_c[((c + 1) & 31) * 16 + ((c + 1) >> 5) * 4 + j] = valid ? static_cast<uint8_t>(s1) : 0;
  } else if (valid) {
    const int64_t s_cols = rows / 32;
    co.scales[(col0 + c) * s_cols + row0 / 32 + j] = static_cast<uint8_t>(s0);
    co.scales[(col0 + c + 1) * s_cols + row0 / 32 + j] = static_cast<uint8_t>(s1);
  }
  // The transposed codes go through shared memory so that each output row's 128 bytes
  // leave in one coalesced piece: stage[row][chunk] holds 16-byte chunks, chunk index
  // XOR (row & 7) against bank conflicts; the BF16 tile buffer is reused once every
  // thread has read what it needs of it.
  __syncthreads();
  uint4* stage = reinterpret_cast<uint4*>(&tile[0][0]);
  if (valid) {
    stage[c * 8 + ((2 * j) ^ (c & 7))] = stage_o0[0];
    stage[c * 8 + ((2 * j + 1) ^ (c & 7))] = stage_o0[1];
    stage[(c + 1) * 8 + ((2 * j) ^ ((c + 1) & 7))] = stage_o1[0];
    stage[(c + 1) * 8 + ((2 * j + 1) ^ ((c + 1) & 7))] = stage_o1[1];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (t >> 3) + 32 * i;  // output row = tile column
    const int ch = t & 7;             // 16 tokens per chunk
    if (r < cols_valid && 16 * ch < rows_valid)
      *reinterpret_cast<uint4*>(co.codes + (col0 + r) * rows + row0 + 16 * ch) =
          stage[r * 8 + (ch ^ (r & 7))];
  }
}

}  // namespace mxfp8
