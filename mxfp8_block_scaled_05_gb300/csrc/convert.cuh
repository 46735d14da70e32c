// convert.cuh - BF16 to MXFP8: block maxima, scale bytes and E4M3 codes of 32-element blocks,
// shared by the quantizers and by the kernels that write MXFP8 copies beside their results.
#pragma once

#include <cstdint>

#include "mxfp8.h"

namespace mxfp8 {

constexpr uint32_t kAbs2 = 0x7FFF7FFFu;  // clears both BF16 sign bits of a word

// Per-half maximum of |a| and |b| for two BF16 pairs, NaN winning over every number; the
// sign bits of the result are meaningless (cleared by kAbs2 once per block). Compared with
// clearing both signs and taking an unsigned 16-bit maximum this is one instruction instead
// of three. A BF16 subnormal amax gives scale byte 0 whether or not it is flushed here.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Per-half unsigned 16-bit maximum of two words: on sign-cleared BF16 bits, the exact
// maximum magnitude, subnormals included (the block-wise FP32 scale depends on it).
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Scale byte from the largest |BF16| bits of a block; 0xFF for a NaN/Inf block.
// Floor rule (OCP): floor(log2 amax) - 8 = biased exponent - 135, byte = E - 8.
// Round-up rule: one more when the mantissa of amax exceeds 1.75 (amax > 448 * 2^e), so
// that nothing saturates. Both clamp at byte 0 (e = -127).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits, int rule) {
  if (amax_bits >= 0x7F80u) return 0xFFu;
  int e = static_cast<int>(amax_bits >> 7) - 8;
  if (rule == MXFP8_RULE_CEIL) e += (amax_bits & 0x7Fu) > 0x60u;
  return e > 0 ? static_cast<uint32_t>(e) : 0u;
}

// 2^-e for scale byte s = e + 127, as an FP32 (a normal number for s <= 253; the 0xFF of a
// NaN/Inf block gives -Inf, whose products are discarded).
__device__ __forceinline__ float inv_scale(uint32_t s) {
  return __uint_as_float((254u - s) << 23);
}

// Two elements given as FP32 bit patterns (lo first in memory order) -> 2 bytes: each
// scaled by an IEEE single-precision product rounded to nearest (exact for a power-of-two
// scale), then one RNE-saturating E4M3 conversion of the pair. Two scalar products measured
// slightly faster than one packed mul.rn.f32x2 (whose operands must sit in a register pair).
__device__ __forceinline__ uint32_t e4m3x2_f32bits(uint32_t lo, uint32_t hi, float mul) {
  const float a = __fmul_rn(__uint_as_float(lo), mul);
  const float b = __fmul_rn(__uint_as_float(hi), mul);
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  return c;
}

// Two BF16 pairs (4 elements, memory order lo(w0), hi(w0), lo(w1), hi(w1)) -> 4 bytes.
// A BF16 value's FP32 bit pattern is its 16 bits shifted to the top half.
__device__ __forceinline__ uint32_t e4m3x4(uint32_t w0, uint32_t w1, float mul) {
  return e4m3x2_f32bits(w0 << 16, w0 & 0xFFFF0000u, mul) |
         (e4m3x2_f32bits(w1 << 16, w1 & 0xFFFF0000u, mul) << 16);
}

// The MXFP8 kernels scale by an exact power of two, so they can scale two BF16 values with
// one packed BF16 product (exact: the results lie in [2^-133, 2^9) or are far below E4M3's
// smallest subnormal, and BF16 keeps subnormals) before widening them for the conversion.
// The block-wise kernel's FP32 scale is not a power of two: it keeps the FP32 products.

// BF16 bits of 2^-e for scale byte s = e + 127 (a normal number for s <= 253; the 0xFF of a
// NaN/Inf block gives +Inf, whose products are discarded).
__device__ __forceinline__ uint32_t inv_scale_bf16(uint32_t s) { return ((254u - s) & 0xFFu) << 7; }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two values given as FP32 bit patterns (lo first in memory order) -> 2 bytes, one
// RNE-saturating E4M3 conversion of the pair.
__device__ __forceinline__ uint32_t e4m3x2_of(uint32_t lo, uint32_t hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(c) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
  return c;
}

// Two BF16 pairs (4 elements, memory order lo(w0), hi(w0), lo(w1), hi(w1)) scaled by the
// BF16 pair mul2 (2^-e in both halves) -> 4 bytes.
__device__ __forceinline__ uint32_t e4m3x4_pow2(uint32_t w0, uint32_t w1, uint32_t mul2) {
  const uint32_t v0 = mul_bf16x2(w0, mul2), v1 = mul_bf16x2(w1, mul2);
  return e4m3x2_of(v0 << 16, v0 & 0xFFFF0000u) | (e4m3x2_of(v1 << 16, v1 & 0xFFFF0000u) << 16);
}

// A BF16 pair times a pair of powers of two, widened to FP32 in one expression each. Exact; -0 is
// added, so that -0 stays -0. Where the pairs are a lane's neighbouring columns this is 1 to 2%
// faster than the packed product and two unpackings (a row copy of 69504 x 2048: 33.4 and 33.9
// us); where they are pairs of rows it makes no difference.
__device__ __forceinline__ void scale_bf16x2(uint32_t w, uint32_t mul2, float& lo, float& hi) {
  asm("{\n\t.reg .b16 a, b, m, n;\n\t"
      "mov.b32 {a, b}, %2;\n\tmov.b32 {m, n}, %3;\n\t"
      "fma.rn.f32.bf16 %0, a, m, %4;\n\tfma.rn.f32.bf16 %1, b, n, %4;\n\t}"
      : "=f"(lo), "=f"(hi) : "r"(w), "r"(mul2), "f"(-0.0f));
}

// Four FP32 values to 4 E4M3 codes, the first lowest.
__device__ __forceinline__ uint32_t e4m3x4_f32(float a, float b, float c, float d) {
  uint32_t o;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(o) : "f"(a), "f"(b), "f"(c), "f"(d));
  return o;
}

// 32 bytes global store in one instruction (the address must be 32-byte aligned).
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&o)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"l"(p), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]),
                 "r"(o[6]), "r"(o[7]) : "memory");
}

// The same 4 elements of a NaN/Inf block: 0x7F with each element's own sign. Blocks like
// this take a separate branch after the normal conversion, which stays free of selects.
__device__ __forceinline__ uint32_t nan4(uint32_t w0, uint32_t w1) {
  const uint32_t s0 = (w0 >> 8) & 0x80u, s1 = (w0 >> 24) & 0x80u;
  const uint32_t s2 = (w1 >> 8) & 0x80u, s3 = (w1 >> 24) & 0x80u;
  return (0x7Fu | s0) | ((0x7Fu | s1) << 8) | ((0x7Fu | s2) << 16) | ((0x7Fu | s3) << 24);
}

}  // namespace mxfp8
