// swiglu.cu - the gated activation between a block's two projections, with its input kept in 8
// bits for the backward pass.
//
// "End-to-End MXFP8 RL on Blackwell" (verl blog post): gate_up_proj and down_proj are MXFP8
// layers (section "The grid, byte for byte"), and memory is what decides micro-batch sizes
// (section "A controlled sweep"). Kept as BF16 the activation's input takes 4 bytes for each
// value of h; kept as MXFP8 2.0625.
//
// x = [g | u], s = 1 / (1 + e^-g), h = g s u. The checkpoint is x on the MXFP8 grid, row-wise:
// the bytes of mxfp8_quantize_rule with linear scales. From its values g', u':
//   dg = dh u' s' (1 + g' (1 - s')),   du = dh g' s',   h' = g' s' u'
// in FP32, each rounded to BF16 once. e^-g is one ex2.approx (2^-22 relative) of g log2(e) in FP32,
// whose own rounding adds up to |g| 2^-24: 2^-17 at the far end of the range, where BF16 keeps
// 2^-9. Beyond it (s below 2^-126, g below -87.33) s is 0. A gate of -inf gives NaN (-inf * 0).
//
// Bound by memory: forward 4 bytes read and 2 + 2.0625 written for each value of h, backward
// 2 + 2.0625 read and 4 (with h' 6) written: 4096 x 12288 values of h take 59 us forward (6.9 TB/s),
// 61 backward and 76 with h' (6.7 TB/s). A thread holds 16 gates and the 16 ups beside them: half a
// block each, so a block's maximum takes one exchange between neighbours, and every access is 16
// or 32 bytes.

#include <cstdint>
#include <cuda_runtime.h>

#include "convert.cuh"
#include "device.cuh"
#include "internal.h"
#include "mxfp8.h"

namespace mxfp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;   // values of h a thread
constexpr unsigned kFull = 0xFFFFFFFFu;

struct SwigluParams {
  const uint16_t* x;
  const uint16_t* grad;
  int64_t rows, width;
  uint8_t* codes;
  uint8_t* scales;
  uint16_t* h;
  uint16_t* grad_x;
  int rule;
};

// 16 BF16 values: one 32-byte access where the address allows it, else two of 16.
template <bool kWide>
__device__ __forceinline__ void load16(const uint16_t* p, uint32_t (&w)[8]) {
  if constexpr (kWide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = ld_nc_v4(p), b = ld_nc_v4(p + 8);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}

// The same of memory that the kernel itself may overwrite: ordinary loads, since non-coherent ones
// need not stay before the stores to their addresses.
template <bool kWide>
__device__ __forceinline__ void load16_operand(const uint16_t* p, uint32_t (&w)[8]) {
  if constexpr (kWide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p) : "memory");
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}

template <bool kWide>
__device__ __forceinline__ void store16(uint16_t* p, const uint32_t (&w)[8]) {
  if constexpr (kWide) {
    st_global_v8(p, w);
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 1 / (1 + e^-g); 0 where e^-g passes FP32's range.
__device__ __forceinline__ float sigmoid(float g) {
  float t, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(g * -1.44269504088896341f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + t));
  return s;
}

__device__ __forceinline__ float silu_up(float g, float u) { return g * sigmoid(g) * u; }

// The place of a thread's values: `row`, and `c` of its row's width. False past the end (an even
// number of threads, so both halves of a block agree).
struct Place {
  int64_t row;
  int c;
  bool valid;
};

__device__ __forceinline__ Place place(int64_t rows, int64_t width) {
  const uint32_t per_row = static_cast<uint32_t>(width / kPer);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads;   // the same in the CTA
  const int64_t row0 = first / per_row;
  const uint32_t at = static_cast<uint32_t>(first - row0 * per_row) + threadIdx.x;
  Place q;
  q.row = row0 + at / per_row;
  q.c = static_cast<int>(at % per_row) * kPer;
  q.valid = q.row < rows;
  return q;
}

// Half a block's codes and scale: the maximum is the block's, shared with the other half.
__device__ __forceinline__ void keep_half(const uint32_t (&w)[8], uint8_t* codes, uint8_t* scale,
                                          int rule, bool valid) {
  uint32_t m2 = max_abs_bf16x2(
      max_abs_bf16x2(max_abs_bf16x2(w[0], w[1]), max_abs_bf16x2(w[2], w[3])),
      max_abs_bf16x2(max_abs_bf16x2(w[4], w[5]), max_abs_bf16x2(w[6], w[7])));
  m2 = max_abs_bf16x2(m2, __shfl_xor_sync(kFull, m2, 1)) & kAbs2;
  const uint32_t s = scale_byte(max(m2 & 0xFFFFu, m2 >> 16), rule);
  uint4 o;
  if (__builtin_expect(s != 0xFFu, 1)) {
    const uint32_t mul2 = inv_scale_bf16(s) * 0x10001u;
    o = make_uint4(e4m3x4_pow2(w[0], w[1], mul2), e4m3x4_pow2(w[2], w[3], mul2),
                   e4m3x4_pow2(w[4], w[5], mul2), e4m3x4_pow2(w[6], w[7], mul2));
  } else {
    o = make_uint4(nan4(w[0], w[1]), nan4(w[2], w[3]), nan4(w[4], w[5]), nan4(w[6], w[7]));
  }
  if (!valid) return;
  *reinterpret_cast<uint4*>(codes) = o;
  if (!(threadIdx.x & 1)) *scale = static_cast<uint8_t>(s);
}

template <bool kKeep, bool kWide>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const SwigluParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const Place q = place(p.rows, p.width);
  uint32_t g[8], u[8];
  const int64_t at = q.row * 2 * p.width + q.c;
  if (q.valid) {
    load16<kWide>(p.x + at, g);
    load16<kWide>(p.x + at + p.width, u);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = u[i] = 0;
  }
  if constexpr (kKeep) {
    const int64_t block = q.row * (p.width / 16) + q.c / 32;
    keep_half(g, p.codes + at, p.scales + block, p.rule, q.valid);
    keep_half(u, p.codes + at + p.width, p.scales + block + p.width / 32, p.rule, q.valid);
  }
  if (!q.valid) return;
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    h[i] = cvt_bf16x2(silu_up(hi(g[i]), hi(u[i])), silu_up(lo(g[i]), lo(u[i])));
  store16<kWide>(p.h + q.row * p.width + q.c, h);
}

// 2^(s - 127) of a scale byte; NaN for 0xFF.
__device__ __forceinline__ float scale_of(uint32_t s) {
  if (s == 0xFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(s ? s << 23 : 0x00400000u);
}

// Two E4M3 codes (the low 16 bits) as FP32, unscaled.
__device__ __forceinline__ void e4m3x2_values(uint32_t codes, float& a, float& b) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(codes)));
  asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(a), "=f"(b) : "r"(h2));
}

constexpr float kLargest = 3.402823466e38f;   // of FP32

// dg, du and h of a gate, an up and the gradient of h. kFar: where dh u passes FP32, dg need not, as
// its factor is small below zero. Then |dh| and |u| are 1 at least, so that u times the factor, which is
// 2^-126 at least or 0, loses nothing, and passes FP32 only where dg does.
template <bool kFar>
__device__ __forceinline__ void value_grads(float g, float u, float dh, float& dg, float& du,
                                            float& h) {
  const float s = sigmoid(g), silu = g * s;
  const float factor = s * fmaf(g, 1.f - s, 1.f), product = dh * u;
  const bool passed = kFar && fabsf(product) > kLargest && fabsf(dh) <= kLargest;
  dg = passed ? u * factor * dh : product * factor;
  du = dh * silu;
  h = silu * u;
}

// The largest number of FP32 for an infinity; NaN stays.
__device__ __forceinline__ float at_most_largest(float v) {
  asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(v) : "f"(kLargest));
  return v;
}

// A thread's results where one of them is an infinity or NaN, from its operands again, with kFar. Kept
// values past FP32 (the round-up rule keeps BF16 values of 1.9375 x 2^127 and more as 2^128) count as
// its largest number: as infinities they met factors of 0. Two values at a time: the registers are the
// kernel's to have (care in its own loop took 80 us in place of 75, with 51 registers in place of 48).
// Every thread comes here where every gradient is NaN: 296 us.
template <bool kAgain>
__device__ __forceinline__ void grads_again(const SwigluParams& p, const Place& q) {
  const int64_t at = q.row * 2 * p.width + q.c, h_at = q.row * p.width + q.c;
  const int64_t block = q.row * (p.width / 16) + q.c / 32;
  const float gs = scale_of(p.scales[block]), us = scale_of(p.scales[block + p.width / 32]);
#pragma unroll 1
  for (int i = 0; i < kPer; i += 2) {
    const uint32_t d = *reinterpret_cast<const uint32_t*>(p.grad + h_at + i);
    float g[2], u[2], a[2], b[2], c[2];
    e4m3x2_values(*reinterpret_cast<const uint16_t*>(p.codes + at + i), g[0], g[1]);
    e4m3x2_values(*reinterpret_cast<const uint16_t*>(p.codes + at + p.width + i), u[0], u[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      value_grads<true>(at_most_largest(g[j] * gs), at_most_largest(u[j] * us),
                        j ? hi(d) : lo(d), a[j], b[j], c[j]);
    *reinterpret_cast<uint32_t*>(p.grad_x + at + i) = cvt_bf16x2(a[1], a[0]);
    *reinterpret_cast<uint32_t*>(p.grad_x + at + p.width + i) = cvt_bf16x2(b[1], b[0]);
    if (kAgain) *reinterpret_cast<uint32_t*>(p.h + h_at + i) = cvt_bf16x2(c[1], c[0]);
  }
}

template <bool kAgain, bool kWide>
__global__ void __launch_bounds__(kThreads) swiglu_grad_kernel(const SwigluParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const Place q = place(p.rows, p.width);
  if (!q.valid) return;
  const int64_t at = q.row * 2 * p.width + q.c;
  const int64_t block = q.row * (p.width / 16) + q.c / 32;
  uint32_t d[8];
  if constexpr (kAgain) {   // h may stand in the gradient's place
    load16_operand<kWide>(p.grad + q.row * p.width + q.c, d);
  } else {
    load16<kWide>(p.grad + q.row * p.width + q.c, d);
  }
  const uint4 gc = ld_nc_v4(p.codes + at), uc = ld_nc_v4(p.codes + at + p.width);
  const float gs = scale_of(p.scales[block]), us = scale_of(p.scales[block + p.width / 32]);
  const uint32_t gw[4] = {gc.x, gc.y, gc.z, gc.w}, uw[4] = {uc.x, uc.y, uc.z, uc.w};
  uint32_t dg[8], du[8], h[8], top = 0;   // top: the results' largest magnitudes
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float g[2], u[2], a[2], b[2], c[2];
    e4m3x2_values(gw[i / 2] >> (16 * (i & 1)), g[0], g[1]);
    e4m3x2_values(uw[i / 2] >> (16 * (i & 1)), u[0], u[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      value_grads<false>(g[j] * gs, u[j] * us, j ? hi(d[i]) : lo(d[i]), a[j], b[j], c[j]);
    dg[i] = cvt_bf16x2(a[1], a[0]);
    du[i] = cvt_bf16x2(b[1], b[0]);
    top = max_abs_bf16x2(top, max_abs_bf16x2(dg[i], du[i]));
    if (kAgain) {
      h[i] = cvt_bf16x2(c[1], c[0]);
      top = max_abs_bf16x2(top, h[i]);
    }
  }
  top &= kAbs2;
  if (__builtin_expect(max(top & 0xFFFFu, top >> 16) >= 0x7F80u, 0)) {
    grads_again<kAgain>(p, q);
    return;
  }
  store16<kWide>(p.grad_x + at, dg);
  store16<kWide>(p.grad_x + at + p.width, du);
  if constexpr (kAgain) store16<kWide>(p.h + q.row * p.width + q.c, h);
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

cudaError_t launch(void (*k)(const SwigluParams), const SwigluArgs& a, cudaStream_t stream) {
  const int64_t threads = a.rows * (a.width / kPer);
  const int64_t ctas = (threads + kThreads - 1) / kThreads;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  cfg.numAttrs = pdl_attr(&attr[0]);
  const SwigluParams p{static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.grad),
                       a.rows, a.width, static_cast<uint8_t*>(a.codes),
                       static_cast<uint8_t*>(a.scales), static_cast<uint16_t*>(a.h),
                       static_cast<uint16_t*>(a.grad_x), a.rule};
  return cudaLaunchKernelEx(&cfg, k, p);
}

}  // namespace

// width % 32 == 0, so with 32-byte aligned buffers every half row starts on 32 bytes
cudaError_t launch_swiglu(const SwigluArgs& a, cudaStream_t stream) {
  if (a.rows == 0 || a.width == 0) return cudaSuccess;
  const bool wide = aligned32(a.x) && aligned32(a.h);
  auto k = a.codes ? (wide ? swiglu_kernel<true, true> : swiglu_kernel<true, false>)
                   : (wide ? swiglu_kernel<false, true> : swiglu_kernel<false, false>);
  return launch(k, a, stream);
}

cudaError_t launch_swiglu_grad(const SwigluArgs& a, cudaStream_t stream) {
  if (a.rows == 0 || a.width == 0) return cudaSuccess;
  const bool wide = aligned32(a.grad) && aligned32(a.grad_x) && (!a.h || aligned32(a.h));
  auto k = a.h ? (wide ? swiglu_grad_kernel<true, true> : swiglu_grad_kernel<true, false>)
               : (wide ? swiglu_grad_kernel<false, true> : swiglu_grad_kernel<false, false>);
  return launch(k, a, stream);
}

}  // namespace mxfp8
