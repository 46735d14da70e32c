// api.cu - the extern "C" boundary (include/mxfp8.h): argument checks, per-device
// set-up (architecture check, SM count, status word) and dispatch to the launchers.

#include <cstdint>
#include <cstdlib>
#include <atomic>
#include <mutex>

#include <cuda_runtime.h>

#include "internal.h"
#include "mxfp8.h"

namespace mxfp8 {

namespace {

// First error a kernel detected on this device since the host last read it.
__device__ int g_device_status;

// mxfp8_get_device_status takes the word with one atomic exchange on the device, so an
// error latched by a kernel on another stream is either taken by this read or left for the
// next one, never cleared unread. Each call gets its own slot for the taken value, so that
// calls from several host threads do not overwrite each other's result. Slots are handed out
// round robin, so only more than 64 reads in flight at once could share one.
constexpr unsigned kStatusSlots = 64;
__device__ int g_status_taken[kStatusSlots];
std::atomic<unsigned> g_status_slot{0};

__global__ void take_status_kernel(unsigned slot) {
  g_status_taken[slot] = atomicExch(&g_device_status, 0);
}

constexpr int kMaxDevices = 64;

struct DeviceState {
  // set up once per device under g_mu; `ready` is published last (release) and read first
  // (acquire), so a caller that sees it set also sees the fields below
  std::atomic<bool> ready{false};
  bool supported = false;
  int sms = 0;
  int* status = nullptr;
};

DeviceState g_dev[kMaxDevices];
std::mutex g_mu;

// Per-device set-up on first use: capability 10.3 (GB300) required, SM count cached,
// address of the status word looked up. Returns MXFP8_OK or an error code.
int device_state(DeviceState** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MXFP8_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return MXFP8_ERR_CUDA;
  DeviceState& d = g_dev[dev];
  if (!d.ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_mu);
    if (!d.ready.load(std::memory_order_relaxed)) {
      int major = 0, minor = 0, sms = 0;
      if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MXFP8_ERR_CUDA;
      d.supported = (major == 10 && minor == 3);
      d.sms = sms;
      if (d.supported) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return MXFP8_ERR_CUDA;
        d.status = static_cast<int*>(p);
      }
      d.ready.store(true, std::memory_order_release);
    }
  }
  if (!d.supported) return MXFP8_ERR_UNSUPPORTED_ARCH;
  *out = &d;
  return MXFP8_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// a * b * c into *out, false if the product leaves int64 (sizes of impossible tensors).
bool mul3(int64_t a, int64_t b, int64_t c, int64_t* out) {
  int64_t ab = 0;
  return !__builtin_mul_overflow(a, b, &ab) && !__builtin_mul_overflow(ab, c, out);
}

constexpr int64_t kMaxTokenTiles = 65535;  // grid.y limit of the quantizer launch
// grid.y limit of the self-check's reference kernel (32 tokens per CTA row)
constexpr int64_t kMaxSelfcheckTokens = int64_t(32) * 65535;

}  // namespace

int num_sms() {
  int dev = 0;
  cudaGetDevice(&dev);
  return (dev >= 0 && dev < kMaxDevices && g_dev[dev].sms > 0) ? g_dev[dev].sms : 148;
}

int64_t scale_bytes_host(int64_t rows, int64_t cols, int axis, int layout) {
  if (rows < 0 || cols < 0 || rows > INT64_MAX - 127 || cols > INT64_MAX - 127) return -1;
  int64_t s_rows, s_cols;
  if (axis == MXFP8_AXIS_ROW) {
    if (cols % 32) return -1;
    s_rows = rows;
    s_cols = cols / 32;
  } else if (axis == MXFP8_AXIS_COL) {
    if (rows % 32) return -1;
    s_rows = cols;
    s_cols = rows / 32;
  } else {
    return -1;
  }
  int64_t bytes = 0;
  if (layout == MXFP8_SCALES_LINEAR) return mul3(s_rows, s_cols, 1, &bytes) ? bytes : -1;
  if (layout == MXFP8_SCALES_SWIZZLED) {
    if (s_rows == 0 || s_cols == 0) return 0;
    return mul3(cdiv(s_rows, 128), cdiv(s_cols, 4), 512, &bytes) ? bytes : -1;
  }
  return -1;
}

}  // namespace mxfp8

using namespace mxfp8;

extern "C" {

int mxfp8_version(void) { return MXFP8_ABI_VERSION; }

const char* mxfp8_status_string(int status) {
  switch (status) {
    case MXFP8_OK: return "ok";
    case MXFP8_ERR_INVALID_ARG: return "invalid argument";
    case MXFP8_ERR_ALIGNMENT: return "alignment: blocked dim not a multiple of 32 or pointer not 16-byte aligned";
    case MXFP8_ERR_UNSUPPORTED_ARCH: return "unsupported device (needs compute capability 10.3, sm_103a)";
    case MXFP8_ERR_CUDA: return "CUDA call failed";
    case MXFP8_ERR_BAD_OFFSETS: return "expert offsets invalid (must be 0-based, non-decreasing, 32-aligned, end at total_rows)";
    case MXFP8_ERR_BAD_TARGET: return "a target or alternative token is at or past the vocabulary";
    case MXFP8_ERR_BAD_EXPERT: return "an expert id is at or past the number of experts";
    case MXFP8_ERR_TIMEOUT: return "a kernel pipeline wait timed out; its work was abandoned";
    default: return "unknown status";
  }
}

size_t mxfp8_scale_bytes(int64_t rows, int64_t cols, int axis, int scale_layout) {
  const int64_t b = scale_bytes_host(rows, cols, axis, scale_layout);
  return b < 0 ? 0 : static_cast<size_t>(b);
}

size_t mxfp8_grouped_scale_bytes(int64_t total_rows, int64_t cols, int num_experts, int axis) {
  if (total_rows < 0 || cols <= 0 || num_experts <= 0 || total_rows % 32) return 0;
  if (total_rows > INT64_MAX - 127) return 0;
  int64_t bytes = 0;
  const int64_t tiles = cdiv(total_rows, 128) + num_experts;  // bound on sum of ceil(count / 128)
  if (axis == MXFP8_AXIS_ROW) {
    if (cols % 32) return 0;
    return mul3(tiles, cdiv(cols / 32, 4), 512, &bytes) ? static_cast<size_t>(bytes) : 0;
  }
  if (axis == MXFP8_AXIS_COL)
    return mul3(cdiv(cols, 128), tiles, 512, &bytes) ? static_cast<size_t>(bytes) : 0;
  return 0;
}

// axis: MXFP8_AXIS_ROW, MXFP8_AXIS_COL or kAxisBoth (out/scales = row-wise copy,
// out2/scales2 = column-wise copy).
static int quantize_common(const void* src, int64_t batch, int64_t rows, int64_t cols, int axis,
                           void* out, void* scales, void* out2, void* scales2, int layout,
                           const int32_t* offsets, int E, void* stream,
                           int rule = MXFP8_RULE_FLOOR) {
  if (rule != MXFP8_RULE_FLOOR && rule != MXFP8_RULE_CEIL) return MXFP8_ERR_INVALID_ARG;
  if (batch < 0 || rows < 0 || cols < 0) return MXFP8_ERR_INVALID_ARG;
  if (axis != MXFP8_AXIS_ROW && axis != MXFP8_AXIS_COL && axis != kAxisBoth)
    return MXFP8_ERR_INVALID_ARG;
  if (layout != MXFP8_SCALES_LINEAR && layout != MXFP8_SCALES_SWIZZLED)
    return MXFP8_ERR_INVALID_ARG;
  const bool row = axis != MXFP8_AXIS_COL, col = axis != MXFP8_AXIS_ROW;
  if (row && cols % 32) return MXFP8_ERR_ALIGNMENT;
  if (col && (rows % 32 || cols % 8)) return MXFP8_ERR_ALIGNMENT;
  if (batch == 0 || rows == 0 || cols == 0) return MXFP8_OK;
  int64_t elems = 0;  // BF16 input bytes = 2 * elems; the kernels index in int64
  if (!mul3(batch, rows, cols, &elems) || elems > INT64_MAX / 2) return MXFP8_ERR_INVALID_ARG;
  if (!src || !out || !scales) return MXFP8_ERR_INVALID_ARG;
  if (axis == kAxisBoth && (!out2 || !scales2)) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(src) || !aligned16(out) || (out2 && !aligned16(out2)))
    return MXFP8_ERR_ALIGNMENT;
  if (layout == MXFP8_SCALES_SWIZZLED && (!aligned16(scales) || (scales2 && !aligned16(scales2))))
    return MXFP8_ERR_ALIGNMENT;
  if (batch > 65535) return MXFP8_ERR_INVALID_ARG;
  const int64_t token_tiles = cdiv(rows, 128) + (offsets ? E : 0);
  if (token_tiles > kMaxTokenTiles || cdiv(cols, 128) > 0x7FFFFFFF) return MXFP8_ERR_INVALID_ARG;
  DeviceState* d = nullptr;
  const int st = device_state(&d);
  if (st != MXFP8_OK) return st;
  QuantizeArgs a{};
  a.src = src;
  a.batch = batch;
  a.rows = rows;
  a.cols = cols;
  a.axis = axis;
  a.layout = layout;
  a.offsets = offsets;
  a.num_experts = E;
  a.rule = rule;
  a.status = d->status;
  if (row) {
    a.out = out;
    a.scales = scales;
    a.scale_item_bytes = scale_bytes_host(rows, cols, MXFP8_AXIS_ROW, layout);
  }
  if (col) {
    a.out_col = axis == kAxisBoth ? out2 : out;
    a.scales_col = axis == kAxisBoth ? scales2 : scales;
    a.scale_item_bytes_col = scale_bytes_host(rows, cols, MXFP8_AXIS_COL, layout);
  }
  return launch_quantize(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MXFP8_OK
                                                                               : MXFP8_ERR_CUDA;
}

int mxfp8_quantize(const void* src_dev, int64_t rows, int64_t cols, int axis, void* out_dev,
                   void* scales_dev, int scale_layout, void* stream) {
  if (axis != MXFP8_AXIS_ROW && axis != MXFP8_AXIS_COL) return MXFP8_ERR_INVALID_ARG;
  return quantize_common(src_dev, 1, rows, cols, axis, out_dev, scales_dev, nullptr, nullptr,
                         scale_layout, nullptr, 0, stream);
}

int mxfp8_quantize_rule(const void* src_dev, int64_t rows, int64_t cols, int axis,
                        void* out_dev, void* scales_dev, int scale_layout, int scale_rule,
                        void* stream) {
  if (axis != MXFP8_AXIS_ROW && axis != MXFP8_AXIS_COL) return MXFP8_ERR_INVALID_ARG;
  return quantize_common(src_dev, 1, rows, cols, axis, out_dev, scales_dev, nullptr, nullptr,
                         scale_layout, nullptr, 0, stream, scale_rule);
}

int mxfp8_quantize_dual(const void* src_dev, int64_t rows, int64_t cols, void* row_out_dev,
                        void* row_scales_dev, void* col_out_dev, void* col_scales_dev,
                        int scale_layout, void* stream) {
  return quantize_common(src_dev, 1, rows, cols, kAxisBoth, row_out_dev, row_scales_dev,
                         col_out_dev, col_scales_dev, scale_layout, nullptr, 0, stream);
}

int mxfp8_quantize_dual_multi(const mxfp8_dual_job* jobs, int num_jobs, int scale_layout,
                              void* stream) {
  if (!jobs || num_jobs < 1 || num_jobs > MXFP8_MAX_DUAL_JOBS) return MXFP8_ERR_INVALID_ARG;
  if (scale_layout != MXFP8_SCALES_LINEAR && scale_layout != MXFP8_SCALES_SWIZZLED)
    return MXFP8_ERR_INVALID_ARG;
  static_assert(MXFP8_MAX_DUAL_JOBS <= kMaxQuantizeJobs, "job table too small");
  QuantizeJobs q{};
  q.n = num_jobs;
  q.layout = scale_layout;
  int64_t tiles = 0;
  for (int i = 0; i < num_jobs; ++i) {
    const mxfp8_dual_job& j = jobs[i];
    // the same checks as mxfp8_quantize_dual
    if (j.rows < 0 || j.cols < 0) return MXFP8_ERR_INVALID_ARG;
    if (j.rows % 32 || j.cols % 32) return MXFP8_ERR_ALIGNMENT;
    if (j.rows == 0 || j.cols == 0) continue;
    if (!j.src || !j.row_out || !j.row_scales || !j.col_out || !j.col_scales)
      return MXFP8_ERR_INVALID_ARG;
    if (!aligned16(j.src) || !aligned16(j.row_out) || !aligned16(j.col_out))
      return MXFP8_ERR_ALIGNMENT;
    if (scale_layout == MXFP8_SCALES_SWIZZLED &&
        (!aligned16(j.row_scales) || !aligned16(j.col_scales)))
      return MXFP8_ERR_ALIGNMENT;
    if (cdiv(j.rows, 128) > kMaxTokenTiles || cdiv(j.cols, 128) > 0x7FFFFFFF)
      return MXFP8_ERR_INVALID_ARG;
    tiles += cdiv(j.rows, 128) * cdiv(j.cols, 128);
    q.src[i] = j.src;
    q.rows[i] = j.rows;
    q.cols[i] = j.cols;
    q.out[i] = j.row_out;
    q.scales[i] = j.row_scales;
    q.out_col[i] = j.col_out;
    q.scales_col[i] = j.col_scales;
  }
  if (tiles > 0x7FFFFFFF) return MXFP8_ERR_INVALID_ARG;
  if (tiles == 0) return MXFP8_OK;
  DeviceState* d = nullptr;
  const int st = device_state(&d);
  if (st != MXFP8_OK) return st;
  q.status = d->status;
  return launch_quantize_jobs(q, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MXFP8_OK
             : MXFP8_ERR_CUDA;
}

size_t mxfp8_blockwise_scale_count(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || cols % 8) return 0;
  if (rows > INT64_MAX - 127 || cols > INT64_MAX - 127) return 0;
  int64_t n = 0;
  return mul3(cdiv(rows, 128), cdiv(cols, 128), 1, &n) ? static_cast<size_t>(n) : 0;
}

int mxfp8_quantize_blockwise(const void* src_dev, int64_t rows, int64_t cols, void* out_dev,
                             float* scale_inv_dev, int scale_type, void* stream) {
  if (scale_type != MXFP8_BW_SCALE_FP32 && scale_type != MXFP8_BW_SCALE_POW2)
    return MXFP8_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0) return MXFP8_ERR_INVALID_ARG;
  if (cols % 8) return MXFP8_ERR_ALIGNMENT;
  if (rows == 0 || cols == 0) return MXFP8_OK;
  if (!src_dev || !out_dev || !scale_inv_dev) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(src_dev) || !aligned16(out_dev) ||
      (reinterpret_cast<uintptr_t>(scale_inv_dev) & 3u))
    return MXFP8_ERR_ALIGNMENT;
  if (cdiv(rows, 128) > 65535 || cdiv(cols, 128) > 0x7FFFFFFF) return MXFP8_ERR_INVALID_ARG;
  DeviceState* d = nullptr;
  const int st = device_state(&d);
  if (st != MXFP8_OK) return st;
  return launch_blockwise(src_dev, rows, cols, out_dev, scale_inv_dev,
                          scale_type == MXFP8_BW_SCALE_POW2,
                          static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MXFP8_OK
             : MXFP8_ERR_CUDA;
}

static int blockwise_1d(const void* src, int64_t rows, int64_t cols, void* row_out,
                        float* row_inv, void* col_out, float* col_inv, bool row, bool col,
                        bool two_d, int scale_type, void* stream) {
  if (scale_type != MXFP8_BW_SCALE_FP32 && scale_type != MXFP8_BW_SCALE_POW2)
    return MXFP8_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0) return MXFP8_ERR_INVALID_ARG;
  if (cols % (row ? 16 : 8) || (two_d && rows % 16)) return MXFP8_ERR_ALIGNMENT;
  if (rows == 0 || cols == 0) return MXFP8_OK;
  if (!src || (row && (!row_out || !row_inv)) || (col && (!col_out || !col_inv)))
    return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(src) || (row && !aligned16(row_out)) || (col && !aligned16(col_out)) ||
      (row && !aligned4(row_inv)) || (col && !aligned4(col_inv)))
    return MXFP8_ERR_ALIGNMENT;
  if (cdiv(rows, 128) > kMaxTokenTiles || cols > 0x7FFFFF00) return MXFP8_ERR_INVALID_ARG;
  DeviceState* d = nullptr;
  const int st = device_state(&d);
  if (st != MXFP8_OK) return st;
  const BlockwiseArgs a{src, rows, cols, row ? row_out : nullptr, row_inv,
                        col ? col_out : nullptr, col_inv, two_d,
                        scale_type == MXFP8_BW_SCALE_POW2};
  return launch_blockwise_tiles(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MXFP8_OK
             : MXFP8_ERR_CUDA;
}

int mxfp8_quantize_blockwise_1d(const void* src_dev, int64_t rows, int64_t cols, int axis,
                                void* out_dev, float* scale_inv_dev, int scale_type,
                                void* stream) {
  if (axis != MXFP8_AXIS_ROW && axis != MXFP8_AXIS_COL) return MXFP8_ERR_INVALID_ARG;
  const bool row = axis == MXFP8_AXIS_ROW;
  return blockwise_1d(src_dev, rows, cols, out_dev, scale_inv_dev, out_dev, scale_inv_dev, row,
                      !row, false, scale_type, stream);
}

int mxfp8_quantize_blockwise_1d_dual(const void* src_dev, int64_t rows, int64_t cols,
                                     void* row_out_dev, float* row_scale_inv_dev,
                                     void* col_out_dev, float* col_scale_inv_dev,
                                     int scale_type, void* stream) {
  return blockwise_1d(src_dev, rows, cols, row_out_dev, row_scale_inv_dev, col_out_dev,
                      col_scale_inv_dev, true, true, false, scale_type, stream);
}

int mxfp8_quantize_blockwise_dual(const void* src_dev, int64_t rows, int64_t cols,
                                  void* out_dev, float* scale_inv_dev, void* out_t_dev,
                                  float* scale_inv_t_dev, int scale_type, void* stream) {
  return blockwise_1d(src_dev, rows, cols, out_dev, scale_inv_dev, out_t_dev, scale_inv_t_dev,
                      true, true, true, scale_type, stream);
}

int mxfp8_quantize_batched(const void* src_dev, int64_t batch, int64_t rows, int64_t cols,
                           int axis, void* out_dev, void* scales_dev, int scale_layout,
                           void* stream) {
  if (axis != MXFP8_AXIS_ROW && axis != MXFP8_AXIS_COL) return MXFP8_ERR_INVALID_ARG;
  return quantize_common(src_dev, batch, rows, cols, axis, out_dev, scales_dev, nullptr, nullptr,
                         scale_layout, nullptr, 0, stream);
}

int mxfp8_quantize_grouped(const void* src_dev, int64_t total_rows, int64_t cols, int axis,
                           const int32_t* expert_offsets_dev, int num_experts, void* out_dev,
                           void* scales_dev, void* stream) {
  if (num_experts <= 0 || num_experts > 1024 || !expert_offsets_dev) return MXFP8_ERR_INVALID_ARG;
  if (axis != MXFP8_AXIS_ROW && axis != MXFP8_AXIS_COL) return MXFP8_ERR_INVALID_ARG;
  if (total_rows % 32) return MXFP8_ERR_ALIGNMENT;
  return quantize_common(src_dev, 1, total_rows, cols, axis, out_dev, scales_dev, nullptr,
                         nullptr, MXFP8_SCALES_SWIZZLED, expert_offsets_dev, num_experts, stream);
}

int mxfp8_quantize_grouped_dual(const void* src_dev, int64_t total_rows, int64_t cols,
                                const int32_t* expert_offsets_dev, int num_experts,
                                void* row_out_dev, void* row_scales_dev, void* col_out_dev,
                                void* col_scales_dev, void* stream) {
  if (num_experts <= 0 || num_experts > 1024 || !expert_offsets_dev) return MXFP8_ERR_INVALID_ARG;
  if (total_rows % 32) return MXFP8_ERR_ALIGNMENT;
  return quantize_common(src_dev, 1, total_rows, cols, kAxisBoth, row_out_dev, row_scales_dev,
                         col_out_dev, col_scales_dev, MXFP8_SCALES_SWIZZLED, expert_offsets_dev,
                         num_experts, stream);
}

// C = 0 for a reduction over nothing (K = 0, or no tokens for a grouped wgrad): `elems`
// output elements zero-filled on the stream; C must be valid and 16-byte aligned.
static int zero_fill_output(void* C, int64_t elems, int out_dtype, void* stream) {
  if (!C) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(C)) return MXFP8_ERR_ALIGNMENT;
  int64_t bytes = 0;
  if (!mul3(elems, out_dtype == MXFP8_OUT_FP32 ? 4 : 2, 1, &bytes)) return MXFP8_ERR_INVALID_ARG;
  DeviceState* d = nullptr;
  const int st = device_state(&d);
  if (st != MXFP8_OK) return st;
  return cudaMemsetAsync(C, 0, static_cast<size_t>(bytes), static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? MXFP8_OK
             : MXFP8_ERR_CUDA;
}

static int gemm_checks(const void* A, const void* sA, const void* B, const void* sB, void* C,
                       int op, int out_dtype) {
  if (!A || !sA || !B || !sB || !C) return MXFP8_ERR_INVALID_ARG;
  if (op < MXFP8_OP_FPROP || op > MXFP8_OP_WGRAD) return MXFP8_ERR_INVALID_ARG;
  if (out_dtype != MXFP8_OUT_BF16 && out_dtype != MXFP8_OUT_FP32) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(sA) || !aligned16(B) || !aligned16(sB) || !aligned16(C))
    return MXFP8_ERR_ALIGNMENT;
  return MXFP8_OK;
}

int mxfp8_gemm(const void* A_dev, const void* sA_dev, const void* B_dev, const void* sB_dev,
               void* C_dev, int64_t M, int64_t N, int64_t K, int op, int out_dtype,
               void* stream) {
  return mxfp8_gemm_ws(A_dev, sA_dev, B_dev, sB_dev, C_dev, M, N, K, op, out_dtype, nullptr,
                       0, stream);
}

size_t mxfp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int op, int out_dtype) {
  if (M <= 0 || N <= 0 || K <= 0 || M > 0x7FFFFF00 || N > 0x7FFFFF00 || K > 0x7FFFFF00)
    return 0;
  if (op < MXFP8_OP_FPROP || op > MXFP8_OP_WGRAD) return 0;
  if (out_dtype != MXFP8_OUT_BF16 && out_dtype != MXFP8_OUT_FP32) return 0;
  DeviceState* d = nullptr;
  if (device_state(&d) != MXFP8_OK) return 0;
  return gemm_workspace_bytes(M, N, K, out_dtype);
}

int mxfp8_gemm_ws(const void* A_dev, const void* sA_dev, const void* B_dev, const void* sB_dev,
                  void* C_dev, int64_t M, int64_t N, int64_t K, int op, int out_dtype,
                  void* workspace_dev, size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0) return MXFP8_ERR_INVALID_ARG;
  if (M > 0x7FFFFF00 || N > 0x7FFFFF00 || K > 0x7FFFFF00) return MXFP8_ERR_INVALID_ARG;
  if (K % 32 || M % 16 || N % 16) return MXFP8_ERR_ALIGNMENT;
  if (op < MXFP8_OP_FPROP || op > MXFP8_OP_WGRAD) return MXFP8_ERR_INVALID_ARG;
  if (out_dtype != MXFP8_OUT_BF16 && out_dtype != MXFP8_OUT_FP32) return MXFP8_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return MXFP8_OK;  // an empty output: nothing to read or write
  if (K == 0) return zero_fill_output(C_dev, M * N, out_dtype, stream);  // the empty sum
  int st = gemm_checks(A_dev, sA_dev, B_dev, sB_dev, C_dev, op, out_dtype);
  if (st != MXFP8_OK) return st;
  if (workspace_dev && (reinterpret_cast<uintptr_t>(workspace_dev) & 31))
    return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  GemmArgs a{A_dev, sA_dev, B_dev, sB_dev, C_dev, M, N, K, op, out_dtype, nullptr, 0, 0,
             d->status, workspace_dev, workspace_dev ? workspace_bytes : 0};
  return launch_gemm(a, static_cast<cudaStream_t>(stream));
}

int mxfp8_blockwise_gemm(const void* A_dev, const float* sA_dev, const void* B_dev,
                         const float* sB_dev, void* C_dev, int64_t M, int64_t N, int64_t K,
                         int op, int out_dtype, void* stream) {
  return mxfp8_blockwise_gemm_ws(A_dev, sA_dev, B_dev, sB_dev, C_dev, M, N, K, op, out_dtype,
                                 nullptr, 0, stream);
}

size_t mxfp8_blockwise_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int out_dtype) {
  if (M <= 0 || N <= 0 || K <= 0 || M > 0x7FFFFF00 || N > 0x7FFFFF00 || K > 0x7FFFFF00)
    return 0;
  if (out_dtype != MXFP8_OUT_BF16 && out_dtype != MXFP8_OUT_FP32) return 0;
  DeviceState* d = nullptr;
  if (device_state(&d) != MXFP8_OK) return 0;
  return static_cast<size_t>(
      blockwise_gemm_workspace_bytes(M, N, K, out_dtype == MXFP8_OUT_FP32));
}

int mxfp8_blockwise_gemm_ws(const void* A_dev, const float* sA_dev, const void* B_dev,
                            const float* sB_dev, void* C_dev, int64_t M, int64_t N, int64_t K,
                            int op, int out_dtype, void* workspace_dev, size_t workspace_bytes,
                            void* stream) {
  if (M < 0 || N < 0 || K < 0) return MXFP8_ERR_INVALID_ARG;
  if (M > 0x7FFFFF00 || N > 0x7FFFFF00 || K > 0x7FFFFF00) return MXFP8_ERR_INVALID_ARG;
  if (K % 16 || N % 8) return MXFP8_ERR_ALIGNMENT;
  if (op < MXFP8_OP_FPROP || op > MXFP8_OP_WGRAD) return MXFP8_ERR_INVALID_ARG;
  if (out_dtype != MXFP8_OUT_BF16 && out_dtype != MXFP8_OUT_FP32) return MXFP8_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return MXFP8_OK;
  if (K == 0) return zero_fill_output(C_dev, M * N, out_dtype, stream);
  if (!A_dev || !sA_dev || !B_dev || !sB_dev || !C_dev) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(A_dev) || !aligned16(B_dev) || !aligned16(C_dev) || !aligned4(sA_dev) ||
      !aligned4(sB_dev))
    return MXFP8_ERR_ALIGNMENT;
  if (workspace_dev && !aligned16(workspace_dev)) return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  const int st = device_state(&d);
  if (st != MXFP8_OK) return st;
  const BlockwiseGemmArgs a{A_dev, sA_dev, B_dev, sB_dev, C_dev, M, N, K,
                            op == MXFP8_OP_WGRAD, out_dtype == MXFP8_OUT_FP32, d->status,
                            workspace_dev, workspace_dev ? workspace_bytes : 0};
  return launch_blockwise_gemm(a, static_cast<cudaStream_t>(stream));
}

int mxfp8_grouped_gemm(const void* A_dev, const void* sA_dev, const void* B_dev,
                       const void* sB_dev, void* C_dev, const int32_t* expert_offsets_dev,
                       int num_experts, int64_t total_rows, int64_t N, int64_t K, int op,
                       int out_dtype, void* stream) {
  if (num_experts <= 0 || num_experts > 1024 || !expert_offsets_dev) return MXFP8_ERR_INVALID_ARG;
  if (total_rows < 0 || N < 0 || K < 0) return MXFP8_ERR_INVALID_ARG;
  if (total_rows > 0x7FFFFF00 || N > 0x7FFFFF00 || K > 0x7FFFFF00) return MXFP8_ERR_INVALID_ARG;
  if (total_rows % 32 || K % 32 || N % 16) return MXFP8_ERR_ALIGNMENT;
  if (op < MXFP8_OP_FPROP || op > MXFP8_OP_WGRAD) return MXFP8_ERR_INVALID_ARG;
  if (out_dtype != MXFP8_OUT_BF16 && out_dtype != MXFP8_OUT_FP32) return MXFP8_ERR_INVALID_ARG;
  // Empty cases read no operand, so A, B and their scales may then be empty (NULL), and the
  // offsets are not read: an empty output (N = 0, K = 0 for wgrad, no tokens for fprop and
  // dgrad) is a no-op; a reduction over nothing (no tokens for wgrad, K = 0 for fprop and
  // dgrad) zero-fills C.
  const bool wgrad = op == MXFP8_OP_WGRAD;
  if (N == 0 || (wgrad ? K == 0 : total_rows == 0)) return MXFP8_OK;
  if (wgrad && total_rows == 0) {
    int64_t elems = 0;
    if (!mul3(N, K, num_experts, &elems)) return MXFP8_ERR_INVALID_ARG;
    return zero_fill_output(C_dev, elems, out_dtype, stream);
  }
  if (!wgrad && K == 0) return zero_fill_output(C_dev, total_rows * N, out_dtype, stream);
  int st = gemm_checks(A_dev, sA_dev, B_dev, sB_dev, C_dev, op, out_dtype);
  if (st != MXFP8_OK) return st;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  GemmArgs a{A_dev, sA_dev, B_dev, sB_dev, C_dev, 0, N, K, op, out_dtype,
             expert_offsets_dev, num_experts, total_rows, d->status};
  return launch_grouped_gemm(a, static_cast<cudaStream_t>(stream));
}

size_t mxfp8_selfcheck_workspace_bytes(int64_t tokens, int64_t N, int64_t K) {
  if (tokens <= 0 || N <= 0 || K <= 0 || K % 32 || N % 16 || tokens % 16) return 0;
  const int64_t b = selfcheck_workspace_bytes(tokens, N, K);
  return b < 0 ? 0 : static_cast<size_t>(b);
}

int mxfp8_selfcheck(const void* w_codes_dev, const void* w_scales_dev,
                    const void* ref_codes_dev, const void* ref_scales_dev, int64_t N, int64_t K,
                    const void* x_bf16_dev, int64_t tokens, void* workspace_dev,
                    size_t workspace_bytes, float* rel_err_dev, void* stream) {
  if (!w_codes_dev || !w_scales_dev || !ref_codes_dev || !ref_scales_dev || !x_bf16_dev ||
      !workspace_dev || !rel_err_dev)
    return MXFP8_ERR_INVALID_ARG;
  if (tokens <= 0 || N <= 0 || K <= 0) return MXFP8_ERR_INVALID_ARG;
  if (K % 32 || N % 16 || tokens % 16) return MXFP8_ERR_ALIGNMENT;
  if (tokens > 0x7FFFFF00 || N > 0x7FFFFF00 || K > 0x7FFFFF00) return MXFP8_ERR_INVALID_ARG;
  if (tokens > kMaxSelfcheckTokens) return MXFP8_ERR_INVALID_ARG;
  const int64_t need = selfcheck_workspace_bytes(tokens, N, K);
  if (need < 0 || workspace_bytes < static_cast<size_t>(need)) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(w_codes_dev) || !aligned16(w_scales_dev) || !aligned16(x_bf16_dev) ||
      (reinterpret_cast<uintptr_t>(workspace_dev) & 255u) ||
      (reinterpret_cast<uintptr_t>(rel_err_dev) & 3u))
    return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  const int st = device_state(&d);
  if (st != MXFP8_OK) return st;
  SelfcheckArgs a{w_codes_dev, w_scales_dev, ref_codes_dev, ref_scales_dev, N, K, x_bf16_dev,
                  tokens, workspace_dev, rel_err_dev, d->status};
  return launch_selfcheck(a, static_cast<cudaStream_t>(stream));
}

int mxfp8_selfcheck_noalloc(const void* w_codes_dev, const void* w_scales_dev,
                            const void* ref_codes_dev, const void* ref_scales_dev, int64_t N,
                            int64_t K, const void* x_bf16_dev, int64_t tokens,
                            float* rel_err_dev, void* stream) {
  if (!w_codes_dev || !w_scales_dev || !ref_codes_dev || !ref_scales_dev || !x_bf16_dev ||
      !rel_err_dev)
    return MXFP8_ERR_INVALID_ARG;
  if (tokens <= 0 || N <= 0 || K <= 0) return MXFP8_ERR_INVALID_ARG;
  if (K % 32 || N % 16 || tokens % 16) return MXFP8_ERR_ALIGNMENT;
  if (tokens > 0x7FFFFF00 || N > 0x7FFFFF00 || K > 0x7FFFFF00) return MXFP8_ERR_INVALID_ARG;
  if (tokens > kMaxSelfcheckTokens) return MXFP8_ERR_INVALID_ARG;
  const int64_t need = selfcheck_workspace_bytes(tokens, N, K);
  if (need < 0 || need > kSelfcheckNoallocMaxBytes) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(w_codes_dev) || !aligned16(w_scales_dev) || !aligned16(x_bf16_dev) ||
      (reinterpret_cast<uintptr_t>(rel_err_dev) & 3u))
    return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  int st = device_state(&d);
  if (st != MXFP8_OK) return st;
  void* ws = nullptr;
  st = selfcheck_noalloc_workspace(&ws);
  if (st != MXFP8_OK) return st;
  SelfcheckArgs a{w_codes_dev, w_scales_dev, ref_codes_dev, ref_scales_dev, N, K, x_bf16_dev,
                  tokens, ws, rel_err_dev, d->status};
  return launch_selfcheck(a, static_cast<cudaStream_t>(stream));
}

// Checks that both log probability calls share; *inv_t gets 1 / temperature.
static int logprob_checks(int dtype, int64_t rows, int64_t vocab, int64_t ld,
                          double temperature, int top, float* inv_t) {
  if (dtype != MXFP8_OUT_BF16 && dtype != MXFP8_OUT_FP32) return MXFP8_ERR_INVALID_ARG;
  if (rows < 0 || vocab <= 0 || vocab > 0x7FFFFFFF || ld < vocab) return MXFP8_ERR_INVALID_ARG;
  if (top < 0 || top > MXFP8_MAX_TOP) return MXFP8_ERR_INVALID_ARG;
  int64_t bytes = 0;
  if (!mul3(rows, ld, 4, &bytes)) return MXFP8_ERR_INVALID_ARG;
  if (!(temperature > 0)) return MXFP8_ERR_INVALID_ARG;  // NaN too
  const double inv = 1.0 / temperature;
  if (!(inv >= 1.2e-38 && inv <= 2.0e38)) return MXFP8_ERR_INVALID_ARG;  // log2(e) / T fits too
  *inv_t = static_cast<float>(inv);
  return MXFP8_OK;
}

int mxfp8_token_logprobs(const void* logits_dev, int logits_dtype, int64_t rows,
                         int64_t vocab, int64_t ld, const int64_t* targets_dev,
                         double temperature, float* logprob_dev, float* entropy_dev,
                         float* stats_dev, int top, float* top_logprob_dev,
                         int64_t* top_id_dev, void* stream) {
  float inv_t = 0.f;
  int st = logprob_checks(logits_dtype, rows, vocab, ld, temperature, top, &inv_t);
  if (st != MXFP8_OK) return st;
  if (rows == 0) return MXFP8_OK;
  if (!logits_dev || !targets_dev || !logprob_dev || !entropy_dev || !stats_dev ||
      (top && (!top_logprob_dev || !top_id_dev)))
    return MXFP8_ERR_INVALID_ARG;
  const bool fp32 = logits_dtype == MXFP8_OUT_FP32;
  if ((reinterpret_cast<uintptr_t>(logits_dev) & (fp32 ? 3u : 1u)) || !aligned8(targets_dev) ||
      !aligned4(logprob_dev) || !aligned4(entropy_dev) || !aligned4(stats_dev) ||
      (top && (!aligned4(top_logprob_dev) || !aligned8(top_id_dev))))
    return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  const LogprobArgs a{logits_dev, rows, vocab, ld, fp32, targets_dev, inv_t, logprob_dev,
                      entropy_dev, stats_dev, top, top_logprob_dev, top_id_dev, d->status};
  const cudaError_t e = launch_logprob(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXFP8_OK
                          : e == cudaErrorInvalidValue ? MXFP8_ERR_INVALID_ARG : MXFP8_ERR_CUDA;
}

int mxfp8_token_logprobs_backward(const void* logits_dev, int logits_dtype, int64_t rows,
                                  int64_t vocab, int64_t ld, const int64_t* targets_dev,
                                  double temperature, const float* stats_dev,
                                  const float* entropy_dev, const float* grad_logprob_dev,
                                  const float* grad_entropy_dev, int top,
                                  const int64_t* top_id_dev, const float* grad_top_dev,
                                  void* grad_logits_dev, int64_t grad_ld, void* stream) {
  float inv_t = 0.f;
  int st = logprob_checks(logits_dtype, rows, vocab, ld, temperature, top, &inv_t);
  if (st != MXFP8_OK) return st;
  int64_t bytes = 0;
  if (grad_ld < vocab || !mul3(rows, grad_ld, 4, &bytes)) return MXFP8_ERR_INVALID_ARG;
  if (rows == 0) return MXFP8_OK;
  if (!logits_dev || !targets_dev || !stats_dev || !entropy_dev || !grad_logprob_dev ||
      !grad_logits_dev || (top && (!top_id_dev || !grad_top_dev)))
    return MXFP8_ERR_INVALID_ARG;
  if (grad_logits_dev == logits_dev && grad_ld != ld) return MXFP8_ERR_INVALID_ARG;
  const bool fp32 = logits_dtype == MXFP8_OUT_FP32;
  if (((reinterpret_cast<uintptr_t>(logits_dev) | reinterpret_cast<uintptr_t>(grad_logits_dev)) &
       (fp32 ? 3u : 1u)) ||
      !aligned8(targets_dev) || !aligned4(stats_dev) || !aligned4(entropy_dev) ||
      !aligned4(grad_logprob_dev) || !aligned4(grad_entropy_dev) ||
      (top && (!aligned8(top_id_dev) || !aligned4(grad_top_dev))))
    return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  const LogprobGradArgs a{logits_dev, rows, vocab, ld, fp32, targets_dev, inv_t, stats_dev,
                          entropy_dev, grad_logprob_dev, grad_entropy_dev, top, top_id_dev,
                          grad_top_dev, grad_logits_dev, grad_ld, d->status};
  const cudaError_t e = launch_logprob_grad(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXFP8_OK
                          : e == cudaErrorInvalidValue ? MXFP8_ERR_INVALID_ARG : MXFP8_ERR_CUDA;
}

constexpr int64_t kMaxRouted = 0x7FFFFF00;  // entries, and rows of all segments together

int64_t mxfp8_route_rows(int64_t tokens, int top_k, int num_experts) {
  int64_t n = 0;
  if (tokens < 0 || top_k < 1 || num_experts < 1 || num_experts > 1024) return 0;
  if (!mul3(tokens, top_k, 1, &n) || n > kMaxRouted) return 0;
  const int64_t rows = (n + 31 * (n < num_experts ? n : num_experts)) / 32 * 32;
  return rows <= kMaxRouted ? rows : 0;
}

// Checks that the calls on a plan share; *entries gets tokens * top_k.
static int plan_checks(int64_t tokens, int top_k, int64_t rows, int64_t* entries) {
  if (tokens < 0 || top_k < 1 || rows < 0 || rows > kMaxRouted) return MXFP8_ERR_INVALID_ARG;
  if (!mul3(tokens, top_k, 1, entries) || *entries > kMaxRouted) return MXFP8_ERR_INVALID_ARG;
  return rows % 32 ? MXFP8_ERR_ALIGNMENT : MXFP8_OK;
}

int mxfp8_route(const int64_t* ids_dev, int64_t tokens, int top_k, int num_experts,
                int64_t total_rows, int32_t* offsets_dev, int32_t* row_of_dev,
                int32_t* entry_of_dev, void* stream) {
  int64_t n = 0;
  int st = plan_checks(tokens, top_k, total_rows, &n);
  if (st != MXFP8_OK) return st;
  if (num_experts < 1 || num_experts > 1024) return MXFP8_ERR_INVALID_ARG;
  if (!offsets_dev || (n && (!ids_dev || !row_of_dev)) || (total_rows && !entry_of_dev))
    return MXFP8_ERR_INVALID_ARG;
  if (!aligned8(ids_dev) || !aligned4(offsets_dev) || !aligned4(row_of_dev) ||
      !aligned4(entry_of_dev))
    return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  const RouteArgs a{ids_dev, n, num_experts, total_rows, offsets_dev, row_of_dev, entry_of_dev,
                    d->status};
  return launch_route(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MXFP8_OK
                                                                           : MXFP8_ERR_CUDA;
}

// Checks of the calls that move rows: sizes in FP32 bytes must fit in int64.
static int rows_checks(int dtype, int64_t tokens, int64_t cols, int top_k, int64_t rows) {
  int64_t n = 0, bytes = 0;
  if (dtype != MXFP8_OUT_BF16 && dtype != MXFP8_OUT_FP32) return MXFP8_ERR_INVALID_ARG;
  // 65535 pieces of 32 columns, the smallest that a launch takes
  if (cols < 0 || cols > int64_t{65535} * 32) return MXFP8_ERR_INVALID_ARG;
  const int st = plan_checks(tokens, top_k, rows, &n);
  if (st != MXFP8_OK) return st;
  if (!mul3(tokens, cols, 4, &bytes) || !mul3(rows, cols, 4, &bytes)) return MXFP8_ERR_INVALID_ARG;
  return MXFP8_OK;
}

int mxfp8_dispatch(const void* x_dev, int dtype, int64_t tokens, int64_t cols, int top_k,
                   const float* weights_dev, const int32_t* row_of_dev,
                   const int32_t* entry_of_dev, int64_t total_rows, void* out_dev,
                   void* stream) {
  int st = rows_checks(dtype, tokens, cols, top_k, total_rows);
  if (st != MXFP8_OK) return st;
  if (total_rows == 0 || cols == 0) return MXFP8_OK;
  if (!entry_of_dev || !out_dev || (tokens && (!x_dev || !row_of_dev)))
    return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(x_dev) || !aligned16(out_dev) || !aligned4(weights_dev) ||
      !aligned4(row_of_dev) || !aligned4(entry_of_dev))
    return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  RowsArgs a{};
  a.src = x_dev;
  a.weights = weights_dev;
  a.row_of = row_of_dev;
  a.entry_of = entry_of_dev;
  a.tokens = tokens;
  a.cols = cols;
  a.rows = total_rows;
  a.k = top_k;
  a.fp32 = dtype == MXFP8_OUT_FP32;
  a.out = out_dev;
  a.status = d->status;
  return launch_dispatch(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MXFP8_OK
                                                                              : MXFP8_ERR_CUDA;
}

int mxfp8_quantize_dispatch(const void* x_dev, int64_t tokens, int64_t cols, int top_k,
                            const float* weights_dev, const int32_t* row_of_dev,
                            const int32_t* entry_of_dev, int64_t total_rows,
                            const int32_t* offsets_dev, int num_experts,
                            void* row_out_dev, void* row_scales_dev, void* col_out_dev,
                            void* col_scales_dev, void* stream) {
  const bool row = row_out_dev || row_scales_dev, col = col_out_dev || col_scales_dev;
  int64_t n = 0, elems = 0;
  int st = plan_checks(tokens, top_k, total_rows, &n);
  if (st != MXFP8_OK) return st;
  if (num_experts < 1 || num_experts > 1024 || cols < 0) return MXFP8_ERR_INVALID_ARG;
  if (cols % (row ? 32 : 8)) return MXFP8_ERR_ALIGNMENT;
  if (total_rows == 0 || cols == 0) return MXFP8_OK;
  if (!mul3(total_rows, cols, 4, &elems) || !mul3(tokens, cols, 1, &elems))
    return MXFP8_ERR_INVALID_ARG;
  if (elems >= int64_t{1} << 35) return MXFP8_ERR_INVALID_ARG;   // rows' places in 32 bits
  if ((!row && !col) || (row && (!row_out_dev || !row_scales_dev)) ||
      (col && (!col_out_dev || !col_scales_dev)) || !entry_of_dev || !offsets_dev ||
      (tokens && (!x_dev || !row_of_dev)))
    return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(x_dev) || !aligned16(row_out_dev) || !aligned16(row_scales_dev) ||
      !aligned16(col_out_dev) || !aligned16(col_scales_dev) || !aligned4(weights_dev) ||
      !aligned4(row_of_dev) || !aligned4(entry_of_dev) || !aligned4(offsets_dev))
    return MXFP8_ERR_ALIGNMENT;
  if (cdiv(total_rows, 128) + num_experts > kMaxTokenTiles || cdiv(cols, 128) > 0x7FFFFFFF)
    return MXFP8_ERR_INVALID_ARG;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  const QuantizeDispatchArgs a{x_dev, tokens, top_k, weights_dev, row_of_dev, entry_of_dev,
                               offsets_dev, num_experts, total_rows, cols, row_out_dev,
                               row_scales_dev, col_out_dev, col_scales_dev, d->status};
  return launch_quantize_dispatch(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MXFP8_OK
             : MXFP8_ERR_CUDA;
}

int mxfp8_combine(const void* y_dev, int dtype, int64_t total_rows, int64_t cols, int64_t tokens,
                  int top_k, const float* weights_dev, const int32_t* row_of_dev, void* out_dev,
                  void* stream) {
  int st = rows_checks(dtype, tokens, cols, top_k, total_rows);
  if (st != MXFP8_OK) return st;
  if (tokens == 0 || cols == 0) return MXFP8_OK;
  if (!row_of_dev || !out_dev || (total_rows && !y_dev)) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(y_dev) || !aligned16(out_dev) || !aligned4(weights_dev) || !aligned4(row_of_dev))
    return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  RowsArgs a{};
  a.src = y_dev;
  a.weights = weights_dev;
  a.row_of = row_of_dev;
  a.tokens = tokens;
  a.cols = cols;
  a.rows = total_rows;
  a.k = top_k;
  a.fp32 = dtype == MXFP8_OUT_FP32;
  a.out = out_dev;
  a.status = d->status;
  return launch_combine(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MXFP8_OK
                                                                             : MXFP8_ERR_CUDA;
}

int mxfp8_combine_backward(const void* grad_out_dev, const void* y_dev, int dtype,
                           int64_t tokens, int64_t cols, int top_k, const float* weights_dev,
                           const int32_t* row_of_dev, const int32_t* entry_of_dev,
                           int64_t total_rows, void* grad_y_dev, float* grad_weights_dev,
                           void* stream) {
  int st = rows_checks(dtype, tokens, cols, top_k, total_rows);
  if (st != MXFP8_OK) return st;
  const bool rows_out = grad_y_dev && total_rows && cols;   // something to write there
  if (tokens == 0 && !rows_out) return MXFP8_OK;
  if (tokens && (!weights_dev || !row_of_dev || !grad_weights_dev ||
                 (cols && (!grad_out_dev || (total_rows && !y_dev)))))
    return MXFP8_ERR_INVALID_ARG;
  if (rows_out && !entry_of_dev) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(grad_out_dev) || !aligned16(y_dev) || !aligned16(grad_y_dev) ||
      !aligned4(weights_dev) || !aligned4(row_of_dev) || !aligned4(entry_of_dev) ||
      !aligned4(grad_weights_dev))
    return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  RowsArgs a{};
  a.src = grad_out_dev;
  a.y = y_dev;
  a.weights = weights_dev;
  a.row_of = row_of_dev;
  a.entry_of = entry_of_dev;
  a.tokens = tokens;
  a.cols = cols;
  a.rows = total_rows;
  a.k = top_k;
  a.fp32 = dtype == MXFP8_OUT_FP32;
  a.out = rows_out ? grad_y_dev : nullptr;
  a.grad_w = grad_weights_dev;
  a.status = d->status;
  return launch_combine_grad(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MXFP8_OK
             : MXFP8_ERR_CUDA;
}

// Sizes of the gated activation: bytes of [rows][2 width] BF16 fit in int64.
static int swiglu_checks(int64_t rows, int64_t width) {
  int64_t bytes = 0;
  if (rows < 0 || width < 0 || width > kMaxRouted / 2) return MXFP8_ERR_INVALID_ARG;
  if (!mul3(rows, width, 4, &bytes)) return MXFP8_ERR_INVALID_ARG;
  if (width % 32) return MXFP8_ERR_ALIGNMENT;
  // 2^31 - 1 CTAs of 256 threads, 16 values each
  return rows * (width / 16) > int64_t{0x7FFFFFFF} * 256 ? MXFP8_ERR_INVALID_ARG : MXFP8_OK;
}

int mxfp8_swiglu(const void* x_dev, int64_t rows, int64_t width, void* h_dev, void* codes_dev,
                 void* scales_dev, int scale_rule, void* stream) {
  int st = swiglu_checks(rows, width);
  if (st != MXFP8_OK) return st;
  if (scale_rule != MXFP8_RULE_FLOOR && scale_rule != MXFP8_RULE_CEIL)
    return MXFP8_ERR_INVALID_ARG;
  if (rows == 0 || width == 0) return MXFP8_OK;
  if (!x_dev || !h_dev || !codes_dev != !scales_dev) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(x_dev) || !aligned16(h_dev) || !aligned16(codes_dev)) return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  SwigluArgs a{};
  a.x = x_dev;
  a.rows = rows;
  a.width = width;
  a.rule = scale_rule;
  a.codes = codes_dev;
  a.scales = scales_dev;
  a.h = h_dev;
  return launch_swiglu(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MXFP8_OK
                                                                            : MXFP8_ERR_CUDA;
}

int mxfp8_swiglu_backward(const void* grad_h_dev, const void* codes_dev, const void* scales_dev,
                          int64_t rows, int64_t width, void* grad_x_dev, void* h_dev,
                          void* stream) {
  int st = swiglu_checks(rows, width);
  if (st != MXFP8_OK) return st;
  if (rows == 0 || width == 0) return MXFP8_OK;
  if (!grad_h_dev || !codes_dev || !scales_dev || !grad_x_dev) return MXFP8_ERR_INVALID_ARG;
  if (!aligned16(grad_h_dev) || !aligned16(codes_dev) || !aligned16(grad_x_dev) ||
      !aligned16(h_dev))
    return MXFP8_ERR_ALIGNMENT;
  DeviceState* d = nullptr;
  st = device_state(&d);
  if (st != MXFP8_OK) return st;
  SwigluArgs a{};
  a.grad = grad_h_dev;
  a.rows = rows;
  a.width = width;
  a.codes = const_cast<void*>(codes_dev);
  a.scales = const_cast<void*>(scales_dev);
  a.h = h_dev;
  a.grad_x = grad_x_dev;
  return launch_swiglu_grad(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MXFP8_OK
                                                                                 : MXFP8_ERR_CUDA;
}

int mxfp8_set_wait_limit_ns(uint64_t ns) {
  set_wait_limit_ns(ns);
  return MXFP8_OK;
}

int mxfp8_get_device_status(void* stream) {
  DeviceState* d = nullptr;
  const int st = device_state(&d);
  if (st != MXFP8_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned slot = g_status_slot.fetch_add(1, std::memory_order_relaxed) % kStatusSlots;
  void* args[] = {const_cast<unsigned*>(&slot)};  // enqueued after the stream's earlier work
  if (cudaLaunchKernel(reinterpret_cast<const void*>(take_status_kernel), dim3(1), dim3(1), args,
                       0, s) != cudaSuccess)
    return MXFP8_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_status_taken, sizeof(int), slot * sizeof(int),
                                cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return MXFP8_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return MXFP8_ERR_CUDA;
  return v;
}

}  // extern "C"
