// internal.h - host-side interface between the C ABI (api.cu) and the kernel launchers.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mxfp8 {

constexpr int kAxisBoth = 2;  // both copies from one read (row-wise + column-wise)

struct QuantizeArgs {
  const void* src;
  int64_t batch;          // independent matrices (1 for a plain call)
  int64_t rows, cols;     // one matrix
  int axis;               // MXFP8_AXIS_ROW / COL, or kAxisBoth
  void* out;              // ROW or COL output (ROW output when axis == kAxisBoth)
  void* scales;
  int64_t scale_item_bytes;
  void* out_col;          // kAxisBoth: the column-wise output
  void* scales_col;
  int64_t scale_item_bytes_col;
  int layout;             // MXFP8_SCALES_LINEAR / SWIZZLED
  const int32_t* offsets; // grouped call: device [num_experts + 1], else nullptr
  int num_experts;
  int rule;               // MXFP8_RULE_FLOOR / MXFP8_RULE_CEIL
  int* status;            // device status word
};

cudaError_t launch_quantize(const QuantizeArgs& a, cudaStream_t stream);

// Programmatic dependent launch: every kernel of the library is launched with
// programmatic stream serialization (its kernels wait for the previous kernel of the
// stream in the kernel itself), unless the environment sets MXFP8_PDL=0 (read once).
// Writes the launch attribute to *attr and returns 1, or returns 0 when it is off.
int pdl_attr(cudaLaunchAttribute* attr);

// Several dual (row-wise + column-wise) quantizations in one launch.
constexpr int kMaxQuantizeJobs = 8;
struct QuantizeJobs {
  int n;
  int layout;
  const void* src[kMaxQuantizeJobs];
  int64_t rows[kMaxQuantizeJobs], cols[kMaxQuantizeJobs];
  void* out[kMaxQuantizeJobs];
  void* scales[kMaxQuantizeJobs];
  void* out_col[kMaxQuantizeJobs];
  void* scales_col[kMaxQuantizeJobs];
  int* status;
};

cudaError_t launch_quantize_jobs(const QuantizeJobs& j, cudaStream_t stream);

// FP8 block-wise (128 x 128) weight quantization; scale_inv [ceil(rows/128)][ceil(cols/128)].
cudaError_t launch_blockwise(const void* src, int64_t rows, int64_t cols, void* out,
                             float* scale_inv, bool pow2, cudaStream_t stream);

// Operands of the block-wise GEMM from one read of a BF16 matrix: row-wise and / or
// transposed copies with 1 x 128 blocks, or (two_d) both copies with 128 x 128 blocks. A
// null row_out / col_out leaves that copy out.
struct BlockwiseArgs {
  const void* src;
  int64_t rows, cols;
  void* row_out;
  float* row_inv;
  void* col_out;
  float* col_inv;
  bool two_d, pow2;
};

cudaError_t launch_blockwise_tiles(const BlockwiseArgs& a, cudaStream_t stream);

struct GemmArgs {
  const void* A;
  const void* sA;
  const void* B;
  const void* sB;
  void* C;
  int64_t M, N, K;
  int op;
  int out_dtype;
  // grouped call
  const int32_t* offsets;  // nullptr for the dense GEMM
  int num_experts;
  int64_t total_rows;
  int* status;
  // dense call: caller-owned workspace for a split-K last wave (nullptr: none)
  void* workspace = nullptr;
  size_t workspace_bytes = 0;
  // dense call: run only if none of these device words is set (nullptr: always)
  const uint32_t* unless = nullptr;
  int num_unless = 0;
};

// Returns MXFP8_OK or an mxfp8_status code.
int launch_gemm(const GemmArgs& a, cudaStream_t stream);
// Bytes of workspace with which launch_gemm runs this dense GEMM's last wave as split-K
// pieces on the current device (0: it never does).
size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int out_dtype);
int launch_grouped_gemm(const GemmArgs& a, cudaStream_t stream);

// The block-wise GEMM: C [M][N] = deq(A) [M][K] . deq(B) [N][K]^T.
struct BlockwiseGemmArgs {
  const void* A;
  const float* sA;   // [ceil(K/128)][M]
  const void* B;
  const float* sB;   // [ceil(N/128)][ceil(K/128)], or (wgrad) [ceil(K/128)][N]
  void* C;
  int64_t M, N, K;
  bool wgrad, out_fp32;
  int* status;
  void* workspace;   // blockwise_gemm_workspace_bytes(...) bytes, or nullptr
  size_t workspace_bytes;
};

// Returns MXFP8_OK or an mxfp8_status code.
int launch_blockwise_gemm(const BlockwiseGemmArgs& a, cudaStream_t stream);
// Workspace with which power-of-two scales run on the block-scaled MMA (0: never).
int64_t blockwise_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, bool out_fp32);

// Estimated time of launch_gemm on CTA pairs per K stage, in that of one wave of 256-wide tiles.
double dense_gemm_waves(int64_t M, int64_t N, bool fp32);

// Tensor map of a row-major byte matrix [outer][inner] in 128-byte x box_outer boxes with
// the 128-byte swizzle.
bool make_operand_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer,
                      uint32_t box_outer);

// Tensor map of a row-major output [rows][N] for stores of 32-row x 64-byte boxes with the
// 64-byte swizzle.
bool make_store_map(CUtensorMap* map, void* base, int64_t rows, int64_t N, bool fp32);
// MXFP8 scale tiles [row tiles][K tiles][512 bytes], in boxes of `tiles_per_box` row tiles.
bool make_scale_map(CUtensorMap* map, const void* base, int64_t row_tiles, int64_t k_tiles,
                    uint32_t tiles_per_box);

// Limits of pipeline waits, and of waits for work in flight on the way out of a kernel.
uint64_t pipeline_wait_ns();
uint64_t pipeline_drain_ns();

struct SelfcheckArgs {
  const void* w_codes;   // E4M3 [N][K] as the GEMM reads it
  const void* w_scales;  // swizzled scales as the GEMM reads them
  const void* ref_codes;   // canonical synchronized weight, E4M3 [N][K]
  const void* ref_scales;  // its linear scales [N][K/32]
  int64_t N, K;
  const void* x;         // BF16 [T][K]
  int64_t T;
  void* workspace;       // selfcheck_workspace_bytes(T, N, K) bytes
  float* rel_err;        // device, one float
  int* status;
};

int64_t selfcheck_workspace_bytes(int64_t T, int64_t N, int64_t K);

// Size of the fixed workspace behind mxfp8_selfcheck_noalloc (8 MiB).
constexpr int64_t kSelfcheckNoallocMaxBytes = int64_t(8) << 20;
int selfcheck_noalloc_workspace(void** out);
int launch_selfcheck(const SelfcheckArgs& a, cudaStream_t stream);

// Log probabilities of given tokens (logits BF16, or FP32 with fp32 set).
struct LogprobArgs {
  const void* logits;     // [rows][ld], the first `vocab` of each row are read
  int64_t rows, vocab, ld;
  bool fp32;
  const int64_t* targets;
  float inv_t;            // 1 / temperature
  float* logprob;         // [rows]
  float* entropy;         // [rows]
  float* stats;           // [rows][2]: maximum logit, log of the sum
  int top;                // alternatives per row, 0 .. 32
  float* top_logprob;     // [rows][top]
  int64_t* top_id;        // [rows][top]
  int* status;
};

struct LogprobGradArgs {
  const void* logits;
  int64_t rows, vocab, ld;
  bool fp32;
  const int64_t* targets;
  float inv_t;
  const float* stats;
  const float* entropy;
  const float* g_logprob;
  const float* g_entropy;  // or nullptr
  int top;
  const int64_t* top_id;
  const float* g_top;
  void* out;               // [rows][out_ld], the logits' type; may be the logits
  int64_t out_ld;
  int* status;
};

cudaError_t launch_logprob(const LogprobArgs& a, cudaStream_t stream);
cudaError_t launch_logprob_grad(const LogprobGradArgs& a, cudaStream_t stream);

// Entries (token, choice) sorted by expert.
struct RouteArgs {
  const int64_t* ids;     // [entries]
  int64_t entries;        // tokens * top_k
  int num_experts;
  int64_t rows;           // of all segments together
  int32_t* offsets;       // [num_experts + 1]
  int32_t* row_of;        // [entries]
  int32_t* entry_of;      // [rows]
  int* status;
};

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream);

// Rows of tokens to and from the experts' segments (BF16, or FP32 with fp32 set).
struct RowsArgs {
  const void* src;          // dispatch: x [tokens][cols]; combine: y [rows][cols]; gradient: dout
  const void* y;            // gradient: y [rows][cols]
  const float* weights;     // [tokens][k], or nullptr for 1
  const int32_t* row_of;    // [tokens][k]
  const int32_t* entry_of;  // [rows]
  int64_t tokens, cols, rows;
  int k;
  bool fp32;
  void* out;                // [rows][cols], combine: [tokens][cols]; gradient: may be nullptr
  float* grad_w;            // gradient: [tokens][k]
  int* status;
};

cudaError_t launch_dispatch(const RowsArgs& a, cudaStream_t stream);
cudaError_t launch_combine(const RowsArgs& a, cudaStream_t stream);
cudaError_t launch_combine_grad(const RowsArgs& a, cudaStream_t stream);

// Grouped MXFP8 operands from the tokens' rows; a null row_out / col_out leaves that copy out.
struct QuantizeDispatchArgs {
  const void* src;          // BF16 [tokens][cols]
  int64_t tokens;
  int top_k;
  const float* weights;     // [tokens][top_k], or nullptr
  const int32_t* row_of;    // [tokens][top_k]
  const int32_t* entry_of;  // [rows]
  const int32_t* offsets;   // [num_experts + 1]
  int num_experts;
  int64_t rows, cols;
  void* row_out;
  void* row_scales;
  void* col_out;
  void* col_scales;
  int* status;
};

cudaError_t launch_quantize_dispatch(const QuantizeDispatchArgs& a, cudaStream_t stream);

// h = silu(gate) * up of gate_up [rows][2 width], with gate_up kept as row-wise MXFP8 (codes
// null: not kept), and the gradient from that copy.
struct SwigluArgs {
  const void* x;         // forward: BF16 [rows][2 width]
  const void* grad;      // backward: BF16 [rows][width]
  int64_t rows, width;
  int rule;
  void* codes;           // E4M3 [rows][2 width]
  void* scales;          // [rows][2 width / 32]
  void* h;               // BF16 [rows][width]; backward: may be nullptr
  void* grad_x;          // backward: BF16 [rows][2 width]
};

cudaError_t launch_swiglu(const SwigluArgs& a, cudaStream_t stream);
cudaError_t launch_swiglu_grad(const SwigluArgs& a, cudaStream_t stream);

int num_sms();  // of the current device (cached)

// Pipeline wait limit of the GEMM kernels for later launches (0: the default).
void set_wait_limit_ns(uint64_t ns);

}  // namespace mxfp8
