/*
 * mxfp8.h - C ABI of the GB300 (sm_103a) MXFP8 quantizer and block-scaled GEMMs.
 *
 * The method: "End-to-End MXFP8 RL on Blackwell: What Matching Buys, When It Pays Off,
 * and How It Fails" (verl blog post). Section "The pipeline", paragraph "The format":
 * MXFP8 is the OCP microscaling FP8 format - E4M3 elements in blocks of 32 along the
 * reduction dimension, each block sharing one power-of-two E8M0 scale. The learner
 * paragraph of the same section: each linear layer runs three GEMMs (forward, data
 * gradient, weight gradient) on quantized operands, some quantized along the token
 * dimension, with token counts padded to multiples of 32. The weight-synchronization
 * paragraph: the synced weights are the forward GEMM's weight quantization, byte for
 * byte. Section "Where the time goes": scales are rearranged into the layout the GEMM
 * reads; here the quantizer writes that layout directly.
 *
 * Conventions shared by every call:
 *  - Pointers named *_dev are device pointers; the caller allocates and owns every
 *    buffer. The library allocates no device memory in any call. Its only state is a
 *    per-device status word (see mxfp8_get_device_status) and per-device capability
 *    flags, set up on the first call on each device.
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream).
 *    Every compute call only enqueues work on `stream` and returns; none synchronizes
 *    except mxfp8_get_device_status. Kernels are launched with programmatic stream
 *    serialization: one may be scheduled while the previous kernel of its stream is
 *    still running, and it waits inside the kernel, before its first read or write of
 *    global memory, until that kernel has completed. Stream order therefore holds as
 *    for a plain launch, against any kernel before it. MXFP8_PDL=0 in the environment
 *    (read once per process) launches them plainly.
 *  - Return value: an mxfp8_status. Arguments are checked on the host before anything
 *    is enqueued; a failed check returns its code and enqueues nothing. Errors found
 *    by a kernel (bad expert offsets, a pipeline wait that ran out) are latched in the
 *    device status word and read with mxfp8_get_device_status. No call throws.
 *  - Matrices are row-major with packed rows (leading dimension = number of columns).
 *    BF16 and E4M3 tensors must start on a 16-byte boundary, scale tensors too.
 *  - Quantization rule (OCP, floor form): per block of 32, e = max(-127,
 *    floor(log2 amax) - 8); scale byte = e + 127; element = E4M3(v * 2^-e), round to
 *    nearest even, saturating at +-448, sign of zero kept. A block holding a NaN or an
 *    infinity gets scale 0xFF and every element 0x7F | (its sign bit).
 *  - Scale layouts. LINEAR: scales [S_rows][S_cols] row-major, one byte per block.
 *    SWIZZLED: the tensor cores' 128 x 4 tiles - byte offset of scale (r, c) is
 *    ((r / 128) * ceil(S_cols / 4) + c / 4) * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4
 *    + (c % 4); the padding bytes of partial tiles are written as 0x00. The GEMMs read
 *    SWIZZLED scales only.
 */
#ifndef MXFP8_H_
#define MXFP8_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MXFP8_ABI_VERSION 1

typedef enum mxfp8_status {
  MXFP8_OK = 0,
  MXFP8_ERR_INVALID_ARG = 1,      /* null pointer, negative or unsupported size/enum */
  MXFP8_ERR_ALIGNMENT = 2,        /* a blocked dim not a multiple of 32, or a pointer
                                     not 16-byte aligned */
  MXFP8_ERR_UNSUPPORTED_ARCH = 3, /* current device is not compute capability 10.3 */
  MXFP8_ERR_CUDA = 4,             /* a CUDA runtime/driver call failed */
  MXFP8_ERR_BAD_OFFSETS = 5,      /* (device) expert offsets not 0-based, non-decreasing,
                                     32-aligned and ending at total_rows; a routing plan of
                                     more rows than total_rows */
  MXFP8_ERR_TIMEOUT = 6,          /* (device) a pipeline wait in a kernel ran out; the
                                     kernel abandoned its work */
  MXFP8_ERR_BAD_TARGET = 7,       /* (device) a token id at or past the vocabulary */
  MXFP8_ERR_BAD_EXPERT = 8        /* (device) an expert id at or past the number of experts */
} mxfp8_status;

typedef enum mxfp8_axis {
  MXFP8_AXIS_ROW = 0, /* blocks along the contiguous (last) dim: out [rows][cols] */
  MXFP8_AXIS_COL = 1  /* blocks along the first dim, emitted transposed: out [cols][rows] */
} mxfp8_axis;

typedef enum mxfp8_scale_layout {
  MXFP8_SCALES_LINEAR = 0,
  MXFP8_SCALES_SWIZZLED = 1
} mxfp8_scale_layout;

typedef enum mxfp8_scale_rule {
  MXFP8_RULE_FLOOR = 0, /* OCP: e = floor(log2 amax) - 8; the largest elements may saturate */
  MXFP8_RULE_CEIL = 1   /* round-up power of two: smallest e with amax <= 448 * 2^e; never
                           saturates (block-wise FP8 recipes' power-of-two scales) */
} mxfp8_scale_rule;

typedef enum mxfp8_op {
  MXFP8_OP_FPROP = 0, /* Y  = X  . W^T   A = X  rows,  B = W  rows          */
  MXFP8_OP_DGRAD = 1, /* dX = dY . W     A = dY rows,  B = W  cols (= W^T)  */
  MXFP8_OP_WGRAD = 2  /* dW = dY^T . X   A = dY cols,  B = X  cols (tokens) */
} mxfp8_op;

typedef enum mxfp8_out_dtype {
  MXFP8_OUT_BF16 = 0,
  MXFP8_OUT_FP32 = 1
} mxfp8_out_dtype;

/* ABI version of the loaded library (MXFP8_ABI_VERSION). */
int mxfp8_version(void);

/* Static text for a status code; never NULL. */
const char* mxfp8_status_string(int status);

/*
 * Bytes of the scale tensor that mxfp8_quantize writes for a [rows][cols] BF16 input.
 * S_rows x S_cols = rows x cols/32 (ROW) or cols x rows/32 (COL); LINEAR is
 * S_rows * S_cols bytes, SWIZZLED is ceil(S_rows/128) * ceil(S_cols/4) * 512 bytes.
 * Returns 0 for invalid arguments (negative sizes, a blocked dim not a multiple of 32,
 * unknown enums, a size that does not fit in int64).
 */
size_t mxfp8_scale_bytes(int64_t rows, int64_t cols, int axis, int scale_layout);

/*
 * MXFP8-quantize a BF16 matrix ("The pipeline" - "The format"; column-wise copies for
 * the weight-gradient GEMM: the learner paragraph).
 *   src_dev      BF16 [rows][cols], read only.
 *   axis ROW     requires cols % 32 == 0; out_dev E4M3 [rows][cols]; scales for
 *                [rows][cols/32].
 *   axis COL     requires rows % 32 == 0 and cols % 8 == 0; out_dev E4M3 [cols][rows]
 *                (the transpose, blocked along its contiguous dim); scales for
 *                [cols][rows/32].
 *   scales_dev   mxfp8_scale_bytes(rows, cols, axis, scale_layout) bytes, written in
 *                full (padding included).
 * rows == 0 or cols == 0 is a no-op. Deterministic: the same input gives the same bytes
 * from every call, which is what makes the synchronized weights equal the forward
 * weights byte for byte (section "The grid, byte for byte").
 */
int mxfp8_quantize(const void* src_dev, int64_t rows, int64_t cols, int axis,
                   void* out_dev, void* scales_dev, int scale_layout, void* stream);

/*
 * mxfp8_quantize with an explicit scale rule (mxfp8_scale_rule). The pages contrast the
 * MXFP8 grid with block-wise FP8 recipes whose power-of-two scales round the other way
 * (section "A different grid, and drift"); MXFP8_RULE_CEIL produces that grid on the same
 * 1x32 blocks so the two can be compared byte for byte. Bytes differ from the floor rule
 * exactly in blocks whose amax exceeds 448 * 2^e_floor (scale byte one higher there).
 * MXFP8_RULE_FLOOR gives the bytes of mxfp8_quantize.
 */
int mxfp8_quantize_rule(const void* src_dev, int64_t rows, int64_t cols, int axis,
                        void* out_dev, void* scales_dev, int scale_layout, int scale_rule,
                        void* stream);

/*
 * Both copies of one BF16 matrix from a single read of it: the row-wise copy (as
 * mxfp8_quantize ROW) into row_out_dev / row_scales_dev and the column-wise copy (as
 * mxfp8_quantize COL) into col_out_dev / col_scales_dev. The learner needs both for X and
 * dY (forward/dgrad operands blocked along K, wgrad operands blocked along tokens:
 * "The pipeline", learner paragraph). Requires rows % 32 == 0 and cols % 32 == 0. Bytes
 * are identical to the two separate calls.
 */
int mxfp8_quantize_dual(const void* src_dev, int64_t rows, int64_t cols, void* row_out_dev,
                        void* row_scales_dev, void* col_out_dev, void* col_scales_dev,
                        int scale_layout, void* stream);

/*
 * One job of mxfp8_quantize_dual_multi: the arguments of one mxfp8_quantize_dual call.
 * All pointers are device pointers owned by the caller.
 */
typedef struct mxfp8_dual_job {
  const void* src;     /* BF16 [rows][cols] */
  int64_t rows, cols;  /* rows % 32 == 0, cols % 32 == 0 */
  void* row_out;       /* E4M3 [rows][cols] */
  void* row_scales;    /* mxfp8_scale_bytes(rows, cols, MXFP8_AXIS_ROW, layout) bytes */
  void* col_out;       /* E4M3 [cols][rows] */
  void* col_scales;    /* mxfp8_scale_bytes(rows, cols, MXFP8_AXIS_COL, layout) bytes */
} mxfp8_dual_job;

#define MXFP8_MAX_DUAL_JOBS 8

/*
 * Several mxfp8_quantize_dual calls in one launch. The tensors' 128 x 128 tiles form one
 * grid, so a small tensor's partly filled last wave of CTAs is shared with the others
 * instead of running alone. Typical use: a linear layer's activations and weight,
 * quantized together before the forward GEMM. "The pipeline" (learner paragraph) gives
 * the quantized operands; the batching is this library's.
 *   jobs        host array of num_jobs descriptors (1 <= num_jobs <= MXFP8_MAX_DUAL_JOBS),
 *               read during the call only; every job is checked as mxfp8_quantize_dual
 *               checks its arguments, and nothing is launched if one fails. Jobs with
 *               rows == 0 or cols == 0 are skipped.
 * Bytes are identical to one mxfp8_quantize_dual call per job. Outputs of different jobs
 * must not overlap.
 */
int mxfp8_quantize_dual_multi(const mxfp8_dual_job* jobs, int num_jobs, int scale_layout,
                              void* stream);

/* Scale choice of the FP8 block-wise recipe (mxfp8_quantize_blockwise). */
typedef enum {
  MXFP8_BW_SCALE_FP32 = 0, /* quantization factor 448 / amax in single precision */
  MXFP8_BW_SCALE_POW2 = 1  /* power-of-two factor 2^-ceil(log2(amax / 448)) */
} mxfp8_blockwise_scale;

/*
 * Number of float scales mxfp8_quantize_blockwise writes for a [rows][cols] weight:
 * ceil(rows/128) * ceil(cols/128). Returns 0 for invalid arguments, including a count
 * that does not fit in int64.
 */
size_t mxfp8_blockwise_scale_count(int64_t rows, int64_t cols);

/*
 * FP8 block-wise weight quantization, the recipe the pages contrast with MXFP8 ("A
 * different grid, and drift": on Blackwell the block-wise learner must use power-of-two
 * block scales while its sampler uses FP32 scales, so the two sides round the same BF16
 * weight differently; "The pipeline", "The format": TE emulates that recipe with MXFP8
 * GEMMs). One scale per 128 x 128 block (the pages give no block size; 128 x 128 is the
 * block-wise weight recipe's usual one):
 *   amax = max |v| over the block;
 *   s = 448 / amax in IEEE single precision (largest finite float if that overflows),
 *       or 2^-e with e = ceil(log2(amax / 448)) >= -127 for MXFP8_BW_SCALE_POW2;
 *       s = 1 for an all-zero block;
 *   code = E4M3(v * s), the product rounded to single precision, then to nearest even,
 *          saturating at 448;
 *   scale_inv = 1 / s in single precision (exactly 2^e for POW2);
 *   a block holding a NaN or an infinity: scale_inv NaN, codes 0x7F with each sign.
 *   src_dev        BF16 [rows][cols], cols % 8 == 0, 16-byte aligned
 *   out_dev        E4M3 [rows][cols], 16-byte aligned
 *   scale_inv_dev  float [ceil(rows/128)][ceil(cols/128)], 4-byte aligned
 * Errors: MXFP8_ERR_INVALID_ARG (bad scale_type, negative or too large sizes, null
 * pointers), MXFP8_ERR_ALIGNMENT (cols % 8, misaligned pointers).
 */
int mxfp8_quantize_blockwise(const void* src_dev, int64_t rows, int64_t cols, void* out_dev,
                             float* scale_inv_dev, int scale_type, void* stream);

/*
 * FP8 block-wise quantization with 1 x 128 blocks along one axis of a BF16 matrix: the
 * activations and gradients of the block-wise recipe, as mxfp8_blockwise_gemm reads them.
 * The scale and code rule is that of mxfp8_quantize_blockwise, with amax over the 128 (at
 * the edge: fewer) values of a block.
 *   src_dev        BF16 [rows][cols], 16-byte aligned
 *   axis ROW       blocks along the columns; cols % 16 == 0. out_dev E4M3 [rows][cols],
 *                  scale_inv_dev float [ceil(cols/128)][rows].
 *   axis COL       blocks along the rows, emitted transposed; cols % 8 == 0, any number of
 *                  rows. out_dev E4M3 [cols][pitch], pitch = rows rounded up to a multiple
 *                  of 16, the codes past `rows` zero; scale_inv_dev float
 *                  [ceil(rows/128)][cols].
 * Scales lie block-major, so that a GEMM tile's scales of one block are contiguous.
 * rows == 0 or cols == 0 is a no-op. Deterministic.
 * Errors as for mxfp8_quantize_blockwise.
 */
int mxfp8_quantize_blockwise_1d(const void* src_dev, int64_t rows, int64_t cols, int axis,
                                void* out_dev, float* scale_inv_dev, int scale_type,
                                void* stream);

/*
 * mxfp8_quantize_blockwise_1d ROW and COL from one read of the input (cols % 16 == 0):
 * what a learner needs of X and dY. Bytes equal those of the two separate calls.
 */
int mxfp8_quantize_blockwise_1d_dual(const void* src_dev, int64_t rows, int64_t cols,
                                     void* row_out_dev, float* row_scale_inv_dev,
                                     void* col_out_dev, float* col_scale_inv_dev,
                                     int scale_type, void* stream);

/*
 * mxfp8_quantize_blockwise and the transpose of its result from one read (rows % 16 == 0,
 * cols % 16 == 0): the weight as the forward and the data-gradient GEMM read it.
 *   out_dev / scale_inv_dev      as mxfp8_quantize_blockwise writes them
 *   out_t_dev / scale_inv_t_dev  E4M3 [cols][rows], float [ceil(cols/128)][ceil(rows/128)]
 */
int mxfp8_quantize_blockwise_dual(const void* src_dev, int64_t rows, int64_t cols,
                                  void* out_dev, float* scale_inv_dev, void* out_t_dev,
                                  float* scale_inv_t_dev, int scale_type, void* stream);

/*
 * `batch` independent matrices [batch][rows][cols] quantized as by mxfp8_quantize, each
 * with its own scale block of mxfp8_scale_bytes(rows, cols, axis, layout) bytes; the
 * scale blocks are concatenated in batch order. Used for per-expert MoE weights.
 */
int mxfp8_quantize_batched(const void* src_dev, int64_t batch, int64_t rows, int64_t cols,
                           int axis, void* out_dev, void* scales_dev, int scale_layout,
                           void* stream);

/*
 * Capacity (bytes) to allocate for the scales of mxfp8_quantize_grouped on a
 * [total_rows][cols] input split into at most num_experts token segments. It is an
 * upper bound that needs no expert counts on the host:
 *   ROW: (ceil(total_rows/128) + num_experts) * ceil(cols/128) * 512
 *   COL: ceil(cols/128) * (ceil(total_rows/128) + num_experts) * 512
 * Returns 0 for invalid arguments, including a size that does not fit in int64.
 */
size_t mxfp8_grouped_scale_bytes(int64_t total_rows, int64_t cols, int num_experts, int axis);

/*
 * MXFP8-quantize a token-segmented (MoE) BF16 matrix [total_rows][cols]; expert e owns
 * rows [off[e], off[e+1]) (section "A held-out workload, and end to end", Table 4).
 *   expert_offsets_dev  int32 [num_experts + 1] on the device: off[0] = 0,
 *                       non-decreasing, multiples of 32, off[E] = total_rows. Checked
 *                       on the device; a violation latches MXFP8_ERR_BAD_OFFSETS and
 *                       the scales are left unspecified.
 *   axis ROW  out_dev [total_rows][cols] (cols % 32 == 0); scales: expert e's SWIZZLED
 *             block for its [cnt_e][cols/32] scales, rows padded to 128.
 *   axis COL  out_dev [cols][total_rows] (cols % 8 == 0); scales: expert e's SWIZZLED
 *             block for its [cols][cnt_e/32] scales, token blocks padded to 4.
 *   Blocks are concatenated in expert order (empty experts take no bytes) inside
 *   scales_dev, whose capacity is mxfp8_grouped_scale_bytes(...); bytes past the last
 *   block are not written. The element bytes equal those of mxfp8_quantize.
 */
int mxfp8_quantize_grouped(const void* src_dev, int64_t total_rows, int64_t cols, int axis,
                           const int32_t* expert_offsets_dev, int num_experts,
                           void* out_dev, void* scales_dev, void* stream);

/*
 * mxfp8_quantize_grouped ROW and COL from one read of the input (cols % 32 == 0);
 * each copy's scales go to its own buffer, sized by mxfp8_grouped_scale_bytes for its
 * axis.
 */
int mxfp8_quantize_grouped_dual(const void* src_dev, int64_t total_rows, int64_t cols,
                                const int32_t* expert_offsets_dev, int num_experts,
                                void* row_out_dev, void* row_scales_dev, void* col_out_dev,
                                void* col_scales_dev, void* stream);

/*
 * Block-scaled GEMM on tcgen05 (kind::mxf8f6f4, E4M3 x E4M3, UE8M0 scales, FP32
 * accumulation): C[M][N] = sum_k deq(A)[m][k] * deq(B)[n][k] ("The pipeline", learner
 * paragraph: the three GEMMs of a linear layer).
 *   A_dev, sA_dev  E4M3 [M][K] and its SWIZZLED scales (rows M, K/32 blocks);
 *   B_dev, sB_dev  E4M3 [N][K] and its SWIZZLED scales (rows N, K/32 blocks);
 *   C_dev          [M][N], BF16 or FP32 (out_dtype), fully overwritten.
 * Both operands are K-major ("TN"); `op` names which quantized copies are passed
 * (see mxfp8_op) and does not change the arithmetic. Requires K % 32 == 0,
 * M % 16 == 0 and N % 16 == 0. Accuracy: |C - C_exact| <= 2^-9 * sum_k |a_k b_k| per
 * element before the output rounding.
 * Empty sizes read no operand, so A, B and their scales may then be NULL:
 *  - M == 0 or N == 0 writes nothing and returns MXFP8_OK.
 *  - K == 0 zero-fills C, the empty sum; C must then be valid and 16-byte aligned.
 */
int mxfp8_gemm(const void* A_dev, const void* sA_dev, const void* B_dev, const void* sB_dev,
               void* C_dev, int64_t M, int64_t N, int64_t K, int op, int out_dtype,
               void* stream);

/*
 * mxfp8_gemm with a caller-owned device workspace, which lets the GEMM run its last,
 * partial wave of output tiles as split-K pieces. The rest of the tiles run as usual.
 *  - Split-K: each tile of that wave is cut into 3 ranges of K on separate CTA pairs. Two
 *    pieces leave FP32 partial sums in the workspace, and the third adds them before
 *    rounding.
 *  - Without a workspace: that wave runs as half-width tiles. On deep reductions the
 *    pieces finish it sooner.
 *  - Results: either way they meet the mxfp8_gemm accuracy bound. They are not bit-identical
 *    to mxfp8_gemm's, because the FP32 sums are added in another order.
 * Arguments as for mxfp8_gemm, plus:
 *   workspace_dev    device memory, 32-byte aligned, or NULL; the library allocates nothing.
 *   workspace_bytes  its size. Split-K runs only when it is at least
 *                    mxfp8_gemm_workspace_bytes for the same problem, else the call
 *                    proceeds as mxfp8_gemm.
 * The workspace holds the partial sums and one arrival counter per tile, CTA and epilogue
 * warp. It must be zero-filled before its first use. Each launch sets its counters back to
 * zero, so it needs no reset between calls or CUDA-graph replays. There is one exception:
 * after a call that latched MXFP8_ERR_TIMEOUT, zero-fill it again. Only one GEMM may use a
 * workspace at a time, so GEMMs that can run concurrently (other streams) need workspaces of
 * their own.
 * Errors as for mxfp8_gemm, plus MXFP8_ERR_ALIGNMENT for a misaligned workspace. A piece
 * whose partners do not arrive within the pipeline wait limit latches MXFP8_ERR_TIMEOUT.
 */
int mxfp8_gemm_ws(const void* A_dev, const void* sA_dev, const void* B_dev, const void* sB_dev,
                  void* C_dev, int64_t M, int64_t N, int64_t K, int op, int out_dtype,
                  void* workspace_dev, size_t workspace_bytes, void* stream);

/*
 * Workspace bytes with which mxfp8_gemm_ws runs this GEMM's last wave as split-K pieces
 * on the current device. The size depends on the device's SM count. 0 means the GEMM never
 * splits: its last wave is full or too wide, or K is too shallow (fewer than 120 stages of
 * 128, where the half tiles finish first). The same 0 is returned for arguments mxfp8_gemm
 * would refuse, and for an unsupported device.
 */
size_t mxfp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int op, int out_dtype);

/*
 * GEMM of block-wise FP8 operands (tcgen05 kind::f8f6f4, E4M3 x E4M3): C[M][N] =
 * sum_k deq(A)[m][k] * deq(B)[n][k], both operands K-major. The product of each 128-deep
 * block is accumulated by the tensor cores in FP32 and folded, times its two scales, into
 * an FP32 sum in registers, so scales need not be powers of two.
 *   A_dev / sA_dev  E4M3 [M][K] and float [ceil(K/128)][M], 1 x 128 blocks
 *                   (mxfp8_quantize_blockwise_1d)
 *   B_dev / sB_dev  FPROP, DGRAD: E4M3 [N][K] and float [ceil(N/128)][ceil(K/128)],
 *                   128 x 128 blocks (mxfp8_quantize_blockwise, or the transposed copy of
 *                   mxfp8_quantize_blockwise_dual for DGRAD);
 *                   WGRAD: E4M3 [N][K] and float [ceil(K/128)][N], 1 x 128 blocks (K = the
 *                   tokens, padded as the COL copies are)
 *   C_dev           [M][N], BF16 or FP32, fully overwritten
 * Requires K % 16 == 0 and N % 8 == 0; any M (WGRAD too). Accuracy: |C - C_exact| <=
 * 2^-9 * sum_k |a_k b_k| per element before the output rounding for K up to 2^22, and
 * K 2^-31 * sum_k |a_k b_k| beyond (the worst case of an FP32 sum over the blocks), as long as
 * the products of its blocks' two scales, which are formed in FP32, are normal numbers or zero.
 * A NaN scale or code gives NaN in the elements it reaches. Deterministic.
 * Empty sizes: M == 0 or N == 0 writes nothing, K == 0 zero-fills C (the operands may then
 * be NULL).
 * Errors: MXFP8_ERR_INVALID_ARG (negative or too large sizes, unknown enums, null
 * pointers), MXFP8_ERR_ALIGNMENT (K % 16, N % 8, codes or C not 16-byte aligned, scales
 * not 4-byte aligned); a pipeline wait that runs out latches MXFP8_ERR_TIMEOUT.
 */
int mxfp8_blockwise_gemm(const void* A_dev, const float* sA_dev, const void* B_dev,
                         const float* sB_dev, void* C_dev, int64_t M, int64_t N, int64_t K,
                         int op, int out_dtype, void* stream);

/*
 * mxfp8_blockwise_gemm with a caller-owned workspace, which lets it run on the block-scaled
 * MMA of mxfp8_gemm when every scale is a power of two (2^-127 .. 2^127, or NaN): the scale of
 * a block of 128 is then the E8M0 scale of its four blocks of 32. The device finds out: a
 * kernel converts the scales and checks them, then one of the two GEMMs runs and the other
 * returns at once. Both meet the accuracy bound; they are not bit-identical. For an FP32 result
 * the tensor cores sum 512 products at a time, and those sums are added in FP32. For a BF16
 * result they sum all of K, which costs up to K 2^-28 * sum_k |a_k b_k|, so that only reductions
 * of up to 2^17 run that way.
 *   workspace_dev    device memory, 16-byte aligned, or NULL; contents do not matter. One GEMM
 *                    at a time may use it.
 *   workspace_bytes  its size. Below mxfp8_blockwise_gemm_workspace_bytes the call proceeds as
 *                    mxfp8_blockwise_gemm.
 */
int mxfp8_blockwise_gemm_ws(const void* A_dev, const float* sA_dev, const void* B_dev,
                            const float* sB_dev, void* C_dev, int64_t M, int64_t N, int64_t K,
                            int op, int out_dtype, void* workspace_dev, size_t workspace_bytes,
                            void* stream);

/*
 * Workspace bytes of mxfp8_blockwise_gemm_ws for one problem; 0 where neither a forward (or data
 * gradient) nor a weight gradient of these sizes would use one: the block-scaled MMA is tried
 * where it is estimated to save power-of-two scales at least the 7 us that the conversion and the
 * check cost others. 0 too for a BF16 result of a reduction longer than 2^17, invalid arguments
 * or no supported device.
 */
size_t mxfp8_blockwise_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int out_dtype);

/*
 * Grouped (MoE expert) block-scaled GEMMs over token segments off[e] .. off[e+1]
 * (expert_offsets_dev as for mxfp8_quantize_grouped).
 *   op FPROP / DGRAD:  A [total_rows][K] with grouped ROW scales (one block per expert,
 *                      as written by mxfp8_quantize_grouped ROW); B [E][N][K] with
 *                      batched SWIZZLED scales (mxfp8_quantize_batched); C
 *                      [total_rows][N]: rows of expert e get A_e . B[e]^T. C rows of
 *                      no expert (none when off[E] = total_rows) are not written.
 *   op WGRAD:          A [N][total_rows] and B [K][total_rows] (column-wise copies,
 *                      grouped COL scales); C [E][N][K], C[e] = A[:, seg e] .
 *                      B[:, seg e]^T; an expert with no tokens gets C[e] = 0.
 * Requires K % 32 == 0, N % 16 == 0, total_rows % 32 == 0, and for WGRAD K % 16 == 0.
 * Empty sizes read no operand and run no kernel: A, B and their scales may then be NULL,
 * and the offsets are not read.
 *  - An empty output is a no-op that returns MXFP8_OK: N == 0, or K == 0 for WGRAD, or
 *    total_rows == 0 (no routed tokens) for FPROP / DGRAD.
 *  - A reduction over nothing zero-fills C, which must then be valid and 16-byte aligned:
 *    WGRAD with total_rows == 0, or FPROP / DGRAD with K == 0.
 */
int mxfp8_grouped_gemm(const void* A_dev, const void* sA_dev, const void* B_dev,
                       const void* sB_dev, void* C_dev, const int32_t* expert_offsets_dev,
                       int num_experts, int64_t total_rows, int64_t N, int64_t K, int op,
                       int out_dtype, void* stream);

/*
 * Workspace bytes mxfp8_selfcheck needs for `tokens` random input rows against an
 * [N][K] weight (0 for invalid sizes: tokens % 16, N % 16 and K % 32 must be 0, and the
 * size must fit in 64 bits).
 */
size_t mxfp8_selfcheck_workspace_bytes(int64_t tokens, int64_t N, int64_t K);

/*
 * Post-synchronization self-check of one quantized weight (section "Correctness: how it
 * fails", the post-sync self-check, condition C3). The BF16 input x [tokens][K] is
 * quantized and multiplied, by this library's kernels, with the weight exactly as the
 * GEMM reads it: w_codes_dev (E4M3 [N][K]) and w_scales_dev (SWIZZLED), i.e. the derived
 * layout - one dense layer, or one expert's slice of a batched expert weight. The result
 * is compared with a reference that multiplies the BF16 input with the canonical
 * synchronized weight, ref_codes_dev (E4M3 [N][K]) and ref_scales_dev (LINEAR
 * [N][K/32]), dequantized, with FP32 accumulation. Writes
 * ||Y - Y_ref||_F / ||Y_ref||_F to *rel_err_dev (device float). A healthy weight gives a
 * few percent (the activations' quantization error); a derived layout that is stale or
 * misplaced relative to the synchronized weight gives order 1; the pages' tolerance is
 * 0.25. Requires tokens % 16 == 0, N % 16 == 0, K % 32 == 0 and tokens <= 2097120;
 * sizes whose workspace would not fit in 64 bits are invalid (MXFP8_ERR_INVALID_ARG).
 *   workspace_dev  caller-owned, >= mxfp8_selfcheck_workspace_bytes(tokens, N, K)
 *                  bytes, 256-byte aligned; holds the quantized input, the FP32 output
 *                  and the two reduction sums. Overwritten.
 * Asynchronous on `stream` like the other calls.
 */
int mxfp8_selfcheck(const void* w_codes_dev, const void* w_scales_dev,
                    const void* ref_codes_dev, const void* ref_scales_dev, int64_t N, int64_t K,
                    const void* x_bf16_dev, int64_t tokens, void* workspace_dev,
                    size_t workspace_bytes, float* rel_err_dev, void* stream);

/*
 * mxfp8_selfcheck without a caller-provided workspace, for callers that cannot allocate
 * device memory when the check runs - for instance a serving engine's post-update hook
 * running while the engine's caching allocator holds all free device memory, or a
 * plugin that has no handle to the host framework's allocator. This entry point has no
 * counterpart on the pages; it exists for those callers.
 *   Arguments and result as mxfp8_selfcheck. The workspace is a fixed 8 MiB array
 *   inside the library (every device that loads the library holds it until the process
 *   exits), so mxfp8_selfcheck_workspace_bytes(tokens, N, K) must not exceed
 *   8 MiB (8388608 bytes); larger sizes return MXFP8_ERR_INVALID_ARG.
 *   No device memory is allocated and no allocating library routine is called.
 *   The first call on a device looks up the array's device address on that device
 *   (under a lock, so host threads may make their first calls at the same time); make
 *   that first call before any stream capture.
 *   All calls share the one array: calls that overlap on the GPU (other streams, other
 *   host threads) race on it and must be serialised by the caller. Every call
 *   rewrites what it reads, and clears its two reduction sums itself.
 */
int mxfp8_selfcheck_noalloc(const void* w_codes_dev, const void* w_scales_dev,
                            const void* ref_codes_dev, const void* ref_scales_dev, int64_t N,
                            int64_t K, const void* x_bf16_dev, int64_t tokens,
                            float* rel_err_dev, void* stream);

#define MXFP8_MAX_TOP 32

/*
 * Log probabilities of given tokens: for each row of logits x, with temperature T,
 * m = max x and log_sum = log sum_v exp((x_v - m) / T),
 *   logprob = (x_target - m) / T - log_sum,
 *   entropy = -sum_v p_v log p_v,  p = softmax(x / T),
 * and the `top` likeliest tokens. The pages measure the drift between sampler and learner by
 * these log probabilities (section "A different grid, and drift").
 *   logits_dev       BF16 or FP32 (logits_dtype: MXFP8_OUT_BF16 / MXFP8_OUT_FP32)
 *                    [rows][ld], aligned to its element; the first `vocab` values of each
 *                    row are read, ld >= vocab
 *   targets_dev      int64 [rows]. A negative target is not scored: its logprob is 0. One
 *                    at or past vocab gives NaN and latches MXFP8_ERR_BAD_TARGET.
 *   logprob_dev      float [rows]
 *   entropy_dev      float [rows]
 *   stats_dev        float [rows][2]: m and log_sum, which the gradient call reads
 *   top              0 .. MXFP8_MAX_TOP
 *   top_logprob_dev  float [rows][top], falling; NULL if top == 0
 *   top_id_dev       int64 [rows][top]; equal logits: the lowest token first. Where fewer
 *                    than `top` logits are above -inf: -1, with log probability -inf.
 * Masks: a logit of -inf has probability 0. A row whose logits are all -inf has log
 * probability -inf (0 if not scored), entropy 0, stats (-inf, 0) and no top tokens. A row
 * holding a NaN or +inf gives NaN (top_id -1).
 * Sums are FP32: log_sum is off by at most (max(256, vocab / 256) + 64) 2^-24 + 2^-20.
 * Deterministic. rows == 0 is a no-op.
 * Errors: MXFP8_ERR_INVALID_ARG (negative sizes, vocab == 0 or above 2^31 - 1, ld < vocab,
 * a temperature that is not positive or whose reciprocal is not a finite, normal float, top
 * out of range, unknown dtype, null pointers), MXFP8_ERR_ALIGNMENT.
 */
int mxfp8_token_logprobs(const void* logits_dev, int logits_dtype, int64_t rows,
                         int64_t vocab, int64_t ld, const int64_t* targets_dev,
                         double temperature, float* logprob_dev, float* entropy_dev,
                         float* stats_dev, int top, float* top_logprob_dev,
                         int64_t* top_id_dev, void* stream);

/*
 * Gradient of the three results of mxfp8_token_logprobs with respect to the logits:
 *   dx_v = (1/T) [ g 1(v = target) + sum_j gt_j 1(v = id_j)
 *                  - p_v (g + sum_j gt_j + h (log p_v + entropy)) ]
 *   targets_dev, stats_dev, entropy_dev, top_id_dev   as that call read or wrote them
 *   grad_logprob_dev  g, float [rows] (not read where the target is negative: 0)
 *   grad_entropy_dev  h, float [rows], or NULL for 0
 *   grad_top_dev      gt, float [rows][top]; NULL, as top_id_dev, if top == 0. A negative
 *                     id is skipped, and its gt is not read. One at or past vocab, like such
 *                     a target, makes the row NaN and latches MXFP8_ERR_BAD_TARGET.
 *   grad_logits_dev   the logits' dtype, [rows][grad_ld], its first `vocab` columns
 *                     written; may be the logits' own buffer (then grad_ld == ld), else
 *                     the two may not overlap. Where its rows start at another place within
 *                     16 bytes than the logits' (another alignment, or pitches that differ by
 *                     no multiple of 16 bytes), values go one at a time: 2 to 3 times slower
 * A row whose logits are all -inf gets zeros, whatever its g, h and gt. Errors as above.
 */
int mxfp8_token_logprobs_backward(const void* logits_dev, int logits_dtype, int64_t rows,
                                  int64_t vocab, int64_t ld, const int64_t* targets_dev,
                                  double temperature, const float* stats_dev,
                                  const float* entropy_dev, const float* grad_logprob_dev,
                                  const float* grad_entropy_dev, int top,
                                  const int64_t* top_id_dev, const float* grad_top_dev,
                                  void* grad_logits_dev, int64_t grad_ld, void* stream);

/*
 * Routing of tokens to experts: what makes the token segments that the grouped calls read, and
 * takes their results back. Entry i = t * top_k + j is token t's j-th choice of an expert. A
 * plan is three int32 arrays that mxfp8_route writes:
 *   offsets   [num_experts + 1], the segments as mxfp8_quantize_grouped and mxfp8_grouped_gemm
 *             take them: starts at 0, multiples of 32, ends at total_rows
 *   row_of    [tokens * top_k], the segment row of each entry, -1 for an entry of no expert
 *   entry_of  [total_rows], the entry of each row, -1 for a padding row
 * The pages pad token segments to multiples of 32 (section "The pipeline", learner paragraph) and
 * train a mixture of experts (section "A held-out workload, and end to end", Table 4); how tokens
 * get to their experts is this library's.
 */

/*
 * A number of rows that the segments of any choice fit in: tokens * top_k, plus 31 rows of
 * padding for each expert that can be in use, rounded down to a multiple of 32. 0 for no entries and
 * for invalid arguments (negative tokens, top_k < 1, num_experts outside 1 .. 1024, or a result
 * above 2^31 - 256).
 */
int64_t mxfp8_route_rows(int64_t tokens, int top_k, int num_experts);

/*
 * Sorts the entries by expert. Entries of an expert keep their order, so the plan does not
 * depend on timing.
 *   ids_dev      int64 [tokens][top_k], 8-byte aligned. A negative id is an entry of no expert
 *                (a dropped token, a padding token). One at or past num_experts is treated so
 *                too, and latches MXFP8_ERR_BAD_EXPERT. A token may name an expert twice.
 *   total_rows   a multiple of 32: mxfp8_route_rows, or fewer where the caller knows the counts.
 *                The last expert's segment takes the rows that are left over, as padding. If the
 *                segments need more, the plan is one of no entries (offsets 0 .. 0, total_rows;
 *                all else -1) and MXFP8_ERR_BAD_OFFSETS is latched.
 *   offsets_dev, row_of_dev, entry_of_dev   the plan, written in full
 * tokens * top_k up to 2^31 - 256, num_experts 1 .. 1024. No entries: ids_dev and row_of_dev may
 * be NULL; total_rows == 0: entry_of_dev too.
 */
int mxfp8_route(const int64_t* ids_dev, int64_t tokens, int top_k, int num_experts,
                int64_t total_rows, int32_t* offsets_dev, int32_t* row_of_dev,
                int32_t* entry_of_dev, void* stream);

/*
 * Copies the tokens' rows into the segments: out[row_of[i]] = w_i x[i / top_k]; padding rows
 * become zero. The gradient of x is mxfp8_combine without weights; that of the weights is the
 * inner products mxfp8_combine_backward gives.
 *   x_dev        [tokens][cols], BF16 or FP32 (dtype: MXFP8_OUT_BF16 / MXFP8_OUT_FP32)
 *   weights_dev  float [tokens][top_k], or NULL for 1 (the values then move unchanged). Products
 *                are FP32, rounded once.
 *   out_dev      [total_rows][cols], of x's type, written in full; may not overlap x
 * Up to 2097120 cols (65535 * 32); rows of a multiple of 16 bytes are the fastest, of an odd
 * number of BF16 values the slowest. x and out start on 16 bytes. A plan whose rows do not fit
 * total_rows is not followed there: MXFP8_ERR_BAD_OFFSETS is latched and the row skipped. Of a plan
 * that mxfp8_route did not write, no two entries may share a row, and row_of and entry_of agree.
 */
int mxfp8_dispatch(const void* x_dev, int dtype, int64_t tokens, int64_t cols, int top_k,
                   const float* weights_dev, const int32_t* row_of_dev,
                   const int32_t* entry_of_dev, int64_t total_rows, void* out_dev, void* stream);

/*
 * mxfp8_dispatch of BF16 rows straight into the grouped GEMMs' MXFP8 operands: the bytes are
 * those of mxfp8_quantize_grouped on the dispatched rows, which are never written.
 *   row_out_dev, row_scales_dev   the ROW copy, E4M3 [total_rows][cols]; cols % 32 == 0
 *   col_out_dev, col_scales_dev   the COL copy, E4M3 [cols][total_rows]; cols % 8 == 0
 * Either copy may be left out (both its pointers NULL), not both. Scale buffers hold
 * mxfp8_grouped_scale_bytes(total_rows, cols, num_experts, axis) bytes and are written in full:
 * zeros follow the last block. Invalid offsets latch MXFP8_ERR_BAD_OFFSETS and write nothing.
 * total_rows == 0 or cols == 0 is a no-op. tokens * cols below 2^35, at most 65535 - num_experts
 * tiles of 128 rows. x and all four outputs start on 16 bytes; none overlaps another.
 */
int mxfp8_quantize_dispatch(const void* x_dev, int64_t tokens, int64_t cols, int top_k,
                            const float* weights_dev, const int32_t* row_of_dev,
                            const int32_t* entry_of_dev, int64_t total_rows,
                            const int32_t* offsets_dev, int num_experts,
                            void* row_out_dev, void* row_scales_dev, void* col_out_dev,
                            void* col_scales_dev, void* stream);

/*
 * Sums the segments' rows back to their tokens: out[t] = sum_j w_i y[row_of[i]], i = t top_k + j,
 * over the entries that have a row (none: zeros; their weights are not read). FP32 sums in the order
 * of j, rounded once. Without weights this is the gradient of mxfp8_dispatch without weights.
 *   y_dev        [total_rows][cols], BF16 or FP32
 *   weights_dev  float [tokens][top_k], or NULL for 1
 *   out_dev      [tokens][cols], of y's type; may not overlap y
 * Sizes, alignment and errors as for mxfp8_dispatch.
 */
int mxfp8_combine(const void* y_dev, int dtype, int64_t total_rows, int64_t cols, int64_t tokens,
                  int top_k, const float* weights_dev, const int32_t* row_of_dev, void* out_dev,
                  void* stream);

/*
 * Gradients of mxfp8_combine: grad_y[row_of[i]] = w_i grad_out[t] (zeros in padding rows), and
 * grad_weights[i] = <grad_out[t], y[row_of[i]]> (0 for an entry without a row), FP32 sums.
 *   grad_out_dev      [tokens][cols], of y's type
 *   grad_y_dev        [total_rows][cols], of y's type, written in full, or NULL where only the
 *                     weights' gradient is wanted (entry_of_dev may then be NULL): the rows'
 *                     gradient also comes from mxfp8_quantize_dispatch(grad_out, weights), on the
 *                     MXFP8 grid. May be y itself, else the two may not overlap. It may not
 *                     overlap grad_out.
 *   grad_weights_dev  float [tokens][top_k]
 */
int mxfp8_combine_backward(const void* grad_out_dev, const void* y_dev, int dtype,
                           int64_t tokens, int64_t cols, int top_k, const float* weights_dev,
                           const int32_t* row_of_dev, const int32_t* entry_of_dev,
                           int64_t total_rows, void* grad_y_dev, float* grad_weights_dev,
                           void* stream);

/*
 * The gated activation h = silu(g) * u, silu(g) = g / (1 + e^-g), of x = [g | u], with x kept in 8
 * bits for the backward pass (2.0625 bytes for each value of h, 4 as BF16).
 *   x_dev       BF16 [rows][2 * width], width % 32 == 0
 *   h_dev       BF16 [rows][width], from x itself, rounded once
 *   codes_dev   E4M3 [rows][2 * width], scales_dev [rows][2 * width / 32]: the bytes of
 *               mxfp8_quantize_rule(x, ROW, LINEAR, scale_rule); both NULL: not kept.
 *               MXFP8_RULE_CEIL saturates nothing: every value of a block is then within 2^-4 of
 *               itself or within 2^-17 of the block's largest where that is 2^-120 or more (within
 *               2^-137 where it is less). BF16's largest numbers, from 1.9375 * 2^127, are kept as
 *               2^128.
 * A gate of -inf gives NaN; sigmoids below 2^-126 are 0.
 * All buffers start on 16 bytes (scales_dev anywhere), and no two overlap. rows == 0 or width == 0
 * is a no-op.
 */
int mxfp8_swiglu(const void* x_dev, int64_t rows, int64_t width, void* h_dev, void* codes_dev,
                 void* scales_dev, int scale_rule, void* stream);

/*
 * Gradient of mxfp8_swiglu from what it kept: with g, u the kept values, s = 1 / (1 + e^-g),
 *   grad_x = [grad_h u s (1 + g (1 - s)) | grad_h g s], and h = g s u again,
 * FP32, each rounded to BF16 once. A kept value of 2^128 or more counts as FP32's largest number. A
 * block kept with a NaN scale gives NaN.
 *   grad_h_dev  BF16 [rows][width]
 *   grad_x_dev  BF16 [rows][2 * width]; may not overlap the inputs
 *   h_dev       BF16 [rows][width], or NULL: not wanted. May be grad_h itself.
 */
int mxfp8_swiglu_backward(const void* grad_h_dev, const void* codes_dev, const void* scales_dev,
                          int64_t rows, int64_t width, void* grad_x_dev, void* h_dev,
                          void* stream);

/*
 * Sets how long a GEMM kernel's pipeline waits (a stage's copies, the tensor cores, the
 * accumulator hand-over) may take before the kernel gives up, for every GEMM launched
 * after the call, in any host thread: `ns` nanoseconds, or the default for ns == 0
 * (MXFP8_WAIT_LIMIT_MS from the environment, else 4 s). Failure detection (the post's
 * section "Correctness: how it fails" lists the failures a pipeline must not hang on): a
 * kernel whose wait runs out latches MXFP8_ERR_TIMEOUT, stops issuing work, waits for the
 * copies and tensor-core operations it has in flight (for at least 2 s, independently of
 * this limit), frees its tensor memory and returns; its outputs are then unspecified. A
 * limit shorter than a tile's computation makes every GEMM time out, which is how the
 * tests exercise that path. The pages have no counterpart for this call. Returns MXFP8_OK.
 */
int mxfp8_set_wait_limit_ns(uint64_t ns);

/*
 * Synchronizes `stream`, then returns and clears the current device's status word:
 * MXFP8_OK, or the first device-side error latched since the last call
 * (MXFP8_ERR_BAD_OFFSETS, MXFP8_ERR_TIMEOUT, MXFP8_ERR_BAD_TARGET, MXFP8_ERR_BAD_EXPERT), or
 * MXFP8_ERR_CUDA if the synchronization itself failed. The word is read and cleared in one atomic
 * exchange, enqueued on `stream` after its earlier work. An error that a kernel on another stream
 * latches concurrently is reported by this call or by the next one; it is never cleared unread.
 */
int mxfp8_get_device_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_H_ */
