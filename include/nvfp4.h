/*
 * nvfp4.h - C ABI of libnvfp4: NVFP4 block quantization and block-scaled GEMMs on MI355X.
 *
 * The format (from "Nemotron NVFP4" explainer, ai.thesatyajit.com, section "What NVFP4
 * actually is"): every element is a 4-bit E2M1 float (1 sign, 2 exponent, 1 mantissa bit),
 * every 16 consecutive elements share one FP8 E4M3 scale, and the whole tensor shares one
 * FP32 scale, 4.5 bits per element in total. Activations and gradients use 1x16 blocks,
 * weights use 16x16 blocks (artiverse.ca "NVIDIA's 4-bit floating point pushes AI training
 * limits", stabilizer paragraph); gradients are rounded stochastically, everything else to
 * nearest (same page; explainer section "Why 4-bit training normally falls apart - and the
 * three fixes"); the weight-gradient GEMM's operands go through a 16-point random-sign
 * Hadamard transform first (same explainer section).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers on the current HIP device. The caller
 *     allocates every buffer and owns it; the library allocates nothing and keeps no state
 *     between calls, so calls are re-entrant on different streams.
 *   - All work is enqueued asynchronously on `hip_stream` (a hipStream_t; NULL = the null
 *     stream). The library never synchronizes; a device fault surfaces at the caller's next
 *     synchronization.
 *   - Arguments are validated on the host before anything is enqueued. On any non-OK status
 *     nothing was enqueued (except NVFP4_ERR_HIP, where a launch itself failed) and
 *     nvfp4_last_error() describes the problem (thread-local string).
 *   - Device-resident arguments (segment/offset tables, amax values) cannot be checked on the
 *     host; their preconditions are stated per function. Violating them gives unspecified
 *     output but never an out-of-bounds access: kernels clamp table lookups.
 *   - Non-finite inputs (Inf/NaN) are outside the contract: outputs are unspecified, the
 *     kernels still terminate normally.
 *   - Empty tensors are valid: with no rows (or an output without rows or columns) nothing is
 *     read or written and the buffer pointers may be NULL; the amax of an empty tensor is 0
 *     (amax_out is still written).
 *
 * NVFP4 tensor layout (nvfp4_tensor), for a logical matrix [rows, cols] quantized along cols:
 *   codes        uint8 [rows, cols/2] row-major; element 2i in the low nibble, 2i+1 in the
 *                high nibble; nibble = sign<<3 | exponent<<1 | mantissa (E2M1, bias 1).
 *   scales       uint8 [rows, cols/16] row-major E4M3 (OCP "FN": bias 7, max 448) codes.
 *                A 16x16 weight tile stores its one scale in each of its 16 rows.
 *   global_scale float [nseg] decode scale s_dec = amax/2688 per segment (1.0 if amax = 0).
 *   Dequantized value: e2m1(code) * e4m3(scale) * global_scale[segment of row].
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NVFP4_OK = 0,
  NVFP4_ERR_INVALID = -1,      /* bad pointer, shape, enum or size                     */
  NVFP4_ERR_UNSUPPORTED = -2,  /* valid request this library does not implement        */
  NVFP4_ERR_WORKSPACE = -3,    /* workspace missing or smaller than nvfp4_workspace_size */
  NVFP4_ERR_HIP = -4           /* a HIP launch failed (message holds hipGetErrorString) */
} nvfp4_status;

typedef enum { NVFP4_IN_BF16 = 0, NVFP4_IN_FP32 = 1 } nvfp4_dtype;
typedef enum { NVFP4_BLOCK_1X16 = 0, NVFP4_BLOCK_16X16 = 1 } nvfp4_block;
typedef enum { NVFP4_ROUND_RN = 0, NVFP4_ROUND_SR = 1 } nvfp4_round;
typedef enum {
  NVFP4_OP_QUANTIZE = 0, NVFP4_OP_RHT_QUANTIZE = 1, NVFP4_OP_GEMM = 2,
  NVFP4_OP_GROUPED_GEMM = 3, NVFP4_OP_AMAX_PAIR = 4, NVFP4_OP_GEMM_EX = 5, NVFP4_OP_ADAMW = 6,
  NVFP4_OP_GEMM_ACT = 7, NVFP4_OP_ACT_GRAD = 8, NVFP4_OP_NORM_GRAD = 9, NVFP4_OP_MOE_SORT = 10,
  NVFP4_OP_HEAD_LOSS = 11, NVFP4_OP_HEAD_GRAD = 12
} nvfp4_op;
/* Output of nvfp4_gemm_ex: FP32, FP32 added to what D holds, or BF16. */
typedef enum { NVFP4_OUT_FP32 = 0, NVFP4_OUT_FP32_ACCUMULATE = 1, NVFP4_OUT_BF16 = 2 } nvfp4_out;

typedef struct nvfp4_tensor {
  uint8_t* codes;        /* device, [rows, cols/2]                       */
  uint8_t* scales;       /* device, [rows, cols/16]                      */
  float* global_scale;   /* device, [nseg] (1 for an unsegmented tensor) */
  int64_t rows;
  int64_t cols;          /* the quantized (contraction) dimension, % 16 == 0 */
} nvfp4_tensor;

/* MXFP4 tensor [rows, cols] quantized along cols: codes as nvfp4_tensor, one E8M0 scale per
 * 32 elements (value 2^(code - 127)), no tensor-level scale. The scales are stored K step by
 * K step: scale j of row r (elements 32j .. 32j+31) at byte ((j / 4) * rows + r) * 4 + j % 4,
 * ceil(cols/128) * rows * 4 bytes, so the four scales of one 128-element step of all rows are
 * contiguous (one DMA request per 32 rows in the GEMM, conflict-free reads in LDS); bytes past
 * a row's last block (cols % 128 != 0) are left unwritten. */
typedef struct mxfp4_tensor {
  uint8_t* codes;        /* device, [rows, cols/2]                     */
  uint8_t* scales;       /* device, [ceil(cols/128), rows, 4] (above)  */
  int64_t rows;
  int64_t cols;          /* % 32 == 0 */
} mxfp4_tensor;

/* A matrix [rows, cols] in 8 bits, as the optimizer's 8-bit states: E4M3 codes and one power of two
 * per 32 consecutive elements of a row (the last block of a row may be shorter), E8M0 code e + 127. */
typedef struct nvfp4_fp8_tensor {
  uint8_t* codes;        /* device, [rows, cols], 16-byte aligned */
  uint8_t* scales;       /* device, [rows, ceil(cols/32)]         */
  int64_t rows;
  int64_t cols;
} nvfp4_fp8_tensor;

/*
 * nvfp4_quantize - two-level block quantization of x[rows, cols] along cols.
 * Defined by: "Nemotron NVFP4" explainer, "What NVFP4 actually is" (E2M1 elements, one E4M3
 * scale per 16 elements, one FP32 tensor scale) and "Why 4-bit training normally falls
 * apart - and the three fixes" (2D weight blocks; stochastic rounding for gradients).
 *
 *   x         device BF16 or FP32 (dt), element (r, c) at x[r*ld + c]; ld >= cols.
 *   blk       NVFP4_BLOCK_1X16 (scale per 16 consecutive elements of a row) or
 *             NVFP4_BLOCK_16X16 (one scale per aligned 16x16 tile; rows % 16 == 0).
 *   rnd       NVFP4_ROUND_RN, or NVFP4_ROUND_SR (1x16 only): element j of the block with
 *             row-major index b uses byte j%4 of word j/4 of Philox4x32-10 with key
 *             (lo32 seed, hi32 seed) and counter (lo32 b, hi32 b, lo32 offset, hi32 offset);
 *             it rounds up iff frac + byte/256 >= 1.
 *   segments  NULL (nseg must be 1) or device int64[nseg+1] row offsets with
 *             segments[0] = 0 <= ... <= segments[nseg] <= rows (non-decreasing; multiples
 *             of 16 for 16X16). Each segment gets its own amax and global scale (expert
 *             stacks of a mixture-of-experts layer). Rows from segments[nseg] on (nvfp4_moe_sort
 *             can leave some, which nvfp4_moe_gather fills with zeros) count as the last segment's,
 *             in its amax too.
 *   amax_in   NULL, or device float[nseg] holding max|x| per segment; then the amax pass is
 *             skipped and no workspace is needed.
 *   out       codes/scales/global_scale as documented above; out->rows == rows,
 *             out->cols == cols.
 *   out_t     NULL, or (16X16) a second tensor receiving the quantization of x^T ([cols, rows]
 *             along rows): the same tile scales and codes, transposed. With segments (a
 *             stack of nseg expert weights) they must be nseg equal blocks of n = rows/nseg
 *             rows (n % 16 == 0; the table must match) and out_t is [nseg*cols, n]: rows
 *             g*cols .. hold expert g's transpose, with global_scale[g] (the operand of the
 *             grouped activation-gradient GEMM).
 *   workspace device scratch of at least nvfp4_workspace_size(NVFP4_OP_QUANTIZE, rows,
 *             cols, nseg) bytes, 256-byte aligned; may be NULL when amax_in is given.
 * Errors: NVFP4_ERR_INVALID (null pointers, cols % 16, rows % 16 for 16X16, ld < cols, bad
 * enum, nseg < 1, segments == NULL with nseg != 1, out_t without 16X16, tensor shape
 * mismatch), NVFP4_ERR_UNSUPPORTED (SR with 16X16, out_t with unequal or misaligned segments),
 * NVFP4_ERR_WORKSPACE, NVFP4_ERR_HIP.
 */
int nvfp4_quantize(const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols, int64_t ld,
                   nvfp4_block blk, nvfp4_round rnd, uint64_t seed, uint64_t offset,
                   const int64_t* segments, int64_t nseg, const float* amax_in,
                   nvfp4_tensor* out, nvfp4_tensor* out_t,
                   void* workspace, size_t ws_bytes, void* hip_stream);

/*
 * nvfp4_quantize_noalloc - nvfp4_quantize for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid allocation. Same
 * arguments, results and errors as nvfp4_quantize minus the workspace: the amax pass keeps its
 * partial (or per-segment) maxima in a static device array of the library, 64 KiB per device,
 * held until the process ends. The call allocates nothing (its first call on a device looks up
 * that device's array once); anything that must start at zero is cleared by a kernel, not a
 * memset, so the call can be captured in a graph.
 *   nseg       at most 16384 (NVFP4_ERR_UNSUPPORTED beyond, nothing enqueued).
 * Every call on one device shares that device's array: calls that overlap on one device (on
 * different streams, or from several threads without ordering) race and give unspecified
 * results. Calls ordered on one stream are safe.
 */
int nvfp4_quantize_noalloc(const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols, int64_t ld,
                           nvfp4_block blk, nvfp4_round rnd, uint64_t seed, uint64_t offset,
                           const int64_t* segments, int64_t nseg, const float* amax_in,
                           nvfp4_tensor* out, nvfp4_tensor* out_t, void* hip_stream);

/*
 * nvfp4_rht_quantize - random Hadamard transform along tokens, then 1x16 quantization of
 * the transposed result. Defined by: "Nemotron NVFP4" explainer, "Why 4-bit training
 * normally falls apart - and the three fixes" (a random Hadamard matrix on the wgrad inputs,
 * undone analytically inside the GEMM) and thelatentdaily "What matters for NVFP4
 * training?", "A methodological warning" (random sign vectors of the rotations).
 *
 *   x          device BF16/FP32 [tokens, cols], element (t, c) at x[t*ld + c];
 *              tokens % 16 == 0.
 *   sign_mask  bit j set => sign -1 on element j of every 16-token block. Both operands of
 *              one wgrad GEMM must use the same mask so that the transform cancels.
 *   transform  for column c and block t: y_i = rn32(1/4 * sum_j H[i][j] s_j x[16t+j, c]),
 *              H[i][j] = (-1)^popcount(i & j): the exact sum rounded once to FP32 (nearest,
 *              ties to even), +0 for an exactly zero sum, for every input (blocks of any
 *              exponent spread; a sum beyond the FP32 range gives infinity).
 *   out        tensor [cols, tokens]: row c holds column c's transformed values quantized in
 *              1x16 blocks along tokens (out->rows == cols, out->cols == tokens).
 *   rnd/seed/offset as for nvfp4_quantize (SR block index is over the output [cols, tokens]).
 *   segments   NULL (nseg must be 1) or device int64[nseg+1] TOKEN offsets, multiples of 16,
 *              non-decreasing from 0 to at most tokens (those behind count as the last
 *              segment's, as in nvfp4_quantize): the tokens routed to each expert of a
 *              mixture-of-experts layer, whose weight gradients are separate GEMMs over their
 *              own tokens (nvfp4_grouped_gemm_k). Each token range gets its own amax (over its
 *              transformed values) and global scale: out->global_scale[nseg]; out's column
 *              range of segment g uses global_scale[g]. A 16-token block belongs to the
 *              segment of its first token; unchecked device data, never an out-of-bounds
 *              access.
 *   amax_in    NULL or device float[nseg] = max|y| of the transformed values per segment.
 *   workspace  >= nvfp4_workspace_size(NVFP4_OP_RHT_QUANTIZE, tokens, cols, nseg) bytes
 *              unless amax_in is given.
 * Errors: as nvfp4_quantize (tokens % 16, cols < 1, ld < cols, nseg < 1, segments == NULL
 * with nseg != 1, ...).
 */
int nvfp4_rht_quantize(const void* x, nvfp4_dtype dt, int64_t tokens, int64_t cols, int64_t ld,
                       uint16_t sign_mask, nvfp4_round rnd, uint64_t seed, uint64_t offset,
                       const int64_t* segments, int64_t nseg, const float* amax_in,
                       nvfp4_tensor* out, void* workspace, size_t ws_bytes, void* hip_stream);

/*
 * mxfp4_quantize - MXFP4 quantization of x[rows, cols] along cols, the format the pages set
 * against NVFP4 ("Nemotron NVFP4" explainer, "What NVFP4 actually is": E2M1 elements, one
 * power-of-two E8M0 scale per 32 elements, 4.25 bits per element, no tensor scale). The
 * scale rule is the OCP Microscaling v1.0 conversion: shared exponent e = floor(log2(block
 * amax)) - 2 clamped to [-127, 127] (-127 for an all-zero block), element = E2M1(x * 2^-e)
 * rounded to nearest even (RN) or stochastically with the Philox bytes of nvfp4_quantize's SR
 * (16-element half-block index b = (row*cols + col)/16), saturating at 6. One pass, no
 * workspace.
 *   x    device BF16 or FP32 (dt), element (r, c) at x[r*ld + c]; 16-byte aligned, ld a
 *        multiple of 16 bytes' worth of elements.
 *   out  codes/scales, out->rows == rows, out->cols == cols (cols % 32 == 0).
 * Errors: NVFP4_ERR_INVALID (null pointers, shapes, enums), NVFP4_ERR_UNSUPPORTED (alignment),
 * NVFP4_ERR_HIP.
 */
int mxfp4_quantize(const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols, int64_t ld,
                   nvfp4_round rnd, uint64_t seed, uint64_t offset, mxfp4_tensor* out,
                   void* hip_stream);

/*
 * mxfp4_quantize_columns - MXFP4 quantization of x's columns: out [cols, rows] holds x^T
 * quantized along its rows, exactly mxfp4_quantize of the transposed tensor (same scale rule,
 * rounding and SR counters, with the half-block index b = (out_row*rows + out_col)/16 of the
 * output), without materializing x^T. The activation- and weight-gradient GEMMs contract W,
 * dY and X over their other dimension ("Nemotron NVFP4" explainer, "What NVFP4 actually is":
 * the MXFP4 comparison format, 32-element blocks along the contraction).
 *   x    device BF16 or FP32 [rows, cols], element (r, c) at x[r*ld + c]; element pairs aligned
 *        (ld any); rows % 32 == 0.
 *   out  out->rows == cols, out->cols == rows; codes 16-byte, scales 8-byte aligned.
 * Errors: NVFP4_ERR_INVALID (null pointers, shapes, rows % 32, enums, alignment of out),
 * NVFP4_ERR_UNSUPPORTED (misaligned x), NVFP4_ERR_HIP.
 */
int mxfp4_quantize_columns(const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols, int64_t ld,
                           nvfp4_round rnd, uint64_t seed, uint64_t offset, mxfp4_tensor* out,
                           void* hip_stream);

/*
 * mxfp4_gemm - D[M, N] (FP32, row stride ldd) = A[M, K] * B[N, K]^T with both operands MXFP4
 * (mxfp4_quantize along K): the comparison format of the pages ("Nemotron NVFP4" explainer,
 * "What NVFP4 actually is") on gfx950's block-scaled FP4 matrix instruction, which applies
 * the E8M0 scales of each 32-element block itself. Products exact, FP32 accumulation.
 *   A: rows = M, cols = K; B: rows = N, cols = K (same K, K % 128 == 0); ldd >= N; each
 *   operand's codes below 2 GiB, codes 16-byte and scales 4-byte aligned.
 * Errors: NVFP4_ERR_INVALID (null pointers, K mismatch, cols % 32, ldd < N, alignment),
 * NVFP4_ERR_UNSUPPORTED (K % 128, operand size), NVFP4_ERR_HIP.
 */
int mxfp4_gemm(const mxfp4_tensor* A, const mxfp4_tensor* B, float* D, int64_t ldd, void* hip_stream);

/*
 * nvfp4_rht_rows_quantize - the rowwise random-sign Hadamard transform then 1x16 quantization
 * along the rows: every 16-element block of a row goes through y = 1/4 * H16 * diag(s) * v
 * (the butterfly and rounding of nvfp4_rht_quantize, signs from sign_mask) and is quantized
 * as nvfp4_quantize's 1x16 blocks, with the tensor scale from max|y|. This is the activation
 * gradient of the Mosaic variant's activation-gradient GEMM (thelatentdaily "What matters for
 * NVFP4 training?": Hadamard transforms on both backward GEMMs, 1D weight quantization): with
 * B = nvfp4_rht_quantize(W, same mask) (W^T transformed along the output features), the
 * product of the two equals dY * W since the transform is orthogonal.
 *   x          device BF16/FP32 [rows, cols], cols % 16 == 0, 16-byte aligned rows.
 *   rnd, seed, offset  as nvfp4_quantize (block index b = row*(cols/16) + col/16).
 *   amax_in    NULL or device float[1] = max|y| (nvfp4_amax with rht = 2); then no workspace.
 *   out        [rows, cols], global_scale[1].
 *   workspace  nvfp4_workspace_size(NVFP4_OP_QUANTIZE, rows, cols, 1) bytes when amax_in is NULL.
 * Errors: NVFP4_ERR_INVALID, NVFP4_ERR_UNSUPPORTED (alignment), NVFP4_ERR_WORKSPACE, NVFP4_ERR_HIP.
 */
int nvfp4_rht_rows_quantize(const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols, int64_t ld,
                            uint16_t sign_mask, nvfp4_round rnd, uint64_t seed, uint64_t offset,
                            const float* amax_in, nvfp4_tensor* out, void* workspace, size_t ws_bytes,
                            void* hip_stream);

/*
 * nvfp4_gemm - D[M, N] (FP32, row stride ldd) = A[M, K] * B[N, K]^T with both operands
 * NVFP4 (each quantized along K), products accumulated in FP32, scaled by
 * A->global_scale[0] * B->global_scale[0]. Covers the forward, activation-gradient and
 * weight-gradient GEMMs of a linear layer (artiverse.ca "NVIDIA's 4-bit floating point
 * pushes AI training limits", paragraph on which parts run in 4-bit).
 *   A: rows = M, cols = K; B: rows = N, cols = K (same K, % 16 == 0); ldd >= N.
 * Errors: NVFP4_ERR_INVALID (null pointers, K mismatch, K % 16, ldd < N),
 * NVFP4_ERR_UNSUPPORTED (an operand's codes above 2 GiB: the kernels use 32-bit buffer
 * offsets; the same limit holds for every GEMM entry point), NVFP4_ERR_HIP.
 */
int nvfp4_gemm(const nvfp4_tensor* A, const nvfp4_tensor* B, float* D, int64_t ldd,
               void* hip_stream);

/*
 * nvfp4_gemm_ex - nvfp4_gemm with the outputs a linear layer needs around its three GEMMs
 * (artiverse.ca "NVIDIA's 4-bit floating point pushes AI training limits", paragraph on which
 * parts run in 4-bit: the GEMMs take NVFP4 operands, the layer's other tensors stay in higher
 * precision): the forward output and the activation gradient handed on in BF16, the weight
 * gradient accumulated into an FP32 main gradient, and the output's amax produced by the GEMM
 * itself, so the next quantization of D (amax_in) is a single pass.
 *   A, B       as nvfp4_gemm (rows M and N, same K, % 16 == 0).
 *   D          device [M, N] with row stride ldd >= N elements:
 *              NVFP4_OUT_FP32             float, D = s_A s_B A B^T (as nvfp4_gemm);
 *              NVFP4_OUT_FP32_ACCUMULATE  float, D = D + s_A s_B A B^T (one FP32 addition per
 *                                         element; D must hold finite values);
 *              NVFP4_OUT_BF16             bfloat16 bits (uint16), the FP32 result rounded to
 *                                         nearest, ties to even.
 *   amax_out   NULL, or device float[1] receiving max |D| over the values as stored (after the
 *              BF16 rounding; after the addition when accumulating). The library clears it.
 *   workspace  device scratch of nvfp4_workspace_size(NVFP4_OP_GEMM_EX, M, N, 1) bytes, sized
 *              for the current device, 256-byte aligned (0 bytes, NULL allowed, when the
 *              tiles fill whole rounds of the device's compute units, or leave a last round of
 *              at most a quarter of them, which is then computed as 64-column quarters of its
 *              tiles over all of K): a partial last round of more than a quarter and at most
 *              half of the compute units is split along K and the two halves' sums meet there
 *              (lower half first), so D is reproducible.
 * The result is deterministic for a given device. Errors: NVFP4_ERR_INVALID (null pointers,
 * K mismatch, K % 16, ldd < N, bad kind, misaligned D), NVFP4_ERR_WORKSPACE, NVFP4_ERR_HIP.
 */
int nvfp4_gemm_ex(const nvfp4_tensor* A, const nvfp4_tensor* B, void* D, int64_t ldd, nvfp4_out out_kind,
                  float* amax_out, void* workspace, size_t ws_bytes, void* hip_stream);

/* Element functions of nvfp4_gemm_act and nvfp4_act_grad. RELU2 max(z, 0)^2; GELU in its tanh
 * form, z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))); SILU z / (1 + exp(-z)). */
typedef enum { NVFP4_ACT_NONE = 0, NVFP4_ACT_RELU2 = 1, NVFP4_ACT_GELU = 2, NVFP4_ACT_SILU = 3 } nvfp4_act;

/*
 * nvfp4_gemm_act - a linear layer's forward product with what follows it, in the GEMM's epilogue
 * (artiverse.ca "NVIDIA's 4-bit floating point pushes AI training limits", paragraph on which
 * parts run in 4-bit: the GEMM takes NVFP4 operands; bias, activation and residual stay in higher
 * precision):
 *   Z = s_A s_B A B^T + bias (FP32);   D = BF16(act(Z) + residual)
 *   A, B       as nvfp4_gemm (rows M and N, same K, % 16 == 0). M may be a whole batch or the few
 *              rows of a generation step.
 *   D          device BF16 bits [M, N], row stride ldd >= N.
 *   bias       NULL, or device BF16 or FP32 (bias_dt) [N].
 *   residual   NULL, or device BF16 [M, N], row stride ldr >= N; may be D itself (same stride).
 *   preact     NULL, or device BF16 [M, N], row stride ldp >= N, receiving BF16(Z): what
 *              nvfp4_act_grad needs. Overlaps no other argument.
 *   amax_out   NULL, or device float[1] receiving max|D| over the values as stored (the amax_in of
 *              D's next quantization). The library clears it.
 *   workspace  nvfp4_workspace_size(NVFP4_OP_GEMM_ACT, M, N, K) bytes, 256-byte aligned (NULL
 *              allowed for 0 bytes): partial sums, and for a K that is not a multiple of 64 both
 *              operands with zeros up to one.
 * The result is deterministic for a given device. Errors: NVFP4_ERR_INVALID (null pointers, K
 * mismatch, K % 16, a stride below N, bad enum, misaligned buffers), NVFP4_ERR_UNSUPPORTED
 * (operand size), NVFP4_ERR_WORKSPACE, NVFP4_ERR_HIP.
 */
int nvfp4_gemm_act(const nvfp4_tensor* A, const nvfp4_tensor* B, uint16_t* D, int64_t ldd, const void* bias,
                   nvfp4_dtype bias_dt, nvfp4_act act, const uint16_t* residual, int64_t ldr, uint16_t* preact,
                   int64_t ldp, float* amax_out, void* workspace, size_t ws_bytes, void* hip_stream);

/*
 * nvfp4_act_grad - the backward of nvfp4_gemm_act's bias and activation (artiverse.ca "NVIDIA's
 * 4-bit floating point pushes AI training limits", as above) from one read of the gradient; the
 * residual's gradient is dY itself, and dZ feeds the two gradient GEMMs:
 *   dZ = BF16(dY * act'(Z));   dbias[n] = sum over m of dY * act'(Z)   (FP32, before the rounding)
 *   dy         device BF16 or FP32 (dt) [M, N], row stride ldy >= N.
 *   z          the forward's preact, device BF16 [M, N], row stride ldz >= N; NULL with
 *              NVFP4_ACT_NONE.
 *   dz         NULL (the bias gradient alone), or device BF16 [M, N], row stride lddz >= N,
 *              overlapping no input.
 *   dbias      NULL, or device float[N]: overwritten, or with accumulate != 0 added to (one FP32
 *              addition per element). The sums run in a fixed order.
 *   workspace  nvfp4_workspace_size(NVFP4_OP_ACT_GRAD, M, N, 1) bytes, 256-byte aligned; may be
 *              NULL without dbias.
 * Errors: NVFP4_ERR_INVALID (null pointers, shapes, strides, enums, misaligned buffers, neither dz
 * nor dbias), NVFP4_ERR_WORKSPACE, NVFP4_ERR_HIP.
 */
int nvfp4_act_grad(const void* dy, nvfp4_dtype dt, int64_t M, int64_t N, int64_t ldy, const uint16_t* z,
                   int64_t ldz, nvfp4_act act, uint16_t* dz, int64_t lddz, float* dbias, int accumulate,
                   void* workspace, size_t ws_bytes, void* hip_stream);

/*
 * nvfp4_grouped_gemm - one GEMM per group (mixture-of-experts expert GEMMs; "Nemotron
 * NVFP4" explainer, "The model underneath" and "The honest part: this is not end-to-end
 * FP4": the expert GEMMs carry most of the compute and run in NVFP4).
 *   m_offsets  device int64[G+1], 0 = m_offsets[0] <= ... <= m_offsets[G] <= A->rows; rows behind the last
 *              group (nvfp4_moe_sort can leave some) are in no product, D's stay as they are.
 *   A          [sum M_g, K], global_scale[G] (one per group, as produced by nvfp4_quantize
 *              with segments = m_offsets).
 *   B          [G*N, K] stacked per-group weights, global_scale[G].
 *   D          [sum M_g, N] FP32, row stride ldd: rows of group g hold A_g * B_g^T scaled by
 *              A->global_scale[g] * B->global_scale[g]. Empty groups are allowed.
 *   workspace  may be NULL (nvfp4_workspace_size returns 0 for this op).
 * Errors: NVFP4_ERR_INVALID (G < 1, B->rows != G*N, K mismatch, ...), NVFP4_ERR_HIP.
 */
int nvfp4_grouped_gemm(int64_t G, const int64_t* m_offsets, const nvfp4_tensor* A,
                       const nvfp4_tensor* B, int64_t N, float* D, int64_t ldd,
                       void* workspace, size_t ws_bytes, void* hip_stream);

/*
 * nvfp4_grouped_gemm_k - GEMMs grouped along the contraction dimension, as the MoE weight
 * gradient needs: expert g's gradient sums over the tokens routed to it ("Nemotron NVFP4"
 * explainer, "The model underneath": expert layers; "Why 4-bit training normally falls apart -
 * and the three fixes": the weight-gradient GEMM). For g < G:
 *   D[g*M + m, n] = A.global_scale[g] * B.global_scale[g] *
 *                   sum over k in [k_offsets[g], k_offsets[g+1]) of a[m, k] * b[n, k]
 * with a, b the E2M1 x E4M3 values, FP32 accumulation.
 *   A          NVFP4 [M, K], B NVFP4 [N, K], quantized along K, each with global_scale[G]
 *              (one per group of K).
 *   k_offsets  device int64[G+1], non-decreasing, multiples of 64 (unchecked device data:
 *              values are clamped into [0, K]; misaligned ones give unspecified output).
 *   D          device FP32 [G*M, N] with row stride ldd >= N; an empty group writes zeros.
 * Errors: NVFP4_ERR_INVALID (G < 1, NULL pointers, K mismatch, ldd < N), NVFP4_ERR_UNSUPPORTED
 * (K % 64 != 0), NVFP4_ERR_HIP.
 */
int nvfp4_grouped_gemm_k(int64_t G, const int64_t* k_offsets, const nvfp4_tensor* A,
                         const nvfp4_tensor* B, float* D, int64_t ldd, void* hip_stream);

/*
 * nvfp4_amax - max|x| of x[rows, cols] (row stride ld), per row segment, into device
 * amax_out[nseg]: the first level of the two-level scale ("Nemotron NVFP4" explainer, "What
 * NVFP4 actually is": one FP32 scale per tensor). With rht = 1 the maximum is taken over the
 * Hadamard-transformed tensor of nvfp4_rht_quantize (rows = tokens; segments are token
 * ranges as there, multiples of 16); with rht = 2 over the rowwise-transformed tensor of
 * nvfp4_rht_rows_quantize (no segments). Useful to precompute amax_in.
 *   workspace  device scratch of nvfp4_workspace_size(rht == 1 ? NVFP4_OP_RHT_QUANTIZE :
 *              NVFP4_OP_QUANTIZE, rows, cols, nseg) bytes, 256-byte aligned, for the partial
 *              maxima of an unsegmented tensor; may be NULL with segments (amax_out[nseg] is
 *              then written directly).
 * Errors: as nvfp4_quantize; NVFP4_ERR_UNSUPPORTED for rht = 2 with segments.
 */
int nvfp4_amax(const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols, int64_t ld,
               const int64_t* segments, int64_t nseg, int rht, uint16_t sign_mask,
               float* amax_out, void* workspace, size_t ws_bytes, void* hip_stream);

/*
 * nvfp4_amax_pair - both tensor maxima of x[tokens, cols] (row stride ld) from one read:
 * amax_out[0] = max|x| (the tensor scale of its 1x16 quantization, as nvfp4_amax with
 * rht = 0) and amax_out[1] = max|y| over the Hadamard-transformed tensor of
 * nvfp4_rht_quantize with this sign_mask (as nvfp4_amax with rht = 1). A tensor that feeds
 * both an fprop/dgrad GEMM and the wgrad GEMM is quantized both ways ("Nemotron NVFP4"
 * explainer, "Why 4-bit training normally falls apart - and the three fixes": only the wgrad
 * operands are transformed); each value can be passed as amax_in of the matching quantize.
 *   x          device, BF16 or FP32; tokens % 16 == 0; element pairs aligned (ld any).
 *   amax_out   device float[2].
 *   workspace  device scratch of nvfp4_workspace_size(NVFP4_OP_AMAX_PAIR, ...) bytes,
 *              256-byte aligned.
 * Both values are exact maxima, so they equal the two nvfp4_amax results bit for bit.
 * Errors: NVFP4_ERR_INVALID (NULL pointer, bad dtype/shape, tokens % 16 != 0),
 * NVFP4_ERR_UNSUPPORTED (misaligned x), NVFP4_ERR_WORKSPACE, NVFP4_ERR_HIP.
 */
int nvfp4_amax_pair(const void* x, nvfp4_dtype dt, int64_t tokens, int64_t cols, int64_t ld,
                    uint16_t sign_mask, float* amax_out, void* workspace, size_t ws_bytes,
                    void* hip_stream);

/* How a routed expert's score comes from the router's logits. */
typedef enum { NVFP4_SCORE_SOFTMAX = 0, NVFP4_SCORE_SIGMOID = 1 } nvfp4_score;

/* A mixture-of-experts layer: the router and the experts' NVFP4 weights, quantized along their
 * columns with one tensor scale per expert (nvfp4_quantize with segments, 1x16 or 16x16). */
typedef struct nvfp4_moe {
  int64_t experts, hidden, ffn;  /* experts 1 .. 512; hidden, ffn multiples of 16               */
  int64_t top_k;                 /* experts per token, 1 .. min(16, experts)                    */
  const void* router;            /* device BF16 or FP32 (router_dt) [experts, hidden]           */
  nvfp4_dtype router_dt;
  nvfp4_tensor w1;               /* [experts*ffn, hidden]; gated: [experts*2*ffn, hidden], each
                                    expert's ffn gate rows before its ffn up rows               */
  nvfp4_tensor w2;               /* [experts*hidden, ffn]; global_scale[experts], as w1's       */
  nvfp4_act act;
  int gated;                     /* h = act(gate x) * (up x) instead of act(w1 x)               */
  nvfp4_score score;
  int renormalize;               /* scores divided by their sum over the token's experts        */
  float routed_scale;            /* factor on every routing weight                              */
} nvfp4_moe;

/*
 * nvfp4_moe_tokens - a whole mixture-of-experts layer for a few tokens, a generation step's batch
 * ("Nemotron NVFP4" explainer, "The model underneath": expert layers, and "The honest part: this is
 * not end-to-end FP4": the expert weights are what runs in NVFP4). x and y are BF16; h is held
 * with the 11 significant bits of FP16 (its range by powers of two beside it), sums are FP32:
 *   l = x router^T (FP32);  the top_k largest of a token's l pick its experts, ties the lowest
 *   s = softmax(l) over all experts, or 1 / (1 + exp(-l));  w = s * routed_scale, or with
 *   renormalize s / (sum over the token's experts of s + 1e-20) * routed_scale
 *   y = BF16(sum over the token's experts of w * w2 h),  h = act(w1 x) or act(gate x) * (up x)
 *   x          device BF16 [tokens, hidden], row stride ldx >= hidden; tokens 0 .. 64 (larger batches:
 *              nvfp4_quantize with segments and nvfp4_grouped_gemm).
 *   y          device BF16 [tokens, hidden], row stride ldy >= hidden; overlaps no input.
 *   ids_out, weights_out   NULL, or device int32 / float [tokens, top_k]: the experts, largest logit
 *              first, and w.
 *   workspace  nvfp4_moe_workspace_size(moe, tokens) bytes (that of more tokens serves fewer),
 *              256-byte aligned. Its first nvfp4_moe_workspace_size(moe, 0) bytes have to be zero
 *              before the first call and are zero again after each; calls that share a workspace
 *              have to be ordered.
 * A token's result does not depend on the other tokens of the call, nor on the order in which
 * workgroups finish. Non-finite values of one token stay with that token. Errors:
 * NVFP4_ERR_INVALID (null or misaligned pointers, shapes, strides, enums), NVFP4_ERR_UNSUPPORTED
 * (more than 64 tokens, 512 experts or top_k 16, hidden or ffn above 2^18, an expert matrix's codes
 * above 2 GiB), NVFP4_ERR_WORKSPACE, NVFP4_ERR_HIP.
 */
int nvfp4_moe_tokens(const nvfp4_moe* moe, const uint16_t* x, int64_t tokens, int64_t ldx, uint16_t* y, int64_t ldy,
                     int32_t* ids_out, float* weights_out, void* workspace, size_t ws_bytes, void* hip_stream);

/* Bytes of nvfp4_moe_tokens' workspace for `tokens` tokens; with tokens = 0 those that have to be
 * zero at first. 0 for a bad argument. */
size_t nvfp4_moe_workspace_size(const nvfp4_moe* moe, int64_t tokens);

/* How the two running means of AdamW are held: FP32, or 8 bits (below). */
typedef enum { NVFP4_STATE_FP32 = 0, NVFP4_STATE_8BIT = 1 } nvfp4_state;

/* One tensor of an AdamW step: n elements, contiguous. Every output may be its input (the usual
 * in-place step) or a buffer that overlaps no input and no other output. */
typedef struct nvfp4_adamw_tensor {
  int64_t n;                   /* elements, >= 0                                            */
  const void* grad;            /* device BF16 or FP32 (grad_dt) [n]                         */
  const float* p;              /* device FP32 [n]: the parameter (a BF16 weight's master copy) */
  float* p_out;                /* device FP32 [n]                                           */
  uint16_t* w_out;             /* NULL, or device BF16 [n]: p_out rounded to nearest even   */
  const void* m;               /* FP32 [n], or E4M3 codes uint8 [n]                         */
  const void* v;               /* FP32 [n], or E4M3 codes uint8 [n] of sqrt(v)              */
  void* m_out;
  void* v_out;
  const uint8_t* m_scale;      /* 8-bit states: E8M0 per 32 elements, uint8 [ceil(n/32)]    */
  const uint8_t* v_scale;
  uint8_t* m_scale_out;
  uint8_t* v_scale_out;
  float weight_decay;          /* decoupled decay of this tensor (0 for biases and norms)   */
  nvfp4_dtype grad_dt;
} nvfp4_adamw_tensor;

typedef struct nvfp4_adamw_hyper {
  double lr, beta1, beta2, eps;  /* 0 <= beta < 1, eps > 0                                   */
  int64_t step;                  /* 1 for the first step (bias correction, random bytes)     */
  double max_norm;               /* > 0: clip the gradient's norm over all tensors; 0: do not */
  uint64_t seed;                 /* of the 8-bit states' stochastic rounding                 */
} nvfp4_adamw_hyper;

/*
 * nvfp4_adamw - one AdamW step over many tensors at once (the optimizer states and the master
 * weights stay in high precision around the 4-bit GEMMs: artiverse.ca "NVIDIA's 4-bit floating
 * point pushes AI training limits", paragraph on which parts run in 4-bit). The gradient is the
 * FP32 main gradient that nvfp4_gemm_ex accumulates, or a BF16 one. Per element, in FP32:
 *   g  = c * grad,  c = min(1, max_norm / (norm + 1e-6)) with max_norm > 0, else 1
 *   m' = beta1 m + (1 - beta1) g;   v' = beta2 v + (1 - beta2) g^2
 *   p' = p (1 - lr weight_decay) - lr / (1 - beta1^step) * m' / (sqrt(v' / (1 - beta2^step)) + eps)
 * norm = sqrt(sum of grad^2 over all tensors), summed in a fixed order: eight consecutive squares
 * in FP32, those sums in binary64. A gradient above 1.8e19 (eight neighbours above 6.5e18) therefore
 * makes it infinite, and one below 2.6e-23 adds nothing. With max_norm > 0 a norm that is infinite or
 * NaN makes the step write back what it read (w_out = BF16(p)); without it gradients that are not
 * finite, or whose square is not, are outside the contract.
 *
 * NVFP4_STATE_8BIT holds m and r = sqrt(v) as E4M3 codes with one scale 2^e per 32 consecutive
 * elements (E8M0 code e + 127; e is the smallest exponent with max|x| <= 448 * 2^e, at least
 * -117; code 0 and value 0 for an all-zero block). A value y = |x| 2^-e is rounded up to the next
 * E4M3 value iff its fraction of the gap + h/65536 >= 1; rounding never makes a nonzero r 0 (an r
 * below 2^-75 has a square below FP32 and ends as sqrt((1 - beta2) g^2)). Element
 * 8b + j (j < 8) of tensor i takes for h the 16 bits of half j % 2 (low first) of word j / 2 of
 * Philox4x32-10 with key (lo32 seed, hi32 seed) and counter (lo32 b, hi32 b, lo32 step, i), the
 * same h for m and r.
 *
 *   table      device copy of the bytes that nvfp4_adamw_table wrote for these tensors, 16-byte
 *              aligned, and the count, chunks and state of that call.
 *   norm_out   NULL, or device float[1] receiving norm (max_norm > 0 only).
 *   amax_out   NULL, or device float[count] receiving max|w_out| (max|p_out| where w_out is
 *              NULL) of each tensor: the amax_in of the weight's next nvfp4_quantize.
 *   workspace  nvfp4_workspace_size(NVFP4_OP_ADAMW, 0, 0, 0) bytes, 256-byte aligned; may be NULL
 *              with max_norm = 0.
 * The result is deterministic. Errors: NVFP4_ERR_INVALID (NULL table, count or chunks out of
 * range, hyperparameters out of range, bad enum), NVFP4_ERR_WORKSPACE, NVFP4_ERR_HIP.
 */
int nvfp4_adamw(const void* table, int64_t count, int64_t chunks, nvfp4_state state,
                const nvfp4_adamw_hyper* hyper, float* norm_out, float* amax_out,
                void* workspace, size_t ws_bytes, void* hip_stream);

/* Bytes of the table of `count` tensors (their n alone is read), 0 for a bad argument. */
size_t nvfp4_adamw_table_size(const nvfp4_adamw_tensor* tensors, int64_t count);

/*
 * nvfp4_adamw_table - checks the tensors and writes their table (the optimizer side of artiverse.ca
 * "NVIDIA's 4-bit floating point pushes AI training limits", as above) to HOST memory: the caller
 * copies it to the device once and keeps it for as long as the tensors stay where they are.
 * Nothing is enqueued.
 *   tensors    host array [count], count >= 1.
 *   table      host memory of at least nvfp4_adamw_table_size bytes.
 *   chunks     receives the value to pass to nvfp4_adamw.
 * Errors: NVFP4_ERR_INVALID (NULL or misaligned pointers with n > 0, n < 0, bad dtype or state,
 * table_bytes too small), NVFP4_ERR_UNSUPPORTED (more than 2^31 - 1 chunks of 2048 elements).
 */
int nvfp4_adamw_table(const nvfp4_adamw_tensor* tensors, int64_t count, nvfp4_state state, void* table,
                      size_t table_bytes, int64_t* chunks);

/*
 * nvfp4_fp8_quantize - an activation held in 8 bits from the forward to the backward pass (1.03 bytes
 * per element instead of 2; artiverse.ca "NVIDIA's 4-bit floating point pushes AI training limits",
 * paragraph on which parts run in 4-bit: what is kept beside the 4-bit products is of higher
 * precision). For each block of 32 elements e is the smallest exponent, at least -117, with
 * max|x| <= 448 * 2^e (code 0 for an all-zero block), and an element is E4M3(x * 2^-e), to nearest
 * even: within 2^-4 of its value, or within 2^-10 * 2^e. A block that holds an infinity or a NaN becomes NaNs
 * (scale code 255, codes 0x7F); a value above 1.9375 * 2^127 rounds to an infinity.
 *   x    device BF16 or FP32 (dt) [rows, cols], row stride ld >= cols.
 * Errors: NVFP4_ERR_INVALID (null or misaligned pointers, shapes, enum), NVFP4_ERR_HIP.
 */
int nvfp4_fp8_quantize(const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols, int64_t ld, nvfp4_fp8_tensor* out,
                       void* hip_stream);

/* nvfp4_fp8_dequantize - y[rows, cols] (BF16, row stride ld): the values of nvfp4_fp8_quantize's codes,
 * exactly ("Nemotron NVFP4" explainer, "What NVFP4 actually is", the element-times-scale form). Errors as there. */
int nvfp4_fp8_dequantize(const nvfp4_fp8_tensor* q, uint16_t* y, int64_t ld, void* hip_stream);

/*
 * nvfp4_rht_quantize_fp8 - nvfp4_rht_quantize of an activation held in 8 bits: the weight gradient's operand
 * ("Nemotron NVFP4" explainer, "Why 4-bit training normally falls apart - and the three fixes"). The
 * result is bit for bit that of nvfp4_rht_quantize on the BF16 tensor of nvfp4_fp8_dequantize.
 * Arguments, workspace (NVFP4_OP_RHT_QUANTIZE) and errors as there; x->rows % 16 == 0.
 */
int nvfp4_rht_quantize_fp8(const nvfp4_fp8_tensor* x, uint16_t sign_mask, nvfp4_round rnd, uint64_t seed, uint64_t offset,
                           const int64_t* segments, int64_t nseg, const float* amax_in, nvfp4_tensor* out, void* workspace,
                           size_t ws_bytes, void* hip_stream);

/*
 * nvfp4_act_grad_fp8 - nvfp4_act_grad with the pre-activation held in 8 bits (the same passages); M and N
 * are z's. An activation other than NVFP4_ACT_NONE. Results as nvfp4_act_grad's on the dequantized z.
 * Arguments, workspace (NVFP4_OP_ACT_GRAD) and errors as there.
 */
int nvfp4_act_grad_fp8(const void* dy, nvfp4_dtype dt, int64_t ldy, const nvfp4_fp8_tensor* z, nvfp4_act act, uint16_t* dz,
                       int64_t lddz, float* dbias, int accumulate, void* workspace, size_t ws_bytes, void* hip_stream);

/*
 * nvfp4_rms_norm - the norm in front of a layer, with the residual's addition before it (norms stay in
 * higher precision around the 4-bit products: artiverse.ca "NVIDIA's 4-bit floating point pushes AI
 * training limits", paragraph on which parts run in 4-bit). In FP32:
 *   h = x + residual, stored in residual_out in the stream's type;  s = 1 / sqrt(mean over a row of h^2 + eps), h as
 *   stored;  y = BF16(h s weight), and/or in 8 bits (nvfp4_fp8_quantize of the unrounded h s weight)
 *   x, residual, residual_out   device BF16 or FP32 (dt, all alike) [rows, cols], row strides >= cols. residual may be
 *              NULL (h = x), residual_out too. residual_out may be x or residual themselves (same stride).
 *   weight     device BF16 or FP32 (weight_dt) [cols].
 *   y          NULL, or device BF16, row stride ldy >= cols.   y8: NULL, or an 8-bit tensor [rows, cols].
 *   amax_out   NULL, or device float[1] receiving max|y| over the BF16 values: the amax_in of y's quantization.
 * Other outputs overlap no input; buffers that begin at the same address with unequal row strides are refused.
 * cols 1 .. 16384 (NVFP4_ERR_UNSUPPORTED above), eps at least 2^-126. Values whose squares leave FP32 are outside the contract.
 * Errors: NVFP4_ERR_INVALID (null or misaligned pointers, shapes, strides, enums, neither y nor y8), NVFP4_ERR_HIP.
 */
int nvfp4_rms_norm(const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols, int64_t ldx, const void* weight, nvfp4_dtype weight_dt,
                   float eps, const void* residual, int64_t ldr, void* residual_out, int64_t ldro, uint16_t* y, int64_t ldy,
                   nvfp4_fp8_tensor* y8, float* amax_out, void* hip_stream);

/*
 * nvfp4_rms_norm_grad - its backward (the same passage), one read of each input, in FP32:
 *   dx = s (u - h s mean(u h s)) + dresidual,  u = dy weight;   dweight[n] = sum over rows of dy h s
 * dx is the gradient of x and of residual alike. s is computed from h again.
 *   dy         device BF16 or FP32 (dy_dt) [rows, cols].
 *   h          the forward's residual_out (x without a residual), BF16 or FP32 (dt).
 *   dresidual  NULL, or the gradient that reached h on its own way (dt).   dx: dt; may be dresidual itself (same stride).
 *   dweight    NULL, or device float[cols]: overwritten, or with accumulate != 0 added to. Summed in a fixed order.
 *   workspace  nvfp4_workspace_size(NVFP4_OP_NORM_GRAD, rows, cols, 1) bytes, 256-byte aligned; NULL without dweight.
 * Errors: as nvfp4_rms_norm, NVFP4_ERR_WORKSPACE.
 */
int nvfp4_rms_norm_grad(const void* dy, nvfp4_dtype dy_dt, int64_t rows, int64_t cols, int64_t lddy, const void* h, nvfp4_dtype dt,
                        int64_t ldh, const void* weight, nvfp4_dtype weight_dt, float eps, const void* dresidual, int64_t lddr,
                        void* dx, int64_t lddx, float* dweight, int accumulate, void* workspace, size_t ws_bytes, void* hip_stream);

/* Rows that hold tokens * top_k pairs sorted by expert, each expert's run padded to a multiple of align,
 * whatever the routing: a multiple of align; -1 for a bad argument or 2^31 and more ("Nemotron NVFP4" explainer, "The model underneath"). */
int64_t nvfp4_moe_sorted_rows(int64_t tokens, int64_t top_k, int64_t experts, int64_t align);

/*
 * nvfp4_moe_sort - the order in which tokens go through the grouped expert products ("Nemotron NVFP4"
 * explainer, "The model underneath": expert layers). Pair p = t * top_k + j is token t's j-th expert.
 *   ids        device int32 [tokens, top_k]; an id outside 0 .. experts - 1 is a dropped pair.
 *   offsets    device int64 [experts + 1]: expert e's rows are offsets[e] .. offsets[e + 1] - 1, its pairs in
 *              ascending order first, then rows without a pair up to a multiple of align (64 for
 *              nvfp4_grouped_gemm_k, whose k_offsets these are, 1 for no padding). Multiples of align.
 *   row_of     device int32 [tokens, top_k]: the pair's row, -1 where dropped.
 *   pair_of    device int32 [rows]: the row's pair, -1 where there is none, the rows from
 *              offsets[experts] on among them.
 *   rows       at least nvfp4_moe_sorted_rows(tokens, top_k, experts, align).
 *   workspace  nvfp4_workspace_size(NVFP4_OP_MOE_SORT, tokens * top_k, experts, 1) bytes, 256-byte aligned.
 * Errors: NVFP4_ERR_INVALID (null or misaligned pointers, sizes), NVFP4_ERR_UNSUPPORTED (more than 1024 experts,
 * 2^31 or more pairs or rows), NVFP4_ERR_WORKSPACE, NVFP4_ERR_HIP.
 */
int nvfp4_moe_sort(const int32_t* ids, int64_t tokens, int64_t top_k, int64_t experts, int64_t align, int64_t rows, int64_t* offsets,
                   int32_t* row_of, int32_t* pair_of, void* workspace, size_t ws_bytes, void* hip_stream);

/*
 * nvfp4_moe_gather - out[row] = x[t] for the pair of each row (times weights[t, j] where given), zeros in rows
 * without one: the grouped products' operand before its quantization ("The model underneath", as above). Its gradient is
 * nvfp4_moe_combine without weights.
 *   x, out     device BF16 or FP32 (dt, alike) [tokens, hidden] and [rows, hidden]; out overlaps no input.
 *   weights    NULL, or device float [tokens, top_k].
 * pair_of is device data: a value that is no pair counts as none. Errors: NVFP4_ERR_INVALID, NVFP4_ERR_UNSUPPORTED (2^26 rows or pairs, 2^35
 * elements and more), NVFP4_ERR_HIP.
 */
int nvfp4_moe_gather(const void* x, nvfp4_dtype dt, int64_t tokens, int64_t hidden, int64_t ldx, const int32_t* pair_of, int64_t rows,
                     int64_t top_k, const float* weights, void* out, int64_t ldo, void* hip_stream);

/*
 * nvfp4_moe_combine - out[t] = sum over j, in order, of weights[t, j] * y[row_of[t, j]] (1 without weights; FP32,
 * rounded once): the experts' outputs back in the tokens' order ("The model underneath", as above). Dropped pairs add nothing.
 *   y          device BF16 or FP32 (dt) [rows, hidden], as nvfp4_grouped_gemm leaves it.
 *   out        device BF16 or FP32 (out_dt) [tokens, hidden], overlapping no input.
 * row_of is device data: a value outside 0 .. rows - 1 is a dropped pair. Errors: as nvfp4_moe_gather.
 */
int nvfp4_moe_combine(const void* y, nvfp4_dtype dt, int64_t rows, int64_t hidden, int64_t ldy, const int32_t* row_of, int64_t tokens,
                      int64_t top_k, const float* weights, void* out, nvfp4_dtype out_dt, int64_t ldo, void* hip_stream);

/*
 * nvfp4_moe_combine_grad - the backward of nvfp4_moe_combine ("The model underneath", as above):
 *   dy[row] = weights[t, j] * dout[t], zeros in rows without a pair;   dweights[t, j] = <dout[t], y[row]>, 0 where dropped
 *   dout, dy   device BF16 or FP32 (out_dt, alike) [tokens, hidden] and [rows, hidden].
 *   y          device BF16 or FP32 (dt) [rows, hidden]; NULL without dweights.
 *   dy, dweights   either may be NULL; dweights: device float [tokens, top_k].
 * Errors: as nvfp4_moe_gather.
 */
int nvfp4_moe_combine_grad(const void* dout, nvfp4_dtype out_dt, int64_t tokens, int64_t hidden, int64_t lddo, const void* y, nvfp4_dtype dt,
                           int64_t rows, int64_t ldy, const int32_t* row_of, const int32_t* pair_of, int64_t top_k, const float* weights,
                           void* dy, int64_t lddy, float* dweights, void* hip_stream);

/*
 * nvfp4_linear_cross_entropy - the softmax cross entropy of a language model's output head, whose logits
 * x w^T are never stored (the output head stays in BF16: artiverse.ca "NVIDIA's 4-bit floating point pushes AI training
 * limits", paragraph on which parts run in 4-bit). With FP32 products and sums:
 *   lse[t] = log(sum over v of exp(l[t, v])),  l = x w^T;   loss[t] = lse[t] - l[t, targets[t]]
 *   x, w       device BF16 [tokens, hidden] and [vocab, hidden], 16-byte aligned, row strides multiples of 8; hidden
 *              a multiple of 16.
 *   targets    device int64 [tokens]. A target outside 0 .. vocab - 1 does not count: loss 0.
 *   loss, lse  device float [tokens]; one of them may be NULL. lse is what the backward needs.
 *   workspace  nvfp4_workspace_size(NVFP4_OP_HEAD_LOSS, tokens, vocab, hidden) bytes, 256-byte aligned.
 * Errors: NVFP4_ERR_INVALID (null or misaligned pointers, shapes, strides), NVFP4_ERR_UNSUPPORTED (row strides of
 * 2^22 elements and more, more than 2^21 tokens, 2^34 elements of x, 2^38 logits or elements of w and more), NVFP4_ERR_WORKSPACE, NVFP4_ERR_HIP.
 */
int nvfp4_linear_cross_entropy(const uint16_t* x, int64_t tokens, int64_t ldx, const uint16_t* w, int64_t vocab, int64_t ldw, int64_t hidden,
                               const int64_t* targets, float* loss, float* lse, void* workspace, size_t ws_bytes, void* hip_stream);

/*
 * nvfp4_linear_cross_entropy_grad - its backward (the same passage). The logits are computed again, in pieces of the
 * vocabulary:
 *   G[t, v] = grad[t] exp(l[t, v] - lse[t]), the target's grad[t] (exp(l - lse) - 1), held in BF16 (the target's, mostly the
 *   largest, with what that leaves of it), 0 for a token that does not count (whose x has to be finite all the same: 0 x is in dw's sums)
 *   dx = BF16(G w);   dw = G^T x
 *   lse        the forward's.   grad: device float [tokens], the gradient of each token's loss.
 *   dx         NULL, or device BF16 [tokens, hidden], row stride lddx >= hidden.
 *   dw         NULL, or device [vocab, hidden], row stride lddw >= hidden: FP32, FP32 added to what it holds, or BF16
 *              (dw_kind), each the FP32 sum of addends that carry G's rounding (2^-8 of each). dx and dw overlap no input.
 *   workspace  nvfp4_workspace_size(NVFP4_OP_HEAD_GRAD, tokens, vocab, hidden) bytes, 256-byte aligned.
 * The result is deterministic. lse is rounded at its size, so the target's G is off by up to 2^-24 |lse| grad: much of it
 * for a token that is nearly sure of its target; nvfp4_linear_cross_entropy_grad_ex takes the loss too. Errors: as nvfp4_linear_cross_entropy.
 */
int nvfp4_linear_cross_entropy_grad(const uint16_t* x, int64_t tokens, int64_t ldx, const uint16_t* w, int64_t vocab, int64_t ldw,
                                    int64_t hidden, const int64_t* targets, const float* lse, const float* grad, uint16_t* dx, int64_t lddx,
                                    void* dw, nvfp4_out dw_kind, int64_t lddw, void* workspace, size_t ws_bytes, void* hip_stream);

/* nvfp4_linear_cross_entropy_grad_ex - the same with loss (NULL, or the forward's, device float [tokens]): the target's G is then
 * grad[t] (exp(-loss[t]) - 1), which keeps its digits however small the loss is (the same passage). Errors as there. */
int nvfp4_linear_cross_entropy_grad_ex(const uint16_t* x, int64_t tokens, int64_t ldx, const uint16_t* w, int64_t vocab, int64_t ldw,
                                       int64_t hidden, const int64_t* targets, const float* lse, const float* loss, const float* grad,
                                       uint16_t* dx, int64_t lddx, void* dw, nvfp4_out dw_kind, int64_t lddw, void* workspace, size_t ws_bytes,
                                       void* hip_stream);

/* Bytes of device workspace `op` needs for the given shape (0 if none). The library allocates
 * no memory itself (caller-owned buffers, see the conventions above), so the partial maxima of
 * the tensor amax (the FP32 tensor scale of "Nemotron NVFP4" explainer, "What NVFP4 actually
 * is") and the K-split partial sums of nvfp4_gemm_ex live in a workspace the caller sizes with
 * this call. ops: nvfp4_op; rows/cols/nseg as in the call the workspace is for (for
 * NVFP4_OP_GEMM_ACT: M, N, K; for NVFP4_OP_ACT_GRAD: M, N, 1; for the later ops as their calls say). */
size_t nvfp4_workspace_size(int op, int64_t rows, int64_t cols, int64_t nseg);

/* Thread-local description of the last non-OK status returned on this thread: the error
 * behaviour shared by every entry point (host validation before anything is enqueued). The
 * string stays valid until the thread's next failing call. */
const char* nvfp4_last_error(void);

/*
 * nvfp4_dequantize - test helper: the decoded value of every element, the two-level scale of
 * "Nemotron NVFP4" explainer, "What NVFP4 actually is" (E2M1 element times its block's E4M3
 * scale times the tensor's FP32 scale): y[r, c] = rn32(e2m1 * e4m3 * global_scale[segment(r)])
 * (e2m1 * e4m3 is exact), y FP32 [rows, cols] contiguous. segments as for nvfp4_quantize
 * (NULL, nseg = 1 allowed). Errors: NVFP4_ERR_INVALID (null pointers, shapes), NVFP4_ERR_HIP.
 */
int nvfp4_dequantize(const nvfp4_tensor* q, const int64_t* segments, int64_t nseg, float* y,
                     void* hip_stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_H */
