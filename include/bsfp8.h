/*
 * bsfp8.h -- block-scaled FP8 grouped quantize and GEMMs for MoE expert layers (gfx950).
 *
 * C ABI of libbsfp8.so.  The library computes, on one GPU, the three steps of the expert-layer
 * path that the following pages turn on:
 *   - DeepGEMM issue #365, "Non-deterministic numerical problem of
 *     k_grouped_fp8_gemm_nt_contiguous" (reproducer: per-channel cast, K-major pack,
 *     k-grouped weight-gradient GEMM with a 1 x 128 fp32 scale recipe, determinism stress);
 *   - TransformerEngine issue #3484, "NaN expert weight gradients at num_groups == 1 with a
 *     padded token buffer for SReLU" (MXFP8 1x32 block scaling, padded token buffers, wgrad
 *     accumulated into an fp32 main_grad, expected behaviour: padding never matters);
 *   - TransformerEngine PR #3224, "Improve device-init grouped linear module with single
 *     grouped weight support" (per-group scale strides in grouped quantize, output reuse,
 *     zero-row early return, device-resident split sizes).
 * and, around them, what a training or serving step of such a layer runs next to its GEMMs: the gated projection
 * with its activation and quantize in one kernel, the norms before and after a block with its gate and residual sum,
 * their gradients, the AdamW step over all parameters, the router with the tokens' way to their experts and back, and
 * activations kept in 8 bits for the backward pass.
 *
 * Conventions for every entry point:
 *   - All data pointers are DEVICE pointers owned by the caller.  The library allocates
 *     nothing, keeps no global mutable state, and is reentrant.  Every call is asynchronous
 *     on `stream` (a hipStream_t; NULL = the default stream) with no host synchronization and
 *     no device-to-host copy; it may be captured in a HIP graph.
 *   - Groups: `split_sizes` is a device int32 array of `num_groups` row counts k_e.  Group e
 *     owns rows [off_e, off_e + k_e) of a token buffer of `capacity_rows` rows, where
 *     off_e = k_0 + ... + k_{e-1}.  Rows at or past T = sum(k_e) are padding: they are never
 *     read and may hold any bits.  num_groups == 1, empty groups and groups of any size
 *     (no alignment of k_e is required) take the same code path.
 *   - Padded group extents (the colwise layouts): Kp_e = 128 * ceil(k_e / 128) and
 *     P_e = Kp_0 + ... + Kp_{e-1}.
 *   - Host-checkable errors return a negative BSFP8_ERR_* code before anything is launched.
 *     Data errors that only the device can see (a negative k_e, or T > capacity_rows) set bits
 *     in `*status` (when `status` is not NULL) with a bitwise OR; the kernels of that call then
 *     write nothing at all.  The library never clears `*status`.
 *   - Results are deterministic: no atomics on data, no split-K; repeated calls on the same
 *     inputs give bitwise identical outputs.
 */
#ifndef BSFP8_H
#define BSFP8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Quantization recipes. */
#define BSFP8_RECIPE_MX_1X32_E8M0 1       /* e4m3 data, one E8M0 power-of-two scale per 32 values */
#define BSFP8_RECIPE_PER_CHANNEL_128_F32 2 /* e4m3 data, one fp32 scale per channel per 128 rows */
#define BSFP8_RECIPE_MXFP4_1X32_E8M0 3     /* e2m1 data (two per byte), one E8M0 scale per 32 values */

/*
 * GEMM arithmetic modifier, OR-ed into the recipe argument of the three GEMM calls only:
 * BSFP8_RECIPE_MX_1X32_E8M0 | BSFP8_GEMM_FP8_MFMA multiplies the same MXFP8 operands on the
 * scaled FP8 MFMA (v_mfma_scale_f32_32x32x64_f8f6f4, codes and E8M0 bytes as they are) instead
 * of widening them exactly to bf16.  Twice the MFMA rate, but the instruction does not sum the
 * products of 8 consecutive K values exactly (smaller products are cut to a window under the
 * largest, toward zero): on MXFP8-quantized Gaussian data the relative Frobenius error is about
 * 1.5e-5 instead of about 1e-7, above the 1e-5 bound the widened path meets.  For callers that
 * accept that error; the widened path stays the default.  Other recipes, and the quantize
 * calls, reject the modifier (BSFP8_ERR_RECIPE).
 */
#define BSFP8_GEMM_FP8_MFMA 0x100

/* Layout selection bits for bsfp8_grouped_quantize. */
#define BSFP8_ROWWISE 1 /* blocks along a row (channels); used by the forward GEMM */
#define BSFP8_COLWISE 2 /* blocks along the token axis within each group; used by wgrad */

/* Activations of bsfp8_grouped_act_quantize. */
#define BSFP8_ACT_SRELU 1      /* y = p * max(h, 0)^2 (scaled squared ReLU) */
#define BSFP8_ACT_SRELU_GRAD 2 /* g = dy * p * 2 max(h, 0) (its gradient with respect to h) */
#define BSFP8_ACT_SWIGLU 3     /* y = p * silu(a) * b, (a | b) the halves of fc1's output row */
#define BSFP8_ACT_SWIGLU_GRAD 4 /* (da | db): the gradient of the scaled SwiGLU */

/* Output element types of bsfp8_grouped_gemm_fprop. */
#define BSFP8_OUT_F32 0
#define BSFP8_OUT_BF16 1

/* Device status bits. */
#define BSFP8_STATUS_NEGATIVE_SPLIT 1u   /* some k_e < 0 */
#define BSFP8_STATUS_EXCEEDS_CAPACITY 2u /* sum(k_e) > capacity_rows */

/* Return codes. */
#define BSFP8_OK 0
#define BSFP8_ERR_NULL_POINTER (-1)  /* a required pointer is NULL */
#define BSFP8_ERR_NUM_GROUPS (-2)    /* num_groups <= 0 or > BSFP8_MAX_GROUPS */
#define BSFP8_ERR_RECIPE (-3)        /* unknown recipe */
#define BSFP8_ERR_SHAPE (-4)         /* a dimension is negative or not a multiple of 32 */
#define BSFP8_ERR_ALIGNMENT (-5)     /* a pointer is not 16-byte aligned */
#define BSFP8_ERR_LAYOUT (-6)        /* layout/recipe combination not supported */
#define BSFP8_ERR_ARGUMENT (-7)      /* other invalid argument (flags, zero_amax_scale) */
#define BSFP8_ERR_LAUNCH (-8)        /* the HIP runtime refused a launch */

#define BSFP8_MAX_GROUPS 1024

/* ----------------------------------------------------------------------------------------- */
/* Buffer sizes.  Pure host functions; they return 0 for invalid arguments.                   */
/* ----------------------------------------------------------------------------------------- */

/* Upper bound of sum(Kp_e) over all valid split sizes: 128 * floor((R + 127 * E) / 128). */
int64_t bsfp8_colwise_rows_bound(int64_t capacity_rows, int32_t num_groups);
/* Bytes of a colwise data buffer: cols * bsfp8_colwise_rows_bound(R, E) (half that for MXFP4). */
size_t bsfp8_colwise_data_bytes(int64_t capacity_rows, int64_t cols, int32_t num_groups, int recipe);
/* Bytes of a colwise scale buffer: rows_bound * cols / 32 (MX, MXFP4) or rows_bound * cols / 128 * 4. */
size_t bsfp8_colwise_scale_bytes(int64_t capacity_rows, int64_t cols, int32_t num_groups, int recipe);
/* Bytes of rowwise data (rows * cols for MXFP8, rows * cols / 2 for MXFP4; 0 for the
 * per-channel recipe, which has no rowwise layout) and of its E8M0 scales (rows * cols / 32). */
size_t bsfp8_rowwise_data_bytes(int64_t rows, int64_t cols, int recipe);
size_t bsfp8_rowwise_scale_bytes(int64_t rows, int64_t cols);

/* ----------------------------------------------------------------------------------------- */
/* Grouped quantize: bf16 -> e4m3 / e2m1 with block scales (DeepGEMM #365 reproducer,         */
/* per-channel cast; TE #3484 MXFP8 block scaling, and the 4-bit quantizer its additional     */
/* context says the same gated paths accept; TE PR #3224, per-member columnwise scale strides). */
/* ----------------------------------------------------------------------------------------- */
/*
 * in_bf16         [capacity_rows][cols] bf16, row-major.
 * split_sizes     device int32[num_groups]; may be NULL only when which == BSFP8_ROWWISE,
 *                 meaning that all capacity_rows rows are live (e.g. a weight [E*N][K]).
 * which           BSFP8_ROWWISE, BSFP8_COLWISE or both (rowwise needs an MX recipe).
 * zero_amax_scale per-channel recipe only: the scale used when a block's amax is 0 (the
 *                 reproducer's sf_val, default 1e-30); must be finite and >= 0.
 *
 * MX 1x32 E8M0 (both layouts): for a block of up to 32 live values with maximum magnitude
 *   amax, e is the smallest integer in [-127, 127] with amax <= 448 * 2^e (amax == 0 gives
 *   -127); the scale byte is e + 127 and each value v becomes e4m3(v * 2^-e).
 * Per-channel 128 (colwise only): for a block of up to 128 live rows of one channel,
 *   sf = fp32(amax / 448); sf == 0 becomes zero_amax_scale; sf = max(sf, 1e-30);
 *   each value v becomes e4m3(fp32(v * fp32(1 / sf))); the fp32 sf is stored.
 * e4m3 is OCP E4M3FN, round to nearest even, sign kept (both recipes keep |v| <= 448).
 * MXFP4 1x32 E8M0 (both layouts): as MXFP8 with 6 in place of 448 (e is the smallest integer in
 *   [-127, 127] with amax <= 6 * 2^e) and each value becoming e2m1(v * 2^-e): OCP FP4 E2M1
 *   (0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives), round to nearest even, sign kept.  The codes of
 *   elements 2i and 2i + 1 along the contiguous axis share a byte, 2i in bits 3..0.
 *
 * Outputs (all caller-allocated; only the requested ones may be non-NULL).  The offsets below
 * count data elements; for MXFP4 element i is a nibble of byte i / 2 (see above).
 *   row_q  [capacity_rows][cols] e4m3: row r, column c at r*cols + c      (live rows only)
 *   row_s  [cols/32][capacity_rows] E8M0: row r, block b at b*capacity_rows + r (live rows only)
 *   col_q  bsfp8_colwise_data_bytes(): group e, row t < Kp_e, column c at
 *          cols*P_e + c*Kp_e + t (each group's rows transposed, token axis contiguous);
 *          lanes k_e <= t < Kp_e hold 0x00.
 *   col_s  MX : E8M0 byte (e, b, c) at cols*P_e/32 + b*cols + c, b < Kp_e/32
 *               (a block with no live row holds byte 0);
 *          PC : fp32 (e, b, c) at cols*P_e/128 + b*cols + c, b < Kp_e/128.
 *   Blocks restart at every group start; a partial block takes its amax over live rows only.
 *   Bytes of col_q / col_s past cols*sum(Kp_e) are not written.
 * noop_flag       NULL, or a device fp32 scalar read by the kernels when they run (TE PR #3224,
 *                 group_quantize output reuse: the noop flag of the FP8 block-scaling path).  A
 *                 nonzero value makes the call a no-op on the device: no output byte and no status
 *                 bit is written, so storage filled by an earlier call (a cached quantized weight)
 *                 is reused as it stands.  Zero (or NULL) quantizes as usual, overwriting the
 *                 caller's pre-allocated outputs in place.  The flag is read on the device, so one
 *                 captured graph serves both the first microbatch (flag 0) and the rest (flag 1).
 *                 4-byte aligned.
 * capacity_rows == 0 returns BSFP8_OK without touching any pointer.
 */
int bsfp8_grouped_quantize(const void* in_bf16, int64_t capacity_rows, int64_t cols,
                           const int32_t* split_sizes, int32_t num_groups, int recipe, int which,
                           float zero_amax_scale, uint8_t* row_q, uint8_t* row_s, uint8_t* col_q,
                           void* col_s, const float* noop_flag, uint32_t* status, void* stream);

/* ----------------------------------------------------------------------------------------- */
/* Activation fused with the grouped quantize (TE #3484 reproducer: fc1 -> ScaledSReLU -> fc2   */
/* with per-token probs; its additional context names the ScaledSwiGLU family beside it; the  */
/* formulas are the usual scaled squared ReLU and scaled SwiGLU).                             */
/* ----------------------------------------------------------------------------------------- */
/*
 * SReLU (activation 1, 2): cols is the row length of h and of the output.
 *   h_bf16   [capacity_rows][cols] bf16: fc1's output (forward) or fc1's output saved for the
 *            backward (BSFP8_ACT_SRELU_GRAD).
 *   dy_bf16  [capacity_rows][cols] bf16, the gradient arriving at the activation's output
 *            (BSFP8_ACT_SRELU_GRAD only; NULL otherwise).
 *   BSFP8_ACT_SRELU:      y = (r * r) * p
 *   BSFP8_ACT_SRELU_GRAD: g = ((2 * r) * p) * dy
 *   with r = h for h > 0 and +0 otherwise.
 * SwiGLU (activation 3, 4): cols is the GLU width F; h_bf16 is [capacity_rows][2F] with
 *   a = columns [0, F) and b = [F, 2F) of each row; dy_bf16 [capacity_rows][F] (gradient only).
 *   With t = exp2s(-a * log2(e)), sg = 1 / (1 + t), s = a * sg:
 *   BSFP8_ACT_SWIGLU:      y = (s * b) * p, quantized as [capacity_rows][F]
 *   BSFP8_ACT_SWIGLU_GRAD: q = dy * p; da = (q * b) * (sg * (1 + a * (1 - sg))); db = q * s,
 *                          quantized as [capacity_rows][2F] = (da | db)
 *   exp2s is a stated fp32 2^x: x clamped to [-126, 126], k = floor(x + 1/2), r = x - k, the
 *   degree-7 Taylor polynomial of exp(r ln 2) with fp32 coefficients (ln 2)^n / n! in Horner
 *   form, times 2^k (relative error below 3e-7; reproducible bit for bit on any IEEE machine).
 * probs      device fp32 [capacity_rows]: the token's routing probability p, or NULL for p = 1.
 * Every operation is rounded to fp32 in the order written (no fused multiply-add); division is
 * correctly rounded.  The fp32 values of the live rows are quantized the way
 * bsfp8_grouped_quantize quantizes a bf16 input, for recipe BSFP8_RECIPE_MX_1X32_E8M0 or
 * BSFP8_RECIPE_MXFP4_1X32_E8M0, into the same layouts (rowwise for the next GEMM's forward,
 * colwise for its weight gradient), sized by the size queries for the output's shape:
 * [capacity_rows][cols] (SReLU), [capacity_rows][F] (SwiGLU) or [capacity_rows][2F] (its
 * gradient).
 * split_sizes is required; rows at or past sum(split_sizes) (of h, dy and probs) are never read.
 * Outputs, status and errors as bsfp8_grouped_quantize; capacity_rows == 0 returns BSFP8_OK
 * without touching any pointer.
 */
int bsfp8_grouped_act_quantize(int activation, const void* h_bf16, const float* probs,
                               const void* dy_bf16, int64_t capacity_rows, int64_t cols,
                               const int32_t* split_sizes, int32_t num_groups, int recipe, int which,
                               uint8_t* row_q, uint8_t* row_s, uint8_t* col_q, void* col_s,
                               uint32_t* status, void* stream);

/* ----------------------------------------------------------------------------------------- */
/* k-grouped weight-gradient GEMM (DeepGEMM #365, k_grouped_fp8_gemm_nt_contiguous; TE #3484, */
/* accumulate into an fp32 main_grad; the contraction runs over each group's tokens only).    */
/* All three recipes, and MXFP8 with BSFP8_GEMM_FP8_MFMA.                                     */
/* ----------------------------------------------------------------------------------------- */
/*
 * dy_col_q, dy_col_s  colwise output of bsfp8_grouped_quantize for dy [capacity_rows][n]
 * x_col_q,  x_col_s   colwise output for x [capacity_rows][h], same split_sizes and recipe
 * out                 fp32 [num_groups][n][h]:
 *     dW[e][i][j] = sum_{t < k_e} deq(dy)[off_e + t][i] * deq(x)[off_e + t][j]
 *   accumulate == 0 : out[e] = dW[e]           (an empty group gets zeros)
 *   accumulate == 1 : out[e] = out[e] + dW[e]  (one fp32 add per element; an empty group's
 *                                               slice is neither read nor written)
 * MX recipe: every e4m3 value is widened exactly with its E8M0 scale folded in; products
 *   accumulate in fp32.
 * Per-channel recipe: each 128-row block's unit-scale partial sum p is folded in as
 *   acc = fma(p, sdy_i * sx_j, acc) in block order.
 * MXFP4 recipe: the scaled fp4 MFMA takes the codes and E8M0 scales as they are (its sums of
 *   e2m1 products within a block are exact); products accumulate in fp32.
 * MX | BSFP8_GEMM_FP8_MFMA: the scaled fp8 MFMA takes the e4m3 codes and E8M0 scales as they
 *   are; results accumulate in fp32 across instructions, with the in-instruction error above.
 * n and h must be multiples of 32, h at most 2^21; capacity_rows + 127 must stay below
 * 2^24 - 128 (BSFP8_ERR_SHAPE otherwise): the kernels address an operand tile and a 128-row
 * output block with 32-bit offsets.
 */
int bsfp8_grouped_gemm_wgrad(const uint8_t* dy_col_q, const void* dy_col_s, int64_t n,
                             const uint8_t* x_col_q, const void* x_col_s, int64_t h,
                             const int32_t* split_sizes, int32_t num_groups, int64_t capacity_rows,
                             int recipe, float* out, int accumulate, uint32_t* status, void* stream);

/* ----------------------------------------------------------------------------------------- */
/* m-grouped forward GEMM (TE PR #3224, grouped GEMM over a single grouped weight; the token   */
/* axis is a free dimension).  recipe: BSFP8_RECIPE_MX_1X32_E8M0 (optionally with             */
/* BSFP8_GEMM_FP8_MFMA) or BSFP8_RECIPE_MXFP4_1X32_E8M0.                                      */
/* ----------------------------------------------------------------------------------------- */
/*
 * x_row_q, x_row_s  rowwise output of bsfp8_grouped_quantize for x [capacity_rows][k]
 *                   (the same recipe as the weight's)
 * w_q, w_s          rowwise output for the weight [num_groups * n][k] (split_sizes NULL):
 *                   expert e's row j is buffer row e*n + j; scales [k/32][num_groups * n]
 * out               [capacity_rows][n], fp32 or bf16 (round to nearest even from fp32):
 *     out[off_e + t][j] = sum_c deq(x)[off_e + t][c] * deq(W_e)[j][c]   for t < k_e
 *   rows at or past sum(k_e) are not written.
 * k and n must be multiples of 32, k below 2^24 - 128, n at most 2^21 (BSFP8_ERR_SHAPE
 * otherwise).  capacity_rows == 0 returns BSFP8_OK
 * without touching any pointer.
 */
int bsfp8_grouped_gemm_fprop(const uint8_t* x_row_q, const uint8_t* x_row_s, int64_t capacity_rows,
                             int64_t k, const uint8_t* w_q, const uint8_t* w_s, int64_t n,
                             const int32_t* split_sizes, int32_t num_groups, int recipe, void* out,
                             int out_dtype, uint32_t* status, void* stream);

/* ----------------------------------------------------------------------------------------- */
/* m-grouped data-gradient GEMM (the remaining GEMM of the expert backward beside wgrad and    */
/* fprop: TE #3484 scope -- the token axis is a free dimension of everything but wgrad).      */
/* recipe: BSFP8_RECIPE_MX_1X32_E8M0 (optionally with BSFP8_GEMM_FP8_MFMA) or                */
/* BSFP8_RECIPE_MXFP4_1X32_E8M0.                                                             */
/* ----------------------------------------------------------------------------------------- */
/*
 * dy_row_q, dy_row_s  rowwise output of bsfp8_grouped_quantize for dy [capacity_rows][n]
 * w_col_q, w_col_s    colwise output of bsfp8_grouped_quantize for the weight viewed as
 *                     [num_groups * n][k] with split sizes n, ..., n (num_groups of them): the
 *                     32-blocks run along n inside each expert, so expert e's matrix is
 *                     transposed in the buffer -- output channel j, contraction index c at
 *                     element k*np*e + j*np + c with np = 128 * ceil(n / 128); E8M0 (e, b, j) at
 *                     k*np*e/32 + b*k + j (bsfp8_colwise_data_bytes / _scale_bytes with
 *                     capacity_rows = num_groups * n give the sizes)
 * out                 [capacity_rows][k], fp32 or bf16 (round to nearest even from fp32):
 *     out[off_e + t][j] = sum_c deq(dy)[off_e + t][c] * deq(W_e)[c][j]   for t < k_e
 *   rows at or past sum(k_e) are not written.
 * n and k must be multiples of 32, n at most 2^24 - 256, k at most 2^21 (BSFP8_ERR_SHAPE
 * otherwise).  capacity_rows == 0 returns BSFP8_OK without touching any pointer.
 */
int bsfp8_grouped_gemm_dgrad(const uint8_t* dy_row_q, const uint8_t* dy_row_s, int64_t capacity_rows,
                             int64_t n, const uint8_t* w_col_q, const void* w_col_s, int64_t k,
                             const int32_t* split_sizes, int32_t num_groups, int recipe, void* out,
                             int out_dtype, uint32_t* status, void* stream);

/* ----------------------------------------------------------------------------------------- */
/* The gated feed-forward projection in one kernel: both projections, the activation, the      */
/* routing probability and the quantize of the result; and its gradient.  recipe:             */
/* BSFP8_RECIPE_MX_1X32_E8M0.                                                                 */
/* ----------------------------------------------------------------------------------------- */
/*
 * For the live rows t of expert e, products accumulated in fp32 (operands widened exactly):
 *     a = x[t] W1_e[0 .. ffn)^T,  b = x[t] W1_e[ffn .. 2 ffn)^T,  y = probs[t] * silu(a) * b
 * with silu(a) = a / (1 + exp(-a)) in fp32, from the unrounded a and b (y within (1.25 |a| + 12) 2^-24 of its value at
 * these a and b).
 * x_row_q, x_row_s  rowwise output of bsfp8_grouped_quantize for x [capacity_rows][hidden]
 * w_q, w_s          rowwise output for W1 [num_groups * 2 ffn][hidden] (split_sizes NULL): expert e's
 *                   a rows, then its b rows
 * probs             fp32 [capacity_rows], or NULL (1)
 * ab                bf16 [capacity_rows][2 ffn], (a | b) kept for the gradient, or NULL
 * y                 [capacity_rows][ffn] of y_dtype (BSFP8_OUT_F32 or BSFP8_OUT_BF16), or NULL
 * which, row_q, row_s, col_q, col_s   y quantized from its fp32 values, laid out as
 *                   bsfp8_grouped_quantize does for [capacity_rows][ffn]; which == 0: none
 * At least one of ab, y and the quantized layouts is asked for.  In the quantized layouts of both directions a value
 * that is not finite has a NaN code; a NaN leaves its block's scale to the block's other values (bsfp8_grouped_quantize
 * gives such a block the scale of an infinity, 2^120).  Rows at or past sum(k_e) are not
 * written.  hidden and ffn are multiples of 32, hidden at most 2^22, ffn at most 2^20.
 * capacity_rows == 0 returns BSFP8_OK without touching any pointer.
 */
int bsfp8_grouped_gemm_swiglu(const uint8_t* x_row_q, const uint8_t* x_row_s, int64_t capacity_rows,
                              int64_t hidden, const uint8_t* w_q, const uint8_t* w_s, int64_t ffn,
                              const float* probs, const int32_t* split_sizes, int32_t num_groups,
                              int recipe, void* ab, void* y, int y_dtype, int which, uint8_t* row_q,
                              uint8_t* row_s, uint8_t* col_q, uint8_t* col_s, uint32_t* status,
                              void* stream);

/*
 * Its gradient, through the second projection: with dh = dy[t] W2_e (fp32), sg = 1 / (1 + exp(-a)),
 *     da = dh * probs * b * sg * (1 + a * (1 - sg))      db = dh * probs * a * sg
 *     dprobs[t] = sum over the ffn channels of dh * a * sg * b
 * dy_row_q, dy_row_s  rowwise output of bsfp8_grouped_quantize for dy [capacity_rows][hidden]
 * w_col_q, w_col_s    W2 viewed as [num_groups * hidden][ffn], colwise with split sizes hidden, ...,
 *                     as bsfp8_grouped_gemm_dgrad takes it
 * ab                  as the forward kept it
 * dab                 bf16 [capacity_rows][2 ffn], (da | db), or NULL
 * which, row_q, ...   (da | db) quantized from its fp32 values, for [capacity_rows][2 ffn]
 * dprobs              fp32 [capacity_rows] or NULL; the parts of the tile columns are summed in order
 * workspace           bsfp8_grouped_gemm_swiglu_grad_workspace_bytes() bytes of device memory, needed
 *                     with dprobs (0 bytes: may be NULL)
 * At least one of dab, the quantized layouts and dprobs is asked for.
 */
size_t bsfp8_grouped_gemm_swiglu_grad_workspace_bytes(int64_t capacity_rows, int64_t ffn,
                                                      int32_t num_groups);
int bsfp8_grouped_gemm_swiglu_grad(const uint8_t* dy_row_q, const uint8_t* dy_row_s,
                                   int64_t capacity_rows, int64_t hidden, const uint8_t* w_col_q,
                                   const uint8_t* w_col_s, int64_t ffn, const void* ab,
                                   const float* probs, const int32_t* split_sizes, int32_t num_groups,
                                   int recipe, void* dab, int which, uint8_t* row_q, uint8_t* row_s,
                                   uint8_t* col_q, uint8_t* col_s, float* dprobs, void* workspace,
                                   uint32_t* status, void* stream);

/* ----------------------------------------------------------------------------------------- */
/* Norms before and after a block, fused with the block's gate and the residual sum.          */
/* ----------------------------------------------------------------------------------------- */

/* Element types of the residual stream, of parameters and of gradients. */
#define BSFP8_F32 0
#define BSFP8_BF16 1

/* Gates of a block's output. */
#define BSFP8_GATE_NONE 0
#define BSFP8_GATE_CHANNEL 1 /* gate[cols] */
#define BSFP8_GATE_TOKEN 2   /* gate[rows] */

/*
 * For each of `rows` rows of `cols` channels, in fp32:
 *     z = y * rstd_y * (post_weight + weight_offset),   rstd_y = 1 / sqrt(mean(y^2) + eps)
 *     r = x_scale * x + y_scale * gate * z
 *     n = r * rstd_r * (pre_weight + weight_offset),    rstd_r = 1 / sqrt(mean(r^2) + eps)
 * x            [rows][cols] of stream_dtype (BSFP8_F32 or BSFP8_BF16): the residual stream
 * y            [rows][cols] bf16, the block's output, or NULL (r = x_scale * x)
 * post_weight  fp32 [cols], the norm after the block, or NULL (z = y)
 * pre_weight   fp32 [cols], the norm before the next block, or NULL (no n)
 * gate         fp32, as gate_kind says (NULL for BSFP8_GATE_NONE)
 * r            [rows][cols] of stream_dtype; may be x itself, and may be NULL where pre_weight is given
 * n            [rows][cols] bf16 (required with pre_weight, NULL without)
 * rstd_y, rstd_r  fp32 [rows], kept for the gradient, or NULL
 * r and n are each rounded once from the fp32 values (n from r before its rounding).  A row of zeros
 * with eps == 0 gives NaN, and a mean square below 2^-126 has the precision of a subnormal fp32.  Any rows and
 * any cols in [1, 32768]; data pointers aligned to 16 bytes, each array contiguous.  Without y,
 * post_weight and gate must be NULL.
 * rows == 0 returns BSFP8_OK without touching any pointer.
 */
int bsfp8_residual_norm(int64_t rows, int64_t cols, const void* x, int stream_dtype, const void* y,
                        const float* post_weight, const float* pre_weight, const float* gate,
                        int gate_kind, float x_scale, float y_scale, float eps, float weight_offset,
                        void* r, void* n, float* rstd_y, float* rstd_r, void* stream);

/*
 * Its gradient.  With rh = r * rstd_r, yh = y * rstd_y (yh = y without post_weight):
 *     g1 = dn * (pre_weight + weight_offset)
 *     d  = dr + rstd_r * (g1 - rh * mean(g1 * rh))       dx = x_scale * d
 *     t  = y_scale * d, dz = gate * t
 *     g2 = dz * (post_weight + weight_offset)            dy = rstd_y * (g2 - yh * mean(g2 * yh))
 *                                                        (dy = dz without post_weight)
 *     dpre_weight = sum over rows of dn * rh             dpost_weight = sum over rows of dz * yh
 *     dgate = sum of t * z over the rows (BSFP8_GATE_CHANNEL) or the channels (BSFP8_GATE_TOKEN)
 * dn           [rows][cols] bf16, the gradient at n, or NULL (then r, rstd_r, pre_weight are NULL too)
 * dr           [rows][cols] of stream_dtype, the gradient at r, or NULL; dn or dr is given
 * r, rstd_r, rstd_y   as the forward left them (rstd_y with post_weight)
 * dx           [rows][cols] of stream_dtype or NULL; may be dr itself
 * dy           [rows][cols] bf16 or NULL; may be dn itself
 * dpre_weight, dpost_weight, dgate   fp32 or NULL; accumulate == 1 adds to the weights' and the
 *              channel gate's (one fp32 add each), a token gate's gradient is always stored
 * workspace    bsfp8_residual_norm_grad_workspace_bytes() bytes of device memory, needed when
 *              dpre_weight, dpost_weight or a channel gate's dgate is asked for
 * Sums over rows are taken in a fixed order.  rows == 0: the stored sums become zero.
 */
size_t bsfp8_residual_norm_grad_workspace_bytes(int64_t rows, int64_t cols);
int bsfp8_residual_norm_grad(int64_t rows, int64_t cols, int stream_dtype, const void* dn, const void* dr,
                             const void* r, const float* rstd_r, const float* pre_weight, const void* y,
                             const float* rstd_y, const float* post_weight, const float* gate,
                             int gate_kind, float x_scale, float y_scale, float weight_offset, void* dx,
                             void* dy, float* dpre_weight, float* dpost_weight, float* dgate,
                             int accumulate, void* workspace, void* stream);

/* ----------------------------------------------------------------------------------------- */
/* AdamW over many tensors in one launch, states in fp32 or in 8 bits.                        */
/* ----------------------------------------------------------------------------------------- */
/*
 * For each element, every operation rounded to fp32 in the order written (the scalars that depend
 * on lr and step are formed in fp64 and rounded once):
 *     g = grad * grad_scale
 *     m = m * beta1 + g * (1 - beta1)
 *     v = v * beta2 + g * g * (1 - beta2)
 *     p = p * (1 - lr * weight_decay) - m / (sqrt(v) * (1 - beta2^step)^(-1/2) + eps)
 *                                         * (lr / (1 - beta1^step))
 * BSFP8_STATE_F32: m and v are fp32 arrays.
 * BSFP8_STATE_8BIT: m and u = sqrt(v) are e4m3 arrays; every 128 consecutive elements of a tensor
 *   (the last block may be shorter) share one fp32 scale sf = max(amax * (1/448), 1e-30), a code
 *   standing for code * sf.  New states are stored as e4m3(m * (1 / sf)), a u that is not zero as at
 *   least the smallest code, 2^-9; p uses them unrounded.  Zeroed codes and scales are a valid start.
 *   bsfp8_adamw_step rounds to nearest: while another element holds its block's scale, a state that
 *   changes by less than half a code's step (3 to 6 percent) a step stays where it is.  sqrt(v) loses
 *   1 - sqrt(beta2) a step, so under nearest rounding it does not follow gradients that become smaller
 *   (the element's updates stay small) and lags behind ones that grow, and the lowest
 *   codes of m do not vanish when its gradients stop.  bsfp8_adamw_step_stochastic is for training.
 * Non-finite gradients enter the states (8-bit: an infinite one makes its block's scale infinite, and all 128
 * elements NaN in the next step); noop_flag is for skipping such a step.
 */
#define BSFP8_STATE_F32 0
#define BSFP8_STATE_8BIT 1

typedef struct bsfp8_adamw_tensor {
  void* param;              /* fp32 or bf16, updated */
  const void* grad;         /* fp32 or bf16 */
  void* exp_avg;            /* m: fp32, or e4m3 codes */
  void* exp_avg_sq;         /* v: fp32, or e4m3 codes of sqrt(v) */
  float* exp_avg_scale;     /* 8-bit states: fp32 [ceil(numel / 128)]; else NULL */
  float* exp_avg_sq_scale;  /* the same */
  void* copy;               /* bf16 copy of the new param, or NULL */
  int64_t numel;            /* >= 0 */
  float lr_scale;           /* this tensor's factor on lr */
  float decay_scale;        /* this tensor's factor on weight_decay */
} bsfp8_adamw_tensor;

/* Bytes of a plan for tensors of these sizes and the number of its chunks (a kernel argument);
 * 0 (and *num_chunks 0) for invalid arguments.  Host only. */
size_t bsfp8_adamw_plan_bytes(const int64_t* numels, int32_t num_tensors, int64_t* num_chunks);
/* Writes the plan into HOST memory; the caller copies it to the device (16-byte aligned) once and
 * keeps it while the tensors stay where they are.  Element pointers need only their element's
 * alignment.  Checks every tensor: BSFP8_ERR_NULL_POINTER, _SHAPE, _ALIGNMENT. */
int bsfp8_adamw_plan(const bsfp8_adamw_tensor* tensors, int32_t num_tensors, int param_dtype,
                     int grad_dtype, int state, void* host_plan, size_t host_plan_bytes);
/*
 * One step over the plan's tensors (param_dtype, grad_dtype, state and the counts as it was made with).
 * lr >= 0, 0 <= beta1, beta2 < 1, eps >= 0, weight_decay >= 0, step >= 1 (BSFP8_ERR_ARGUMENT).
 * lr_dev, step_dev  NULL, or device scalars that replace lr and step, read when the kernel runs (a
 *                   captured graph is replayed with new values); the same bounds hold for them, which
 *                   are not checked there
 * grad_scale        NULL (1), or a device fp32 scalar (clipping, loss scale)
 * noop_flag         NULL, or a device fp32 scalar: nonzero leaves everything as it is
 */
int bsfp8_adamw_step(const void* device_plan, int32_t num_tensors, int64_t num_chunks, int param_dtype,
                     int grad_dtype, int state, double lr, double beta1, double beta2, double eps,
                     double weight_decay, int64_t step, const float* lr_dev, const int32_t* step_dev,
                     const float* grad_scale, const float* noop_flag, void* stream);
/*
 * The same step with stochastic rounding of 8-bit states: each goes to one of the two e4m3 values around it,
 * with the probability that makes the expected state the unrounded one; a state that is a code stays.  The
 * random bits are a function of seed, step, the tensor's index in the plan and the element alone: the same
 * arguments give the same states.  p and copy are those of bsfp8_adamw_step.  With BSFP8_STATE_F32 nothing
 * is rounded and seed has no effect.
 */
int bsfp8_adamw_step_stochastic(const void* device_plan, int32_t num_tensors, int64_t num_chunks, int param_dtype,
                                int grad_dtype, int state, double lr, double beta1, double beta2, double eps,
                                double weight_decay, int64_t step, const float* lr_dev, const int32_t* step_dev,
                                const float* grad_scale, const float* noop_flag, uint64_t seed, void* stream);

/* ----------------------------------------------------------------------------------------- */
/* Tokens to their experts and back: the router's choice, the sort by expert, the rows        */
/* gathered for the grouped calls above, and their weighted sum.                              */
/* ----------------------------------------------------------------------------------------- */

/* Scores of the router. */
#define BSFP8_ROUTE_SOFTMAX 1
#define BSFP8_ROUTE_SIGMOID 2

#define BSFP8_MAX_TOP_K 32

/*
 * The top_k experts of each of `tokens` tokens and their probabilities, in fp32:
 *     BSFP8_ROUTE_SOFTMAX:  s[t][e] = exp(l[t][e]) / sum_i exp(l[t][i])          key = l + bias
 *     BSFP8_ROUTE_SIGMOID:  s[t][e] = 1 / (1 + exp2s(-l[t][e] * log2(e)))        key = s + bias
 *   with exp2s as stated at bsfp8_grouped_act_quantize (each operation rounded in the order written, so that the
 *   choice is the same on every IEEE machine).
 * logits    [tokens][num_experts] of logits_dtype (BSFP8_F32 or BSFP8_BF16).  A logit or key of -infinity masks the
 *           expert for that token: it is not chosen, and a logit of -infinity has the score 0.
 * bias      fp32 [num_experts], moves the choice alone, or NULL (0)
 * experts   int32 [tokens][top_k]: the experts of the largest keys, the largest first, the lowest index first among
 *           equals (+0 equals -0, a NaN key comes before all others); -1 where fewer than top_k are open
 * probs     fp32 [tokens][top_k]: scale * s of the chosen (0 beside -1); with renormalize == 1
 *           scale * s / (sum of the chosen s)
 * score_sum fp32 [num_experts] or NULL: sum of s[t][e] over the tokens, added in a fixed order
 * workspace bsfp8_route_topk_workspace_bytes() bytes of device memory, needed with score_sum
 * 1 <= num_experts <= BSFP8_MAX_GROUPS, 1 <= top_k <= min(num_experts, BSFP8_MAX_TOP_K), tokens * top_k <= 2^30.  The
 * logits begin at a multiple of 16 bytes, rows of any length follow one another.  tokens == 0 writes nothing but zeros
 * to score_sum.
 */
size_t bsfp8_route_topk_workspace_bytes(int64_t tokens, int32_t num_experts);
int bsfp8_route_topk(const void* logits, int logits_dtype, int64_t tokens, int32_t num_experts, int32_t top_k,
                     int scoring, const float* bias, int renormalize, float scale, float* probs, int32_t* experts,
                     float* score_sum, void* workspace, void* stream);

/*
 * Its gradient: dlogits [tokens][num_experts] of logits_dtype, the gradient of
 *     sum probs[t][j] * dprobs[t][j] + sum_e dscore_sum[e] * score_sum[e]
 * with respect to the logits, the choice held.  experts as the forward wrote them (an entry outside
 * [0, num_experts) is no choice; of an expert that stands twice both parts are added); dprobs fp32 [tokens][top_k];
 * dscore_sum fp32 [num_experts] or NULL (0).
 */
int bsfp8_route_topk_grad(const float* dprobs, const void* logits, int logits_dtype, const int32_t* experts,
                          int64_t tokens, int32_t num_experts, int32_t top_k, int scoring, int renormalize, float scale,
                          const float* dscore_sum, void* dlogits, void* stream);

/*
 * The choices c = t * top_k + j sorted by their experts, those of one expert in the order of c.  A choice whose expert
 * lies outside [0, num_experts) is dropped (no expert: -1; under expert parallelism: another rank's, with the first
 * local expert's index taken off).
 * experts      int32 [tokens][top_k]
 * probs        fp32 [tokens][top_k] or NULL
 * split_sizes  int32 [num_experts]: rows of each expert
 * rows         int32 [tokens][top_k]: the row of each choice, -1 if dropped
 * choices      int32 [tokens * top_k]: the choice of each row, -1 past the last row
 * row_probs    fp32 [tokens * top_k]: probs of each row's choice, 0 past the last row; NULL without probs
 * workspace    bsfp8_dispatch_plan_workspace_bytes() bytes of device memory (0 for few choices: may be NULL)
 * tokens * top_k <= 2^30.  tokens == 0 writes zeros to split_sizes.
 */
size_t bsfp8_dispatch_plan_workspace_bytes(int64_t tokens, int32_t top_k, int32_t num_experts);
int bsfp8_dispatch_plan(const int32_t* experts, const float* probs, int64_t tokens, int32_t top_k, int32_t num_experts,
                        int32_t* split_sizes, int32_t* rows, int32_t* choices, float* row_probs, void* workspace,
                        void* stream);

/*
 * Rows of tokens for their experts: out[rows[t][j]] = weights[t][j] * x[t], rounded once from fp32.
 * x        [tokens][cols] of dtype (BSFP8_F32 or BSFP8_BF16); out [capacity_rows][cols] of dtype
 * rows     int32 [tokens][top_k], as bsfp8_dispatch_plan writes them; one outside [0, capacity_rows) is skipped
 * weights  fp32 [tokens][top_k], or NULL (1: the rows are copied bit for bit)
 * Rows of out that no choice has are not written; no two choices have one row.  1 <= cols <= 2^24,
 * tokens * top_k <= 2^30, capacity_rows <= 2^31 - 1, and x is below 2^35 elements with cols rounded up to 8 2^n (above
 * 1024: to a multiple of 1024).  This is also the gradient of bsfp8_combine without weights.
 */
int bsfp8_dispatch(const void* x, int dtype, int64_t tokens, int64_t cols, const int32_t* rows, int32_t top_k,
                   const float* weights, void* out, int64_t capacity_rows, void* stream);

/*
 * The same rows straight into the quantized layouts of bsfp8_grouped_quantize for [capacity_rows][cols]: the bytes
 * that it writes for the rows of bsfp8_dispatch, except that weighted rows are quantized from their fp32 products.
 * x_bf16    [tokens][cols] bf16
 * choices   int32 [capacity_rows], as bsfp8_dispatch_plan writes them.  Rows at or past sum(split_sizes) are not written; a
 *           row before it whose choice lies outside [0, tokens * top_k) is one of zeros
 * recipe    BSFP8_RECIPE_MX_1X32_E8M0 or BSFP8_RECIPE_MXFP4_1X32_E8M0
 * split_sizes  as bsfp8_dispatch_plan writes them
 * capacity_rows + 127 must stay below 2^24 - 128, as for bsfp8_grouped_gemm_wgrad, here and in the two calls below that
 * quantize activations (the kernels address a group's channels with 32-bit offsets); BSFP8_ERR_SHAPE otherwise.
 */
int bsfp8_dispatch_quantize(const void* x_bf16, int64_t tokens, int64_t cols, const int32_t* choices, int32_t top_k,
                            const float* weights, int64_t capacity_rows, const int32_t* split_sizes,
                            int32_t num_groups, int recipe, int which, uint8_t* row_q, uint8_t* row_s, uint8_t* col_q,
                            uint8_t* col_s, uint32_t* status, void* stream);

/*
 * The experts' rows back at their tokens: out[t] = add[t] + sum_j weights[t][j] * y[rows[t][j]], the sum over j in fp32
 * in the order of j, rounded once.
 * y       [capacity_rows][cols] of dtype; a row outside [0, capacity_rows) counts as zero and is not read
 * weights fp32 [tokens][top_k] or NULL (1: this is the gradient of bsfp8_dispatch without weights)
 * add     [tokens][cols] of dtype or NULL (0); may be out itself
 * out     [tokens][cols] of dtype; its size bounded as x above
 */
int bsfp8_combine(const void* y, int dtype, int64_t capacity_rows, int64_t cols, const int32_t* rows, int64_t tokens,
                  int32_t top_k, const float* weights, const void* add, void* out, void* stream);

/*
 * Its gradient: dy[rows[t][j]] = weights[t][j] * dout[t] and dweights[t][j] = sum over the channels of
 * dout[t] * y[rows[t][j]] (0 for a choice without a row), the sum in fp32 in a fixed order.  (With x in place of dout
 * and the rows' gradient in place of y, dweights is that of a weighted bsfp8_dispatch, whose dx is bsfp8_combine of the
 * rows' gradient with the same weights.)
 * dout      [tokens][cols] of dtype
 * y         [capacity_rows][cols] of dtype, needed for dweights
 * dy        [capacity_rows][cols] of dtype or NULL; may be y itself.  Rows that no choice has are not written; no two
 *           choices have one row
 * dweights  fp32 [tokens][top_k] or NULL
 */
int bsfp8_combine_grad(const void* dout, int dtype, int64_t tokens, int64_t cols, const void* y, int64_t capacity_rows,
                       const int32_t* rows, int32_t top_k, const float* weights, void* dy, float* dweights,
                       void* stream);

/* ----------------------------------------------------------------------------------------- */
/* Activations kept in 8 bits for the backward pass.                                          */
/* ----------------------------------------------------------------------------------------- */
/*
 * bsfp8_grouped_act_quantize (activation BSFP8_ACT_SRELU or BSFP8_ACT_SWIGLU, the same bytes), and in the same pass its
 * input h, kept for the gradient in 8 bits: the bytes that bsfp8_grouped_quantize writes for h with
 * BSFP8_RECIPE_MX_1X32_E8M0 and BSFP8_ROWWISE.
 * kept_q, kept_s  those of [capacity_rows][cols] (SReLU) or [capacity_rows][2 cols] (SwiGLU)
 * cols is at most 2^21.
 */
int bsfp8_grouped_act_checkpoint(int activation, const void* h_bf16, const float* probs, int64_t capacity_rows,
                                 int64_t cols, const int32_t* split_sizes, int32_t num_groups, int recipe, int which,
                                 uint8_t* row_q, uint8_t* row_s, uint8_t* col_q, uint8_t* col_s, uint8_t* kept_q,
                                 uint8_t* kept_s, uint32_t* status, void* stream);

/*
 * The gradient from what was kept.  With h the values that kept_q and kept_s stand for, r = max(h, 0),
 * sg = 1 / (1 + exp2s(-a * log2(e))), in fp32, by the operations of bsfp8_grouped_act_quantize in their order (the bytes
 * that it writes for the gradient, and for the activation, of these values; a NaN has an MXFP8 NaN code, where the scale is
 * that of its block's other values, and gives an MXFP4 block the scale of an infinity):
 *     SReLU:   g = 2 r p dy                          quantized as [capacity_rows][cols]
 *              v = r^2
 *     SwiGLU:  (da | db) = (dy p b sg (1 + a (1 - sg)) | dy p a sg)        as [capacity_rows][2 cols]
 *              v = a sg b
 * which, row_q, ...   layouts of the gradient (recipe BSFP8_RECIPE_MX_1X32_E8M0 or BSFP8_RECIPE_MXFP4_1X32_E8M0); 0: none
 * y_col_q, y_col_s    NULL, or the activation p v again, in the colwise layout of [capacity_rows][cols] (same recipe):
 *                     the operand of the second projection's weight gradient, so that the forward need not keep it
 * dprobs     fp32 [capacity_rows] or NULL: sum over the channels of dy v, in a fixed order (live rows only)
 * workspace  bsfp8_grouped_act_checkpoint_grad_workspace_bytes() bytes of device memory, needed with dprobs
 * kept_q, kept_s, probs, dy as in the forward; dy_bf16 [capacity_rows][cols].  Some output is asked for.
 */
size_t bsfp8_grouped_act_checkpoint_grad_workspace_bytes(int64_t capacity_rows, int64_t cols);
int bsfp8_grouped_act_checkpoint_grad(int activation, const uint8_t* kept_q, const uint8_t* kept_s, const float* probs,
                                      const void* dy_bf16, int64_t capacity_rows, int64_t cols,
                                      const int32_t* split_sizes, int32_t num_groups, int recipe, int which,
                                      uint8_t* row_q, uint8_t* row_s, uint8_t* col_q, uint8_t* col_s, uint8_t* y_col_q,
                                      uint8_t* y_col_s, float* dprobs, void* workspace, uint32_t* status, void* stream);

/* Static description of a return code. */
const char* bsfp8_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* BSFP8_H */
