// C ABI of libbsfp8: argument validation, buffer-size queries and launches on the caller's
// stream.  Every host-checkable error is reported before any HIP call is made, so these
// checks run (and are tested) on machines without a GPU.  Nothing here allocates, and the
// library holds no mutable state.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/bsfp8.h"
#include <string.h>

#include "adamw_plan.hpp"
#include "group_layout.hpp"
#include "norm_layout.hpp"

namespace bsfp8 {
int launch_grouped_quantize(const void* in, int64_t R, int64_t C, const int32_t* splits, int E, int recipe,
                            int which, float zas, uint8_t* row_q, uint8_t* row_s, uint8_t* col_q, void* col_s,
                            const float* noop_flag, uint32_t* status, hipStream_t stream);
int launch_grouped_act_quantize(int act, const void* h, const float* probs, const void* dy, int64_t R, int64_t C,
                                const int32_t* splits, int E, int recipe, int which, uint8_t* row_q, uint8_t* row_s,
                                uint8_t* col_q, void* col_s, uint32_t* status, hipStream_t stream);
int launch_grouped_gemm_wgrad(const uint8_t* dy_q, const void* dy_s, int64_t n, const uint8_t* x_q, const void* x_s,
                              int64_t h, const int32_t* splits, int E, int64_t R, int recipe, float* out,
                              int accumulate, uint32_t* status, hipStream_t stream);
int launch_grouped_gemm_fprop(const uint8_t* x_q, const uint8_t* x_s, int64_t R, int64_t K, const uint8_t* w_q,
                              const uint8_t* w_s, int64_t N, const int32_t* splits, int E, int recipe, void* out,
                              int out_dtype, uint32_t* status, hipStream_t stream);
int launch_grouped_gemm_dgrad(const uint8_t* dy_q, const uint8_t* dy_s, int64_t R, int64_t n, const uint8_t* w_q,
                              const void* w_s, int64_t k, const int32_t* splits, int E, int recipe, void* out,
                              int out_dtype, uint32_t* status, hipStream_t stream);
int launch_grouped_gemm_swiglu(const uint8_t* x_q, const uint8_t* x_s, int64_t R, int64_t hidden, const uint8_t* w_q,
                               const uint8_t* w_s, int64_t F, const float* probs, const int32_t* splits, int E,
                               void* ab, void* y, int y_f32, uint8_t* row_q, uint8_t* row_s, uint8_t* col_q,
                               uint8_t* col_s, uint32_t* status, hipStream_t stream);
int launch_grouped_gemm_swiglu_grad(const uint8_t* dy_q, const uint8_t* dy_s, int64_t R, int64_t hidden,
                                    const uint8_t* w_q, const uint8_t* w_s, int64_t F, const void* ab,
                                    const float* probs, const int32_t* splits, int E, void* dab, uint8_t* row_q,
                                    uint8_t* row_s, uint8_t* col_q, uint8_t* col_s, float* dprobs, float* workspace,
                                    uint32_t* status, hipStream_t stream);
size_t glu_grad_workspace_bytes(int64_t R, int64_t F, int E);
int launch_residual_norm(int64_t R, int64_t C, const void* x, int x_f32, const void* y, const float* post_w,
                         const float* pre_w, const float* gate, int gate_kind, float x_scale, float y_scale, float eps,
                         float offset, void* r, void* n, float* rstd_y, float* rstd_r, hipStream_t stream);
int launch_residual_norm_grad(int64_t R, int64_t C, int x_f32, const void* dn, const void* dr, const void* r,
                              const float* rstd_r, const float* pre_w, const void* y, const float* rstd_y,
                              const float* post_w, const float* gate, int gate_kind, float x_scale, float y_scale,
                              float offset, void* dx, void* dy, float* dpre_w, float* dpost_w, float* dgate,
                              int accumulate, float* workspace, hipStream_t stream);
int launch_adamw(const void* plan, int32_t num_tensors, int64_t chunks, int p_f32, int g_f32, int q8, double lr,
                 double beta1, double beta2, double eps, double decay, int64_t step, const float* lr_dev,
                 const int32_t* step_dev, const float* grad_scale, const float* noop_flag, const uint64_t* seed,
                 hipStream_t stream);
}  // namespace bsfp8

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool valid_recipe(int r) {
  return r == BSFP8_RECIPE_MX_1X32_E8M0 || r == BSFP8_RECIPE_PER_CHANNEL_128_F32 || r == BSFP8_RECIPE_MXFP4_1X32_E8M0;
}
// recipes with E8M0 block scales (both layouts; the only ones the m-grouped GEMMs take)
bool mx_recipe(int r) { return r == BSFP8_RECIPE_MX_1X32_E8M0 || r == BSFP8_RECIPE_MXFP4_1X32_E8M0; }
// the recipe argument of the GEMM calls: a data recipe, or MXFP8 on the scaled fp8 MFMA
bool wgrad_recipe(int r) { return valid_recipe(r) || r == (BSFP8_RECIPE_MX_1X32_E8M0 | BSFP8_GEMM_FP8_MFMA); }
bool mgrouped_recipe(int r) { return mx_recipe(r) || r == (BSFP8_RECIPE_MX_1X32_E8M0 | BSFP8_GEMM_FP8_MFMA); }
// data elements per byte
int64_t per_byte(int r) { return r == BSFP8_RECIPE_MXFP4_1X32_E8M0 ? 2 : 1; }
bool valid_groups(int32_t e) { return e > 0 && e <= BSFP8_MAX_GROUPS; }
// dims must be positive multiples of 32 and small enough that byte offsets fit in int64
bool valid_dim(int64_t d) { return d > 0 && d % 32 == 0 && d <= (int64_t(1) << 40); }
// The GEMM kernels address a 256-row operand tile with 32-bit offsets: 256 * row length must
// stay below 2^32, i.e. a K extent (k for fprop, a group's padded rows for wgrad) below 2^24.
constexpr int64_t kMaxKExtent = (int64_t(1) << 24) - 128;
// The GEMM epilogues address a 128-row block of the output with 32-bit byte offsets and mark
// lanes past the last column with offsets from 2^31 up: 128 * 4 * (output row length) must stay
// below 2^31.
constexpr int64_t kMaxOutCols = int64_t(1) << 21;
bool aligned_to(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
bool valid_dtype(int d) { return d == BSFP8_F32 || d == BSFP8_BF16; }
bool finite_nonnegative(double v) { return isfinite(v) && v >= 0.0; }
// rows and columns of the residual norms: every element offset fits in int64
bool valid_norm_shape(int64_t rows, int64_t cols) {
  return rows >= 0 && rows <= (int64_t(1) << 40) && cols >= 1 && cols <= bsfp8::kNormMaxCols;
}
// the block's output, its norm and its gate, as both directions take them
int check_norm_block(const void* y, const float* post_w, const float* gate, int gate_kind) {
  if (gate_kind < BSFP8_GATE_NONE || gate_kind > BSFP8_GATE_TOKEN) return BSFP8_ERR_ARGUMENT;
  if (gate_kind != BSFP8_GATE_NONE && gate == nullptr) return BSFP8_ERR_NULL_POINTER;
  if (gate_kind == BSFP8_GATE_NONE && gate != nullptr) return BSFP8_ERR_ARGUMENT;
  if (y == nullptr && (post_w != nullptr || gate != nullptr)) return BSFP8_ERR_ARGUMENT;
  return BSFP8_OK;
}

// quantized outputs of a gated projection: the pointers of the layouts asked for
int check_glu_quantized(int which, const void* row_q, const void* row_s, const void* col_q, const void* col_s) {
  if ((which & BSFP8_ROWWISE) && (row_q == nullptr || row_s == nullptr)) return BSFP8_ERR_NULL_POINTER;
  if ((which & BSFP8_COLWISE) && (col_q == nullptr || col_s == nullptr)) return BSFP8_ERR_NULL_POINTER;
  if ((which & BSFP8_ROWWISE) && (!aligned16(row_q) || !aligned16(row_s))) return BSFP8_ERR_ALIGNMENT;
  if ((which & BSFP8_COLWISE) && (!aligned16(col_q) || !aligned16(col_s))) return BSFP8_ERR_ALIGNMENT;
  return BSFP8_OK;
}
// the gated projections' loads mark offsets past a 256-row tile by 2^31
constexpr int64_t kMaxGluHidden = int64_t(1) << 22;
// what both directions of a gated projection need of their sizes
int check_glu_shape(int64_t capacity_rows, int64_t hidden, int64_t ffn, int32_t num_groups, int recipe, int which) {
  if (!valid_recipe(recipe & ~BSFP8_GEMM_FP8_MFMA)) return BSFP8_ERR_RECIPE;
  if (recipe != BSFP8_RECIPE_MX_1X32_E8M0) return BSFP8_ERR_LAYOUT;
  if (!valid_groups(num_groups)) return BSFP8_ERR_NUM_GROUPS;
  if (!valid_dim(hidden) || !valid_dim(ffn) || capacity_rows < 0 || capacity_rows > (int64_t(1) << 31) ||
      hidden > kMaxGluHidden || 2 * ffn > kMaxOutCols)
    return BSFP8_ERR_SHAPE;
  if ((which & ~(BSFP8_ROWWISE | BSFP8_COLWISE)) != 0) return BSFP8_ERR_ARGUMENT;
  return BSFP8_OK;
}

// an AdamW step; seed: NULL, or that of the 8-bit states' stochastic rounding
int adamw_step(const void* device_plan, int32_t num_tensors, int64_t num_chunks, int param_dtype, int grad_dtype,
               int state, double lr, double beta1, double beta2, double eps, double weight_decay, int64_t step,
               const float* lr_dev, const int32_t* step_dev, const float* grad_scale, const float* noop_flag,
               const uint64_t* seed, void* stream) {
  if (!valid_dtype(param_dtype) || !valid_dtype(grad_dtype) || (state != BSFP8_STATE_F32 && state != BSFP8_STATE_8BIT))
    return BSFP8_ERR_ARGUMENT;
  if (!finite_nonnegative(lr) || !finite_nonnegative(eps) || !finite_nonnegative(weight_decay) ||
      !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || step < 1)
    return BSFP8_ERR_ARGUMENT;
  if (num_tensors <= 0 || num_chunks < 0 || num_chunks > 0x7fffffff) return BSFP8_ERR_SHAPE;
  if (num_chunks == 0) return BSFP8_OK;  // only empty tensors
  if (device_plan == nullptr) return BSFP8_ERR_NULL_POINTER;
  if (!aligned16(device_plan) || !aligned4(lr_dev) || !aligned4(step_dev) || !aligned4(grad_scale) ||
      !aligned4(noop_flag))
    return BSFP8_ERR_ALIGNMENT;
  return bsfp8::launch_adamw(device_plan, num_tensors, num_chunks, param_dtype == BSFP8_F32, grad_dtype == BSFP8_F32,
                             state == BSFP8_STATE_8BIT, lr, beta1, beta2, eps, weight_decay, step, lr_dev, step_dev,
                             grad_scale, noop_flag, seed, (hipStream_t)stream);
}

}  // namespace

extern "C" {

int64_t bsfp8_colwise_rows_bound(int64_t capacity_rows, int32_t num_groups) {
  if (capacity_rows < 0 || !valid_groups(num_groups)) return 0;
  return bsfp8::col_rows_bound(capacity_rows, num_groups);
}

size_t bsfp8_colwise_data_bytes(int64_t capacity_rows, int64_t cols, int32_t num_groups, int recipe) {
  if (!valid_dim(cols) || !valid_recipe(recipe)) return 0;
  return (size_t)bsfp8_colwise_rows_bound(capacity_rows, num_groups) * (size_t)(cols / per_byte(recipe));
}

size_t bsfp8_colwise_scale_bytes(int64_t capacity_rows, int64_t cols, int32_t num_groups, int recipe) {
  if (!valid_dim(cols) || !valid_recipe(recipe)) return 0;
  const size_t rows = (size_t)bsfp8_colwise_rows_bound(capacity_rows, num_groups);
  if (mx_recipe(recipe)) return rows / 32 * (size_t)cols;
  return rows / 128 * (size_t)cols * sizeof(float);
}

size_t bsfp8_rowwise_data_bytes(int64_t rows, int64_t cols, int recipe) {
  if (rows < 0 || !valid_dim(cols) || !mx_recipe(recipe)) return 0;
  return (size_t)rows * (size_t)(cols / per_byte(recipe));
}

size_t bsfp8_rowwise_scale_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || !valid_dim(cols)) return 0;
  return (size_t)rows * (size_t)(cols / 32);
}

int bsfp8_grouped_quantize(const void* in_bf16, int64_t capacity_rows, int64_t cols, const int32_t* split_sizes,
                           int32_t num_groups, int recipe, int which, float zero_amax_scale, uint8_t* row_q,
                           uint8_t* row_s, uint8_t* col_q, void* col_s, const float* noop_flag, uint32_t* status,
                           void* stream) {
  if (!valid_recipe(recipe)) return BSFP8_ERR_RECIPE;
  if (which <= 0 || (which & ~(BSFP8_ROWWISE | BSFP8_COLWISE)) != 0) return BSFP8_ERR_ARGUMENT;
  if ((which & BSFP8_ROWWISE) && !mx_recipe(recipe)) return BSFP8_ERR_LAYOUT;
  if (capacity_rows < 0 || !valid_dim(cols)) return BSFP8_ERR_SHAPE;
  if (recipe == BSFP8_RECIPE_PER_CHANNEL_128_F32 && !(isfinite(zero_amax_scale) && zero_amax_scale >= 0.0f))
    return BSFP8_ERR_ARGUMENT;
  if (split_sizes == nullptr && (which & BSFP8_COLWISE)) return BSFP8_ERR_NULL_POINTER;
  if (split_sizes != nullptr && !valid_groups(num_groups)) return BSFP8_ERR_NUM_GROUPS;
  if (capacity_rows == 0) return BSFP8_OK;  // nothing to read or write
  if (in_bf16 == nullptr) return BSFP8_ERR_NULL_POINTER;
  if ((which & BSFP8_ROWWISE) && (row_q == nullptr || row_s == nullptr)) return BSFP8_ERR_NULL_POINTER;
  if ((which & BSFP8_COLWISE) && (col_q == nullptr || col_s == nullptr)) return BSFP8_ERR_NULL_POINTER;
  if (!aligned16(in_bf16) || !aligned4(split_sizes) || !aligned4(noop_flag) || !aligned4(status))
    return BSFP8_ERR_ALIGNMENT;
  if ((which & BSFP8_ROWWISE) && (!aligned16(row_q) || !aligned16(row_s))) return BSFP8_ERR_ALIGNMENT;
  if ((which & BSFP8_COLWISE) && (!aligned16(col_q) || !aligned16(col_s))) return BSFP8_ERR_ALIGNMENT;
  return bsfp8::launch_grouped_quantize(in_bf16, capacity_rows, cols, split_sizes, split_sizes ? num_groups : 0,
                                        recipe, which, zero_amax_scale, (which & BSFP8_ROWWISE) ? row_q : nullptr,
                                        (which & BSFP8_ROWWISE) ? row_s : nullptr,
                                        (which & BSFP8_COLWISE) ? col_q : nullptr,
                                        (which & BSFP8_COLWISE) ? col_s : nullptr, noop_flag, status,
                                        (hipStream_t)stream);
}

int bsfp8_grouped_act_quantize(int activation, const void* h_bf16, const float* probs, const void* dy_bf16,
                               int64_t capacity_rows, int64_t cols, const int32_t* split_sizes, int32_t num_groups,
                               int recipe, int which, uint8_t* row_q, uint8_t* row_s, uint8_t* col_q, void* col_s,
                               uint32_t* status, void* stream) {
  if (activation < BSFP8_ACT_SRELU || activation > BSFP8_ACT_SWIGLU_GRAD) return BSFP8_ERR_ARGUMENT;
  const bool grad = activation == BSFP8_ACT_SRELU_GRAD || activation == BSFP8_ACT_SWIGLU_GRAD;
  if (!valid_recipe(recipe)) return BSFP8_ERR_RECIPE;
  if (!mx_recipe(recipe)) return BSFP8_ERR_LAYOUT;
  if (which <= 0 || (which & ~(BSFP8_ROWWISE | BSFP8_COLWISE)) != 0) return BSFP8_ERR_ARGUMENT;
  if (capacity_rows < 0 || !valid_dim(cols)) return BSFP8_ERR_SHAPE;
  if (split_sizes == nullptr) return BSFP8_ERR_NULL_POINTER;
  if (!valid_groups(num_groups)) return BSFP8_ERR_NUM_GROUPS;
  if (capacity_rows == 0) return BSFP8_OK;  // nothing to read or write
  if (h_bf16 == nullptr || (grad && dy_bf16 == nullptr)) return BSFP8_ERR_NULL_POINTER;
  if ((which & BSFP8_ROWWISE) && (row_q == nullptr || row_s == nullptr)) return BSFP8_ERR_NULL_POINTER;
  if ((which & BSFP8_COLWISE) && (col_q == nullptr || col_s == nullptr)) return BSFP8_ERR_NULL_POINTER;
  if (!aligned16(h_bf16) || !aligned16(dy_bf16) || !aligned4(probs) || !aligned4(split_sizes) || !aligned4(status))
    return BSFP8_ERR_ALIGNMENT;
  if ((which & BSFP8_ROWWISE) && (!aligned16(row_q) || !aligned16(row_s))) return BSFP8_ERR_ALIGNMENT;
  if ((which & BSFP8_COLWISE) && (!aligned16(col_q) || !aligned16(col_s))) return BSFP8_ERR_ALIGNMENT;
  return bsfp8::launch_grouped_act_quantize(activation, h_bf16, probs, grad ? dy_bf16 : nullptr, capacity_rows,
                                            cols, split_sizes, num_groups, recipe, which,
                                            (which & BSFP8_ROWWISE) ? row_q : nullptr,
                                            (which & BSFP8_ROWWISE) ? row_s : nullptr,
                                            (which & BSFP8_COLWISE) ? col_q : nullptr,
                                            (which & BSFP8_COLWISE) ? col_s : nullptr, status, (hipStream_t)stream);
}

int bsfp8_grouped_gemm_wgrad(const uint8_t* dy_col_q, const void* dy_col_s, int64_t n, const uint8_t* x_col_q,
                             const void* x_col_s, int64_t h, const int32_t* split_sizes, int32_t num_groups,
                             int64_t capacity_rows, int recipe, float* out, int accumulate, uint32_t* status,
                             void* stream) {
  if (!wgrad_recipe(recipe)) return BSFP8_ERR_RECIPE;
  if (!valid_groups(num_groups)) return BSFP8_ERR_NUM_GROUPS;
  if (!valid_dim(n) || !valid_dim(h) || capacity_rows < 0) return BSFP8_ERR_SHAPE;
  if (capacity_rows + 127 > kMaxKExtent || h > kMaxOutCols) return BSFP8_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return BSFP8_ERR_ARGUMENT;
  if (split_sizes == nullptr || out == nullptr) return BSFP8_ERR_NULL_POINTER;
  // the operands are read only when some group is non-empty, which needs capacity_rows > 0
  if (capacity_rows > 0 && (dy_col_q == nullptr || dy_col_s == nullptr || x_col_q == nullptr || x_col_s == nullptr))
    return BSFP8_ERR_NULL_POINTER;
  if (!aligned16(dy_col_q) || !aligned16(x_col_q) || !aligned16(dy_col_s) || !aligned16(x_col_s) ||
      !aligned16(out) || !aligned4(split_sizes) || !aligned4(status))
    return BSFP8_ERR_ALIGNMENT;
  return bsfp8::launch_grouped_gemm_wgrad(dy_col_q, dy_col_s, n, x_col_q, x_col_s, h, split_sizes, num_groups,
                                          capacity_rows, recipe, out, accumulate, status, (hipStream_t)stream);
}

int bsfp8_grouped_gemm_fprop(const uint8_t* x_row_q, const uint8_t* x_row_s, int64_t capacity_rows, int64_t k,
                             const uint8_t* w_q, const uint8_t* w_s, int64_t n, const int32_t* split_sizes,
                             int32_t num_groups, int recipe, void* out, int out_dtype, uint32_t* status,
                             void* stream) {
  if (!mgrouped_recipe(recipe)) return BSFP8_ERR_RECIPE;
  if (!valid_groups(num_groups)) return BSFP8_ERR_NUM_GROUPS;
  if (!valid_dim(k) || !valid_dim(n) || capacity_rows < 0 || k > kMaxKExtent || n > kMaxOutCols)
    return BSFP8_ERR_SHAPE;
  if (out_dtype != BSFP8_OUT_F32 && out_dtype != BSFP8_OUT_BF16) return BSFP8_ERR_ARGUMENT;
  if (capacity_rows == 0) return BSFP8_OK;  // zero-row early return: nothing is dereferenced
  if (x_row_q == nullptr || x_row_s == nullptr || w_q == nullptr || w_s == nullptr || split_sizes == nullptr ||
      out == nullptr)
    return BSFP8_ERR_NULL_POINTER;
  if (!aligned16(x_row_q) || !aligned16(x_row_s) || !aligned16(w_q) || !aligned16(w_s) || !aligned16(out) ||
      !aligned4(split_sizes) || !aligned4(status))
    return BSFP8_ERR_ALIGNMENT;
  return bsfp8::launch_grouped_gemm_fprop(x_row_q, x_row_s, capacity_rows, k, w_q, w_s, n, split_sizes, num_groups,
                                          recipe, out, out_dtype, status, (hipStream_t)stream);
}

int bsfp8_grouped_gemm_dgrad(const uint8_t* dy_row_q, const uint8_t* dy_row_s, int64_t capacity_rows, int64_t n,
                             const uint8_t* w_col_q, const void* w_col_s, int64_t k, const int32_t* split_sizes,
                             int32_t num_groups, int recipe, void* out, int out_dtype, uint32_t* status,
                             void* stream) {
  if (!mgrouped_recipe(recipe)) return BSFP8_ERR_RECIPE;
  if (!valid_groups(num_groups)) return BSFP8_ERR_NUM_GROUPS;
  // the weight rows are n rounded up to 128: that padded length bounds the 32-bit tile offsets
  if (!valid_dim(n) || !valid_dim(k) || capacity_rows < 0 || n + 127 > kMaxKExtent || k > kMaxOutCols)
    return BSFP8_ERR_SHAPE;
  if (out_dtype != BSFP8_OUT_F32 && out_dtype != BSFP8_OUT_BF16) return BSFP8_ERR_ARGUMENT;
  if (capacity_rows == 0) return BSFP8_OK;  // zero-row early return: nothing is dereferenced
  if (dy_row_q == nullptr || dy_row_s == nullptr || w_col_q == nullptr || w_col_s == nullptr ||
      split_sizes == nullptr || out == nullptr)
    return BSFP8_ERR_NULL_POINTER;
  if (!aligned16(dy_row_q) || !aligned16(dy_row_s) || !aligned16(w_col_q) || !aligned16(w_col_s) || !aligned16(out) ||
      !aligned4(split_sizes) || !aligned4(status))
    return BSFP8_ERR_ALIGNMENT;
  return bsfp8::launch_grouped_gemm_dgrad(dy_row_q, dy_row_s, capacity_rows, n, w_col_q, w_col_s, k, split_sizes,
                                          num_groups, recipe, out, out_dtype, status, (hipStream_t)stream);
}

int bsfp8_grouped_gemm_swiglu(const uint8_t* x_row_q, const uint8_t* x_row_s, int64_t capacity_rows, int64_t hidden,
                              const uint8_t* w_q, const uint8_t* w_s, int64_t ffn, const float* probs,
                              const int32_t* split_sizes, int32_t num_groups, int recipe, void* ab, void* y,
                              int y_dtype, int which, uint8_t* row_q, uint8_t* row_s, uint8_t* col_q, uint8_t* col_s,
                              uint32_t* status, void* stream) {
  int rc = check_glu_shape(capacity_rows, hidden, ffn, num_groups, recipe, which);
  if (rc != BSFP8_OK) return rc;
  if (y_dtype != BSFP8_OUT_F32 && y_dtype != BSFP8_OUT_BF16) return BSFP8_ERR_ARGUMENT;
  if (capacity_rows == 0) return BSFP8_OK;
  if (ab == nullptr && y == nullptr && which == 0) return BSFP8_ERR_ARGUMENT;
  if (x_row_q == nullptr || x_row_s == nullptr || w_q == nullptr || w_s == nullptr || split_sizes == nullptr)
    return BSFP8_ERR_NULL_POINTER;
  if (!aligned16(x_row_q) || !aligned16(x_row_s) || !aligned16(w_q) || !aligned16(w_s) || !aligned4(probs) ||
      !aligned4(split_sizes) || !aligned16(ab) || !aligned16(y) || !aligned4(status))
    return BSFP8_ERR_ALIGNMENT;
  rc = check_glu_quantized(which, row_q, row_s, col_q, col_s);
  if (rc != BSFP8_OK) return rc;
  const bool row = (which & BSFP8_ROWWISE) != 0, col = (which & BSFP8_COLWISE) != 0;
  return bsfp8::launch_grouped_gemm_swiglu(x_row_q, x_row_s, capacity_rows, hidden, w_q, w_s, ffn, probs, split_sizes,
                                           num_groups, ab, y, y_dtype == BSFP8_OUT_F32, row ? row_q : nullptr,
                                           row ? row_s : nullptr, col ? col_q : nullptr, col ? col_s : nullptr,
                                           status, (hipStream_t)stream);
}

size_t bsfp8_grouped_gemm_swiglu_grad_workspace_bytes(int64_t capacity_rows, int64_t ffn, int32_t num_groups) {
  if (check_glu_shape(capacity_rows, 32, ffn, num_groups, BSFP8_RECIPE_MX_1X32_E8M0, 0) != BSFP8_OK) return 0;
  return bsfp8::glu_grad_workspace_bytes(capacity_rows, ffn, num_groups);
}

int bsfp8_grouped_gemm_swiglu_grad(const uint8_t* dy_row_q, const uint8_t* dy_row_s, int64_t capacity_rows,
                                   int64_t hidden, const uint8_t* w_col_q, const uint8_t* w_col_s, int64_t ffn,
                                   const void* ab, const float* probs, const int32_t* split_sizes,
                                   int32_t num_groups, int recipe, void* dab, int which, uint8_t* row_q,
                                   uint8_t* row_s, uint8_t* col_q, uint8_t* col_s, float* dprobs, void* workspace,
                                   uint32_t* status, void* stream) {
  int rc = check_glu_shape(capacity_rows, hidden, ffn, num_groups, recipe, which);
  if (rc != BSFP8_OK) return rc;
  if (capacity_rows == 0) return BSFP8_OK;
  if (dab == nullptr && which == 0 && dprobs == nullptr) return BSFP8_ERR_ARGUMENT;
  if (dy_row_q == nullptr || dy_row_s == nullptr || w_col_q == nullptr || w_col_s == nullptr || ab == nullptr ||
      split_sizes == nullptr)
    return BSFP8_ERR_NULL_POINTER;
  if (dprobs != nullptr && workspace == nullptr &&
      bsfp8::glu_grad_workspace_bytes(capacity_rows, ffn, num_groups) > 0)
    return BSFP8_ERR_NULL_POINTER;
  if (!aligned16(dy_row_q) || !aligned16(dy_row_s) || !aligned16(w_col_q) || !aligned16(w_col_s) || !aligned16(ab) ||
      !aligned4(probs) || !aligned4(split_sizes) || !aligned16(dab) || !aligned4(dprobs) || !aligned16(workspace) ||
      !aligned4(status))
    return BSFP8_ERR_ALIGNMENT;
  rc = check_glu_quantized(which, row_q, row_s, col_q, col_s);
  if (rc != BSFP8_OK) return rc;
  const bool row = (which & BSFP8_ROWWISE) != 0, col = (which & BSFP8_COLWISE) != 0;
  return bsfp8::launch_grouped_gemm_swiglu_grad(
      dy_row_q, dy_row_s, capacity_rows, hidden, w_col_q, w_col_s, ffn, ab, probs, split_sizes, num_groups, dab,
      row ? row_q : nullptr, row ? row_s : nullptr, col ? col_q : nullptr, col ? col_s : nullptr, dprobs,
      (float*)workspace, status, (hipStream_t)stream);
}

int bsfp8_residual_norm(int64_t rows, int64_t cols, const void* x, int stream_dtype, const void* y,
                        const float* post_weight, const float* pre_weight, const float* gate, int gate_kind,
                        float x_scale, float y_scale, float eps, float weight_offset, void* r, void* n, float* rstd_y,
                        float* rstd_r, void* stream) {
  if (!valid_norm_shape(rows, cols)) return BSFP8_ERR_SHAPE;
  if (!valid_dtype(stream_dtype) || !isfinite(x_scale) || !isfinite(y_scale) || !isfinite(weight_offset) ||
      !finite_nonnegative(eps))
    return BSFP8_ERR_ARGUMENT;
  if (rows == 0) return BSFP8_OK;
  const int rc = check_norm_block(y, post_weight, gate, gate_kind);
  if (rc != BSFP8_OK) return rc;
  if (x == nullptr || (pre_weight != nullptr && n == nullptr) || (pre_weight == nullptr && r == nullptr))
    return BSFP8_ERR_NULL_POINTER;
  if (pre_weight == nullptr && (n != nullptr || rstd_r != nullptr)) return BSFP8_ERR_ARGUMENT;
  if (post_weight == nullptr && rstd_y != nullptr) return BSFP8_ERR_ARGUMENT;
  if (!aligned16(x) || !aligned16(y) || !aligned16(post_weight) || !aligned16(pre_weight) || !aligned16(gate) ||
      !aligned16(r) || !aligned16(n) || !aligned4(rstd_y) || !aligned4(rstd_r))
    return BSFP8_ERR_ALIGNMENT;
  return bsfp8::launch_residual_norm(rows, cols, x, stream_dtype == BSFP8_F32, y, post_weight, pre_weight, gate,
                                     gate_kind, x_scale, y_scale, eps, weight_offset, r, n, rstd_y, rstd_r,
                                     (hipStream_t)stream);
}

size_t bsfp8_residual_norm_grad_workspace_bytes(int64_t rows, int64_t cols) {
  if (!valid_norm_shape(rows, cols)) return 0;
  return (size_t)bsfp8::norm_grad_slots(rows, cols) * 2 * (size_t)cols * sizeof(float);
}

int bsfp8_residual_norm_grad(int64_t rows, int64_t cols, int stream_dtype, const void* dn, const void* dr,
                             const void* r, const float* rstd_r, const float* pre_weight, const void* y,
                             const float* rstd_y, const float* post_weight, const float* gate, int gate_kind,
                             float x_scale, float y_scale, float weight_offset, void* dx, void* dy,
                             float* dpre_weight, float* dpost_weight, float* dgate, int accumulate, void* workspace,
                             void* stream) {
  if (!valid_norm_shape(rows, cols)) return BSFP8_ERR_SHAPE;
  if (!valid_dtype(stream_dtype) || !isfinite(x_scale) || !isfinite(y_scale) || !isfinite(weight_offset) ||
      (accumulate != 0 && accumulate != 1))
    return BSFP8_ERR_ARGUMENT;
  const bool sums = dpre_weight != nullptr || dpost_weight != nullptr ||
                    (gate_kind == BSFP8_GATE_CHANNEL && dgate != nullptr);
  if (rows > 0) {
    const int rc = check_norm_block(y, post_weight, gate, gate_kind);
    if (rc != BSFP8_OK) return rc;
    if (dn == nullptr && dr == nullptr) return BSFP8_ERR_NULL_POINTER;
    if (dn != nullptr && (r == nullptr || rstd_r == nullptr || pre_weight == nullptr)) return BSFP8_ERR_NULL_POINTER;
    if (post_weight != nullptr && rstd_y == nullptr) return BSFP8_ERR_NULL_POINTER;
    if (sums && workspace == nullptr) return BSFP8_ERR_NULL_POINTER;
  } else if (gate_kind < BSFP8_GATE_NONE || gate_kind > BSFP8_GATE_TOKEN) {
    return BSFP8_ERR_ARGUMENT;
  }
  // a gradient of what the call has none of
  if (rows > 0 && ((dn == nullptr && (dpre_weight != nullptr || r != nullptr || rstd_r != nullptr ||
                                      pre_weight != nullptr)) ||
                   (y == nullptr && dy != nullptr) || (post_weight == nullptr && dpost_weight != nullptr)))
    return BSFP8_ERR_ARGUMENT;
  if (gate_kind == BSFP8_GATE_NONE && dgate != nullptr) return BSFP8_ERR_ARGUMENT;
  if (!aligned16(dn) || !aligned16(dr) || !aligned16(r) || !aligned16(pre_weight) || !aligned16(y) ||
      !aligned16(post_weight) || !aligned16(gate) || !aligned16(dx) || !aligned16(dy) || !aligned16(dpre_weight) ||
      !aligned16(dpost_weight) || !aligned16(dgate) || !aligned16(workspace) || !aligned4(rstd_r) || !aligned4(rstd_y))
    return BSFP8_ERR_ALIGNMENT;
  return bsfp8::launch_residual_norm_grad(rows, cols, stream_dtype == BSFP8_F32, dn, dr, r, rstd_r, pre_weight, y,
                                          rstd_y, post_weight, gate, gate_kind, x_scale, y_scale, weight_offset, dx,
                                          dy, dpre_weight, dpost_weight, dgate, accumulate, (float*)workspace,
                                          (hipStream_t)stream);
}

size_t bsfp8_adamw_plan_bytes(const int64_t* numels, int32_t num_tensors, int64_t* num_chunks) {
  int64_t chunks = 0;
  bool ok = numels != nullptr && num_tensors > 0;
  for (int32_t i = 0; ok && i < num_tensors; ++i) {
    ok = numels[i] >= 0 && numels[i] <= (int64_t(1) << 40);
    if (ok) chunks += bsfp8::adam_chunks_of(numels[i]);
    ok = ok && chunks <= 0x7fffffff;
  }
  if (!ok) chunks = 0;
  if (num_chunks != nullptr) *num_chunks = chunks;
  return ok ? (size_t)(bsfp8::adam_table_bytes(num_tensors) + chunks * (int64_t)sizeof(bsfp8::AdamChunk)) : 0;
}

int bsfp8_adamw_plan(const bsfp8_adamw_tensor* tensors, int32_t num_tensors, int param_dtype, int grad_dtype,
                     int state, void* host_plan, size_t host_plan_bytes) {
  if (tensors == nullptr || host_plan == nullptr) return BSFP8_ERR_NULL_POINTER;
  if (!valid_dtype(param_dtype) || !valid_dtype(grad_dtype) || (state != BSFP8_STATE_F32 && state != BSFP8_STATE_8BIT))
    return BSFP8_ERR_ARGUMENT;
  if (num_tensors <= 0) return BSFP8_ERR_SHAPE;
  const bool q8 = state == BSFP8_STATE_8BIT;
  const int pb = param_dtype == BSFP8_F32 ? 4 : 2, gb = grad_dtype == BSFP8_F32 ? 4 : 2, sb = q8 ? 1 : 4;
  int64_t chunks = 0;
  for (int32_t i = 0; i < num_tensors; ++i) {
    const bsfp8_adamw_tensor& t = tensors[i];
    if (t.numel < 0 || t.numel > (int64_t(1) << 40)) return BSFP8_ERR_SHAPE;
    chunks += bsfp8::adam_chunks_of(t.numel);
    if (chunks > 0x7fffffff) return BSFP8_ERR_SHAPE;
    if (!isfinite(t.lr_scale) || !isfinite(t.decay_scale)) return BSFP8_ERR_ARGUMENT;
    if (t.numel == 0) continue;
    if (t.param == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr ||
        (q8 && (t.exp_avg_scale == nullptr || t.exp_avg_sq_scale == nullptr)))
      return BSFP8_ERR_NULL_POINTER;
    if (!aligned_to(t.param, pb) || !aligned_to(t.grad, gb) || !aligned_to(t.exp_avg, sb) ||
        !aligned_to(t.exp_avg_sq, sb) || !aligned_to(t.copy, 2) ||
        (q8 && (!aligned4(t.exp_avg_scale) || !aligned4(t.exp_avg_sq_scale))))
      return BSFP8_ERR_ALIGNMENT;
  }
  const int64_t table = bsfp8::adam_table_bytes(num_tensors);
  if (host_plan_bytes < (size_t)(table + chunks * (int64_t)sizeof(bsfp8::AdamChunk))) return BSFP8_ERR_SHAPE;
  memset(host_plan, 0, (size_t)table);
  memcpy(host_plan, tensors, (size_t)num_tensors * sizeof(bsfp8_adamw_tensor));
  uint8_t* at = (uint8_t*)host_plan + table;
  for (int32_t i = 0; i < num_tensors; ++i) {
    const int64_t n = bsfp8::adam_chunks_of(tensors[i].numel);
    for (int64_t j = 0; j < n; ++j, at += sizeof(bsfp8::AdamChunk)) {
      const bsfp8::AdamChunk c{i, (int32_t)j};
      memcpy(at, &c, sizeof(c));
    }
  }
  return BSFP8_OK;
}

int bsfp8_adamw_step(const void* device_plan, int32_t num_tensors, int64_t num_chunks, int param_dtype,
                     int grad_dtype, int state, double lr, double beta1, double beta2, double eps,
                     double weight_decay, int64_t step, const float* lr_dev, const int32_t* step_dev,
                     const float* grad_scale, const float* noop_flag, void* stream) {
  return adamw_step(device_plan, num_tensors, num_chunks, param_dtype, grad_dtype, state, lr, beta1, beta2, eps,
                    weight_decay, step, lr_dev, step_dev, grad_scale, noop_flag, nullptr, stream);
}

int bsfp8_adamw_step_stochastic(const void* device_plan, int32_t num_tensors, int64_t num_chunks, int param_dtype,
                                int grad_dtype, int state, double lr, double beta1, double beta2, double eps,
                                double weight_decay, int64_t step, const float* lr_dev, const int32_t* step_dev,
                                const float* grad_scale, const float* noop_flag, uint64_t seed, void* stream) {
  return adamw_step(device_plan, num_tensors, num_chunks, param_dtype, grad_dtype, state, lr, beta1, beta2, eps,
                    weight_decay, step, lr_dev, step_dev, grad_scale, noop_flag, &seed, stream);
}

const char* bsfp8_strerror(int code) {
  switch (code) {
    case BSFP8_OK: return "success";
    case BSFP8_ERR_NULL_POINTER: return "a required pointer is NULL";
    case BSFP8_ERR_NUM_GROUPS: return "num_groups must be in [1, 1024]";
    case BSFP8_ERR_RECIPE: return "unknown recipe";
    case BSFP8_ERR_SHAPE: return "a dimension is negative, not a multiple of 32, or too large";
    case BSFP8_ERR_ALIGNMENT: return "a pointer is not 16-byte aligned";
    case BSFP8_ERR_LAYOUT: return "rowwise layout needs an MX 1x32 E8M0 recipe (MXFP8 or MXFP4)";
    case BSFP8_ERR_ARGUMENT: return "invalid argument";
    case BSFP8_ERR_LAUNCH: return "kernel launch failed";
    default: return "unknown error code";
  }
}

}  // extern "C"
