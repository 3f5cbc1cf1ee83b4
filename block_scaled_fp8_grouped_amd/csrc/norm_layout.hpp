// Launch shapes of the residual-norm kernels, shared by the launchers and the workspace query.
#pragma once

#include <stdint.h>

namespace bsfp8 {

constexpr int64_t kNormMaxCols = 32768;  // 1024 threads x 4 chunks x 8 elements
constexpr int64_t kNormCus = 256;

// Up to 512 columns a row is one wave's, 4 rows to a workgroup; above, a workgroup's of as many waves as
// the row needs at `vpt` chunks of 8 elements per thread.
struct NormShape {
  bool wave;
  int vpt, threads;
};

inline NormShape norm_shape(int64_t cols) {
  if (cols <= 512) return {true, 1, 256};
  const int vpt = cols <= 8192 ? 1 : cols <= 16384 ? 2 : 4;
  return {false, vpt, 64 * (int)((cols + 512 * vpt - 1) / (512 * vpt))};
}

// Workgroups: as many as fill the chip with `waves` waves per CU, each walking every gridDim-th set of
// `rows_at_once` rows (per wave or per workgroup).
inline int64_t norm_fill(int64_t rows, int64_t cols, int64_t waves, int rows_at_once) {
  const NormShape s = norm_shape(cols);
  const int64_t rpb = (s.wave ? 4 : 1) * rows_at_once, need = (rows + rpb - 1) / rpb, per = waves / (s.threads / 64);
  const int64_t most = kNormCus * (per < 1 ? 1 : per);
  return need < most ? need : most;
}

// Forward: four times what the chip holds at once (28 waves per CU), so that no CU is left with one more row
// than the others for long (32768 x 7168: 352 us, once 366, a row per workgroup 419).
inline int64_t norm_blocks(int64_t rows, int64_t cols) { return norm_fill(rows, cols, 4 * 28, 1); }

// Rows that the gradient takes at once, and its workgroups, as many as partial rows.
inline int norm_grad_rows(int64_t cols) { return cols >= 8 && cols <= 8192 ? 2 : 1; }
inline int64_t norm_grad_slots(int64_t rows, int64_t cols) { return norm_fill(rows, cols, 16, norm_grad_rows(cols)); }

}  // namespace bsfp8
