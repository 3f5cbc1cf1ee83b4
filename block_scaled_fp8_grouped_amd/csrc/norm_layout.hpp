// Launch shapes of the residual-norm kernels, shared by the launchers and the workspace query.
#pragma once

#include <stdint.h>

namespace bsfp8 {

constexpr int64_t kNormMaxCols = 32768;  // 1024 threads x 4 chunks x 8 elements

// Threads per row and chunks of 8 elements per thread.
struct NormShape {
  int nt, vpt;
};

inline NormShape norm_shape(int64_t cols) {
  const int64_t c = (cols + 7) / 8;  // chunks of a row
  if (c <= 64) return {64, 1};
  if (c <= 128) return {64, 2};
  if (c <= 256) return {256, 1};
  if (c <= 512) return {256, 2};
  if (c <= 1024) return {1024, 1};
  if (c <= 2048) return {1024, 2};
  return {1024, 4};
}

inline int64_t norm_rows_per_block(int64_t cols) {
  const int nt = norm_shape(cols).nt;
  return nt < 256 ? 256 / nt : 1;
}

// Forward: enough workgroups for every CU to hold 8, each walking every gridDim-th row.
inline int64_t norm_blocks(int64_t rows, int64_t cols) {
  const int64_t rpb = norm_rows_per_block(cols), b = (rows + rpb - 1) / rpb;
  return b < 2048 ? b : 2048;
}

// Gradient: as many workgroups as partial rows.
inline int64_t norm_grad_slots(int64_t rows, int64_t cols) {
  const int64_t rpb = norm_rows_per_block(cols), b = (rows + rpb - 1) / rpb;
  const int64_t most = norm_shape(cols).nt >= 1024 ? 512 : 1024;
  return b < most ? b : most;
}

}  // namespace bsfp8
