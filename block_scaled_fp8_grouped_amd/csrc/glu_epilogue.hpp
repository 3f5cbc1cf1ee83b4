// Arithmetic and quantization of the gated projections' epilogues (glu_gemm.hip).
#pragma once

#include "common.hpp"
#include "group_layout.hpp"

namespace bsfp8 {

typedef short v8s __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float to_f32(short b) { return __uint_as_float((uint32_t)(uint16_t)b << 16); }

// Sigmoid in fp32 from the hardware's 2^x and reciprocal (each within 1 ulp; the result within 4,
// below the rounding of every form the outputs are kept in): 2^x beyond fp32's range is inf or 0,
// which gives the limits 0 and 1.
__device__ __forceinline__ float sigmoid_fast(float a) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(a * -1.44269504f));
}

// y = p silu(a) b
__device__ __forceinline__ float swiglu(float a, float b, float p) { return a * sigmoid_fast(a) * b * p; }

// From d, the gradient at the product's output before the activation's probability: the gradients
// of p silu(a) b at a and b, and silu(a) b d, this column's part of the probability's.
__device__ __forceinline__ void swiglu_grad(float a, float b, float p, float d, float& da, float& db, float& dp) {
  const float sg = sigmoid_fast(a), sl = a * sg, q = d * p;
  db = q * sl;
  da = q * b * (sg * (1.0f + a * (1.0f - sg)));
  dp += d * sl * b;
}

// Orders a wave's LDS writes before its own later LDS reads (no other wave is involved).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Where a gated projection's outputs go; any of them may be NULL.  [R][N] outputs, N columns.
struct GluOut {
  void* y;  // bf16 or fp32 [R][N]
  int y_f32;
  uint8_t *row_q, *row_s, *col_q, *col_s;
};

// 8 consecutive columns of a row: kept in the row-major output and quantized along the row, the 4
// lanes of a block of 32 columns side by side.  `live` says whether this lane's row and columns exist.
__device__ __forceinline__ void put_row8(const GluOut& o, int64_t R, int64_t N, int64_t row, int64_t col, bool live,
                                         const float* v) {
  if (o.y != nullptr && live) {
    if (o.y_f32) {
      float* p = (float*)o.y + row * N + col;
      *(v4f*)p = v4f{v[0], v[1], v[2], v[3]};
      *(v4f*)(p + 4) = v4f{v[4], v[5], v[6], v[7]};
    } else {
      v8s w;
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = (short)f32_to_bf16(v[k]);
      *(v8s*)((uint16_t*)o.y + row * N + col) = w;
    }
  }
  if (o.row_q != nullptr) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
    const int e = e8m0_exponent(__uint_as_float(m));
    const float s = exp2_neg(e);
    if (live) {
      v2i q;
      q[0] = (int)e4m3x4(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
      q[1] = (int)e4m3x4(v[4] * s, v[5] * s, v[6] * s, v[7] * s);
      *(v2i*)(o.row_q + row * N + col) = q;
      if ((col & 31) == 0) o.row_s[col / 32 * R + row] = (uint8_t)(e + 127);
    }
  }
}

// 32 consecutive tokens (from t, a multiple of 32, inside the group's padded rows) of one channel,
// all in this lane.
__device__ __forceinline__ void put_col32(const GluOut& o, int64_t N, const GroupInfo& g, int64_t t, int64_t col,
                                          bool live, const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 32; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
  const int e = e8m0_exponent(__uint_as_float(m));
  const float s = exp2_neg(e);
  v4i q[2];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    q[k >> 2][k & 3] = (int)e4m3x4(v[4 * k] * s, v[4 * k + 1] * s, v[4 * k + 2] * s, v[4 * k + 3] * s);
  if (live) {
    uint8_t* dst = o.col_q + col_elem(N, g.p, g.kp, col, t);
    *(v4i*)dst = q[0];
    *(v4i*)(dst + 16) = q[1];
    o.col_s[col_e8m0(N, g.p, t / 32, col)] = (uint8_t)(e + 127);
  }
}

}  // namespace bsfp8
