// Arithmetic and quantization of the gated projections' epilogues (glu_gemm.hip).
#pragma once

#include "common.hpp"
#include "group_layout.hpp"

namespace bsfp8 {

typedef short v8s __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float to_f32(short b) { return __uint_as_float((uint32_t)(uint16_t)b << 16); }

// Sigmoid in fp32 from the hardware's 2^x and reciprocal, each within 1 ulp.  The argument of 2^x is rounded, which for
// a < 0 is an error of up to 1.22 |a| units of 2^-24 beside the 5 of the rest: as much as an a off by 1 ulp, where a's own sum
// is off by more.  Below the rounding of bf16 and e4m3 outputs (8 |a| 2^-24 < 2^-9 up to the largest |a| with a sigmoid above 0);
// fp32 outputs of y and dprobs carry it.  2^x beyond fp32's range is inf or 0, which gives the limits 0 and 1; a sigmoid
// below 2^-126 (a < -87.3) may be 0.
__device__ __forceinline__ float sigmoid_fast(float a) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(a * -1.44269504f));
}

// y = p silu(a) b
__device__ __forceinline__ float swiglu(float a, float b, float p) { return a * sigmoid_fast(a) * b * p; }

// From d, the gradient at the product's output before the activation's probability: the gradients
// of p silu(a) b at a and b, and silu(a) b d, this column's part of the probability's.
// silu'(a) = sg (1 + a (1 - sg)) = sg + (s - s sg) with s = a sg.
__device__ __forceinline__ void swiglu_grad(float a, float b, float p, float d, float& da, float& db, float& dp) {
  const float sg = sigmoid_fast(a), sl = a * sg, slope = sg + __builtin_fmaf(-sl, sg, sl);
  const float z = d * sl;
  db = z * p;
  dp = __builtin_fmaf(z, b, dp);
  da = d * p * b * slope;
}

// max(m, |a|, |b|) in one instruction.  NaN operands are passed over: a NaN leaves the scale of its block to the other values
// (the quantize kernels, whose maximum is one of bit patterns, take the scale of an infinity for it).
__device__ __forceinline__ float max3_abs(float m, float a, float b) {
  asm("v_max3_f32 %0, %0, |%1|, |%2|" : "+v"(m) : "v"(a), "v"(b));
  return m;
}

// E8M0 byte of a block with largest magnitude amax: e8m0_exponent(amax) + 127.  Adding 0x1fffff carries into the
// exponent field exactly where the mantissa is above 1.75's, and subnormals end at 0.
__device__ __forceinline__ uint32_t e8m0_byte(float amax) {
  const uint32_t f = (__float_as_uint(amax) + 0x1fffffu) >> 23;
  return f > 8u ? f - 8u : 0u;
}
// Four fp32 -> four e4m3 codes of v / 2^(byte - 127): the conversion divides by its scale operand, of which it uses
// the exponent field alone (0 stands for 2^-127), and rounds as the multiplication by 2^-e and the plain conversion do.  Infinities
// and NaN become NaN codes.
__device__ __forceinline__ uint32_t e4m3x4_scaled(float a, float b, float c, float d, float scale) {
  typedef short v2s __attribute__((ext_vector_type(2)));
  v2s w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true);
  return __builtin_bit_cast(uint32_t, w);
}

// Where a gated projection's outputs go; any of them may be NULL.  [R][N] outputs, N columns.
struct GluOut {
  void* y;  // bf16 or fp32 [R][N]
  int y_f32;
  uint8_t *row_q, *row_s, *col_q, *col_s;
};

// The same at a tile's first row and a first column: uniform bases, so that a lane's place is a 32-bit offset.
struct GluTileOut {
  void* y;
  int y_f32;
  uint8_t *row_q, *row_s, *col_q, *col_s;
  uint32_t N;
  int64_t R, kp;
};
__device__ __forceinline__ GluTileOut glu_tile_out(const GluOut& o, int64_t R, int64_t N, const GroupInfo& g, int64_t row0,
                                                   int64_t col) {
  const int64_t row = g.off + row0, at = row * N + col;
  return {o.y == nullptr ? nullptr : (uint8_t*)o.y + at * (o.y_f32 ? 4 : 2),
          o.y_f32,
          o.row_q == nullptr ? nullptr : o.row_q + at,
          o.row_q == nullptr ? nullptr : o.row_s + col / 32 * R + row,
          o.col_q == nullptr ? nullptr : o.col_q + col_elem(N, g.p, g.kp, col, row0),
          o.col_q == nullptr ? nullptr : o.col_s + col_e8m0(N, g.p, row0 / 32, col),
          (uint32_t)N,
          R,
          g.kp};
}

// 8 consecutive columns of a row (r, c from the tile's own): kept in the row-major output and quantized along the
// row, the 4 lanes of a block of 32 columns side by side.  `live` says whether this lane's row and columns
// exist.
__device__ __forceinline__ void put_row8(const GluTileOut& o, int r, int c, bool live, const float* v) {
  const uint32_t at = (uint32_t)r * o.N + (uint32_t)c;
  if (o.y != nullptr && live) {
    if (o.y_f32) {
      float* p = (float*)o.y + at;
      *(v4f*)p = v4f{v[0], v[1], v[2], v[3]};
      *(v4f*)(p + 4) = v4f{v[4], v[5], v[6], v[7]};
    } else {
      v8s w;
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = (short)f32_to_bf16(v[k]);
      *(v8s*)((uint16_t*)o.y + at) = w;
    }
  }
  if (o.row_q != nullptr) {
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k += 2) m = max3_abs(m, v[k], v[k + 1]);
    m = fmaxf(m, __shfl_xor(m, 1, 64));
    m = fmaxf(m, __shfl_xor(m, 2, 64));
    const uint32_t byte = e8m0_byte(m);
    const float s = __uint_as_float(byte << 23);
    if (live) {
      v2i q;
      q[0] = (int)e4m3x4_scaled(v[0], v[1], v[2], v[3], s);
      q[1] = (int)e4m3x4_scaled(v[4], v[5], v[6], v[7], s);
      *(v2i*)(o.row_q + at) = q;
      if ((c & 31) == 0) o.row_s[(c >> 5) * o.R + r] = (uint8_t)byte;
    }
  }
}

// 32 consecutive tokens of one channel (t, a multiple of 32, and c from the tile's own; inside the group's padded
// rows), all in this lane.
__device__ __forceinline__ void put_col32(const GluTileOut& o, int t, int c, bool live, const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; k += 2) m = max3_abs(m, v[k], v[k + 1]);
  const uint32_t byte = e8m0_byte(m);
  const float s = __uint_as_float(byte << 23);
  v4i q[2];
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k >> 2][k & 3] = (int)e4m3x4_scaled(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3], s);
  if (live) {
    uint8_t* dst = o.col_q + (c * o.kp + t);
    *(v4i*)dst = q[0];
    *(v4i*)(dst + 16) = q[1];
    o.col_s[(uint32_t)(t >> 5) * o.N + (uint32_t)c] = (uint8_t)byte;
  }
}

}  // namespace bsfp8
