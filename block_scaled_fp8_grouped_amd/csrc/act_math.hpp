// The activations between an expert's two projections, in fp32 with every rounding stated (include/bsfp8.h), shared
// by the kernels that quantize them.
#pragma once

#include "common.hpp"

namespace bsfp8 {

// 2^x in fp32 by a stated algorithm every IEEE fp32 machine reproduces bit for bit: x clamped to
// [-126, 126]; k = floor(x + 1/2), r = x - k (exact); the degree-7 Taylor polynomial of
// exp(r ln 2) (coefficients (ln 2)^n / n! in fp32, Horner order, no fused multiply-add) times 2^k.
__device__ __forceinline__ float exp2_clamped(float x) {
  const float kf = floorf(x + 0.5f);  // an integer in [-126, 126]: exact as fp32 and as int
  const int k = (int)kf;
  const float r = x - kf;
  float poly = 1.52527338e-05f;
  poly = poly * r + 0.000154035304f;
  poly = poly * r + 0.00133335581f;
  poly = poly * r + 0.00961812911f;
  poly = poly * r + 0.0555041087f;
  poly = poly * r + 0.240226507f;
  poly = poly * r + 0.693147182f;
  poly = poly * r + 1.0f;
  return ldexpf(poly, k);
}
__device__ __forceinline__ float exp2_stated(float x) {
  return exp2_clamped(x > 126.0f ? 126.0f : (x < -126.0f ? -126.0f : x));
}

// The activations between fc1 and fc2 (TE #3484: fc1 -> ScaledSReLU / ScaledSwiGLU -> fc2 with
// per-token probs), in fp32, each operation rounded in the order written:
//   ACT 1: r = max(h, 0) (+0 for h <= 0);  y = (r * r) * p
//   ACT 2: its gradient                     g = ((2 * r) * p) * dy
//   ACT 3: sg = 1 / (1 + 2^(-a log2 e)), s = a * sg;  y = (s * b) * p
// (the division correctly rounded: recip_rn equals it on the [1, 2^126] that 1 + 2^x spans here)
template <int ACT>
__device__ __forceinline__ float act_value(float h, float b, float p, float d) {
  if constexpr (ACT <= 2) {
    const float r = h > 0.0f ? h : 0.0f;
    if constexpr (ACT == 1) {
      const float r2 = r * r;
      return r2 * p;
    } else {
      const float tp = (2.0f * r) * p;
      return tp * d;
    }
  } else {
    const float t = exp2_stated(-h * 1.44269502f);
    const float den = 1.0f + t;  // in [1, 2^126]: t <= 2^126 after the clamp
    const float sg = recip_rn(den);
    const float sl = h * sg;
    const float sb = sl * b;
    return sb * p;
  }
}

//   ACT 4: the gradient of ACT 3, q = dy * p:  da = (q * b) * (sg * (1 + a * (1 - sg))),  db = q * s
// (sg and s shared by the two outputs of one element)
__device__ __forceinline__ void glu_grad(float a, float b, float p, float d, float& da, float& db) {
  const float t = exp2_stated(-a * 1.44269502f);
  const float den = 1.0f + t;  // in [1, 2^126]
  const float sg = recip_rn(den);
  const float sl = a * sg;
  const float q = d * p;
  db = q * sl;
  const float u = 1.0f - sg;
  const float v = a * u;
  const float w = 1.0f + v;
  const float ds = sg * w;
  const float qb = q * b;
  da = qb * ds;
}

}  // namespace bsfp8
