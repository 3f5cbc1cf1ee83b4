// AdamW over many tensors in one launch (gfx950).  include/bsfp8.h states the formulas.
//
// Bound by HBM: every element's parameter, gradient and states are read once and written once
// (fp32 master weights and states with a bf16 copy: 30 bytes an element; 8-bit states: 18).  The
// plan, laid out once by the caller, holds the tensors' addresses and one entry per chunk of
// kAdamChunk elements, so tensors of one element and of billions share a launch and a workgroup
// finds its work with two loads.
//
// 8-bit states: m and u = sqrt(v) as e4m3, one fp32 scale (largest magnitude times 1/448) per 128
// consecutive elements of a tensor.  u instead of v: v spans the square of the gradients' range,
// u's codes keep 2^17 of it with 4 significant bits each, and u is what the update divides by.  A
// scale in fp32 rather than a power of two: the block's largest state is then always the code 448
// and decays with the scale step by step, where a power-of-two scale would leave the code itself
// to decay, which by less than half a code's step a time it cannot.  The update itself uses m and
// u before they are rounded.
//
// Every operation is rounded to fp32 in the order written.
#include "adamw_plan.hpp"
#include "common.hpp"

namespace bsfp8 {

struct AdamArgs {
  const AdamTensor* tensors;
  const AdamChunk* chunks;
  double lr, decay, log_beta1, log_beta2, step;
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
  const float *lr_dev, *grad_scale, *noop_flag;
  const int32_t* step_dev;
};

__device__ __forceinline__ float val(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float val(float f) { return f; }
__device__ __forceinline__ void put(float f, uint16_t& o) { o = f32_to_bf16(f); }
__device__ __forceinline__ void put(float f, float& o) { o = f; }

// 4 elements at p, n of them live (the rest read as 0); any alignment of the element's size.
template <class T>
__device__ __forceinline__ void load4(const T* p, int n, float* v) {
  T t[4] = {};
  if (n >= 4) {
    __builtin_memcpy(t, p, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) t[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = val(t[i]);
}
template <class T>
__device__ __forceinline__ void store4(T* p, int n, const float* v) {
  T t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) put(v[i], t[i]);
  if (n >= 4) {
    __builtin_memcpy(p, t, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = t[i];
  }
}
// 4 e4m3 codes
__device__ __forceinline__ void load4_codes(const uint8_t* p, int n, float* v) {
  uint32_t w = 0;
  if (n >= 4) {
    __builtin_memcpy(&w, p, 4);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) w |= (uint32_t)p[i] << (8 * i);
  }
  v[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
  v[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
  v[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
  v[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
}
__device__ __forceinline__ void store4_codes(uint8_t* p, int n, const float* v) {
  const uint32_t w = e4m3x4(v[0], v[1], v[2], v[3]);
  if (n >= 4) {
    __builtin_memcpy(p, &w, 4);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = (uint8_t)(w >> (8 * i));
  }
}

// The scale of a block of 128 elements held 4 to a lane by 32 lanes.
__device__ __forceinline__ float block_scale(const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  return fmaxf(m * (1.0f / 448.0f), 1e-30f);
}

template <class PT, class GT, bool Q8>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(AdamArgs a) {
  if (a.noop_flag != nullptr && *a.noop_flag != 0.0f) return;
  const AdamChunk ch = a.chunks[blockIdx.x];
  const AdamTensor& tn = a.tensors[ch.tensor];
  const double lr = (a.lr_dev != nullptr ? (double)*a.lr_dev : a.lr) * (double)tn.lr_scale;
  const double t = a.step_dev != nullptr ? (double)*a.step_dev : a.step;
  const double c1 = 1.0 - exp(t * a.log_beta1), c2 = 1.0 - exp(t * a.log_beta2);
  const float keep = (float)(1.0 - lr * a.decay * (double)tn.decay_scale);
  const float step_size = (float)(lr / c1), root = (float)(1.0 / sqrt(c2));
  const float gs = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
  const int64_t first = (int64_t)ch.index * kAdamChunk;
  PT* __restrict__ const param = (PT*)tn.param;
  const GT* __restrict__ const grad = (const GT*)tn.grad;
  uint16_t* __restrict__ const copy = (uint16_t*)tn.copy;

#pragma unroll
  for (int u = 0; u < kAdamChunk / (4 * kAdamThreads); ++u) {
    const int64_t at = first + 4 * (u * kAdamThreads + (int)threadIdx.x);
    const int64_t left = tn.numel - at;
    const int n = left > 4 ? 4 : (int)left;  // <= 0: nothing of this lane's is live
    float p[4], g[4], m[4], v[4], root_v[4];
    load4(param + at, n, p);
    load4(grad + at, n, g);
    if constexpr (Q8) {
      const int64_t blk = at / 128;
      load4_codes((const uint8_t*)tn.exp_avg + at, n, m);
      load4_codes((const uint8_t*)tn.exp_avg_sq + at, n, v);
      const float sm = n > 0 ? tn.exp_avg_scale[blk] : 0.0f, sv = n > 0 ? tn.exp_avg_sq_scale[blk] : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] *= sm;
        v[i] *= sv;
        v[i] *= v[i];
      }
    } else {
      load4((const float*)tn.exp_avg + at, n, m);
      load4((const float*)tn.exp_avg_sq + at, n, v);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float gi = g[i] * gs;
      m[i] = m[i] * a.beta1 + gi * a.one_minus_beta1;
      v[i] = v[i] * a.beta2 + gi * gi * a.one_minus_beta2;
      root_v[i] = sqrtf(v[i]);
      p[i] = p[i] * keep - m[i] / (root_v[i] * root + a.eps) * step_size;
    }
    store4(param + at, n, p);
    if (copy != nullptr) store4(copy + at, n, p);
    if constexpr (Q8) {
      // lanes past the tensor's end hold zeros, which leave their block's largest as it is
      const float sm = block_scale(m), sv = block_scale(root_v);
      const float im = 1.0f / sm, iv = 1.0f / sv;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] *= im;
        root_v[i] *= iv;
      }
      store4_codes((uint8_t*)tn.exp_avg + at, n, m);
      store4_codes((uint8_t*)tn.exp_avg_sq + at, n, root_v);
      if ((threadIdx.x & 31) == 0 && n > 0) {
        tn.exp_avg_scale[at / 128] = sm;
        tn.exp_avg_sq_scale[at / 128] = sv;
      }
    } else {
      store4((float*)tn.exp_avg + at, n, m);
      store4((float*)tn.exp_avg_sq + at, n, v);
    }
  }
}

int launch_adamw(const void* plan, int32_t num_tensors, int64_t chunks, int p_f32, int g_f32, int q8, double lr,
                 double beta1, double beta2, double eps, double decay, int64_t step, const float* lr_dev,
                 const int32_t* step_dev, const float* grad_scale, const float* noop_flag, hipStream_t stream) {
  AdamArgs a{};
  a.tensors = (const AdamTensor*)plan;
  a.chunks = (const AdamChunk*)((const uint8_t*)plan + adam_table_bytes(num_tensors));
  a.lr = lr;
  a.decay = decay;
  a.log_beta1 = log(beta1);
  a.log_beta2 = log(beta2);
  a.step = (double)step;
  a.beta1 = (float)beta1;
  a.one_minus_beta1 = (float)(1.0 - beta1);
  a.beta2 = (float)beta2;
  a.one_minus_beta2 = (float)(1.0 - beta2);
  a.eps = (float)eps;
  a.lr_dev = lr_dev;
  a.step_dev = step_dev;
  a.grad_scale = grad_scale;
  a.noop_flag = noop_flag;
  const dim3 grid((unsigned)chunks), block(kAdamThreads);
#define BSFP8_ADAM(P, G, Q) hipLaunchKernelGGL((adamw_kernel<P, G, Q>), grid, block, 0, stream, a)
  if (p_f32) {
    if (g_f32) {
      if (q8) BSFP8_ADAM(float, float, true);
      else BSFP8_ADAM(float, float, false);
    } else {
      if (q8) BSFP8_ADAM(float, uint16_t, true);
      else BSFP8_ADAM(float, uint16_t, false);
    }
  } else {
    if (g_f32) {
      if (q8) BSFP8_ADAM(uint16_t, float, true);
      else BSFP8_ADAM(uint16_t, float, false);
    } else {
      if (q8) BSFP8_ADAM(uint16_t, uint16_t, true);
      else BSFP8_ADAM(uint16_t, uint16_t, false);
    }
  }
#undef BSFP8_ADAM
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
