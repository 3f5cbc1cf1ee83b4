// Norms before and after a block, fused with the block's gate and the residual sum, and their
// gradient (gfx950).  include/bsfp8.h states the formulas.
//
// Both passes are bound by HBM: the forward reads x and y and writes r and n, the gradient reads
// dn, dr, r and y and writes dx and dy, each once.  A row is held in registers from its loads to
// its stores (chunks of 8 elements per thread, NT threads per row), so the row's two reductions
// (mean y^2, then mean r^2; in the gradient mean(g1 rh), then mean(g2 yh)) cost no second read.
//
// The weights' gradients are sums over all rows.  Each workgroup walks every gridDim-th row with
// its columns' sums in registers, writes one partial row per sum into the caller's workspace, and
// a second launch adds the partial rows in a fixed order: no atomics, the same bits every time.
//
// Rows of any length and any 2- or 4-byte alignment take the same path: a thread's 8 elements are
// moved as one unaligned vector, the last chunk of a row whose length is not a multiple of 8 by
// element.
#include "common.hpp"
#include "norm_layout.hpp"

namespace bsfp8 {

struct NormArgs {
  int64_t R, C;
  const void* x;          // residual stream in (forward), [R][C]
  const uint16_t* y;      // block output [R][C] bf16, or NULL
  const float *post_w, *pre_w, *gate;
  int gate_kind;
  float x_scale, y_scale, eps, offset;
  void* r;                // forward: residual stream out; gradient: as saved by the forward
  uint16_t* n;
  float *rstd_y, *rstd_r;
  // gradient
  const uint16_t* dn;
  const void* dr;
  void* dx;
  uint16_t* dy;
  float *dgate, *partial;  // dgate: per token; partial: [slots][3][C] (dpre, dpost, dgate per channel)
  int need;                // sums to keep: 1 dpre, 2 dpost, 4 dgate per channel
};

__device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float to_f32(float f) { return f; }
__device__ __forceinline__ void from_f32(float f, uint16_t& o) { o = f32_to_bf16(f); }
__device__ __forceinline__ void from_f32(float f, float& o) { o = f; }

// 8 elements at p (n of them exist; the others read as 0), any alignment of the element's size.
template <class T>
__device__ __forceinline__ void load8(const T* p, int n, float* v) {
  if (n >= 8) {
    T t[8];
    __builtin_memcpy(t, p, sizeof(t));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
}
template <class T>
__device__ __forceinline__ void store8(T* p, int n, const float* v) {
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) from_f32(v[i], t[i]);
  if (n >= 8) {
    __builtin_memcpy(p, t, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = t[i];
  }
}

// Sum of K values over the NT threads of a row, the same bits in every thread.  `sm` holds two
// alternating buffers, so one barrier per reduction is enough: a buffer is written again two
// reductions later, after the barrier of the one between.
template <int NT, int K>
struct RowSum {
  static constexpr int NW = NT / 64;
  float (*sm)[K][NW > 1 ? NW : 1];
  int turn = 0;
  __device__ __forceinline__ void operator()(float* v) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) v[k] += __shfl_xor(v[k], d, 64);
    if constexpr (NW > 1) {
      const int w = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) sm[turn][k][w] = v[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NW; ++i) s += sm[turn][k][i];
        v[k] = s;
      }
      turn ^= 1;
    }
  }
};

__device__ __forceinline__ float rstd_of(float sum, float inv_c, float eps) {
  return 1.0f / sqrtf(sum * inv_c + eps);
}

template <class XT, int NT, int VPT>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void residual_norm_kernel(NormArgs a) {
  constexpr int RPB = NT < 256 ? 256 / NT : 1;  // rows per workgroup
  __shared__ float sm[2][1][NT / 64];
  RowSum<NT, 1> row_sum{sm};
  const int t = threadIdx.x % NT;
  const float inv_c = 1.0f / (float)a.C;
  const int C = (int)a.C;
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / NT; row < a.R; row += (int64_t)gridDim.x * RPB) {
    const int64_t base = row * a.C;
    float x[VPT][8], y[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * NT) * 8;
      load8((const XT*)a.x + base + c, C - c, x[i]);
      if (a.y != nullptr) load8(a.y + base + c, C - c, y[i]);
    }
    if (a.y != nullptr) {
      float s = a.y_scale;
      if (a.gate_kind == BSFP8_GATE_TOKEN) s *= a.gate[row];
      if (a.post_w != nullptr) {
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) q += y[i][e] * y[i][e];
        row_sum(&q);
        const float ry = rstd_of(q, inv_c, a.eps);
        if (t == 0 && a.rstd_y != nullptr) a.rstd_y[row] = ry;
        s *= ry;
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * NT) * 8;
        float w[8];
        if (a.post_w != nullptr) {
          load8(a.post_w + c, C - c, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][e] *= w[e] + a.offset;
        }
        if (a.gate_kind == BSFP8_GATE_CHANNEL) {
          load8(a.gate + c, C - c, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = a.x_scale * x[i][e] + s * y[i][e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] *= a.x_scale;
    }
    if (a.r != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * NT) * 8;
        store8((XT*)a.r + base + c, C - c, x[i]);
      }
    }
    if (a.pre_w != nullptr) {
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) q += x[i][e] * x[i][e];
      row_sum(&q);
      const float rr = rstd_of(q, inv_c, a.eps);
      if (t == 0 && a.rstd_r != nullptr) a.rstd_r[row] = rr;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * NT) * 8;
        float w[8];
        load8(a.pre_w + c, C - c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * rr * (w[e] + a.offset);
        store8(a.n + base + c, C - c, x[i]);
      }
    }
  }
}

template <class XT, int NT, int VPT>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void residual_norm_grad_kernel(NormArgs a) {
  constexpr int RPB = NT < 256 ? 256 / NT : 1;
  __shared__ float sm1[2][1][NT / 64], sm2[2][2][NT / 64];
  RowSum<NT, 1> row_sum{sm1};
  RowSum<NT, 2> row_sum2{sm2};
  const int t = threadIdx.x % NT;
  const float inv_c = 1.0f / (float)a.C;
  const int C = (int)a.C;
  float sum_pre[VPT][8], sum_post[VPT][8], sum_gate[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum_pre[i][e] = sum_post[i][e] = sum_gate[i][e] = 0.0f;

  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / NT; row < a.R; row += (int64_t)gridDim.x * RPB) {
    const int64_t base = row * a.C;
    float d[VPT][8], y[VPT][8];
    float g[VPT][8], rh[VPT][8];
    float rr = 0.0f, ry = 1.0f;
    if (a.dn != nullptr) rr = a.rstd_r[row];
    if (a.y != nullptr && a.post_w != nullptr) ry = a.rstd_y[row];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * NT) * 8;
      if (a.dn != nullptr) {
        load8(a.dn + base + c, C - c, g[i]);
        load8((const XT*)a.r + base + c, C - c, rh[i]);
      }
      if (a.dr != nullptr) {
        load8((const XT*)a.dr + base + c, C - c, d[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[i][e] = 0.0f;
      }
      if (a.y != nullptr) load8(a.y + base + c, C - c, y[i]);
    }
    // through the norm before the next block: d = dr + rr (g1 - rh mean(g1 rh))
    if (a.dn != nullptr) {
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * NT) * 8;
        float w[8];
        load8(a.pre_w + c, C - c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          rh[i][e] *= rr;
          sum_pre[i][e] += g[i][e] * rh[i][e];
          g[i][e] *= w[e] + a.offset;
          q += g[i][e] * rh[i][e];
        }
      }
      row_sum(&q);
      q *= inv_c;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[i][e] += rr * (g[i][e] - rh[i][e] * q);
    }
    if (a.dx != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * NT) * 8;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = a.x_scale * d[i][e];
        store8((XT*)a.dx + base + c, C - c, o);
      }
    }
    if (a.y == nullptr) continue;
    // through the gate and the norm after the block
    const float gt = a.gate_kind == BSFP8_GATE_TOKEN ? a.gate[row] : 1.0f;
    float q[2] = {0.0f, 0.0f};  // sum g2 yh, sum t z
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * NT) * 8;
      float w[8], gc[8];
      if (a.post_w != nullptr) {
        load8(a.post_w + c, C - c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] += a.offset;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
      }
      if (a.gate_kind == BSFP8_GATE_CHANNEL) {
        load8(a.gate + c, C - c, gc);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) gc[e] = gt;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float yh = y[i][e] * ry;
        const float back = a.y_scale * d[i][e];
        const float dz = gc[e] * back;
        const float bz = back * yh * w[e];
        sum_gate[i][e] += bz;
        sum_post[i][e] += dz * yh;
        q[1] += bz;
        y[i][e] = yh;
        d[i][e] = dz * w[e];  // g2
        q[0] += d[i][e] * yh;
      }
    }
    if (a.post_w != nullptr || (a.gate_kind == BSFP8_GATE_TOKEN && a.dgate != nullptr)) {
      row_sum2(q);
      if (a.gate_kind == BSFP8_GATE_TOKEN && a.dgate != nullptr && t == 0) a.dgate[row] = q[1];
    }
    if (a.dy != nullptr) {
      const float c2 = a.post_w != nullptr ? q[0] * inv_c : 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * NT) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) d[i][e] = ry * (d[i][e] - y[i][e] * c2);
        store8(a.dy + base + c, C - c, d[i]);
      }
    }
  }
  if (a.need == 0) return;

  // this workgroup's partial rows; the RPB row lanes of a narrow row are added in order first
  float* out = a.partial + (int64_t)blockIdx.x * 3 * a.C;
  __shared__ float tot[RPB > 1 ? NT * VPT * 8 : 1];
  auto put = [&](int which, float (&s)[VPT][8]) {
    if constexpr (RPB > 1) {
      for (int w = 0; w < RPB; ++w) {
        if ((int)(threadIdx.x / NT) == w) {
#pragma unroll
          for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float* p = &tot[(t + i * NT) * 8 + e];
              *p = w == 0 ? s[i][e] : *p + s[i][e];
            }
        }
        __syncthreads();
      }
      for (int c = threadIdx.x; c < C; c += 256) out[which * a.C + c] = tot[c];
      __syncthreads();
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * NT) * 8;
        store8(out + which * a.C + c, C - c, s[i]);
      }
    }
  };
  if (a.need & 1) put(0, sum_pre);
  if (a.need & 2) put(1, sum_post);
  if (a.need & 4) put(2, sum_gate);
}

// Sums of the partial rows: 64 columns per workgroup, its 4 waves take every fourth slot, and the
// four sums are added in order.
struct NormReduceArgs {
  int64_t C;
  int slots, accumulate;
  const float* partial;
  float* out[3];
};

__global__ __launch_bounds__(256) void residual_norm_reduce_kernel(NormReduceArgs a) {
  __shared__ float sm[4][64];
  const int which = blockIdx.y, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  float* out = a.out[which];
  if (out == nullptr) return;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < a.C) {
    const float* p = a.partial + which * a.C + c;
#pragma unroll 8
    for (int k = w; k < a.slots; k += 4) s += p[(int64_t)k * 3 * a.C];
  }
  sm[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < a.C) {
    const float v = ((sm[0][lane] + sm[1][lane]) + sm[2][lane]) + sm[3][lane];
    out[c] = a.accumulate ? out[c] + v : v;
  }
}

// ------------------------------------------------------------------------------------------
// Launchers
// ------------------------------------------------------------------------------------------

template <class XT, bool GRAD, int NT, int VPT>
static int launch_norm(const NormArgs& a, int64_t blocks, hipStream_t stream) {
  constexpr int threads = NT < 256 ? 256 : NT;
  if constexpr (GRAD)
    hipLaunchKernelGGL((residual_norm_grad_kernel<XT, NT, VPT>), dim3((unsigned)blocks), dim3(threads), 0, stream, a);
  else
    hipLaunchKernelGGL((residual_norm_kernel<XT, NT, VPT>), dim3((unsigned)blocks), dim3(threads), 0, stream, a);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

template <class XT, bool GRAD>
static int dispatch_norm(const NormArgs& a, hipStream_t stream) {
  const NormShape s = norm_shape(a.C);
  const int64_t blocks = GRAD ? norm_grad_slots(a.R, a.C) : norm_blocks(a.R, a.C);
#define BSFP8_NORM(NT_, VPT_) \
  if (s.nt == NT_ && s.vpt == VPT_) return launch_norm<XT, GRAD, NT_, VPT_>(a, blocks, stream)
  BSFP8_NORM(64, 1);
  BSFP8_NORM(64, 2);
  BSFP8_NORM(256, 1);
  BSFP8_NORM(256, 2);
  BSFP8_NORM(1024, 1);
  BSFP8_NORM(1024, 2);
  BSFP8_NORM(1024, 4);
#undef BSFP8_NORM
  return BSFP8_ERR_SHAPE;
}

int launch_residual_norm(int64_t R, int64_t C, const void* x, int x_f32, const void* y, const float* post_w,
                         const float* pre_w, const float* gate, int gate_kind, float x_scale, float y_scale, float eps,
                         float offset, void* r, void* n, float* rstd_y, float* rstd_r, hipStream_t stream) {
  NormArgs a{};
  a.R = R;
  a.C = C;
  a.x = x;
  a.y = (const uint16_t*)y;
  a.post_w = post_w;
  a.pre_w = pre_w;
  a.gate = gate;
  a.gate_kind = gate_kind;
  a.x_scale = x_scale;
  a.y_scale = y_scale;
  a.eps = eps;
  a.offset = offset;
  a.r = r;
  a.n = (uint16_t*)n;
  a.rstd_y = rstd_y;
  a.rstd_r = rstd_r;
  return x_f32 ? dispatch_norm<float, false>(a, stream) : dispatch_norm<uint16_t, false>(a, stream);
}

int launch_residual_norm_grad(int64_t R, int64_t C, int x_f32, const void* dn, const void* dr, const void* r,
                              const float* rstd_r, const float* pre_w, const void* y, const float* rstd_y,
                              const float* post_w, const float* gate, int gate_kind, float x_scale, float y_scale,
                              float offset, void* dx, void* dy, float* dpre_w, float* dpost_w, float* dgate,
                              int accumulate, float* workspace, hipStream_t stream) {
  NormArgs a{};
  a.R = R;
  a.C = C;
  a.y = (const uint16_t*)y;
  a.post_w = post_w;
  a.pre_w = pre_w;
  a.gate = gate;
  a.gate_kind = gate_kind;
  a.x_scale = x_scale;
  a.y_scale = y_scale;
  a.offset = offset;
  a.r = const_cast<void*>(r);
  a.rstd_y = const_cast<float*>(rstd_y);
  a.rstd_r = const_cast<float*>(rstd_r);
  a.dn = (const uint16_t*)dn;
  a.dr = dr;
  a.dx = dx;
  a.dy = (uint16_t*)dy;
  const bool channel = gate_kind == BSFP8_GATE_CHANNEL;
  a.dgate = channel ? nullptr : dgate;
  a.partial = workspace;
  a.need = (dpre_w ? 1 : 0) | (dpost_w ? 2 : 0) | (channel && dgate ? 4 : 0);
  if (R > 0) {
    const int rc = x_f32 ? dispatch_norm<float, true>(a, stream) : dispatch_norm<uint16_t, true>(a, stream);
    if (rc != BSFP8_OK) return rc;
  }
  if (a.need == 0) return BSFP8_OK;
  NormReduceArgs b{};
  b.C = C;
  b.slots = (int)norm_grad_slots(R, C);
  b.accumulate = accumulate;
  b.partial = workspace;
  b.out[0] = dpre_w;
  b.out[1] = dpost_w;
  b.out[2] = channel ? dgate : nullptr;
  hipLaunchKernelGGL(residual_norm_reduce_kernel, dim3((unsigned)((C + 63) / 64), 3), dim3(256), 0, stream, b);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
