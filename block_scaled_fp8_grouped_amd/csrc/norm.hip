// Norms before and after a block, fused with the block's gate and the residual sum, and their
// gradient (gfx950).  include/bsfp8.h states the formulas.
//
// Both passes are bound by HBM: the forward reads x and y and writes r and n, the gradient reads
// dn, dr, r and y and writes dx and dy, each once.  A row is held in registers from its loads to
// its stores (8 elements per thread up to 8192 columns, as many waves as the row needs), so the
// row's two reductions cost no second read.  Workgroups walk every gridDim-th row, so that the
// weights are loaded once and held (post_weight, its offset and a channel's gate as one factor), and
// the next row's loads are in flight while this one is reduced: without that, one barrier after the
// other leaves the memory idle (7168 columns: forward 500 us, gradient 880 us on 32768 rows).
//
// The weights' gradients are sums over all rows.  Each workgroup keeps its columns' sums in
// registers, writes one partial row per sum into the caller's workspace, and a second launch adds the
// partial rows in a fixed order: no atomics, the same bits every time.  The gradients of
// post_weight and of a channel's gate are one sum, S = sum of y_scale d yh, times the other factor.
//
// Rows of any length and any 2- or 4-byte alignment take the same path: a thread's 8 elements are
// moved as one unaligned vector, the last chunk of a row whose length is not a multiple of 8 by
// element.
#include <type_traits>

#include "common.hpp"
#include "norm_layout.hpp"
#include "row_io.hpp"

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
  float *dgate, *partial;  // dgate: per token; partial: [slots][2][C] (the pre_weight sum, the y sum)
  int need;                // sums to keep: 1 the pre_weight sum, 2 the y sum
  bool stream;             // row outputs past the caches
};

// Sums of K values over the threads of a row, the same bits in every thread: a wave (WAVE), or the
// workgroup's up to 16 waves through LDS.  `sm` holds two alternating buffers, so one barrier per reduction is
// enough: a buffer is written again two reductions later, after the barrier of the one between.
template <bool WAVE, int K>
struct RowSum {
  float (*sm)[K][16];
  int turn = 0;
  __device__ __forceinline__ explicit RowSum(float (*buffers)[K][16]) : sm(buffers) {
    if constexpr (!WAVE) {
      if (threadIdx.x < 32 * K) sm[0][0][threadIdx.x] = 0.0f;  // the waves that are not there
      __syncthreads();
    }
  }
  __device__ __forceinline__ void operator()(float (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    if constexpr (WAVE) {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v[k]), 63));
    } else {
      if ((threadIdx.x & 63) == 63)
#pragma unroll
        for (int k = 0; k < K; ++k) sm[turn][k][threadIdx.x >> 6] = v[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v4f s = *(const v4f*)&sm[turn][k][0];
#pragma unroll
        for (int i = 1; i < 4; ++i) s += *(const v4f*)&sm[turn][k][4 * i];
        v[k] = (s[0] + s[1]) + (s[2] + s[3]);
      }
      turn ^= 1;
    }
  }
};

// The hardware's reciprocal square root, within 1 ulp of fp32.  It takes subnormal numbers for zero: small arguments (an
// eps below 2^-100 and a row that is smaller still) are scaled by an even power of two.
__device__ __forceinline__ float rstd_of(float sum, float inv_c, float eps) {
  const float v = sum * inv_c + eps;
  const bool small = v < 0x1p-100f;
  return __builtin_amdgcn_rsqf(small ? v * 0x1p100f : v) * (small ? 0x1p50f : 1.0f);
}

// The factors of 8 columns: pre_weight + offset, and (post_weight + offset) times a channel's gate.
__device__ __forceinline__ void load_factors(const NormArgs& a, int c, int n, float* wq, float* wp) {
#pragma unroll
  for (int e = 0; e < 8; ++e) wq[e] = wp[e] = 1.0f;
  if (a.pre_w != nullptr) {
    load8(a.pre_w + c, n, wq);
#pragma unroll
    for (int e = 0; e < 8; ++e) wq[e] += a.offset;
  }
  if (a.post_w != nullptr) {
    load8(a.post_w + c, n, wp);
#pragma unroll
    for (int e = 0; e < 8; ++e) wp[e] += a.offset;
  }
  if (a.gate_kind == BSFP8_GATE_CHANNEL) {
    float g[8];
    load8(a.gate + c, n, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) wp[e] *= g[e];
  }
}

// WAVE: a row per wave, 4 rows per workgroup of 256; else a row per workgroup.  VPT chunks of 8 elements
// per thread; with one, the factors are held and the next row is fetched ahead.
template <class XT, bool WAVE, int VPT>
__global__ __launch_bounds__(WAVE ? 256 : 1024, VPT == 1 ? 7 : 4) void residual_norm_kernel(NormArgs a) {
  constexpr bool AHEAD = VPT == 1;
  const int NT = WAVE ? 64 : blockDim.x, RPB = WAVE ? 4 : 1;
  __shared__ __attribute__((aligned(16))) float sm[2][1][16];
  RowSum<WAVE, 1> row_sum(sm);
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const float inv_c = 1.0f / (float)a.C;
  const int C = (int)a.C;
  const bool has_y = a.y != nullptr;
  float wq[VPT][8], wp[VPT][8];
  if constexpr (AHEAD) load_factors(a, t * 8, C - t * 8, wq[0], wp[0]);
  Raw8<XT> xr[VPT];
  Raw8<uint16_t> yr[VPT];
  float gate = 1.0f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * NT) * 8;
      xr[i].load((const XT*)a.x + row * a.C + c, C - c);
      if (has_y) yr[i].load(a.y + row * a.C + c, C - c);
    }
    if (a.gate_kind == BSFP8_GATE_TOKEN) gate = a.gate[row];
  };
  const int64_t stride = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + (WAVE ? threadIdx.x >> 6 : 0);
  if (AHEAD && row < a.R) fetch(row);
  for (; row < a.R; row += stride) {
    const int64_t base = row * a.C;
    if constexpr (!AHEAD) fetch(row);
    float x[VPT][8], y[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[i][e] = a.x_scale * xr[i][e];
        if (has_y) y[i][e] = yr[i][e];
      }
    float s = a.y_scale * gate;
    if (AHEAD && row + stride < a.R) fetch(row + stride);
    if (has_y) {
      if (a.post_w != nullptr) {
        float q[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) q[0] = __builtin_fmaf(y[i][e], y[i][e], q[0]);
        row_sum(q);
        const float ry = rstd_of(q[0], inv_c, a.eps);
        if (t == 0 && a.rstd_y != nullptr) a.rstd_y[row] = ry;
        s *= ry;
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if constexpr (!AHEAD) load_factors(a, (t + i * NT) * 8, C - (t + i * NT) * 8, wq[i], wp[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = __builtin_fmaf(s, y[i][e] * wp[i][e], x[i][e]);
      }
    } else if constexpr (!AHEAD) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) load_factors(a, (t + i * NT) * 8, C - (t + i * NT) * 8, wq[i], wp[i]);
    }
    if (a.r != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * NT) * 8;
        store8((XT*)a.r + base + c, C - c, x[i], a.stream);
      }
    }
    if (a.pre_w != nullptr) {
      float q[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) q[0] = __builtin_fmaf(x[i][e], x[i][e], q[0]);
      row_sum(q);
      const float rr = rstd_of(q[0], inv_c, a.eps);
      if (t == 0 && a.rstd_r != nullptr) a.rstd_r[row] = rr;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * NT) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * rr * wq[i][e];
        store8(a.n + base + c, C - c, x[i], a.stream);
      }
    }
  }
}

// ROWS rows at a time: their loads are in flight together and their reductions share a barrier.  With two,
// the last thread of a row whose length is not a multiple of 8 takes the row's last 8 elements instead of a
// part of a chunk (loads by element cost more registers than 16 waves leave); the first `shift` of them are
// its neighbour's: their factors are zero here, which keeps them out of the row's sums, what has come from dr
// is dropped, and they are not stored.
template <class XT, bool WAVE, int VPT, int ROWS>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void residual_norm_grad_kernel(NormArgs a) {
  constexpr bool HOLD = VPT == 1;
  constexpr bool WHOLE = ROWS == 2;
  const int NT = WAVE ? 64 : blockDim.x, RPB = WAVE ? 4 * ROWS : ROWS;
  __shared__ __attribute__((aligned(16))) float sm[2][ROWS][16];
  RowSum<WAVE, ROWS> row_sum(sm);
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const float inv_c = 1.0f / (float)a.C;
  const int C = (int)a.C;
  const bool has_n = a.dn != nullptr, has_y = a.y != nullptr;
  float wq[VPT][8], wp[VPT][8], sum_pre[VPT][8], sum_y[VPT][8];
  const bool mine = t * 8 < C;
  const int shift = WHOLE && mine && t * 8 + 8 > C ? t * 8 + 8 - C : 0;
  if constexpr (HOLD) {
    load_factors(a, t * 8 - shift, C - t * 8 + shift, wq[0], wp[0]);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < shift) wq[0][e] = wp[0][e] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum_pre[i][e] = sum_y[i][e] = 0.0f;
  const int64_t stride = (int64_t)gridDim.x * RPB;
  const int wave_row = WAVE ? __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) * ROWS : 0;
  // elements of this thread's chunk i that exist
  auto count = [&](int i, bool live) { return live ? C - (t + i * NT) * 8 : 0; };
  auto put8 = [&](auto* p, int n, const float* v, bool stream) {
    if constexpr (WHOLE) {
      if (n > 0) {
        if (shift == 0) {
          store8(p, 8, v, stream);
        } else {
#pragma unroll
          for (int e = 1; e < 8; ++e)
            if (e >= shift) from_f32(v[e], p[e]);
        }
      }
    } else {
      store8(p, n, v, stream);
    }
  };
  for (int64_t row = (int64_t)blockIdx.x * RPB + wave_row; row < a.R; row += stride) {
    Raw8<uint16_t> n[ROWS][VPT], y[ROWS][VPT];
    Raw8<XT> r[ROWS][VPT], d0[ROWS][VPT];
    float rr[ROWS], ry[ROWS], gate[ROWS], q[ROWS], d[ROWS][VPT][8];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const bool live = row + j < a.R;  // a row that is not there has no columns: zeros, nothing stored
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const uint32_t c = (t + i * NT) * 8 - shift;
        const int64_t base = (row + j) * a.C;
        const int m = count(i, live);
        if constexpr (WHOLE) {
          n[j][i] = y[j][i] = {};
          r[j][i] = d0[j][i] = {};
          if (m > 0) {
            if (has_n) {
              n[j][i].load_all(a.dn + base + c);
              r[j][i].load_all((const XT*)a.r + base + c);
            }
            if (a.dr != nullptr) d0[j][i].load_all((const XT*)a.dr + base + c);
            if (has_y) y[j][i].load_all(a.y + base + c);
          }
        } else {
          if (has_n) {
            n[j][i].load(a.dn + base + c, m);
            r[j][i].load((const XT*)a.r + base + c, m);
          }
          if (a.dr != nullptr) d0[j][i].load((const XT*)a.dr + base + c, m);
          if (has_y) y[j][i].load(a.y + base + c, m);
        }
      }
      rr[j] = has_n && live ? a.rstd_r[row + j] : 0.0f;
      ry[j] = a.post_w == nullptr ? 1.0f : live ? a.rstd_y[row + j] : 0.0f;
      gate[j] = a.gate_kind != BSFP8_GATE_TOKEN ? 1.0f : live ? a.gate[row + j] : 0.0f;
      q[j] = 0.0f;
    }
    if constexpr (!HOLD) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) load_factors(a, (t + i * NT) * 8, C - (t + i * NT) * 8, wq[i], wp[i]);
    }
    // through the norm before the next block: d = dr + rr (g1 - rh mean(g1 rh))
    if (has_n) {
#pragma unroll
      for (int j = 0; j < ROWS; ++j)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float rh = r[j][i][e] * rr[j], nr = n[j][i][e] * rh;
            sum_pre[i][e] += nr;
            q[j] = __builtin_fmaf(nr, wq[i][e], q[j]);
          }
      __builtin_amdgcn_sched_barrier(0);  // (each phase's temporaries end with it: registers)
      row_sum(q);
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const float m = q[j] * inv_c * rr[j];
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[j][i][e] = a.dr != nullptr ? d0[j][i][e] : 0.0f;
          if (has_n)
            d[j][i][e] = __builtin_fmaf(rr[j], __builtin_fmaf(-r[j][i][e], m, n[j][i][e] * wq[i][e]), d[j][i][e]);
        }
        if constexpr (WHOLE) {
          // the neighbour's elements: where dx is dr it may have written them before they were read here, and a zero
          // factor does not keep an infinity out of the row's sum
          if (shift != 0) {
#pragma unroll
            for (int e = 0; e < 7; ++e)
              if (e < shift) d[j][i][e] = 0.0f;
          }
        }
        if (a.dx != nullptr) {
          const uint32_t c = (t + i * NT) * 8 - shift;
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = a.x_scale * d[j][i][e];
          put8((XT*)a.dx + (row + j) * a.C + c, count(i, row + j < a.R), o, a.stream);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!has_y) continue;
    // through the gate and the norm after the block: with t = y_scale d and u = t (post_weight + offset)
    // (channel gate), g2 = (token gate) u and the token gate's gradient is the sum of u yh
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      q[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float back = a.y_scale * d[j][i][e], by = back * (y[j][i][e] * ry[j]);
          sum_y[i][e] = __builtin_fmaf(gate[j], by, sum_y[i][e]);
          q[j] = __builtin_fmaf(by, wp[i][e], q[j]);
          d[j][i][e] = back * wp[i][e];
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    const bool token = a.gate_kind == BSFP8_GATE_TOKEN && a.dgate != nullptr;
    if (a.post_w != nullptr || token) {
      row_sum(q);
      if (token && t == 0) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
          if (row + j < a.R) a.dgate[row + j] = q[j];
      }
    }
    if (a.dy != nullptr) {
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const float m = a.post_w != nullptr ? q[j] * inv_c * ry[j] : 0.0f, k = ry[j] * gate[j];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const uint32_t c = (t + i * NT) * 8 - shift;
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = k * __builtin_fmaf(-y[j][i][e], m, d[j][i][e]);
          put8(a.dy + (row + j) * a.C + c, count(i, row + j < a.R), o, a.stream);
        }
      }
    }
  }
  if (a.need == 0) return;

  // this workgroup's partial rows; the 4 waves' rows are added in order first
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.C;
  __shared__ float tot[WAVE ? 64 * VPT * 8 : 1];
  auto put = [&](int which, float (&s)[VPT][8]) {
    if constexpr (WAVE) {
      for (int w = 0; w < 4; ++w) {
        if ((int)(threadIdx.x >> 6) == w) {
#pragma unroll
          for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float* p = &tot[(t + i * 64) * 8 - shift + e];
              if (e >= shift) *p = w == 0 ? s[i][e] : *p + s[i][e];
            }
        }
        __syncthreads();
      }
      for (int c = threadIdx.x; c < C; c += 256) out[which * a.C + c] = tot[c];
      __syncthreads();
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * NT) * 8 - shift;
        put8(out + which * a.C + c, C - (t + i * NT) * 8, s[i], false);
      }
    }
  };
  if (a.need & 1) put(0, sum_pre);
  if (a.need & 2) put(1, sum_y);
}

// Sums of the partial rows: 64 columns per workgroup, its 16 waves take every 16th slot, and the 16
// sums are added in order.  The y sum times the channel's gate is dpost_weight, times post_weight + offset
// the channel gate's gradient.
struct NormReduceArgs {
  int64_t C;
  int slots, accumulate;
  const float *partial, *post_w, *gate;  // gate: per channel, or NULL
  float offset;
  float *dpre, *dpost, *dgate;
};

__global__ __launch_bounds__(1024) void residual_norm_reduce_kernel(NormReduceArgs a) {
  __shared__ float sm[16][64];
  const int which = blockIdx.y, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (which == 0 ? a.dpre == nullptr : a.dpost == nullptr && a.dgate == nullptr) return;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < a.C) {
    const float* p = a.partial + which * a.C + c;
#pragma unroll 8
    for (int k = w; k < a.slots; k += 16) s += p[(int64_t)k * 2 * a.C];
  }
  sm[w][lane] = s;
  __syncthreads();
  if (w != 0 || c >= a.C) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += sm[i][lane];
  auto put = [&](float* out, float v) {
    if (out != nullptr) out[c] = a.accumulate ? out[c] + v : v;
  };
  if (which == 0) {
    put(a.dpre, s);
  } else {
    put(a.dpost, a.gate != nullptr ? s * a.gate[c] : s);
    if (a.dgate != nullptr) put(a.dgate, a.post_w != nullptr ? s * (a.post_w[c] + a.offset) : s);
  }
}

// ------------------------------------------------------------------------------------------
// Launchers
// ------------------------------------------------------------------------------------------

template <class XT, bool GRAD, bool WAVE, int VPT>
static int launch_norm(const NormArgs& a, int64_t blocks, int threads, hipStream_t stream) {
  const dim3 grid((unsigned)blocks), block(threads);
  if constexpr (!GRAD)
    hipLaunchKernelGGL((residual_norm_kernel<XT, WAVE, VPT>), grid, block, 0, stream, a);
  else if (VPT == 1 && norm_grad_rows(a.C) == 2)
    hipLaunchKernelGGL((residual_norm_grad_kernel<XT, WAVE, VPT, VPT == 1 ? 2 : 1>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((residual_norm_grad_kernel<XT, WAVE, VPT, 1>), grid, block, 0, stream, a);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

// Row outputs of at least this many elements each go past the caches: two of them would fill the last-level
// cache, and the next pass would not find their beginning there (32768 x 7168: gradient 540 -> 513 us).
constexpr int64_t kNormStreamElements = int64_t(1) << 26;

template <class XT, bool GRAD>
static int dispatch_norm(NormArgs& a, hipStream_t stream) {
  a.stream = a.R * a.C >= kNormStreamElements;
  const NormShape s = norm_shape(a.C);
  const int64_t blocks = GRAD ? norm_grad_slots(a.R, a.C) : norm_blocks(a.R, a.C);
  if (s.wave) return launch_norm<XT, GRAD, true, 1>(a, blocks, s.threads, stream);
  if (s.vpt == 1) return launch_norm<XT, GRAD, false, 1>(a, blocks, s.threads, stream);
  if (s.vpt == 2) return launch_norm<XT, GRAD, false, 2>(a, blocks, s.threads, stream);
  return launch_norm<XT, GRAD, false, 4>(a, blocks, s.threads, stream);
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
  a.need = (dpre_w ? 1 : 0) | (dpost_w || (channel && dgate) ? 2 : 0);
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
  b.post_w = post_w;
  b.gate = channel ? gate : nullptr;
  b.offset = offset;
  b.dpre = dpre_w;
  b.dpost = dpost_w;
  b.dgate = channel ? dgate : nullptr;
  hipLaunchKernelGGL(residual_norm_reduce_kernel, dim3((unsigned)((C + 63) / 64), 2), dim3(1024), 0, stream, b);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
