// Rows quantized on their way into the grouped layouts (gfx950): tokens' rows gathered for their experts, and the
// activation between two projections with its input kept in 8 bits, and its gradient from what was kept.
// include/bsfp8.h states the formulas, group_layout.hpp the layouts.
//
// A workgroup of 4 waves walks sub-tiles of 64 rows of one column range, two for each 128 rows of a group's padded extent.
// A thread holds 8 consecutive channels of a row: 4 neighbouring lanes have a block of 32, so the rowwise scale takes
// two moves within a quad and the rowwise codes are stored from the registers the values were computed in; only the
// colwise layout goes through LDS, as fp32, where a thread takes 32 rows of one channel.  The next sub-tile's loads are in
// flight while this one is computed.  The scales of a sub-tile are staged in LDS and stored 64 rows at a time.
#include <type_traits>

#include "act_math.hpp"
#include "common.hpp"
#include "group_layout.hpp"
#include "token_layout.hpp"

namespace bsfp8 {

constexpr int kTThreads = 256;
constexpr int kTRows = 64;

// What a launch does: the rows of tokens, or an activation's forward or gradient.
constexpr int kModeRows = 0, kModeSrelu = 1, kModeSrelu_grad = 2, kModeSwiglu = 3, kModeSwiglu_grad = 4;
constexpr bool mode_grad(int m) { return m == kModeSrelu_grad || m == kModeSwiglu_grad; }
constexpr bool mode_glu(int m) { return m >= kModeSwiglu; }
// input columns of a tile, values quantized rowwise (outputs, then inputs kept), arrays for the colwise layout
constexpr int mode_width(int m) { return mode_grad(m) ? 64 : 128; }
constexpr int mode_outs(int m) { return m == kModeSwiglu_grad ? 2 : 1; }
constexpr int mode_kept(int m) { return m == kModeSrelu ? 1 : m == kModeSwiglu ? 2 : 0; }
constexpr int mode_cols(int m) { return m == kModeSwiglu_grad ? 3 : m == kModeSrelu_grad ? 2 : 1; }

struct TokenQuantArgs {
  const uint16_t* in;      // rows of tokens, or h (forward), or dy (gradient)
  const uint8_t *kq, *ks;  // gradient: what the forward kept
  int64_t R, F;            // capacity rows; width of one half (the columns of x, of the activation, of dy)
  const float* probs;      // of each row; rows of tokens: of each choice
  const int32_t* choices;  // rows of tokens
  int64_t tokens;
  int K;
  const int32_t* splits;
  int E;
  uint8_t *row_q, *row_s, *col_q, *col_s;
  uint8_t *kept_q, *kept_s;    // forward
  uint8_t *ycol_q, *ycol_s;    // gradient
  float* partial;              // gradient: [column tiles][R] parts of dprobs, or NULL
  uint32_t* status;
  int run;  // 128-row tiles per workgroup
};

// Maximum over the 4 lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, false));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, false));
}

// A block's biased exponent from its largest magnitude's bits, and the quantized 8 values of a lane.
template <bool F4>
__device__ __forceinline__ int block_exponent(uint32_t m) {
  return F4 ? e8m0_exponent_fp4(__uint_as_float(m)) : e8m0_exponent(__uint_as_float(m));
}
__device__ __forceinline__ uint32_t largest8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}
template <bool F4>
__device__ __forceinline__ v2i codes8(const float (&v)[8], float s) {
  v2i q = {0, 0};
  if constexpr (F4) {
    q[0] = (int)e2m1x8(v[0] * s, v[1] * s, v[2] * s, v[3] * s, v[4] * s, v[5] * s, v[6] * s, v[7] * s);
  } else {
    q[0] = (int)e4m3x4(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
    q[1] = (int)e4m3x4(v[4] * s, v[5] * s, v[6] * s, v[7] * s);
  }
  return q;
}

__device__ __forceinline__ void unpack8(const v4i& w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo((uint32_t)w[i]);
    v[2 * i + 1] = bf16_hi((uint32_t)w[i]);
  }
}
// 8 e4m3 codes times their block's power of two (byte b: 2^(b - 127); 0 stands for 2^-127, a subnormal number).
__device__ __forceinline__ void unpack_codes(const v2i& w, uint32_t byte, float (&v)[8]) {
  const float two = __uint_as_float(byte == 0 ? 0x400000u : byte << 23);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __builtin_amdgcn_cvt_f32_fp8(w[i], 0) * two;
    v[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(w[i], 1) * two;
    v[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(w[i], 2) * two;
    v[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(w[i], 3) * two;
  }
}

// The sigmoid from the hardware's 2^x and reciprocal (each within an ulp): the gradient of 8-bit values needs no more.
__device__ __forceinline__ float sigmoid_fast(float a) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-a * 1.44269502f));
}

template <int MODE, bool F4>
__global__ __launch_bounds__(kTThreads) void token_quant_kernel(TokenQuantArgs a) {
  constexpr bool GRAD = mode_grad(MODE), GLU = mode_glu(MODE), ROWS = MODE == kModeRows;
  constexpr int W = mode_width(MODE), LPR = W / 8, RPP = kTThreads / LPR, PASSES = kTRows / RPP;
  constexpr int OUTS = mode_outs(MODE), KEPT = mode_kept(MODE), COLS = mode_cols(MODE);
  __shared__ GroupScanSmem<kTThreads> gsm;
  __shared__ __attribute__((aligned(16))) float tile[COLS][kTRows][W];
  __shared__ uint8_t scales[OUTS + KEPT][W / 32][kTRows];

  const int tid = threadIdx.x, ch = tid % LPR, r_of = tid / LPR;
  const int64_t ctiles = (a.F + W - 1) / W;
  const int64_t rt0 = (int64_t)blockIdx.x / ctiles * a.run, c0 = (int64_t)blockIdx.x % ctiles * W;
  const int ncols = (int)(a.F - c0 < W ? a.F - c0 : W);  // a multiple of 32
  const bool live_col = ch * 8 < ncols, row_out = a.row_q != nullptr, col_out = a.col_q != nullptr;
  const int64_t C = a.F * OUTS;  // columns of the output

  // rows of tokens without the colwise layout need no groups: their rows are the ones that have a choice
  GroupInfo g{};
  const bool grouped = !ROWS || col_out;
  if (grouped) {
    const uint32_t flags = group_scan<kTThreads>(a.splits, a.E, a.R, 128, rt0, 0, gsm, g);
    report_status(a.status, flags);
    if (g.e < 0) return;
  }
  struct Sub {
    int64_t row0, p, kp, block;  // first row; the group's packed offset and extent; first 32-row block of the sub-tile
    int live;                    // live rows
  };
  // the sub-tile `half` (0, 1) of 128-row tile rt
  auto place = [&](int64_t rt, int half, Sub& s) -> bool {
    if (!grouped) {
      s.row0 = rt * 128 + half * kTRows;
      s.p = s.kp = s.block = 0;
      const int64_t left = a.R - s.row0;
      s.live = (int)(left < 0 ? 0 : left < kTRows ? left : kTRows);
      return rt * 128 < a.R;
    }
    while (rt >= g.tile + g.kp / 128) {  // past this group (or it is empty)
      g.tile += g.kp / 128;
      g.off += g.k;
      g.p += g.kp;
      if (++g.e >= a.E) return false;
      g.k = a.splits[g.e];  // validated by the scan: 0 <= k, sum <= capacity
      g.kp = col_padded_rows(g.k);
    }
    const int64_t in_group = 128 * (rt - g.tile) + half * kTRows, left = g.k - in_group;
    s.row0 = g.off + in_group;
    s.p = g.p;
    s.kp = g.kp;
    s.block = in_group / 32;
    s.live = (int)(left < 0 ? 0 : left < kTRows ? left : kTRows);
    return true;
  };

  v4i in0[GRAD ? 1 : PASSES], in1[GLU && !GRAD ? PASSES : 1], dy[GRAD ? PASSES : 1];
  v2i kq0[GRAD ? PASSES : 1], kq1[GRAD && GLU ? PASSES : 1];
  uint32_t ks0[GRAD ? PASSES : 1], ks1[GRAD && GLU ? PASSES : 1];
  float prob[PASSES];
  bool there[PASSES];
  auto load = [&](const Sub& s) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * RPP + r_of;
      const int64_t row = s.row0 + r;
      bool ok = r < s.live;
      int64_t src = row;
      float p = 1.0f;
      if constexpr (ROWS) {
        const int64_t c = ok ? (int64_t)a.choices[row] : -1;
        ok = c >= 0 && c < a.tokens * a.K;
        src = ok ? (int64_t)((uint32_t)c / (uint32_t)a.K) : 0;
        if (ok && a.probs != nullptr) p = a.probs[c];
      } else {
        if (ok && a.probs != nullptr) p = a.probs[row];
      }
      there[i] = grouped ? r < s.live : ok;
      ok = ok && live_col;
      prob[i] = ok ? p : 0.0f;
      const int64_t c = c0 + ch * 8;
      if constexpr (!GRAD) {
        in0[i] = v4i{0, 0, 0, 0};
        if constexpr (GLU) in1[i] = v4i{0, 0, 0, 0};
        if (ok) {
          const uint16_t* at = a.in + src * (GLU ? 2 : 1) * a.F + c;
          in0[i] = *(const v4i*)at;
          if constexpr (GLU) in1[i] = *(const v4i*)(at + a.F);
        }
      } else {
        dy[i] = v4i{0, 0, 0, 0};
        kq0[i] = v2i{0, 0};
        ks0[i] = 127;
        if constexpr (GLU) {
          kq1[i] = v2i{0, 0};
          ks1[i] = 127;
        }
        if (ok) {
          dy[i] = *(const v4i*)(a.in + row * a.F + c);
          const uint8_t* q = a.kq + row * (GLU ? 2 : 1) * a.F + c;
          kq0[i] = *(const v2i*)q;
          ks0[i] = a.ks[c / 32 * a.R + row];
          if constexpr (GLU) {
            kq1[i] = *(const v2i*)(q + a.F);
            ks1[i] = a.ks[(a.F + c) / 32 * a.R + row];
          }
        }
      }
    }
  };

  // 8 values of a row into a rowwise layout of `width` columns, their block's scale into the staged scales
  auto put_row = [&](auto f4, uint8_t* q, int64_t width, int64_t row, int64_t c, int r, bool ok, int which,
                     const float(&v)[8]) {
    constexpr bool X4 = decltype(f4)::value;
    const int e = block_exponent<X4>(quad_max(largest8(v)));
    const v2i w = codes8<X4>(v, exp2_neg(e));
    if (ok) {
      if constexpr (X4) *(int*)(q + (row * width + c) / 2) = w[0];
      else *(v2i*)(q + row * width + c) = w;
    }
    if ((ch & 3) == 0) scales[which][ch >> 2][r] = (uint8_t)(e + 127);
  };
  const std::integral_constant<bool, F4> f4;
  const std::integral_constant<bool, false> f8;

  Sub cur;
  if (!place(rt0, 0, cur)) return;
  load(cur);
  for (int step = 0;; ++step) {
    const bool any_col = col_out || (GRAD && a.ycol_q != nullptr);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * RPP + r_of;
      const int64_t row = cur.row0 + r, c = c0 + ch * 8;
      const bool ok = there[i] && live_col;
      const float p = prob[i];
      float y[8], z[GLU && GRAD ? 8 : 1], v[GRAD ? 8 : 1];
      if constexpr (!GRAD) {
        float h[8];
        unpack8(in0[i], h);
        if constexpr (ROWS) {
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = a.probs != nullptr ? h[k] * p : h[k];
        } else if constexpr (!GLU) {
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = act_value<1>(h[k], 0.0f, p, 0.0f);
          put_row(f8, a.kept_q, a.F, row, c, r, ok, OUTS, h);
        } else {
          float b[8];
          unpack8(in1[i], b);
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = act_value<3>(h[k], b[k], p, 0.0f);
          put_row(f8, a.kept_q, 2 * a.F, row, c, r, ok, OUTS, h);
          put_row(f8, a.kept_q, 2 * a.F, row, a.F + c, r, ok, OUTS + 1, b);
        }
      } else {
        float d[8], h[8], part = 0.0f;
        unpack8(dy[i], d);
        unpack_codes(kq0[i], ks0[i], h);
        if constexpr (!GLU) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float x = h[k] > 0.0f ? h[k] : 0.0f, x2 = x * x;
            y[k] = 2.0f * x * p * d[k];
            v[k] = x2 * p;
            part = __builtin_fmaf(d[k], x2, part);
          }
        } else {
          float b[8];
          unpack_codes(kq1[i], ks1[i], b);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float sg = sigmoid_fast(h[k]), sl = h[k] * sg, q = d[k] * p, val = sl * b[k];
            z[k] = q * sl;
            y[k] = q * b[k] * __builtin_fmaf(sl, 1.0f - sg, sg);
            v[k] = val * p;
            part = __builtin_fmaf(d[k], val, part);
          }
        }
        if (a.partial != nullptr) {
#pragma unroll
          for (int m = 1; m < LPR; m <<= 1) part += __shfl_xor(part, m, 64);
          if (ch == 0 && there[i]) a.partial[(int64_t)blockIdx.x % ctiles * a.R + row] = part;
        }
      }
      if (row_out) {
        put_row(f4, a.row_q, C, row, c, r, ok, 0, y);
        if constexpr (GLU && GRAD) put_row(f4, a.row_q, C, row, a.F + c, r, ok, 1, z);
      }
      if (any_col) {
        auto stage = [&](int which, const float(&x)[8]) {
          *(float4*)&tile[which][r][ch * 8] = make_float4(x[0], x[1], x[2], x[3]);
          *(float4*)&tile[which][r][ch * 8 + 4] = make_float4(x[4], x[5], x[6], x[7]);
        };
        stage(0, y);
        if constexpr (GLU && GRAD) stage(1, z);
        if constexpr (GRAD) stage(COLS - 1, v);
      }
    }
    __syncthreads();
    Sub nxt;
    const int ns = step + 1;
    const bool more = ns < 2 * a.run && place(rt0 + ns / 2, ns & 1, nxt);
    const Sub now = cur;
    if (more) load(nxt);
    if (any_col) {
      // a task is 32 rows of one channel of one array
      for (int task = tid; task < COLS * 2 * W; task += kTThreads) {
        const int c = task % W, half = task / W % 2, which = task / (2 * W);
        const bool is_y = GRAD && which == COLS - 1;
        uint8_t* q = is_y ? a.ycol_q : a.col_q;
        if (q == nullptr || c >= ncols) continue;
        const int64_t width = is_y ? a.F : C, oc = c0 + c + (which == 1 && !is_y ? a.F : 0);
        float x[32];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          x[i] = tile[which][32 * half + i][c];
          m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
        }
        const int e = block_exponent<F4>(m);
        const float s = exp2_neg(e);
        const int64_t at = col_elem(width, now.p, now.kp, oc, 32 * (now.block + half));
        if constexpr (F4) {
          v4i w;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float* t = x + 8 * i;
            w[i] = (int)e2m1x8(t[0] * s, t[1] * s, t[2] * s, t[3] * s, t[4] * s, t[5] * s, t[6] * s, t[7] * s);
          }
          *(v4i*)(q + at / 2) = w;
        } else {
          v4i w[2];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            w[i >> 2][i & 3] = (int)e4m3x4(x[4 * i] * s, x[4 * i + 1] * s, x[4 * i + 2] * s, x[4 * i + 3] * s);
          *(v4i*)(q + at) = w[0];
          *(v4i*)(q + at + 16) = w[1];
        }
        (is_y ? a.ycol_s : a.col_s)[col_e8m0(width, now.p, now.block + half, oc)] = (uint8_t)(e + 127);
      }
    }
    // the staged scales of the live rows
    for (int i = tid; i < (OUTS + KEPT) * (W / 32) * kTRows; i += kTThreads) {
      const int r = i % kTRows, b = i / kTRows % (W / 32), which = i / (kTRows * (W / 32));
      uint8_t* s = which < OUTS ? a.row_s : a.kept_s;
      if (s == nullptr || r >= now.live || b * 32 >= ncols) continue;
      if constexpr (ROWS) {
        if (!grouped) {
          const int64_t c = a.choices[now.row0 + r];
          if (c < 0 || c >= a.tokens * a.K) continue;
        }
      }
      const int64_t half = which < OUTS ? which : which - OUTS;
      s[((half * a.F + c0) / 32 + b) * a.R + now.row0 + r] = scales[which][b][r];
    }
    if (!more) break;
    __syncthreads();  // the tile and the scales are free for the next sub-tile
    cur = nxt;
  }
}

// dprobs[r] = the parts of the column tiles added in order; rows past the live ones are left as they are.
__global__ __launch_bounds__(256) void token_dprobs_kernel(const float* partial, int64_t R, int64_t tiles,
                                                           const int32_t* splits, int E, float* dprobs) {
  __shared__ int64_t wave_sum_sm[4];
  int64_t live = 0;
  bool bad = false;
  for (int e = threadIdx.x; e < E; e += 256) {
    const int32_t k = splits[e];
    bad |= k < 0;
    live += k;
  }
  live = wave_inclusive_scan(bad ? int64_t(1) << 40 : live);
  if ((threadIdx.x & 63) == 63) wave_sum_sm[threadIdx.x >> 6] = live;
  __syncthreads();
  live = wave_sum_sm[0] + wave_sum_sm[1] + wave_sum_sm[2] + wave_sum_sm[3];
  if (live > R) return;  // sizes that the first launch refused (a negative one counts as more than any capacity)
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (r >= live) return;
  float s = 0.0f;
  for (int64_t t = 0; t < tiles; ++t) s += partial[t * R + r];
  dprobs[r] = s;
}

size_t act_checkpoint_grad_workspace_bytes(int64_t R, int64_t F) {
  return (size_t)((F + 63) / 64) * (size_t)R * sizeof(float);
}

template <int MODE>
static int launch_mode(const TokenQuantArgs& given, bool f4, hipStream_t stream) {
  TokenQuantArgs a = given;
  constexpr int W = mode_width(MODE);
  const bool grouped = MODE != kModeRows || a.col_q != nullptr;
  // sum ceil(k_e / 128) <= floor((R + 127 E) / 128) tiles for any valid sizes
  const int64_t tiles = grouped ? (a.R + 127 * (int64_t)a.E) / 128 : (a.R + 127) / 128, ctiles = (a.F + W - 1) / W;
  // a run of tiles per workgroup on large inputs, so that the sizes are scanned once for it
  const int64_t run = tiles * ctiles / 2048;
  a.run = (int)(run < 1 ? 1 : run > 8 ? 8 : run);
  const int64_t blocks = (tiles + a.run - 1) / a.run * ctiles;
  if (blocks > 0x7fffffff) return BSFP8_ERR_SHAPE;
  if (f4) hipLaunchKernelGGL((token_quant_kernel<MODE, true>), dim3((unsigned)blocks), dim3(kTThreads), 0, stream, a);
  else hipLaunchKernelGGL((token_quant_kernel<MODE, false>), dim3((unsigned)blocks), dim3(kTThreads), 0, stream, a);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

int launch_dispatch_quantize(const void* x, int64_t T, int64_t C, const int32_t* choices, int K, const float* weights,
                             int64_t R, const int32_t* splits, int E, int recipe, uint8_t* row_q, uint8_t* row_s,
                             uint8_t* col_q, uint8_t* col_s, uint32_t* status, hipStream_t stream) {
  TokenQuantArgs a{};
  a.in = (const uint16_t*)x;
  a.R = R;
  a.F = C;
  a.probs = weights;
  a.choices = choices;
  a.tokens = T;
  a.K = K;
  a.splits = splits;
  a.E = E;
  a.row_q = row_q;
  a.row_s = row_s;
  a.col_q = col_q;
  a.col_s = col_s;
  a.status = status;
  return launch_mode<kModeRows>(a, recipe == BSFP8_RECIPE_MXFP4_1X32_E8M0, stream);
}

int launch_act_checkpoint(int act, const void* h, const float* probs, int64_t R, int64_t F, const int32_t* splits, int E,
                          int recipe, uint8_t* row_q, uint8_t* row_s, uint8_t* col_q, uint8_t* col_s, uint8_t* kept_q,
                          uint8_t* kept_s, uint32_t* status, hipStream_t stream) {
  TokenQuantArgs a{};
  a.in = (const uint16_t*)h;
  a.R = R;
  a.F = F;
  a.probs = probs;
  a.splits = splits;
  a.E = E;
  a.row_q = row_q;
  a.row_s = row_s;
  a.col_q = col_q;
  a.col_s = col_s;
  a.kept_q = kept_q;
  a.kept_s = kept_s;
  a.status = status;
  const bool f4 = recipe == BSFP8_RECIPE_MXFP4_1X32_E8M0;
  return act == BSFP8_ACT_SRELU ? launch_mode<kModeSrelu>(a, f4, stream) : launch_mode<kModeSwiglu>(a, f4, stream);
}

int launch_act_checkpoint_grad(int act, const uint8_t* kept_q, const uint8_t* kept_s, const float* probs, const void* dy,
                               int64_t R, int64_t F, const int32_t* splits, int E, int recipe, uint8_t* row_q,
                               uint8_t* row_s, uint8_t* col_q, uint8_t* col_s, uint8_t* ycol_q, uint8_t* ycol_s,
                               float* dprobs, float* workspace, uint32_t* status, hipStream_t stream) {
  TokenQuantArgs a{};
  a.in = (const uint16_t*)dy;
  a.kq = kept_q;
  a.ks = kept_s;
  a.R = R;
  a.F = F;
  a.probs = probs;
  a.splits = splits;
  a.E = E;
  a.row_q = row_q;
  a.row_s = row_s;
  a.col_q = col_q;
  a.col_s = col_s;
  a.ycol_q = ycol_q;
  a.ycol_s = ycol_s;
  a.partial = dprobs != nullptr ? workspace : nullptr;
  a.status = status;
  const bool f4 = recipe == BSFP8_RECIPE_MXFP4_1X32_E8M0;
  const int rc = act == BSFP8_ACT_SRELU ? launch_mode<kModeSrelu_grad>(a, f4, stream)
                                        : launch_mode<kModeSwiglu_grad>(a, f4, stream);
  if (rc != BSFP8_OK || dprobs == nullptr) return rc;
  hipLaunchKernelGGL(token_dprobs_kernel, dim3((unsigned)((R + 255) / 256)), dim3(256), 0, stream, workspace, R,
                     (F + 63) / 64, splits, E, dprobs);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
