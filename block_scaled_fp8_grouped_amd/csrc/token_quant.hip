// Rows quantized on their way into the grouped layouts (gfx950): tokens' rows gathered for their experts, and the
// activation between two projections with its input kept in 8 bits, and its gradient from what was kept.
// include/bsfp8.h states the formulas, group_layout.hpp the layouts.
//
// A wave owns 32 rows of a group (a block of the colwise layout) and walks along their columns, 16 * CH at a time: lane
// l has CH consecutive channels (l % 16) of 8 consecutive rows (l / 16).  So both layouts' blocks are reduced by moves
// between lanes (4 or 8 neighbours along a row; the 4 lanes of a column), a lane's 8 rows of a channel are 8 consecutive
// colwise codes, and nothing goes through LDS: no barrier, and as many waves as registers allow hide the loads of each
// other.  The 4 waves of a workgroup have the 128 rows that share a channel's 128-byte line of codes.  What belongs to a
// row (the choice that it stands for, its probability, its part of dprobs) is held while the wave walks.
#include <type_traits>

#include "act_math.hpp"
#include "common.hpp"
#include "glu_epilogue.hpp"
#include "group_layout.hpp"
#include "token_layout.hpp"

namespace bsfp8 {

constexpr int kTThreads = 256;

// What a launch does: the rows of tokens (as they are, or weighted), or an activation's forward or gradient.
constexpr int kModeRows = 0, kModeWeighted = 1, kModeSrelu = 2, kModeSwiglu = 3, kModeSreluGrad = 4, kModeSwigluGrad = 5;
constexpr bool mode_rows(int m) { return m <= kModeWeighted; }
constexpr bool mode_grad(int m) { return m >= kModeSreluGrad; }
constexpr bool mode_glu(int m) { return m == kModeSwiglu || m == kModeSwigluGrad; }
// channels a lane holds: 4 where three arrays of values (da, db and the activation) have to stay in registers
constexpr int mode_channels(int m) { return mode_grad(m) ? 4 : 8; }

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
  float* partial;              // gradient: [segments][R] parts of dprobs, or NULL
  uint32_t* status;
  int segments, tiles;         // column segments, column tiles in each
};

template <int CTRL>
__device__ __forceinline__ uint32_t lane_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141;  // lane moves within a quad; of 8 lanes, the order reversed

// From each lane's 8 row maxima m the blocks' (over the 4 neighbours of a quad, and with CH == 4 the next quad): lane q of
// its quad gets those of rows q and 4 + q.  Each step halves the values a lane carries, so that a scale is worked out once
// and not by every lane of its block.
template <int CH>
__device__ __forceinline__ void row_block_max(const uint32_t (&m)[8], int ch, uint32_t (&out)[2]) {
  const bool odd = ch & 1, high = ch & 2;
  uint32_t t[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t a = m[2 * k], b = m[2 * k + 1];
    if constexpr (CH == 4) {
      a = max(a, lane_move<kHalfMirror>(a));
      b = max(b, lane_move<kHalfMirror>(b));
    }
    t[k] = max(odd ? b : a, lane_move<kXor1>(odd ? a : b));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    out[k] = max(high ? t[2 * k + 1] : t[2 * k], lane_move<kXor2>(high ? t[2 * k] : t[2 * k + 1]));
}
// Lane q's value of a quad in all of its lanes.
template <int Q>
__device__ __forceinline__ uint32_t quad_lane(uint32_t v) {
  return lane_move<Q * 0x55>(v);
}

// From each lane's 4 column maxima those over the 4 lanes 16 apart: lanes 16 q .. 16 q + 15 get that of column q.
__device__ __forceinline__ uint32_t col_block_max(uint32_t m0, uint32_t m1, uint32_t m2, uint32_t m3) {
  auto p = __builtin_amdgcn_permlane16_swap(m0, m1, false, false);  // rows of 16 lanes: (0 of m0, 0 of m1, 2, 2), (1, 1, 3, 3)
  const uint32_t a = max((uint32_t)p[0], (uint32_t)p[1]);
  p = __builtin_amdgcn_permlane16_swap(m2, m3, false, false);
  const uint32_t b = max((uint32_t)p[0], (uint32_t)p[1]);
  p = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return max((uint32_t)p[0], (uint32_t)p[1]);
}
// The values of lanes 16 q .. 16 q + 15 in all rows of 16 lanes, q = 0 .. 3.
__device__ __forceinline__ void col_broadcast(uint32_t v, uint32_t (&out)[4]) {
  const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)h[0], (uint32_t)h[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)h[1], (uint32_t)h[1], false, false);
  out[0] = (uint32_t)lo[0];
  out[1] = (uint32_t)lo[1];
  out[2] = (uint32_t)hi[0];
  out[3] = (uint32_t)hi[1];
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// A block's scale byte from the bits of its largest magnitude.
template <bool F4>
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  if constexpr (F4) return (uint32_t)(e8m0_exponent_fp4(__uint_as_float(m)) + 127);
  // (e8m0_byte's steps, its lower end by a saturating subtraction)
  return __builtin_elementwise_sub_sat((m + 0x1fffffu) >> 23, 8u);
}
// N (4 or 8) values' codes: 4 to a word, or with F4 8 to a word (N == 4: in its low half).
template <bool F4, int N>
struct Codes {
  uint32_t w[F4 ? 1 : N / 4];
};
template <bool F4, int N>
__device__ __forceinline__ Codes<F4, N> codes_of(const float (&v)[N], uint32_t byte) {
  Codes<F4, N> q;
  if constexpr (F4) {
    const float s = exp2_neg((int)byte - 127);
    if constexpr (N == 8)
      q.w[0] = e2m1x8(v[0] * s, v[1] * s, v[2] * s, v[3] * s, v[4] * s, v[5] * s, v[6] * s, v[7] * s);
    else
      q.w[0] = e2m1x8(v[0] * s, v[1] * s, v[2] * s, v[3] * s, 0.0f, 0.0f, 0.0f, 0.0f);
  } else {
    const float s = __uint_as_float(byte << 23);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) q.w[i] = e4m3x4_scaled(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], s);
  }
  return q;
}

// A lane's 8 rows x CH channels: as fp32, or (bf16 inputs as they are) pairs of channels.  Largest magnitudes are those of
// bit patterns where the bytes have to be grouped_quantize's (a NaN block has an infinity's scale there), and otherwise
// (CH == 4, gradients) fp32 maxima, which pass over a NaN and take the magnitude for nothing.
template <int CH>
struct Values {
  float v[8][CH];
  __device__ __forceinline__ uint32_t row_max(int i) const {
    if constexpr (CH == 4) return __float_as_uint(max3_abs(max3_abs(0.0f, v[i][0], v[i][1]), v[i][2], v[i][3]));
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) m = max(m, magnitude(v[i][c]));
    return m;
  }
  __device__ __forceinline__ void col_max(uint32_t (&m)[CH]) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (CH == 4) {
        float f = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i += 2) f = max3_abs(f, v[i][c], v[i + 1][c]);
        m[c] = __float_as_uint(f);
      } else {
        m[c] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          asm("" : "+v"(v[i][c]));  // (the rows' magnitudes are not kept for this: they would take as many registers again)
          m[c] = max(m[c], magnitude(v[i][c]));
        }
      }
    }
  }
  template <bool F4>
  __device__ __forceinline__ Codes<F4, CH> row_codes(int i, uint32_t byte) const {
    return codes_of<F4, CH>(v[i], byte);
  }
  template <bool F4>
  __device__ __forceinline__ Codes<F4, 8> col_codes(int c, uint32_t byte) const {
    const float x[8] = {v[0][c], v[1][c], v[2][c], v[3][c], v[4][c], v[5][c], v[6][c], v[7][c]};
    return codes_of<F4, 8>(x, byte);
  }
};

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef short v2s __attribute__((ext_vector_type(2)));
typedef uint16_t v2u __attribute__((ext_vector_type(2)));

// Two bf16 pairs -> four e4m3 codes, straight from bf16 (the conversion is exact up to its one rounding, as from fp32).
__device__ __forceinline__ uint32_t e4m3x4_bf16(uint32_t a, uint32_t b, float scale) {
  v2s w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(v2bf, a), scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(v2bf, b), scale, true);
  return __builtin_bit_cast(uint32_t, w);
}
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u, a), __builtin_bit_cast(v2u, b)));
}

struct Pairs {
  uint32_t w[8][4];
  __device__ __forceinline__ uint32_t row_max(int i) const {
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) m = pair_max(m, w[i][c] & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);  // (the bits of fp32)
  }
  __device__ __forceinline__ void col_max(uint32_t (&m)[8]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t p = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        asm("" : "+v"(w[i][c]));
        p = pair_max(p, w[i][c] & 0x7fff7fffu);
      }
      m[2 * c] = p << 16;
      m[2 * c + 1] = p & 0xffff0000u;
    }
  }
  template <bool F4>
  __device__ __forceinline__ Codes<F4, 8> row_codes(int i, uint32_t byte) const {
    if constexpr (F4) {
      float x[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[2 * c] = bf16_lo(w[i][c]);
        x[2 * c + 1] = bf16_hi(w[i][c]);
      }
      return codes_of<F4, 8>(x, byte);
    } else {
      const float s = __uint_as_float(byte << 23);
      return {{e4m3x4_bf16(w[i][0], w[i][1], s), e4m3x4_bf16(w[i][2], w[i][3], s)}};
    }
  }
  template <bool F4>
  __device__ __forceinline__ Codes<F4, 8> col_codes(int c, uint32_t byte) const {
    if constexpr (F4) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = c & 1 ? bf16_hi(w[i][c / 2]) : bf16_lo(w[i][c / 2]);
      return codes_of<F4, 8>(x, byte);
    } else {
      const float s = __uint_as_float(byte << 23);
      uint32_t p[4];  // the channel's rows in pairs
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[i] = __builtin_amdgcn_perm(w[2 * i + 1][c / 2], w[2 * i][c / 2], c & 1 ? 0x07060302u : 0x05040100u);
      return {{e4m3x4_bf16(p[0], p[1], s), e4m3x4_bf16(p[2], p[3], s)}};
    }
  }
};

// Where a wave's values go, and in it a lane's.
struct LanePlace {
  int64_t row0, R;          // (uniform) the wave's first row
  int64_t p, kp, block;     // (uniform) its group's packed offset and extent, its block of 32 rows
  int live;                 // (uniform) its rows that are there, 0 to 32
  int ch, rl;               // lane % 16, lane / 16
  int nl;                   // rows of the lane's 8 that are there
  bool live_col;            // whether its channels exist
};

// Buffers from a uniform address on; a lane's offset of kNowhere or more is dropped (loads: 0).
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)kNowhere, 0x00020000);
}
// The same for row i of every lane's 8, the lane's offset that of its first row: as many bytes as the rows from it on have.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void* p, int i, uint32_t row_bytes, int live) {
  return __builtin_amdgcn_make_buffer_rsrc((uint8_t*)const_cast<void*>(p) + (uint32_t)i * row_bytes, (short)0,
                                           (int)(live > i ? (uint32_t)(live - i) * row_bytes : 0u), 0x00020000);
}
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}
template <bool F4, int N>
__device__ __forceinline__ void store_codes(__amdgpu_buffer_rsrc_t rs, uint32_t off, const Codes<F4, N>& q) {
  if constexpr (F4 && N == 4) __builtin_amdgcn_raw_buffer_store_b16((short)q.w[0], rs, (int)off, 0, 0);
  else if constexpr (F4 || N == 4) __builtin_amdgcn_raw_buffer_store_b32((int)q.w[0], rs, (int)off, 0, 0);
  else __builtin_amdgcn_raw_buffer_store_b64(v2i{(int)q.w[0], (int)q.w[1]}, rs, (int)off, 0, 0);
}

// The values along their rows: codes into q [R][width] from channel c0 on, scales into s [width / 32][R].
template <bool F4, int CH, class V>
__device__ __forceinline__ void put_rows(const LanePlace& l, uint8_t* q, uint8_t* s, uint32_t width, int64_t c0, const V& x) {
  constexpr int PER = F4 ? 2 : 1;
  uint32_t m[8], top[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = x.row_max(i);
  row_block_max<CH>(m, l.ch, top);
  const uint32_t byte[2] = {scale_byte<F4>(top[0]), scale_byte<F4>(top[1])};
  const uint8_t* at = q + (l.row0 * width + c0) / PER;
  const uint32_t off = l.live_col ? (8 * (uint32_t)l.rl * width + (uint32_t)(l.ch * CH)) / PER : kNowhere;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = byte[i >> 2], of = i % 4 == 0 ? quad_lane<0>(b) : i % 4 == 1 ? quad_lane<1>(b) : i % 4 == 2 ? quad_lane<2>(b) : quad_lane<3>(b);
    store_codes<F4, CH>(row_buffer(at, i, width / PER, l.live), off, x.template row_codes<F4>(i, of));
  }
  // a block's first quad has its 8 scales, two a lane
  const int r = l.ch & 3;
  const __amdgpu_buffer_rsrc_t rs = buffer_at(s + c0 / 32 * l.R + l.row0);
  const uint32_t to = (CH == 8 || (l.ch & 4) == 0) && l.live_col ? (uint32_t)(l.ch * CH / 32) * (uint32_t)l.R + 8 * l.rl + r : kNowhere;
  __builtin_amdgcn_raw_buffer_store_b8((char)byte[0], rs, (int)(r < l.nl ? to : kNowhere), 0, 0);
  __builtin_amdgcn_raw_buffer_store_b8((char)byte[1], rs, (int)(4 + r < l.nl ? to : kNowhere), 4, 0);
  __builtin_amdgcn_sched_barrier(0);
}

// A tile's colwise codes wait in LDS until all 4 waves have theirs, so that a channel's 128 rows leave as one line: stored
// from the registers, 8 bytes a lane and a channel's 32 in lanes 16 apart, they took 190 us on 65536 x 4096 against 130 for as
// many rowwise codes.  The 16-byte granules of a channel are permuted by its group of 8 channels, which spreads the lanes of
// a write over the banks.
template <bool F4>
struct ColTile {
  static constexpr int RUN = F4 ? 64 : 128, GRANULES = RUN / 16;  // bytes of a channel's 128 codes
  static __device__ __forceinline__ int swizzle(int channel) { return (channel >> 3) & (GRANULES - 1); }
};

// The values along their columns: codes into a tile's [16 * CH] channels in LDS, scales into the colwise layout of `width`
// channels.
template <bool F4, int CH, class V>
__device__ __forceinline__ void put_cols(const LanePlace& l, int wave, uint8_t* codes, uint8_t* s, int64_t width, int64_t c0,
                                         V& x) {
  typedef ColTile<F4> T;
  uint32_t m[CH];
  x.col_max(m);
  const __amdgpu_buffer_rsrc_t rs = buffer_at(s + col_e8m0(width, l.p, l.block, c0));
  const int at = (32 * wave + 8 * l.rl) / (F4 ? 2 : 1);  // first of the lane's 8 codes in a channel's run
#pragma unroll
  for (int k = 0; k < CH / 4; ++k) {
    const uint32_t mine = scale_byte<F4>(col_block_max(m[4 * k], m[4 * k + 1], m[4 * k + 2], m[4 * k + 3]));
    uint32_t byte[4];
    col_broadcast(mine, byte);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int channel = l.ch * CH + 4 * k + i;
      const Codes<F4, 8> q = x.template col_codes<F4>(4 * k + i, byte[i]);
      __builtin_memcpy(codes + channel * T::RUN + (((at >> 4) ^ T::swizzle(channel)) << 4 | (at & 15)), q.w, sizeof(q.w));
    }
    __builtin_amdgcn_raw_buffer_store_b8((char)mine, rs, (int)(l.live_col ? l.ch * CH + l.rl : (int)kNowhere), 4 * k, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// A tile's codes from LDS to the layout, 16 bytes a lane; `wave0`: the workgroup's first block of 32 rows.
template <bool F4, int W>
__device__ __forceinline__ void flush_cols(const LanePlace& l, int64_t block0, const uint8_t* codes, uint8_t* q, int64_t width,
                                           int64_t c0, int ncols) {
  typedef ColTile<F4> T;
  const __amdgpu_buffer_rsrc_t rs = buffer_at(q + col_elem(width, l.p, l.kp, c0, 32 * block0) / (F4 ? 2 : 1));
  const uint32_t run = (uint32_t)l.kp / (F4 ? 2 : 1);
#pragma unroll
  for (int i = 0; i < W * T::GRANULES / kTThreads; ++i) {
    const int g = i * kTThreads + (int)threadIdx.x, channel = g / T::GRANULES, k = g % T::GRANULES;
    const v4i w = *(const v4i*)(codes + channel * T::RUN + 16 * (k ^ T::swizzle(channel)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, w), rs,
                                           (int)(channel < ncols ? (uint32_t)channel * run + 16u * (uint32_t)k : kNowhere), 0, 0);
  }
}

// A lane's 4 e4m3 codes times their block's power of two, 2^(byte - 127).
__device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t byte, float (&v)[4]) {
  const float scale = __uint_as_float(byte << 23);  // (the conversion takes its exponent field alone: 0 stands for 2^-127)
  const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false), hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
  v[0] = lo[0];
  v[1] = lo[1];
  v[2] = hi[0];
  v[3] = hi[1];
}

// The value is worked out here and now: the compiler would move its last steps to the branch that stores it and hold their
// operands instead, which are more.
__device__ __forceinline__ void keep(float& v) { asm volatile("" : "+v"(v)); }

// 8 consecutive scale bytes of a column of blocks, of which n are there.
__device__ __forceinline__ uint64_t load_bytes(const uint8_t* p, int n) {
  uint64_t b = 0;
  if (n == 8) {
    __builtin_memcpy(&b, p, 8);
  } else {
#pragma unroll 1
    for (int i = 0; i < n; ++i) b |= (uint64_t)p[i] << (8 * i);
  }
  return b;
}

// A lane's inputs of one column tile as they lie in memory.
template <int MODE>
struct TokenInputs;
template <>
struct TokenInputs<kModeRows> {
  Pairs h;
};
template <>
struct TokenInputs<kModeWeighted> : TokenInputs<kModeRows> {};
template <>
struct TokenInputs<kModeSrelu> : TokenInputs<kModeRows> {};
template <>
struct TokenInputs<kModeSwiglu> : TokenInputs<kModeRows> {
  Pairs b;
};
template <>
struct TokenInputs<kModeSreluGrad> {
  uint32_t k0[8];
  v2i dy[8];
  uint64_t s0;
};
template <>
struct TokenInputs<kModeSwigluGrad> : TokenInputs<kModeSreluGrad> {
  uint32_t k1[8];
  uint64_t s1;
};

template <int MODE, bool F4>
__global__ __launch_bounds__(kTThreads) void token_quant_kernel(TokenQuantArgs a) {
  constexpr bool GRAD = mode_grad(MODE), GLU = mode_glu(MODE), ROWS = mode_rows(MODE);
  constexpr int CH = mode_channels(MODE), W = 16 * CH, HALVES = GLU ? 2 : 1, OUTS = GRAD ? HALVES : 1;
  constexpr int ARRAYS = GRAD ? HALVES + 1 : 1;  // of colwise codes: the output's halves, the activation
  __shared__ GroupScanSmem<kTThreads> gsm;
  __shared__ __attribute__((aligned(16))) uint8_t codes[2][ARRAYS][W * ColTile<F4>::RUN];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t rt = blockIdx.x / (uint32_t)a.segments, seg = blockIdx.x % (uint32_t)a.segments;
  const bool row_out = a.row_q != nullptr, col_out = a.col_q != nullptr;
  const uint32_t F = (uint32_t)a.F, wide = F * HALVES, C = F * OUTS;  // columns of x; of h; of the output

  LanePlace l;
  l.ch = lane & 15;
  l.rl = lane >> 4;
  l.R = a.R;
  int64_t left;  // rows from the wave's first on
  // rows of tokens without the colwise layout need no groups: theirs are the rows that have a choice
  if (!ROWS || col_out) {
    GroupInfo g{};
    const uint32_t flags = group_scan<kTThreads>(a.splits, a.E, a.R, 128, rt, 0, gsm, g);
    report_status(a.status, flags);
    if (g.e < 0) return;
    const int64_t in_group = uniform64(128 * (rt - g.tile) + 32 * wave);
    left = uniform64(g.k) - in_group;
    l.row0 = uniform64(g.off) + in_group;
    l.p = uniform64(g.p);
    l.kp = uniform64(g.kp);
    l.block = in_group / 32;
  } else {
    l.row0 = 128 * rt + 32 * wave;
    left = a.R - l.row0;
    l.p = l.kp = l.block = 0;
  }
  l.live = (int)(left < 0 ? 0 : left < 32 ? left : 32);
  left -= 8 * l.rl;
  l.nl = (int)(left < 0 ? 0 : left < 8 ? left : 8);

  // the source rows and probabilities of a lane's 8 rows
  int64_t src[ROWS ? 8 : 1];
  float prob[8], part[GRAD ? 8 : 1];
  bool ok[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    ok[i] = i < l.nl;
    prob[i] = 1.0f;
    if constexpr (ROWS) {
      const int64_t c = ok[i] ? (int64_t)a.choices[l.row0 + 8 * l.rl + i] : -1;
      ok[i] = c >= 0 && c < a.tokens * a.K;
      src[i] = ok[i] ? (int64_t)((uint32_t)c / (uint32_t)a.K) * F : 0;
      if (MODE == kModeWeighted && ok[i]) prob[i] = a.probs[c];
    } else if (ok[i] && a.probs != nullptr) {
      prob[i] = a.probs[l.row0 + 8 * l.rl + i];
    }
    if constexpr (GRAD) part[i] = 0.0f;
  }
  if constexpr (ROWS) {
    if (!col_out) {  // rows are stored up to the first without a choice
      int n = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) n = ok[i] && n == i ? i + 1 : n;
      l.nl = n;
      l.live = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int m = __builtin_amdgcn_readlane(n, 16 * k);
        l.live = l.live == 8 * k ? 8 * k + m : l.live;
      }
    }
  }

  auto load = [&](int64_t c0, TokenInputs<MODE>& x) {
    const bool live_col = c0 + l.ch * CH < F;
    if constexpr (ROWS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v4i w = {0, 0, 0, 0};
        if (ok[i] && live_col) w = *(const v4i*)(a.in + src[i] + c0 + l.ch * CH);
#pragma unroll
        for (int k = 0; k < 4; ++k) x.h.w[i][k] = (uint32_t)w[k];
      }
    } else if constexpr (!GRAD) {
      const uint32_t off = live_col ? 2 * (8 * (uint32_t)l.rl * wide + (uint32_t)(l.ch * CH)) : kNowhere;
#pragma unroll
      for (int half = 0; half < HALVES; ++half) {
        const uint16_t* at = a.in + l.row0 * wide + half * (int64_t)F + c0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const v4i w = __builtin_bit_cast(
              v4i, __builtin_amdgcn_raw_buffer_load_b128(row_buffer(at, i, 2 * wide, l.live), (int)off, 0, 0));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (GLU) (half ? x.b : x.h).w[i][k] = (uint32_t)w[k];
            else x.h.w[i][k] = (uint32_t)w[k];
          }
        }
      }
    } else {
      const uint32_t off = live_col ? 8 * (uint32_t)l.rl * wide + (uint32_t)(l.ch * CH) : kNowhere;
      const uint32_t dyo = live_col ? 2 * (8 * (uint32_t)l.rl * F + (uint32_t)(l.ch * CH)) : kNowhere;
      const uint8_t* q = a.kq + l.row0 * wide + c0;
      const uint16_t* dy = a.in + l.row0 * F + c0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x.k0[i] = __builtin_amdgcn_raw_buffer_load_b32(row_buffer(q, i, wide, l.live), (int)off, 0, 0);
        if constexpr (GLU) x.k1[i] = __builtin_amdgcn_raw_buffer_load_b32(row_buffer(q + F, i, wide, l.live), (int)off, 0, 0);
        x.dy[i] = __builtin_bit_cast(
            v2i, __builtin_amdgcn_raw_buffer_load_b64(row_buffer(dy, i, 2 * F, l.live), (int)dyo, 0, 0));
      }
      const int nl = live_col ? l.nl : 0;
      const uint8_t* s = a.ks + c0 / 32 * a.R + l.row0 + ((uint64_t)(l.ch * CH / 32) * (uint64_t)a.R + 8 * l.rl);
      x.s0 = load_bytes(s, nl);
      if constexpr (GLU) x.s1 = load_bytes(s + (int64_t)(F / 32) * a.R, nl);
    }
  };

  // (loading a tile ahead costs more waves than it hides: 368 us against 400 on 65536 x 2048 of the SwiGLU's gradient)
  TokenInputs<MODE> x;
  const int64_t begin = seg * a.tiles * W, stop = begin + (int64_t)a.tiles * W, end = stop < F ? stop : F;
  int turn = 0;
  for (int64_t c0 = begin; c0 < end; c0 += W) {
    l.live_col = c0 + l.ch * CH < F;
    load(c0, x);
    if constexpr (MODE == kModeRows) {
            if (row_out) put_rows<F4, 8>(l, a.row_q, a.row_s, C, c0, x.h);
      if (col_out) put_cols<F4, 8>(l, wave, codes[turn][0], a.col_s, C, c0, x.h);
    } else if constexpr (!GRAD) {
      if constexpr (!ROWS) {
        put_rows<false, 8>(l, a.kept_q, a.kept_s, wide, c0, x.h);
        if constexpr (GLU) put_rows<false, 8>(l, a.kept_q, a.kept_s, wide, F + c0, x.b);
      }
      Values<8> y;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = prob[i];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float h = k & 1 ? bf16_hi(x.h.w[i][k / 2]) : bf16_lo(x.h.w[i][k / 2]);
          if constexpr (ROWS) y.v[i][k] = h * p;
          else if constexpr (!GLU) y.v[i][k] = act_value<1>(h, 0.0f, p, 0.0f);
          else y.v[i][k] = act_value<3>(h, k & 1 ? bf16_hi(x.b.w[i][k / 2]) : bf16_lo(x.b.w[i][k / 2]), p, 0.0f);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (row_out) put_rows<F4, 8>(l, a.row_q, a.row_s, C, c0, y);
      if (col_out) put_cols<F4, 8>(l, wave, codes[turn][0], a.col_s, C, c0, y);
    } else {
      Values<4> y, z, v;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float h[4], b[4];
        unpack_codes(x.k0[i], (uint32_t)(x.s0 >> (8 * i)) & 255u, h);
        if constexpr (GLU) unpack_codes(x.k1[i], (uint32_t)(x.s1 >> (8 * i)) & 255u, b);
        const float p = prob[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w = (uint32_t)x.dy[i][k / 2];
          const float d = k & 1 ? bf16_hi(w) : bf16_lo(w);
          if constexpr (!GLU) {
            const float r = h[k] > 0.0f ? h[k] : 0.0f, r2 = r * r;
            y.v[i][k] = 2.0f * r * p * d;
            v.v[i][k] = r2 * p;
            part[i] = __builtin_fmaf(d, r2, part[i]);
          } else {
            float dp = 0.0f;
            swiglu_grad(h[k], b[k], p, d, y.v[i][k], z.v[i][k], dp);
            v.v[i][k] = swiglu(h[k], b[k], p);
            part[i] += dp;
            keep(z.v[i][k]);
          }
          keep(y.v[i][k]);
          keep(v.v[i][k]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (row_out) {
        put_rows<F4, 4>(l, a.row_q, a.row_s, C, c0, y);
        if constexpr (GLU) put_rows<F4, 4>(l, a.row_q, a.row_s, C, F + c0, z);
      }
      if (col_out) {
        put_cols<F4, 4>(l, wave, codes[turn][0], a.col_s, C, c0, y);
        if constexpr (GLU) put_cols<F4, 4>(l, wave, codes[turn][HALVES - 1], a.col_s, C, F + c0, z);
      }
      if (a.ycol_q != nullptr) put_cols<F4, 4>(l, wave, codes[turn][ARRAYS - 1], a.ycol_s, F, c0, v);
    }
    // (two buffers: a wave that fills the one of the tile after next has passed the next tile's barrier, which every wave
    // reaches with its part of this one read)
    if (col_out || (GRAD && a.ycol_q != nullptr)) {
      __syncthreads();
      const int ncols = F - c0 < W ? (int)(F - c0) : W;
      const int64_t block0 = l.block - wave;
      if (col_out) {
        flush_cols<F4, W>(l, block0, codes[turn][0], a.col_q, C, c0, ncols);
        if constexpr (GRAD && GLU) flush_cols<F4, W>(l, block0, codes[turn][1], a.col_q, C, F + c0, ncols);
      }
      if constexpr (GRAD) {
        if (a.ycol_q != nullptr) flush_cols<F4, W>(l, block0, codes[turn][ARRAYS - 1], a.ycol_q, F, c0, ncols);
      }
      turn ^= 1;
    }
  }
  if constexpr (GRAD) {
    if (a.partial != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float s = part[i];
        s += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x128, 0xf, 0xf, false));
        s += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x124, 0xf, 0xf, false));
        s += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x122, 0xf, 0xf, false));
        s += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x121, 0xf, 0xf, false));
        if (l.ch == 0 && i < l.nl) a.partial[seg * a.R + l.row0 + 8 * l.rl + i] = s;
      }
    }
  }
}

// dprobs[r] = the parts of the column segments added in order; rows past the live ones are left as they are.
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

// Column segments of a launch over `rows` row tiles and `cols` column tiles: as many as give 4096 workgroups (16 per CU).
struct TokenSegments {
  int64_t count, tiles;
};
static TokenSegments token_segments(int64_t rows, int64_t cols) {
  int64_t n = (4096 + rows - 1) / (rows < 1 ? 1 : rows);
  n = n < 1 ? 1 : n > cols ? cols : n;
  const int64_t per = (cols + n - 1) / n;
  return {(cols + per - 1) / per, per};
}
static int64_t token_row_tiles(int64_t R, int E) {
  // sum ceil(k_e / 128) <= floor((R + 127 E) / 128) tiles for any valid sizes
  return E > 0 ? (R + 127 * (int64_t)E) / 128 : (R + 127) / 128;
}

size_t act_checkpoint_grad_workspace_bytes(int64_t R, int64_t F) {
  // (at least as many segments as with any number of groups)
  return (size_t)token_segments(token_row_tiles(R, 0), (F + 63) / 64).count * (size_t)R * sizeof(float);
}

template <int MODE>
static int launch_mode(const TokenQuantArgs& given, bool f4, hipStream_t stream) {
  TokenQuantArgs a = given;
  constexpr int W = 16 * mode_channels(MODE);
  const bool grouped = !mode_rows(MODE) || a.col_q != nullptr;
  const int64_t rows = token_row_tiles(a.R, grouped ? a.E : 0);
  const TokenSegments s = token_segments(rows, (a.F + W - 1) / W);
  const int64_t blocks = rows * s.count;
  if (blocks > 0x7fffffff) return BSFP8_ERR_SHAPE;
  a.segments = (int)s.count;
  a.tiles = (int)s.tiles;
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
  const bool f4 = recipe == BSFP8_RECIPE_MXFP4_1X32_E8M0;
  return weights != nullptr ? launch_mode<kModeWeighted>(a, f4, stream) : launch_mode<kModeRows>(a, f4, stream);
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
  const int rc = act == BSFP8_ACT_SRELU ? launch_mode<kModeSreluGrad>(a, f4, stream)
                                        : launch_mode<kModeSwigluGrad>(a, f4, stream);
  if (rc != BSFP8_OK || dprobs == nullptr) return rc;
  const int64_t parts = token_segments(token_row_tiles(R, E), (F + 63) / 64).count;
  hipLaunchKernelGGL(token_dprobs_kernel, dim3((unsigned)((R + 255) / 256)), dim3(256), 0, stream, workspace, R, parts,
                     splits, E, dprobs);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
