// Rows quantized on their way into the grouped layouts (gfx950): tokens' rows gathered for their experts, and the
// activation between two projections with its input kept in 8 bits, and its gradient from what was kept.
// include/bsfp8.h states the formulas, group_layout.hpp the layouts.
//
// A wave owns 32 rows of a group (a block of the colwise layout) and walks along their columns, 128 at a time: lane l has
// 8 consecutive channels (l % 16) of 8 consecutive rows (l / 16).  So both layouts' blocks are reduced by moves between
// lanes (4 neighbours along a row; the 4 lanes of a column), and a row's codes are stored from registers, 128 bytes of a
// row at a time.  A lane's 8 rows of a channel are 8 consecutive colwise codes; those of the 4 waves of a workgroup meet in
// LDS, whence a channel's 128 leave as one line.  What belongs to a row (the choice that it stands for, its probability,
// its part of dprobs) is held while the wave walks.
//
// What bounds them: bytes, which come and go at 6.2 TB/s at best, and the instructions that the conversions to codes in two
// directions take.  65536 gathered rows of 4096 (32 experts, 4 a token) read 134 MB and write 553 MB, 111 us: 169 us.  The
// SwiGLU's gradient of 65536 x 2048 reads 545 MB and writes 690 MB, 200 us: 320 us, at the 256 registers (and 11 spilled)
// that leave two waves a SIMD, and with 25 vector instructions for a sigmoid by the forward's steps (278 us with 4, from the
// hardware's exponential and reciprocal, which put codes next to a border on its other side: 110 of 268 million).  The
// activations' kernels also spill 29 to 162 scalar registers into lanes: a buffer descriptor for each of a lane's 8 rows and each
// array.  Activation and kept input of 4099 x 4128, 88 MB: 14 us of bytes in 22 us, 1320 workgroups at 1024 places.
#include <math.h>

#include <type_traits>

#include "act_math.hpp"
#include "common.hpp"
#include "glu_epilogue.hpp"
#include "group_layout.hpp"
#include "row_io.hpp"

namespace bsfp8 {

// Codes go past the caches (a line's 128 bytes leave together, and none is read again here): 181 -> 170 us on 65536
// gathered rows of 4096, whose tokens then stay in them; 288 -> 279 us on the SwiGLU's gradient (with the
// hardware's sigmoid).  An activation's rowwise codes, which the next product reads, stay in them (SReLU of 4099 x 4128
// 26.9 -> 22.2 us, layers the same).
constexpr int kInCaches = 0, kPastCaches = 2;
constexpr int kTThreads = 256;

// An activation's forward or gradient.
constexpr int kModeSrelu = 0, kModeSwiglu = 1, kModeSreluGrad = 2, kModeSwigluGrad = 3;
constexpr bool mode_grad(int m) { return m >= kModeSreluGrad; }
constexpr bool mode_glu(int m) { return m == kModeSwiglu || m == kModeSwigluGrad; }
constexpr int kTCols = 128;  // channels of a tile: 16 lanes of 8

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
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;  // lane moves within a quad

// From each lane's 8 row maxima m those of the 4 lanes of its quad, which have a block of 32 channels: lane q gets those
// of rows q and 4 + q.  Each step halves the values a lane carries, so that a scale is worked out once and not by every lane of
// its block.
__device__ __forceinline__ void row_block_max(const uint32_t (&m)[8], int ch, uint32_t (&out)[2]) {
  const bool odd = ch & 1, high = ch & 2;
  uint32_t t[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    t[k] = max(odd ? m[2 * k + 1] : m[2 * k], lane_move<kXor1>(odd ? m[2 * k] : m[2 * k + 1]));
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
// 8 values' codes: 4 to a word, with F4 8 to a word.
template <bool F4>
struct Codes {
  uint32_t w[F4 ? 1 : 2];
};
template <bool F4>
__device__ __forceinline__ Codes<F4> codes_of(const float (&v)[8], uint32_t byte) {
  if constexpr (F4) {
    const float s = exp2_neg((int)byte - 127);
    return {{e2m1x8(v[0] * s, v[1] * s, v[2] * s, v[3] * s, v[4] * s, v[5] * s, v[6] * s, v[7] * s)}};
  } else {
    const float s = __uint_as_float(byte << 23);
    return {{e4m3x4_scaled(v[0], v[1], v[2], v[3], s), e4m3x4_scaled(v[4], v[5], v[6], v[7], s)}};
  }
}

// A lane's 8 rows x 8 channels: as fp32, or (bf16 inputs as they are) pairs of channels.  Largest magnitudes are those of
// bit patterns where the bytes have to be grouped_quantize's (a NaN block has an infinity's scale there), or (FLOAT:
// MXFP8 gradients) fp32 maxima, which pass over a NaN, whose code stays one, and take the magnitude for nothing.  e2m1 has no
// NaN: an MXFP4 block shows one by its scale alone.
template <bool FLOAT>
struct Values {
  float v[8][8];
  __device__ __forceinline__ uint32_t row_max(int i) const {
    if constexpr (FLOAT) {
      float f = 0.0f;
#pragma unroll
      for (int c = 0; c < 8; c += 2) f = max3_abs(f, v[i][c], v[i][c + 1]);
      return __float_as_uint(f);
    }
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) m = max(m, magnitude(v[i][c]));
    return m;
  }
  __device__ __forceinline__ void col_max(uint32_t (&m)[8]) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if constexpr (FLOAT) {
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
  __device__ __forceinline__ Codes<F4> row_codes(int i, uint32_t byte) const {
    return codes_of<F4>(v[i], byte);
  }
  template <bool F4>
  __device__ __forceinline__ Codes<F4> col_codes(int c, uint32_t byte) const {
    const float x[8] = {v[0][c], v[1][c], v[2][c], v[3][c], v[4][c], v[5][c], v[6][c], v[7][c]};
    return codes_of<F4>(x, byte);
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
  __device__ __forceinline__ Codes<F4> row_codes(int i, uint32_t byte) const {
    if constexpr (F4) {
      float x[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[2 * c] = bf16_lo(w[i][c]);
        x[2 * c + 1] = bf16_hi(w[i][c]);
      }
      return codes_of<F4>(x, byte);
    } else {
      const float s = __uint_as_float(byte << 23);
      return {{e4m3x4_bf16(w[i][0], w[i][1], s), e4m3x4_bf16(w[i][2], w[i][3], s)}};
    }
  }
  template <bool F4>
  __device__ __forceinline__ Codes<F4> col_codes(int c, uint32_t byte) const {
    if constexpr (F4) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = c & 1 ? bf16_hi(w[i][c / 2]) : bf16_lo(w[i][c / 2]);
      return codes_of<F4>(x, byte);
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
template <int AUX, bool F4>
__device__ __forceinline__ void store_codes(__amdgpu_buffer_rsrc_t rs, uint32_t off, const Codes<F4>& q) {
  if constexpr (F4) __builtin_amdgcn_raw_buffer_store_b32((int)q.w[0], rs, (int)off, 0, AUX);
  else __builtin_amdgcn_raw_buffer_store_b64(v2i{(int)q.w[0], (int)q.w[1]}, rs, (int)off, 0, AUX);
}

// The values along their rows: codes into q [R][width] from channel c0 on, scales into s [width / 32][R].
template <bool F4, int AUX = kPastCaches, class V>
__device__ __forceinline__ void put_rows(const LanePlace& l, uint8_t* q, uint8_t* s, uint32_t width, int64_t c0, const V& x) {
  constexpr int PER = F4 ? 2 : 1;
  uint32_t m[8], top[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = x.row_max(i);
  row_block_max(m, l.ch, top);
  const uint32_t byte[2] = {scale_byte<F4>(top[0]), scale_byte<F4>(top[1])};
  const uint8_t* at = q + (l.row0 * width + c0) / PER;
  const uint32_t off = l.live_col ? (8 * (uint32_t)l.rl * width + (uint32_t)(l.ch * 8)) / PER : kNowhere;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = byte[i >> 2];
    const uint32_t of = i % 4 == 0 ? quad_lane<0>(b) : i % 4 == 1 ? quad_lane<1>(b) : i % 4 == 2 ? quad_lane<2>(b)
                                                                                              : quad_lane<3>(b);
    store_codes<AUX>(row_buffer(at, i, width / PER, l.live), off, x.template row_codes<F4>(i, of));
  }
  // the quad has its block's 8 scales, two a lane
  const int r = l.ch & 3;
  const __amdgpu_buffer_rsrc_t rs = buffer_at(s + c0 / 32 * l.R + l.row0);
  const uint32_t to = l.live_col ? (uint32_t)(l.ch / 4) * (uint32_t)l.R + 8 * l.rl + r : kNowhere;
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

// The values along their columns: codes into a tile's 128 channels in LDS, scales into the colwise layout of `width`
// channels.
template <bool F4, class V>
__device__ __forceinline__ void put_cols(const LanePlace& l, int wave, uint8_t* codes, uint8_t* s, int64_t width, int64_t c0,
                                         V& x) {
  typedef ColTile<F4> T;
  uint32_t m[8];
  x.col_max(m);
  const __amdgpu_buffer_rsrc_t rs = buffer_at(s + col_e8m0(width, l.p, l.block, c0));
  const int at = (32 * wave + 8 * l.rl) / (F4 ? 2 : 1);  // first of the lane's 8 codes in a channel's run
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t mine = scale_byte<F4>(col_block_max(m[4 * k], m[4 * k + 1], m[4 * k + 2], m[4 * k + 3]));
    uint32_t byte[4];
    col_broadcast(mine, byte);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int channel = l.ch * 8 + 4 * k + i;
      const Codes<F4> q = x.template col_codes<F4>(4 * k + i, byte[i]);
      __builtin_memcpy(codes + channel * T::RUN + (((at >> 4) ^ T::swizzle(channel)) << 4 | (at & 15)), q.w, sizeof(q.w));
    }
    __builtin_amdgcn_raw_buffer_store_b8((char)mine, rs, (int)(l.live_col ? l.ch * 8 + l.rl : (int)kNowhere), 4 * k, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// A tile's codes from LDS to the layout, 16 bytes a lane; `block0`: the workgroup's first block of 32 rows.
template <bool F4>
__device__ __forceinline__ void flush_cols(const LanePlace& l, int64_t block0, const uint8_t* codes, uint8_t* q, int64_t width,
                                           int64_t c0, int ncols) {
  typedef ColTile<F4> T;
  const __amdgpu_buffer_rsrc_t rs = buffer_at(q + col_elem(width, l.p, l.kp, c0, 32 * block0) / (F4 ? 2 : 1));
  const uint32_t run = (uint32_t)l.kp / (F4 ? 2 : 1);
#pragma unroll
  for (int i = 0; i < kTCols * T::GRANULES / kTThreads; ++i) {
    const int g = i * kTThreads + (int)threadIdx.x, channel = g / T::GRANULES, k = g % T::GRANULES;
    const v4i w = *(const v4i*)(codes + channel * T::RUN + 16 * (k ^ T::swizzle(channel)));
    const uint32_t to = channel < ncols ? (uint32_t)channel * run + 16u * (uint32_t)k : kNowhere;
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, w), rs, (int)to, 0, kPastCaches);
  }
}

// 8 e4m3 codes times their block's power of two, 2^(byte - 127).
__device__ __forceinline__ void unpack_codes(const v2i& w, uint32_t byte, float (&v)[8]) {
  const float scale = __uint_as_float(byte << 23);  // (the conversion takes its exponent field alone: 0 stands for 2^-127)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((uint32_t)w[i], scale, false);
    const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((uint32_t)w[i], scale, true);
    v[4 * i] = lo[0];
    v[4 * i + 1] = lo[1];
    v[4 * i + 2] = hi[0];
    v[4 * i + 3] = hi[1];
  }
}

// The value is worked out here and now: the compiler would move its last steps to the branch that stores it and hold their
// operands instead, which are more.
template <class T>
__device__ __forceinline__ void keep(T& v) {
  asm volatile("" : "+v"(v));
}

// The sigmoid of act_value's SwiGLU and of glu_grad, step for step, the clamp in one instruction: it takes a bound for a NaN,
// whose products with a stay NaN.
__device__ __forceinline__ float act_sigmoid(float a) {
  return recip_rn(1.0f + exp2_clamped(__builtin_amdgcn_fmed3f(-a * 1.44269502f, -126.0f, 126.0f)));
}

// 8 consecutive scale bytes of a column of blocks, of which n are there.
__device__ __forceinline__ void load_bytes(const uint8_t* p, int n, uint32_t (&out)[2]) {
  out[0] = out[1] = 0;
  if (n == 8) {
    __builtin_memcpy(out, p, 8);
  } else {
    uint64_t b = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) b |= (uint64_t)p[i] << (8 * i);
    out[0] = (uint32_t)b;
    out[1] = (uint32_t)(b >> 32);
  }
}

// A lane's inputs of one column tile as they lie in memory.
template <int MODE>
struct TokenInputs;
template <>
struct TokenInputs<kModeSrelu> {
  Pairs h;
};
template <>
struct TokenInputs<kModeSwiglu> : TokenInputs<kModeSrelu> {
  Pairs b;
};
template <>
struct TokenInputs<kModeSreluGrad> {
  v2i k0[8];
  v4i dy[8];
  uint32_t s0[2];
};
template <>
struct TokenInputs<kModeSwigluGrad> : TokenInputs<kModeSreluGrad> {
  v2i k1[8];
  uint32_t s1[2];
};

__device__ __forceinline__ int wave_total(int v) { return __builtin_amdgcn_readlane(wave_scan32(v), 63); }

// Row tiles (of 128 rows) in an order in which the groups advance side by side, each in proportion to its size: with S tiles
// in the largest group, a group of T has given floor(j T / S) of them by the end of step j, at most one a step.  A token's rows
// lie in several groups, at about the same fraction of each (the plan keeps the tokens' order), so that the tiles in
// flight at a time read the same tokens and find them in the caches.  Every wave works the order out by itself; lane l has
// groups V l .. V l + V - 1.
template <int V>
struct Turns {
  int k[V];         // rows
  uint32_t rate[V]; // tiles a step, in units of 2^-32, rounded up (0: one)
  int off, packed;  // rows before the lane's first group, and padded to 128 (valid sizes: below 2^24 and 2^25)
  int most;         // (uniform) tiles of the largest group

  __device__ __forceinline__ static int tiles(int rows) { return (rows + 127) >> 7; }
  // the sizes, and what is wrong with them
  __device__ __forceinline__ uint32_t read(const int32_t* __restrict__ splits, int E, int64_t capacity) {
    const int lane = threadIdx.x & 63;
    bool negative = false, large = false;
    off = packed = most = 0;
    int64_t rows = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i, v = e < E ? splits[e] : 0;
      negative |= v < 0;
      large |= (int64_t)v > capacity;
      k[i] = v < 0 || (int64_t)v > capacity ? 0 : v;  // below 2^24: a lane's and a wave's sums are below 2^34
      rows += k[i];
      packed += tiles(k[i]);
      most = max(most, tiles(k[i]));
    }
    uint32_t flags = __ballot(negative) != 0 ? BSFP8_STATUS_NEGATIVE_SPLIT : 0u;
    // (in units of 256 rows, rounded down and up, where 32 bits would not do)
    large |= rows > capacity;
    const int low = wave_total((int)(rows >> 8)), part = wave_total((int)(rows & 255));
    if (__ballot(large) != 0 || ((int64_t)low << 8) + part > capacity) flags |= BSFP8_STATUS_EXCEEDS_CAPACITY;
    if (flags) return flags;
    off = wave_scan32((int)rows) - (int)rows;
    packed = 128 * (wave_scan32(packed) - packed);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) most = max(most, __shfl_xor(most, d, 64));
    most = __builtin_amdgcn_readfirstlane(most);
    // T 2^32 / S is a multiple of 1 / S, at least 2^-17, and double is off by less: rounded up rightly.  S times it is T and
    // less than S / 2^32 more, so that the last step ends at T.
#pragma unroll
    for (int i = 0; i < V; ++i)
      rate[i] = tiles(k[i]) == most ? 0u : (uint32_t)ceil((double)tiles(k[i]) * 0x1p32 / (double)most);
    return 0;
  }
  // tiles of the lane's group i, and of all, in the first j steps
  __device__ __forceinline__ int given(int i, int j) const {
    return k[i] == 0 ? 0 : rate[i] == 0u ? j : (int)__umulhi((uint32_t)j, rate[i]);
  }
  __device__ __forceinline__ int until(int j) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) n += given(i, j);
    return wave_total(n);
  }
  // tile m: its group's rows, their first, the packed offset, and which of the group's tiles it is; false past the last
  __device__ __forceinline__ bool find(int m, int& rows, int& first, int& p, int& tile) const {
    int lo = 0, hi = most;  // the step with until(lo) <= m < until(lo + 1)
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (m < until(mid + 1)) hi = mid;
      else lo = mid + 1;
    }
    if (lo == most) return false;
    const int left = m - until(lo);
    int has = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) has += given(i, lo + 1) > given(i, lo);
    const int seen = wave_scan32(has) - has;  // groups of this step before the lane's
    const int who = __builtin_ctzll(__ballot(left >= seen && left < seen + has));
    int n = left - seen, o = off, q = packed, size = 0, at = 0;
    bool done = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = given(i, lo + 1) > given(i, lo);
      if (!done && in && n == 0) {
        size = k[i];
        at = given(i, lo);
        done = true;
      }
      n -= in;
      if (!done) {
        o += k[i];
        q += 128 * tiles(k[i]);
      }
    }
    rows = __builtin_amdgcn_readlane(size, who);
    first = __builtin_amdgcn_readlane(o, who);
    p = __builtin_amdgcn_readlane(q, who);
    tile = __builtin_amdgcn_readlane(at, who);
    return true;
  }
};

// The sum of the sizes where the groups' places do not matter, and what is wrong with them.  Every wave works it out by
// itself; capacity below 2^24.
__device__ __forceinline__ uint32_t live_rows(const int32_t* __restrict__ splits, int E, int capacity, int& total) {
  const int lane = threadIdx.x & 63;
  bool negative = false, large = false;
  int rows = 0;  // a lane's at most 16 sizes, each at most the capacity
  auto read = [&](auto n) {  // all loads in flight
    int v[decltype(n)::value];
#pragma unroll
    for (int i = 0; i < decltype(n)::value; ++i) v[i] = 64 * i + lane < E ? splits[64 * i + lane] : 0;
#pragma unroll
    for (int i = 0; i < decltype(n)::value; ++i) {
      negative |= v[i] < 0;
      large |= v[i] > capacity;
      rows += v[i] < 0 || v[i] > capacity ? 0 : v[i];
    }
  };
  if (E <= 256) read(std::integral_constant<int, 4>());
  else read(std::integral_constant<int, 16>());
  large |= rows > capacity;
  total = wave_total(rows > capacity ? 0 : rows);  // at most 64 times the capacity
  return (__ballot(negative) != 0 ? BSFP8_STATUS_NEGATIVE_SPLIT : 0u) |
         (__ballot(large) != 0 || total > capacity ? BSFP8_STATUS_EXCEEDS_CAPACITY : 0u);
}

// Rows of tokens: a row tile's column segment, the row tiles in the order of Turns (V > 0), or as they lie (V == 0: rowwise
// only, few rows, no need of the groups).
template <bool WEIGHTED, bool F4, int V>
__global__ __launch_bounds__(kTThreads) void dispatch_quantize_kernel(TokenQuantArgs a) {
  constexpr int W = kTCols;
  __shared__ __attribute__((aligned(16))) uint8_t codes[2][W * ColTile<F4>::RUN];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const bool row_out = a.row_q != nullptr, col_out = V > 0 && a.col_q != nullptr;
  const uint32_t F = (uint32_t)a.F;
  const int64_t seg = blockIdx.x % (uint32_t)a.segments, m = blockIdx.x / (uint32_t)a.segments;
  LanePlace l;
  l.ch = lane & 15;
  l.rl = lane >> 4;
  l.R = a.R;
  Turns<V ? V : 1> turns;
  int32_t near[8];  // (V == 0: the lane's choices, asked for beside the sizes)
  if constexpr (V == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = m * 128 + 32 * wave + 8 * l.rl + i;
      near[i] = r < a.R ? a.choices[r] : -1;
    }
  }
  int total = 0;
  const uint32_t flags = V > 0 ? turns.read(a.splits, a.E, a.R) : live_rows(a.splits, a.E, (int)a.R, total);
  report_status(a.status, flags);
  if (flags) return;
  int64_t left;
  if constexpr (V > 0) {
    int rows, first, p, tile;
    if (!turns.find((int)m, rows, first, p, tile)) return;
    const int in_group = 128 * tile + 32 * wave;
    l.row0 = first + in_group;
    l.p = p;
    l.kp = (rows + 127) & ~127;
    l.block = in_group / 32;
    left = rows - in_group;
  } else {
    l.row0 = m * 128 + 32 * wave;
    l.p = l.kp = l.block = 0;
    left = total - l.row0;
  }
  l.live = (int)(left < 0 ? 0 : left < 32 ? left : 32);
  left -= 8 * l.rl;
  l.nl = (int)(left < 0 ? 0 : left < 8 ? left : 8);
  const uint16_t* src[8];
  float weight[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t c = i >= l.nl ? -1 : V == 0 ? near[i] : a.choices[l.row0 + 8 * l.rl + i];
    const bool ok = c >= 0 && c < a.tokens * a.K;  // (another choice: a row of zeros)
    src[i] = ok ? a.in + (int64_t)((uint32_t)c / (uint32_t)a.K) * F + l.ch * 8 : nullptr;
    weight[i] = WEIGHTED && ok ? a.probs[c] : 1.0f;
  }
  int turn = 0;
  const int64_t begin = seg * a.tiles * W, stop = begin + (int64_t)a.tiles * W, end = stop < F ? stop : F;
  for (int64_t c0 = begin; c0 < end; c0 += W) {
    l.live_col = c0 + l.ch * 8 < F;
    Pairs x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v4i w = {0, 0, 0, 0};
      if (src[i] != nullptr && l.live_col) w = *(const v4i*)(src[i] + c0);
#pragma unroll
      for (int k = 0; k < 4; ++k) x.w[i][k] = (uint32_t)w[k];
    }
    auto put = [&](auto& values) {
      if (row_out) put_rows<F4>(l, a.row_q, a.row_s, F, c0, values);
      if (!col_out) return;
      put_cols<F4>(l, wave, codes[turn], a.col_s, F, c0, values);
      __syncthreads();  // (one for two buffers: see the activations' kernel)
      flush_cols<F4>(l, l.block - wave, codes[turn], a.col_q, F, c0, F - c0 < W ? (int)(F - c0) : W);
      turn ^= 1;
    };
    if constexpr (WEIGHTED) {
      Values<false> y;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) y.v[i][k] = (k & 1 ? bf16_hi(x.w[i][k / 2]) : bf16_lo(x.w[i][k / 2])) * weight[i];
      __builtin_amdgcn_sched_barrier(0);
      put(y);
    } else {
      put(x);
    }
  }
}

template <int MODE, bool F4>
__global__ __launch_bounds__(kTThreads, mode_grad(MODE) ? 2 : 1) void act_checkpoint_kernel(TokenQuantArgs a) {
  constexpr bool GRAD = mode_grad(MODE), GLU = mode_glu(MODE);
  constexpr int W = kTCols, HALVES = GLU ? 2 : 1, OUTS = GRAD ? HALVES : 1;
  __shared__ GroupScanSmem<kTThreads> gsm;
  constexpr int BUFFERS = GRAD ? 2 : 1;  // (the forward's one array a tile: SwiGLU of 65536 x 2048 226 us with two, 220 with one)
  __shared__ __attribute__((aligned(16))) uint8_t codes[BUFFERS][W * ColTile<F4>::RUN];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t rt = blockIdx.x / (uint32_t)a.segments, seg = blockIdx.x % (uint32_t)a.segments;
  const bool row_out = a.row_q != nullptr, col_out = a.col_q != nullptr;
  const uint32_t F = (uint32_t)a.F, wide = F * HALVES, C = F * OUTS;  // columns of x; of h; of the output

  LanePlace l;
  l.ch = lane & 15;
  l.rl = lane >> 4;
  l.R = a.R;
  int64_t left;  // rows from the wave's first on
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
  l.live = (int)(left < 0 ? 0 : left < 32 ? left : 32);
  left -= 8 * l.rl;
  l.nl = (int)(left < 0 ? 0 : left < 8 ? left : 8);

  float prob[8], part[GRAD ? 8 : 1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    prob[i] = i < l.nl && a.probs != nullptr ? a.probs[l.row0 + 8 * l.rl + i] : 1.0f;
    if constexpr (GRAD) part[i] = 0.0f;
  }

  auto load = [&](int64_t c0, TokenInputs<MODE>& x) {
    const bool live_col = c0 + l.ch * 8 < F;
    if constexpr (!GRAD) {
      const uint32_t off = live_col ? 2 * (8 * (uint32_t)l.rl * wide + (uint32_t)(l.ch * 8)) : kNowhere;
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
      const uint32_t off = live_col ? 8 * (uint32_t)l.rl * wide + (uint32_t)(l.ch * 8) : kNowhere;
      const uint32_t dyo = live_col ? 2 * (8 * (uint32_t)l.rl * F + (uint32_t)(l.ch * 8)) : kNowhere;
      const uint8_t* q = a.kq + l.row0 * wide + c0;
      const uint16_t* dy = a.in + l.row0 * F + c0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x.k0[i] = __builtin_bit_cast(
            v2i, __builtin_amdgcn_raw_buffer_load_b64(row_buffer(q, i, wide, l.live), (int)off, 0, 0));
        if constexpr (GLU)
          x.k1[i] = __builtin_bit_cast(
              v2i, __builtin_amdgcn_raw_buffer_load_b64(row_buffer(q + F, i, wide, l.live), (int)off, 0, 0));
        x.dy[i] = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(row_buffer(dy, i, 2 * F, l.live), (int)dyo, 0, 0));
      }
      const int nl = live_col ? l.nl : 0;
      const uint8_t* s = a.ks + c0 / 32 * a.R + l.row0 + ((uint64_t)(l.ch * 8 / 32) * (uint64_t)a.R + 8 * l.rl);
      load_bytes(s, nl, x.s0);
      if constexpr (GLU) load_bytes(s + (int64_t)(F / 32) * a.R, nl, x.s1);
    }
  };

  // (a tile asked for ahead takes registers that are worth more as waves: 400 us against 368 when the SwiGLU's gradient of
  // 65536 x 2048 took that, with the hardware's sigmoid)
  TokenInputs<MODE> x;
  int turn = 0;
  const int64_t begin = seg * a.tiles * W, stop = begin + (int64_t)a.tiles * W, end = stop < F ? stop : F;
  // the colwise layout of a tile's values: `half` of the `width` channels from c0 on
  auto cols = [&](uint8_t* q, uint8_t* s, uint32_t width, int64_t c0, int64_t half, auto& values) {
    if (BUFFERS == 1 && c0 != begin) __syncthreads();  // (the tile before is out)
    put_cols<F4>(l, wave, codes[turn], s, width, half + c0, values);
    // (two buffers: a wave that fills the one of the array after next has passed the next one's barrier, which every wave
    // reaches with its part of this one read)
    __syncthreads();
    flush_cols<F4>(l, l.block - wave, codes[turn], q, width, half + c0, F - c0 < W ? (int)(F - c0) : W);
    turn = (turn + 1) % BUFFERS;
  };
  for (int64_t c0 = begin; c0 < end; c0 += W) {
    l.live_col = c0 + l.ch * 8 < F;
    load(c0, x);
    if constexpr (!GRAD) {
      put_rows<false>(l, a.kept_q, a.kept_s, wide, c0, x.h);
      if constexpr (GLU) put_rows<false>(l, a.kept_q, a.kept_s, wide, F + c0, x.b);
      Values<false> y;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = prob[i];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float h = k & 1 ? bf16_hi(x.h.w[i][k / 2]) : bf16_lo(x.h.w[i][k / 2]);
          if constexpr (!GLU) y.v[i][k] = act_value<1>(h, 0.0f, p, 0.0f);
          else y.v[i][k] = act_value<3>(h, k & 1 ? bf16_hi(x.b.w[i][k / 2]) : bf16_lo(x.b.w[i][k / 2]), p, 0.0f);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (row_out) put_rows<F4, kInCaches>(l, a.row_q, a.row_s, C, c0, y);
      if (col_out) cols(a.col_q, a.col_s, C, c0, 0, y);
    } else {
      // one array of values at a time, worked out from the inputs and the sigmoids, which stay
      Values<!F4> y, sg;
      float d[8], h[8], b[8];
      auto inputs = [&](int i) {
        keep(x.k0[i]);
        keep(x.s0[i >> 2]);
        unpack_codes(x.k0[i], x.s0[i >> 2] >> (8 * (i & 3)) & 255u, h);
        if constexpr (GLU) {
          keep(x.k1[i]);
          keep(x.s1[i >> 2]);
          unpack_codes(x.k1[i], x.s1[i >> 2] >> (8 * (i & 3)) & 255u, b);
        }
        keep(x.dy[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = k & 1 ? bf16_hi((uint32_t)x.dy[i][k / 2]) : bf16_lo((uint32_t)x.dy[i][k / 2]);
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // the activation, its part of dprobs
        inputs(i);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float val;
          if constexpr (!GLU) {
            const float r = h[k] > 0.0f ? h[k] : 0.0f;
            val = r * r;
          } else {
            sg.v[i][k] = act_sigmoid(h[k]);
            keep(sg.v[i][k]);
            val = h[k] * sg.v[i][k] * b[k];
          }
          part[i] = __builtin_fmaf(d[k], val, part[i]);
          y.v[i][k] = val * prob[i];
          keep(y.v[i][k]);
        }
        keep(part[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (a.ycol_q != nullptr) cols(a.ycol_q, a.ycol_s, F, c0, 0, y);
      if (row_out || col_out) {
        if constexpr (GLU) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            inputs(i);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              y.v[i][k] = d[k] * prob[i] * (h[k] * sg.v[i][k]);
              keep(y.v[i][k]);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
          if (row_out) put_rows<F4>(l, a.row_q, a.row_s, C, F + c0, y);
          if (col_out) cols(a.col_q, a.col_s, C, c0, F, y);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          inputs(i);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if constexpr (!GLU) {
              const float r = h[k] > 0.0f ? h[k] : 0.0f;
              y.v[i][k] = 2.0f * r * prob[i] * d[k];
            } else {
              const float s = sg.v[i][k];
              y.v[i][k] = d[k] * prob[i] * b[k] * (s * (1.0f + h[k] * (1.0f - s)));
            }
            keep(y.v[i][k]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (row_out) put_rows<F4>(l, a.row_q, a.row_s, C, c0, y);
        if (col_out) cols(a.col_q, a.col_s, C, c0, 0, y);
      }
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

// Column segments of a launch over `rows` row tiles and `cols` column tiles: as many as give kTFill workgroups, or
// twice that for an activation's forward (2048 / 4096 / 8192 workgroups: SReLU of 65536 x 4096 300 / 278 / 264 us, its
// gradient 350 / 335 / 329, SwiGLU's of 65536 x 2048 339 / 319 / 353, 65536 gathered rows of 4096 170 / 170 / 179).
struct TokenSegments {
  int64_t count, tiles;
};
constexpr int64_t kTFill = 4096;
static TokenSegments token_segments(int64_t rows, int64_t cols, int64_t fill = kTFill) {
  int64_t n = (fill + rows - 1) / (rows < 1 ? 1 : rows);
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
  return (size_t)token_segments(token_row_tiles(R, 0), (F + kTCols - 1) / kTCols).count * (size_t)R * sizeof(float);
}

template <int MODE>
static int launch_mode(const TokenQuantArgs& given, bool f4, hipStream_t stream) {
  TokenQuantArgs a = given;
  const int64_t rows = token_row_tiles(a.R, a.E);
  const TokenSegments s = token_segments(rows, (a.F + kTCols - 1) / kTCols, mode_grad(MODE) ? kTFill : 2 * kTFill);
  const int64_t blocks = rows * s.count;
  if (blocks > 0x7fffffff) return BSFP8_ERR_SHAPE;
  a.segments = (int)s.count;
  a.tiles = (int)s.tiles;
  if (f4) hipLaunchKernelGGL((act_checkpoint_kernel<MODE, true>), dim3((unsigned)blocks), dim3(kTThreads), 0, stream, a);
  else hipLaunchKernelGGL((act_checkpoint_kernel<MODE, false>), dim3((unsigned)blocks), dim3(kTThreads), 0, stream, a);
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
  // Rows that need no groups are taken as they lie while they are few: their tokens stay in the caches anyway, and the order
  // of turns takes each workgroup time to work out (rowwise MXFP8, turns / as they lie: 32 rows of 7168 12.1 / 3.9 us, 4096
  // of 4096 13.1 / 7.0, 16384 of 4096 25.8 / 21.4, 32768 of 7168 98.9 / 98.6, 65536 of 4096 109 / 116).
  const bool turns = col_q != nullptr || R >= 32768;
  const int64_t rows = token_row_tiles(R, turns ? E : 0);
  const TokenSegments seg = token_segments(rows, (C + kTCols - 1) / kTCols);
  if (rows * seg.count > 0x7fffffff) return BSFP8_ERR_SHAPE;
  a.segments = (int)seg.count;
  a.tiles = (int)seg.tiles;
  const dim3 grid((unsigned)(rows * seg.count)), block(kTThreads);
  auto go = [&](auto weighted, auto f4) {
    constexpr bool W = decltype(weighted)::value, F4 = decltype(f4)::value;
    if (!turns) hipLaunchKernelGGL((dispatch_quantize_kernel<W, F4, 0>), grid, block, 0, stream, a);
    else if (E <= 64) hipLaunchKernelGGL((dispatch_quantize_kernel<W, F4, 1>), grid, block, 0, stream, a);
    else if (E <= 256) hipLaunchKernelGGL((dispatch_quantize_kernel<W, F4, 4>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((dispatch_quantize_kernel<W, F4, 16>), grid, block, 0, stream, a);
  };
  const std::integral_constant<bool, true> yes;
  const std::integral_constant<bool, false> no;
  const bool f4 = recipe == BSFP8_RECIPE_MXFP4_1X32_E8M0;
  if (weights != nullptr && f4) go(yes, yes);
  else if (weights != nullptr) go(yes, no);
  else if (f4) go(no, yes);
  else go(no, no);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
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
  const int64_t parts = token_segments(token_row_tiles(R, E), (F + kTCols - 1) / kTCols).count;
  hipLaunchKernelGGL(token_dprobs_kernel, dim3((unsigned)((R + 255) / 256)), dim3(256), 0, stream, workspace, R, parts,
                     splits, E, dprobs);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
