// Rows of fp32 or bf16 moved 8 elements at a time, and sums over a wave: what the kernels share that walk
// rows of any length and alignment.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace bsfp8 {

__device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float to_f32(float f) { return f; }
__device__ __forceinline__ void from_f32(float f, uint16_t& o) { o = f32_to_bf16(f); }
__device__ __forceinline__ void from_f32(float f, float& o) { o = f; }

// 8 elements as they lie in memory: n of them exist at p, the others read as 0; any alignment of the
// element's size.
template <class T>
struct Raw8;
template <>
struct Raw8<float> {
  float t[8];
  __device__ __forceinline__ void load_all(const float* p) { __builtin_memcpy(t, p, sizeof(t)); }
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n >= 8) {
      __builtin_memcpy(t, p, sizeof(t));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = i < n ? p[i] : 0.0f;
    }
  }
  __device__ __forceinline__ float operator[](int i) const { return t[i]; }
};
template <>
struct Raw8<uint16_t> {
  uint32_t w[4];  // pairs, so that the compiler keeps them in four registers
  __device__ __forceinline__ void load_all(const uint16_t* p) { __builtin_memcpy(w, p, sizeof(w)); }
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (n >= 8) {
      __builtin_memcpy(w, p, sizeof(w));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ float operator[](int i) const { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
};
template <class T>
__device__ __forceinline__ void load8(const T* p, int n, float* v) {
  Raw8<T> r;
  r.load(p, n);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r[i];
}
// 8 elements past the caches, any alignment of the element's size.
__device__ __forceinline__ void stream8(float* p, const float* t) {
  typedef float V __attribute__((ext_vector_type(4), aligned(4)));
  __builtin_nontemporal_store(V{t[0], t[1], t[2], t[3]}, (V*)p);
  __builtin_nontemporal_store(V{t[4], t[5], t[6], t[7]}, (V*)p + 1);
}
__device__ __forceinline__ void stream8(uint16_t* p, const uint16_t* t) {
  typedef uint16_t V __attribute__((ext_vector_type(8), aligned(2)));
  __builtin_nontemporal_store(V{t[0], t[1], t[2], t[3], t[4], t[5], t[6], t[7]}, (V*)p);
}
template <class T>
__device__ __forceinline__ void store8(T* p, int n, const float* v, bool past_caches = false) {
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) from_f32(v[i], t[i]);
  if (n >= 8) {
    if (past_caches) stream8(p, t);
    else __builtin_memcpy(p, t, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = t[i];
  }
}

// Sum of a wave's 64 values, in lane 63: adds with data-parallel lane moves (a shuffle through LDS takes ten
// times as long).
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](auto ctrl, int rows) {
    constexpr int C = decltype(ctrl)::value;
    const int m = rows == 0xf ? __builtin_amdgcn_update_dpp(0, __float_as_int(v), C, 0xf, 0xf, false)
                              : rows == 0xa ? __builtin_amdgcn_update_dpp(0, __float_as_int(v), C, 0xa, 0xf, false)
                                            : __builtin_amdgcn_update_dpp(0, __float_as_int(v), C, 0xc, 0xf, false);
    v += __int_as_float(m);
  };
  add(std::integral_constant<int, 0x111>(), 0xf);  // the lane 1, 2, 4, 8 below in its row of 16 (0 where none)
  add(std::integral_constant<int, 0x112>(), 0xf);
  add(std::integral_constant<int, 0x114>(), 0xf);
  add(std::integral_constant<int, 0x118>(), 0xf);
  add(std::integral_constant<int, 0x142>(), 0xa);  // lane 15 of the row below, into rows 1 and 3
  add(std::integral_constant<int, 0x143>(), 0xc);  // lane 31, into rows 2 and 3
  return v;
}

// Inclusive sum over a wave, with data-parallel lane moves.
__device__ __forceinline__ int wave_scan32(int v) {
  auto add = [&](auto ctrl, auto rows) {
    v += __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
  };
  using std::integral_constant;
  add(integral_constant<int, 0x111>(), integral_constant<int, 0xf>());  // 1, 2, 4, 8 lanes below in the row of 16
  add(integral_constant<int, 0x112>(), integral_constant<int, 0xf>());
  add(integral_constant<int, 0x114>(), integral_constant<int, 0xf>());
  add(integral_constant<int, 0x118>(), integral_constant<int, 0xf>());
  add(integral_constant<int, 0x142>(), integral_constant<int, 0xa>());  // row 0's total to row 1, 2's to 3
  add(integral_constant<int, 0x143>(), integral_constant<int, 0xc>());  // the first half's total to the second
  return v;
}

}  // namespace bsfp8
