// The router: each token's top_k experts with their probabilities, the sums of the scores, and the gradient of both
// (gfx950).  include/bsfp8.h states the formulas.
//
// A token's logits lie in the registers of 16 lanes (up to 256 experts) or of a wave (up to 1024), V = 1 to 16
// consecutive experts a lane, so that a lane's logits are one wide load and its reductions over a token are moves within
// a row of 16 lanes.  Keys are compared as unsigned numbers whose order is that of the keys (NaN highest, the masked
// lowest, then 0 for the taken).  A choice takes one reduction for the largest key, and where two of a token's keys are
// equal one more for the lowest expert that has it.
//
// What bounds them: 131072 tokens of 128 logits in fp32 are 67 MB, 11 us at 6.2 TB/s.  The choices' comparisons are about
// 35 vector instructions a choice for 4 tokens, so the forward pass is bound by them: 40 us with the sums of the scores, 31
// without, 49 by sigmoid scores with a bias
// (66 with both reductions at every choice; 49 with the scoring and the choices per lane looked up while running, 44 with
// what is taken compared again and not kept as lane masks).  The gradient reads and writes 134 MB, 22 us; a token's
// loads hang on each other (its choices, then their logits), so the next token's are asked for ahead and the chosen
// logits of a row that the lanes hold come from LDS: 33 us (58 without).
#include <math.h>

#include <type_traits>

#include "act_math.hpp"
#include "common.hpp"
#include "row_io.hpp"
#include "token_layout.hpp"

namespace bsfp8 {

struct RouteArgs {
  const void* logits;
  int64_t T;
  int E, K;
  const float* bias;
  int renormalize;
  float scale;
  float* probs;        // forward out; gradient: dprobs in
  int32_t* experts;
  float* partial;      // forward: [blocks][E] sums of the scores, or NULL
  const float* dsum;   // gradient: dscore_sum, or NULL
  void* dlogits;
};

// Reductions over the G lanes of a token; every lane gets the result.
template <int G, class Op>
__device__ __forceinline__ uint32_t over_token(uint32_t v, Op op) {
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));  // the row of 16, turned by 8
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
  if constexpr (G == 64) {
    v = op(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    v = op(v, (uint32_t)__shfl_xor((int)v, 32, 64));
  }
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t max_over(uint32_t v) {
  return over_token<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int G>
__device__ __forceinline__ uint32_t min_over(uint32_t v) {
  return over_token<G>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int G>
__device__ __forceinline__ float sum_over(float v) {
  return __uint_as_float(over_token<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int G>
__device__ __forceinline__ float fmax_over(float v) {
  return __uint_as_float(over_token<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}

// A key as an unsigned number of the same order: +0 where it was -0, NaN above all; -infinity, the key of the masked, is
// kMasked and the lowest, so that 0 stands for the taken.
constexpr uint32_t kMasked = 0x007fffffu;
__device__ __forceinline__ uint32_t ordered(float key) {
  const uint32_t b = __float_as_uint(key + 0.0f);
  return key != key ? 0xffffffffu : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// 1 / (1 + 2^(-l log2 e)) by the stated steps, and 1 - it without the cancellation.
__device__ __forceinline__ float sigmoid_stated(float l, float* other = nullptr) {
  const float t = exp2_stated(-l * 1.44269502f);
  const float s = recip_rn(1.0f + t);
  if (other != nullptr) *other = t * s;
  return s;
}

// exp(x) for x <= 0: the hardware's 2^y, y = x log2(e) rounded, times 1 + (x - y ln 2), which makes good what the rounding took
// (up to |x| 2^-24 of the result, as much as that of x = l - m itself).  What remains is 2 ulp at |x| = 80; below 2^-126 it
// is 0.  A NaN stays one, minus infinity gives 0.
__device__ __forceinline__ float exp_neg(float x) {
  x = __builtin_elementwise_maximum(x, -150.0f);
  const float y = x * 1.44269504f, t = __builtin_amdgcn_exp2f(y);
  return __builtin_fmaf(t, __builtin_fmaf(-y, 0.693147182f, x), t);
}

// V values of a row from e0 on; past its end: -infinity.
template <int V, class T>
__device__ __forceinline__ void load_logits(const T* row, int e0, int E, float (&l)[V]) {
  if (e0 + V <= E) {
    T t[V];
    __builtin_memcpy(t, row + e0, sizeof(t));
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = to_f32(t[v]);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? to_f32(row[e0 + v]) : -INFINITY;
  }
}

// The scores of a token's V logits a lane: s, and for the sigmoid 1 - s (FULL gradients).
template <int G, int V, bool SIGMOID>
__device__ __forceinline__ void scores_of(const float (&l)[V], float (&s)[V], float* other = nullptr) {
  if constexpr (SIGMOID) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o;
      s[v] = sigmoid_stated(l[v], &o);
      if (l[v] == -INFINITY) s[v] = 0.0f;
      if (other != nullptr) other[v] = o;
    }
    return;
  }
  float m = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
  m = fmax_over<G>(m);
  if (m == -INFINITY) m = 0.0f;  // every expert masked: the scores are 0
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = exp_neg(l[v] - m);
    sum += s[v];
  }
  sum = sum_over<G>(sum);
  const float inv = sum == 0.0f ? 0.0f : recip_rn(sum);  // (the largest counts 1 in it)
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] *= inv;
}

// The scores of a lane's P chosen over what they are divided by: ph, and for the sigmoid 1 - s.
template <int G, int P, bool SIGMOID>
__device__ __forceinline__ void chosen_scores(const float (&l)[P], const int (&e)[P], float (&ph)[P], float (&other)[P]) {
  float m = -INFINITY, sum = 0.0f;
  if constexpr (!SIGMOID) {
#pragma unroll
    for (int i = 0; i < P; ++i) m = fmaxf(m, l[i]);
    m = fmax_over<G>(m);
    if (m == -INFINITY) m = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    ph[i] = SIGMOID ? sigmoid_stated(l[i], &other[i]) : expf(l[i] - m);
    if (e[i] < 0 || l[i] == -INFINITY) ph[i] = 0.0f;
    sum += ph[i];
  }
  sum = sum_over<G>(sum);
  const float inv = sum == 0.0f ? 0.0f : SIGMOID ? 1.0f / sum : recip_rn(sum);
#pragma unroll
  for (int i = 0; i < P; ++i) ph[i] *= inv;
}

// P: a lane's choices j = lane, lane + G, ... of a token.
template <class T, int G, int V, int P, bool SIGMOID>
__global__ __launch_bounds__(256) void route_topk_kernel(RouteArgs a) {
  __shared__ float sums[256 / G][G * V + 1];
  __shared__ int taken[256 / G][BSFP8_MAX_TOP_K];
  const int lane = threadIdx.x & (G - 1), group = threadIdx.x / G, e0 = lane * V;
  float total[V];
#pragma unroll
  for (int v = 0; v < V; ++v) total[v] = 0.0f;
  // every lane of a wave walks as many tokens, so that the moves between lanes find them all
  for (int64_t t0 = (int64_t)blockIdx.x * (256 / G); t0 < a.T; t0 += (int64_t)gridDim.x * (256 / G)) {
    const bool live = t0 + group < a.T;
    const int64_t t = live ? t0 + group : a.T - 1;
    const T* row = (const T*)a.logits + t * a.E;
    float l[V], s[V];
    load_logits<V>(row, e0, a.E, l);
    if (SIGMOID || a.partial != nullptr) scores_of<G, V, SIGMOID>(l, s);
    if (a.partial != nullptr && live) {
#pragma unroll
      for (int v = 0; v < V; ++v) total[v] += s[v];
    }
    uint32_t u[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float key = SIGMOID ? s[v] : l[v];
      if (a.bias != nullptr && e0 + v < a.E) key += a.bias[e0 + v];
      if (SIGMOID || a.bias != nullptr) key = l[v] == -INFINITY ? -INFINITY : key;
      u[v] = ordered(key);
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + i * G < a.K) taken[group][lane + i * G] = -1;
    for (int j = 0; j < a.K; ++j) {
      uint32_t best = u[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = u[v] > best ? u[v] : best;
      best = max_over<G>(best);
      const bool open_ = best > kMasked;
      const uint32_t key = open_ ? best : 0xfffffffeu;  // (a number that no key has)
      // one of a token's keys is the largest, unless two are equal: then the lowest expert's is taken
      uint64_t hit[V];
      int found = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        hit[v] = __ballot(u[v] == key);
        found += __popcll(hit[v]);
      }
      if (found * G != __popcll(__ballot(open_))) {
        uint32_t e = 0xffffffffu;
#pragma unroll
        for (int v = V - 1; v >= 0; --v) e = u[v] == key ? (uint32_t)(e0 + v) : e;
        e = min_over<G>(e);
#pragma unroll
        for (int v = 0; v < V; ++v) hit[v] = __ballot(e == (uint32_t)(e0 + v));
      }
      uint64_t lanes = hit[0];
      int at = e0;
#pragma unroll
      for (int v = 1; v < V; ++v) {
        lanes |= hit[v];
        at = __builtin_amdgcn_inverse_ballot_w64(hit[v]) ? e0 + v : at;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) u[v] = __builtin_amdgcn_inverse_ballot_w64(hit[v]) ? 0u : u[v];
      if (__builtin_amdgcn_inverse_ballot_w64(lanes)) taken[group][j] = at;
    }
    wave_lds_order();
    int mine[P];
#pragma unroll
    for (int i = 0; i < P; ++i) mine[i] = lane + i * G < a.K ? taken[group][lane + i * G] : -1;
    wave_lds_order();
    float p[P], other[P], x[P];
    // (the chosen logits are read again: a lane holds other experts' than those it writes)
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = mine[i] >= 0 ? to_f32(row[mine[i]]) : -INFINITY;
    if (a.renormalize) {
      chosen_scores<G, P, SIGMOID>(x, mine, p, other);
    } else {
      float m = l[0], sum = 0.0f;
      if constexpr (!SIGMOID) {
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
        m = fmax_over<G>(m);
        if (m == -INFINITY) m = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += exp_neg(l[v] - m);
        sum = sum_over<G>(sum);
      }
#pragma unroll
      for (int i = 0; i < P; ++i)
        p[i] = mine[i] < 0 ? 0.0f : SIGMOID ? sigmoid_stated(x[i]) : exp_neg(x[i] - m) * recip_rn(sum);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int j = lane + i * G;
      if (live && j < a.K) {
        a.experts[t * a.K + j] = mine[i];
        a.probs[t * a.K + j] = p[i] * a.scale;
      }
    }
  }
  if (a.partial != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v) sums[group][e0 + v] = total[v];
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 256) {
      float s = 0.0f;
      for (int g = 0; g < 256 / G; ++g) s += sums[g][e];
      a.partial[(int64_t)blockIdx.x * a.E + e] = s;
    }
  }
}

// The partial sums of 16 experts added in a fixed order: a workgroup's 64 rows of 16 lanes have every 64th each, 8 loads in
// flight; then the 4 rows of a wave, then the waves.
__global__ __launch_bounds__(1024) void route_sum_kernel(const float* partial, int blocks, int E, float* out) {
  __shared__ float sums[16][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x * 16 + (lane & 15);
  float s = 0.0f;
  if (e < E) {
    for (int b0 = wave * 4 + (lane >> 4); b0 < blocks; b0 += 8 * 64) {
      float n[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) n[u] = b0 + 64 * u < blocks ? partial[(int64_t)(b0 + 64 * u) * E + e] : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += n[u];
    }
  }
  s += __shfl_xor(s, 16, 64);
  s += __shfl_xor(s, 32, 64);
  if (lane < 16) sums[wave][lane] = s;
  __syncthreads();
  if (threadIdx.x < 16 && e < E) {
    s = 0.0f;
    for (int w = 0; w < 16; ++w) s += sums[w][lane];
    out[e] = s;
  }
}

// FULL: every score is needed (the scores' sums have a gradient, or the softmax is not renormalized).
template <class T, int G, int V, int P, bool SIGMOID, bool FULL>
__global__ __launch_bounds__(256) void route_topk_grad_kernel(RouteArgs a) {
  __shared__ int at_sm[256 / G][BSFP8_MAX_TOP_K];
  __shared__ float part_sm[256 / G][BSFP8_MAX_TOP_K];
  __shared__ __attribute__((aligned(16))) float row_sm[256 / G][G * V];
  const int lane = threadIdx.x & (G - 1), group = threadIdx.x / G, e0 = lane * V;
  float dsum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dsum[v] = FULL && a.dsum != nullptr && e0 + v < a.E ? a.dsum[e0 + v] : 0.0f;
  // a token's logits, choices and gradients, asked for before the token before it is worked on
  float next_l[V], next_g[P];
  int next_e[P];
  const int64_t step = (int64_t)gridDim.x * (256 / G);
  auto ask = [&](int64_t t0) {
    const int64_t t = t0 + group < a.T ? t0 + group : a.T - 1;
    if constexpr (FULL) load_logits<V>((const T*)a.logits + t * a.E, e0, a.E, next_l);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int j = lane + i * G;
      next_e[i] = j < a.K ? a.experts[t * a.K + j] : -1;
      next_g[i] = j < a.K ? a.probs[t * a.K + j] : 0.0f;
    }
  };
  ask((int64_t)blockIdx.x * (256 / G));
  for (int64_t t0 = (int64_t)blockIdx.x * (256 / G); t0 < a.T; t0 += step) {
    const bool live = t0 + group < a.T;
    const int64_t t = live ? t0 + group : a.T - 1;
    const T* row = (const T*)a.logits + t * a.E;
    float l[V], s[V], other[V], g[P];
    int e[P];
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = FULL ? next_l[v] : 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      e[i] = next_e[i] < a.E ? next_e[i] : -1;
      g[i] = e[i] >= 0 ? next_g[i] * a.scale : 0.0f;
    }
    ask(t0 + step);
    float* to = &row_sm[group][e0];
    const bool chosen_only = a.renormalize || SIGMOID;
    // the chosen logits: from LDS where the lanes hold the row anyway
    float x[P];
    if constexpr (FULL) {
      if (chosen_only) {
#pragma unroll
        for (int v = 0; v < V; ++v) to[v] = l[v];
        wave_lds_order();
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = e[i] >= 0 ? row_sm[group][e[i]] : -INFINITY;
        wave_lds_order();
      }
      scores_of<G, V, SIGMOID>(l, s, other);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = e[i] >= 0 ? to_f32(row[e[i]]) : -INFINITY;
    }
    // what a choice gives to its expert: at the logit, or (softmax without renormalize) at the score
    const bool at_score = !a.renormalize && !SIGMOID;
    if (a.renormalize) {
      float ph[P], rest[P], mean = 0.0f;
      chosen_scores<G, P, SIGMOID>(x, e, ph, rest);
#pragma unroll
      for (int i = 0; i < P; ++i) mean += g[i] * ph[i];
      mean = sum_over<G>(mean);
#pragma unroll
      for (int i = 0; i < P; ++i) g[i] = e[i] < 0 ? 0.0f : ph[i] * (g[i] - mean) * (SIGMOID ? rest[i] : 1.0f);
    } else if constexpr (SIGMOID) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float rest;
        const float sc = sigmoid_stated(x[i], &rest);
        g[i] = x[i] == -INFINITY ? 0.0f : g[i] * sc * rest;
      }
    }
    // the choices' parts at their experts' places.  Each choice writes its number there first: one that finds another's
    // shares its expert, and the parts are then added choice by choice, in order
    float d[V];
#pragma unroll
    for (int v = 0; v < V; ++v) to[v] = 0.0f;
    wave_lds_order();
    bool alone = true;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (e[i] >= 0) row_sm[group][e[i]] = __int_as_float(lane + i * G);
    wave_lds_order();
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (e[i] >= 0) alone &= __float_as_int(row_sm[group][e[i]]) == lane + i * G;
    wave_lds_order();
    if (__ballot(!alone) == 0) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (e[i] >= 0) row_sm[group][e[i]] = g[i];
      wave_lds_order();
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = to[v];
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int j = lane + i * G;
        if (j < a.K) {
          at_sm[group][j] = e[i];
          part_sm[group][j] = g[i];
        }
      }
      wave_lds_order();
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = 0.0f;
      for (int j = 0; j < a.K; ++j) {
        const int x = at_sm[group][j] - e0;
        const float y = part_sm[group][j];
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] += x == v ? y : 0.0f;
      }
    }
    wave_lds_order();
    if constexpr (FULL) {
      float back[V], mean = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        back[v] = dsum[v];
        if (at_score) {
          back[v] += d[v];
          d[v] = 0.0f;
        }
        mean += s[v] == 0.0f ? 0.0f : back[v] * s[v];
      }
      if constexpr (SIGMOID) {
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] += s[v] == 0.0f ? 0.0f : back[v] * s[v] * other[v];
      } else {
        mean = sum_over<G>(mean);
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] += s[v] == 0.0f ? 0.0f : s[v] * (back[v] - mean);
      }
    }
    if (live) {
      T* out = (T*)a.dlogits + t * a.E + e0;
      T o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) from_f32(d[v], o[v]);
      if (e0 + V <= a.E) {
        __builtin_memcpy(out, o, sizeof(o));
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (e0 + v < a.E) out[v] = o[v];
      }
    }
  }
}

// f with the lanes per token, the experts and the choices per lane that E and K take, and the scoring.  K is at most E: one
// expert a lane leaves one choice a lane, and a wave's lanes have more than 4 experts.
template <class F>
static void for_shape(int E, int K, bool sigmoid, F f) {
  auto scoring = [&](auto g, auto v, auto p) {
    if (sigmoid) f(g, v, p, std::true_type());
    else f(g, v, p, std::false_type());
  };
  auto choices = [&](auto g, auto v) {
    constexpr int G = decltype(g)::value;
    if constexpr (G < BSFP8_MAX_TOP_K && decltype(v)::value > 1) {
      if (K > G) {
        scoring(g, v, std::integral_constant<int, BSFP8_MAX_TOP_K / G>());
        return;
      }
    }
    scoring(g, v, std::integral_constant<int, 1>());
  };
  if (route_lanes(E) == 16) {
    const std::integral_constant<int, 16> g;
    if (E <= 16) choices(g, std::integral_constant<int, 1>());
    else if (E <= 32) choices(g, std::integral_constant<int, 2>());
    else if (E <= 64) choices(g, std::integral_constant<int, 4>());
    else if (E <= 128) choices(g, std::integral_constant<int, 8>());
    else choices(g, std::integral_constant<int, 16>());
  } else {
    const std::integral_constant<int, 64> g;
    if (E <= 512) choices(g, std::integral_constant<int, 8>());
    else choices(g, std::integral_constant<int, 16>());
  }
}

int launch_route_topk(const void* logits, bool f32, int64_t T, int E, int K, bool sigmoid, const float* bias,
                      int renormalize, float scale, float* probs, int32_t* experts, float* score_sum, float* workspace,
                      hipStream_t stream) {
  const int64_t blocks = route_blocks(T, E);
  if (blocks > 0) {
    const RouteArgs a{logits, T, E, K, bias, renormalize, scale, probs, experts,
                      score_sum != nullptr ? workspace : nullptr, nullptr, nullptr};
    const dim3 grid((unsigned)blocks), block(256);
    for_shape(E, K, sigmoid, [&](auto g, auto v, auto p, auto sg) {
      constexpr int G = decltype(g)::value, V = decltype(v)::value, P = decltype(p)::value;
      constexpr bool S = decltype(sg)::value;
      if (f32) hipLaunchKernelGGL((route_topk_kernel<float, G, V, P, S>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((route_topk_kernel<uint16_t, G, V, P, S>), grid, block, 0, stream, a);
    });
    if (hipGetLastError() != hipSuccess) return BSFP8_ERR_LAUNCH;
  }
  if (score_sum == nullptr) return BSFP8_OK;
  hipLaunchKernelGGL(route_sum_kernel, dim3((unsigned)((E + 15) / 16)), dim3(1024), 0, stream, workspace, (int)blocks, E,
                     score_sum);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

int launch_route_topk_grad(const float* dprobs, const void* logits, bool f32, const int32_t* experts, int64_t T, int E,
                           int K, bool sigmoid, int renormalize, float scale, const float* dsum, void* dlogits,
                           hipStream_t stream) {
  const RouteArgs a{logits, T, E, K, nullptr, renormalize, scale, const_cast<float*>(dprobs),
                    const_cast<int32_t*>(experts), nullptr, dsum, dlogits};
  const bool full = dsum != nullptr || (!sigmoid && !renormalize);
  const dim3 grid((unsigned)route_blocks(T, E, true)), block(256);
  for_shape(E, K, sigmoid, [&](auto g, auto v, auto p, auto sg) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value, P = decltype(p)::value;
    constexpr bool S = decltype(sg)::value;
    auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    if (f32 && full) launch(route_topk_grad_kernel<float, G, V, P, S, true>);
    else if (f32) launch(route_topk_grad_kernel<float, G, V, P, S, false>);
    else if (full) launch(route_topk_grad_kernel<uint16_t, G, V, P, S, true>);
    else launch(route_topk_grad_kernel<uint16_t, G, V, P, S, false>);
  });
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
