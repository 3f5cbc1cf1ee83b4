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
// u's codes span 2^18, the upper 2^15 of it with 4 significant bits each, and u is what the update
// divides by; a u below the smallest code is raised to it, so that no update is divided by nothing.  A
// scale in fp32 rather than a power of two: the block's largest state is then always the code 448
// and decays with the scale step by step, where a power-of-two scale would leave the code itself
// to decay.  The update itself uses m and u before they are rounded.
//
// Rounding of the 8-bit states.  To nearest, a code that another element's scale holds up stays where
// it is as long as a step changes its state by less than half a code's step, 3 to 6 percent: u, which
// loses 1 - sqrt(beta2) a step (2.5 percent at 0.95, 0.05 at 0.999), never falls again, and m's lowest
// codes do not either.  Stochastic rounding goes up with the probability of the part cut off: the
// expected state is the unrounded one at any beta.  Its bits are SplitMix64 outputs (Steele, Lea and
// Flood 2014, a bijective mix of a counter) of the caller's seed, the step, the tensor's place in the
// plan and the element, 20 per state: the same call gives the same bits on any launch shape.  A graph
// replayed with a new step_dev takes new ones.
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
  uint64_t seed;  // stochastic rounding
  int64_t num_chunks;
  int per;  // chunks per workgroup
};

__device__ __forceinline__ float val(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float val(float f) { return f; }
__device__ __forceinline__ void put(float f, uint16_t& o) { o = f32_to_bf16(f); }
__device__ __forceinline__ void put(float f, float& o) { o = f; }

// The plan's pointers come from memory, where the compiler cannot know that they are global ones and would use
// flat accesses (which also occupy the LDS counter): T* as a global pointer.
template <class T>
using Global = __attribute__((address_space(1))) T*;
template <class T>
__device__ __forceinline__ Global<T> global(const void* p) {
  return (Global<T>)(uintptr_t)p;
}

// N bytes, any alignment of their elements; NT: past the caches (nothing here is read again before the step
// is over).
template <bool NT, class V>
__device__ __forceinline__ V load_vec(Global<const V> p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool NT, class V>
__device__ __forceinline__ void store_vec(Global<V> p, V v) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <class T>
struct Vec4 {
  typedef T type __attribute__((ext_vector_type(4), aligned(sizeof(T))));
};

// 4 elements at p, n of them live (the rest read as 0); any alignment of the element's size.
template <bool NT, class T>
__device__ __forceinline__ void load4(Global<const T> p, int n, float* v) {
  typename Vec4<T>::type t = {0, 0, 0, 0};
  if (n >= 4) {
    t = load_vec<NT, typename Vec4<T>::type>((Global<const typename Vec4<T>::type>)p);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) t[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = val((T)t[i]);
}
template <bool NT, class T>
__device__ __forceinline__ void store4(Global<T> p, int n, const float* v) {
  T t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) put(v[i], t[i]);
  if (n >= 4) {
    store_vec<NT, typename Vec4<T>::type>((Global<typename Vec4<T>::type>)p,
                                         typename Vec4<T>::type{t[0], t[1], t[2], t[3]});
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = t[i];
  }
}
typedef uint32_t u32_any __attribute__((aligned(1)));
// 4 e4m3 codes
template <bool NT>
__device__ __forceinline__ void load4_codes(Global<const uint8_t> p, int n, float* v) {
  uint32_t w = 0;
  if (n >= 4) {
    w = load_vec<NT, u32_any>((Global<const u32_any>)p);
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
template <bool NT>
__device__ __forceinline__ void store4_codes(Global<uint8_t> p, int n, const float* v) {
  const uint32_t w = e4m3x4(v[0], v[1], v[2], v[3]);
  if (n >= 4) {
    store_vec<NT, u32_any>((Global<u32_any>)p, w);
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

__device__ __forceinline__ uint64_t mix64(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
  z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
  return z ^ (z >> 31);
}
constexpr uint64_t kWeyl = 0x9e3779b97f4a7c15ull;  // the counter's stride (2^64 over the golden ratio, odd)

// w, in units of its block's scale, to a neighbouring e4m3 value, away from zero with the probability of its distance
// from the one below, by 20 random bits: they are added to the 20 of the mantissa that go, and carry with just
// that probability.  Below 2^-6, where the codes are multiples of 2^-9, 2^-6 is added for it, whose mantissa ends there.
// 448, and what is not a number, stay as they are.
__device__ __forceinline__ float round_by(float w, uint32_t r) {
  const float a = fabsf(w), low = a < 0x1p-6f ? 0x1p-6f : 0.0f;
  const float q = __uint_as_float((__float_as_uint(a + low) + r) & 0xfff00000u) - low;
  return a < 448.0f ? copysignf(q, w) : w;
}

// fp32 states: 512 threads, 4 elements each, one chunk per workgroup.  8-bit states: 256 threads, 8 elements
// each, up to 4 chunks per workgroup, which spares most of the scalars' fp64 arithmetic (the larger share
// where an element moves 18 bytes, not 30).  376 million elements (fp32 parameters and gradients, bf16
// copies), fp32 / 8-bit states: 1.81 / 1.10 ms = 6.2 TB/s, what an elementwise pass over large arrays reaches
// (boxes differ: 1.99 / 1.26 ms on others); through the caches, with flat accesses and one chunk of 256
// threads 2.13 / 1.38 ms.  Stochastic rounding: 1271 us where nearest takes 1268; without copies, and with bf16
// parameters and gradients, where an element moves 10 bytes and the arithmetic bounds, 1043 to 843.
template <bool Q8>
constexpr int adam_threads() {
  return Q8 ? 256 : 512;
}

// SR: stochastic rounding of 8-bit states.
template <class PT, class GT, bool Q8, bool NT, bool SR>
__global__ __launch_bounds__(adam_threads<Q8>()) void adamw_kernel(AdamArgs a) {
  constexpr int kThreads = adam_threads<Q8>();
  if (a.noop_flag != nullptr && *a.noop_flag != 0.0f) return;
  const float gs = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
  const double t = a.step_dev != nullptr ? (double)*a.step_dev : a.step;
  const double c1 = 1.0 - exp(t * a.log_beta1), c2 = 1.0 - exp(t * a.log_beta2);
  const float root = (float)(1.0 / sqrt(c2));
  const uint64_t step_key = SR ? mix64(a.seed + kWeyl * (uint64_t)(int64_t)t) : 0;
  uint64_t tensor_key = 0;
  const int64_t from = (int64_t)blockIdx.x * a.per;
  const int64_t to = from + a.per < a.num_chunks ? from + a.per : a.num_chunks;
  int tensor = -1;
  AdamTensor tn{};
  float keep = 0.0f, step_size = 0.0f;
  for (int64_t c = from; c < to; ++c) {
    const AdamChunk ch = a.chunks[c];
    if (ch.tensor != tensor) {
      tensor = ch.tensor;
      tn = a.tensors[tensor];
      if constexpr (SR) tensor_key = mix64(step_key + kWeyl * (uint64_t)tensor);
      const double lr = (a.lr_dev != nullptr ? (double)*a.lr_dev : a.lr) * (double)tn.lr_scale;
      keep = (float)(1.0 - lr * a.decay * (double)tn.decay_scale);
      step_size = (float)(lr / c1);
    }
    const Global<PT> param = global<PT>(tn.param);
    const Global<const GT> grad = global<const GT>(tn.grad);
    const Global<uint16_t> copy = global<uint16_t>(tn.copy);
    const Global<uint8_t> m8 = global<uint8_t>(tn.exp_avg), v8 = global<uint8_t>(tn.exp_avg_sq);
    const Global<float> m32 = global<float>(tn.exp_avg), v32 = global<float>(tn.exp_avg_sq);
    const Global<float> m_scale = global<float>(tn.exp_avg_scale), v_scale = global<float>(tn.exp_avg_sq_scale);
    const int64_t first = (int64_t)ch.index * kAdamChunk;
#pragma unroll
    for (int u = 0; u < kAdamChunk / (4 * kThreads); ++u) {
      const int64_t at = first + 4 * (u * kThreads + (int)threadIdx.x);
      const int64_t left = tn.numel - at;
      const int n = left > 4 ? 4 : (int)left;  // <= 0: nothing of this lane's is live
      float p[4], g[4], m[4], v[4], root_v[4];
      load4<NT, PT>(param + at, n, p);
      load4<NT, GT>(grad + at, n, g);
      if constexpr (Q8) {
        const int64_t blk = at / 128;
        load4_codes<NT>(m8 + at, n, m);
        load4_codes<NT>(v8 + at, n, v);
        const float sm = n > 0 ? m_scale[blk] : 0.0f, sv = n > 0 ? v_scale[blk] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          m[i] *= sm;
          v[i] *= sv;
          v[i] *= v[i];
        }
      } else {
        load4<NT, float>(m32 + at, n, m);
        load4<NT, float>(v32 + at, n, v);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float gi = g[i] * gs;
        m[i] = m[i] * a.beta1 + gi * a.one_minus_beta1;
        v[i] = v[i] * a.beta2 + gi * gi * a.one_minus_beta2;
        root_v[i] = sqrtf(v[i]);
        p[i] = p[i] * keep - m[i] / (root_v[i] * root + a.eps) * step_size;
      }
      store4<NT, PT>(param + at, n, p);
      if (tn.copy != nullptr) store4<NT, uint16_t>(copy + at, n, p);
      if constexpr (Q8) {
        // lanes past the tensor's end hold zeros, which leave their block's largest as it is
        const float sm = block_scale(m), sv = block_scale(root_v);
        const float im = 1.0f / sm, iv = 1.0f / sv;
        bool nonzero[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          nonzero[i] = root_v[i] > 0.0f;
          m[i] *= im;
          root_v[i] *= iv;
        }
        if constexpr (SR) {
          const uint64_t key = tensor_key + kWeyl * (uint64_t)(at / 2);
          const uint64_t bits_m = mix64(key), bits_v = mix64(key + kWeyl);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // (of a 32-bit word for two states; the 8 bits that they share are the lowest of one and the highest of the other)
            const uint32_t wm = (uint32_t)(bits_m >> (32 * (i >> 1))), wv = (uint32_t)(bits_v >> (32 * (i >> 1)));
            m[i] = round_by(m[i], i & 1 ? wm >> 12 : wm & 0xfffffu);
            root_v[i] = round_by(root_v[i], i & 1 ? wv >> 12 : wv & 0xfffffu);
          }
        }
        // A second state that is not zero keeps a code that is not: m, which has a scale of its own, may keep one
        // there, and the next step divides it by this. 
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (nonzero[i] && root_v[i] < 0x1p-9f) root_v[i] = 0x1p-9f;
        store4_codes<NT>(m8 + at, n, m);
        store4_codes<NT>(v8 + at, n, root_v);
        if ((threadIdx.x & 31) == 0 && n > 0) {
          m_scale[at / 128] = sm;
          v_scale[at / 128] = sv;
        }
      } else {
        store4<NT, float>(m32 + at, n, m);
        store4<NT, float>(v32 + at, n, v);
      }
    }
  }
}

// Consecutive chunks per workgroup: one where the chip still has room for more workgroups (a small step's
// time is one chunk's latency).
static int adam_chunks_per_block(bool q8, int64_t chunks) {
  const int64_t per = chunks / (256 * 8), most = q8 ? 4 : 1;
  return (int)(per < 1 ? 1 : per > most ? most : per);
}
// Steps from this many chunks on go past the caches: 8192 chunks are 16 million elements, 300 to 500 MB, as
// much as the last-level cache holds; below, the parameters may still be there when the next pass reads them
// (270,000 elements: 4.9 us through the caches, 5.7 past them).
constexpr int64_t kAdamStreamChunks = 8192;

int launch_adamw(const void* plan, int32_t num_tensors, int64_t chunks, int p_f32, int g_f32, int q8, double lr,
                 double beta1, double beta2, double eps, double decay, int64_t step, const float* lr_dev,
                 const int32_t* step_dev, const float* grad_scale, const float* noop_flag, const uint64_t* seed,
                 hipStream_t stream) {
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
  a.seed = seed != nullptr ? *seed : 0;
  a.grad_scale = grad_scale;
  a.noop_flag = noop_flag;
  a.num_chunks = chunks;
  a.per = adam_chunks_per_block(q8, chunks);
  const dim3 grid((unsigned)((chunks + a.per - 1) / a.per));
  const bool nt = chunks >= kAdamStreamChunks;
  auto go = [&](auto p, auto g) {
    using P = decltype(p);
    using G = decltype(g);
    auto run = [&](auto kernel, int threads) { hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, stream, a); };
    if (!q8) run(nt ? adamw_kernel<P, G, false, true, false> : adamw_kernel<P, G, false, false, false>, adam_threads<false>());
    else if (seed == nullptr)
      run(nt ? adamw_kernel<P, G, true, true, false> : adamw_kernel<P, G, true, false, false>, adam_threads<true>());
    else run(nt ? adamw_kernel<P, G, true, true, true> : adamw_kernel<P, G, true, false, true>, adam_threads<true>());
  };
  if (p_f32) {
    if (g_f32) go(float(), float());
    else go(float(), uint16_t());
  } else {
    if (g_f32) go(uint16_t(), float());
    else go(uint16_t(), uint16_t());
  }
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
