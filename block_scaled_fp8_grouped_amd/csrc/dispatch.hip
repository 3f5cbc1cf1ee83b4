// Tokens to their experts and back (gfx950): the sort of the choices by expert, the rows gathered, their weighted sum
// and its gradient.  include/bsfp8.h states the formulas.
//
// The sort is a counting sort by expert, stable by construction: a workgroup takes a chunk of consecutive choices, each
// of its 16 waves a consecutive part of it, and a choice's row is the sum of the choices of lower experts, those of its
// expert in earlier chunks, in earlier waves and in earlier lanes.  A first launch counts each chunk's choices per
// expert; the second adds up the chunks before its own by itself (no third launch, no wait between workgroups) and
// places.  Up to one chunk of choices takes one launch.
//
// What bounds it: 131072 tokens' 8 choices of 128 are 21 MB, 3.4 us, in two launches: 15 us, of which the second's
// workgroups take 1 for their choices, 3 to add up the chunks' counts, 1 for the bins' begins (2 with all waves in it), 2 to
// rank 4096 choices and 1 to store them.
//
// The row movers walk tokens: a token's row is read once and written (dispatch), or a token's top_k rows are read and
// summed (combine), each byte moved once in rows of cols elements, 8 elements a thread.  All are bound by HBM: 16384 tokens'
// sums of 4 rows of 4096 bf16 with the residual stream 138 us, 130 us of bytes at 6.2 TB/s; the gradient of 16411 tokens' 3
// rows of 2050, which begin at any multiple of 4 bytes, 91 us (69 us of bytes).
#include <type_traits>

#include "common.hpp"
#include "row_io.hpp"
#include "token_layout.hpp"

namespace bsfp8 {

// ---------------------------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanSteps = kPlanUnit / kPlanThreads;  // choices a thread takes at a time

struct PlanArgs {
  const int32_t* experts;
  const float* probs;
  int64_t N;       // choices
  int E;
  int64_t chunk;   // choices per workgroup, a multiple of kPlanUnit
  int chunks;
  int32_t *hist;   // [chunks][plan_hist_row(E)]: choices of each chunk per expert, then the dropped ones
  int32_t *splits, *rows, *choices;
  float* row_probs;
};

__device__ __forceinline__ int plan_bin(int32_t e, int E) { return e < 0 || e >= E ? E : e; }

__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(PlanArgs a) {
  __shared__ int32_t count[kMaxGroups + 1];
  for (int b = threadIdx.x; b <= a.E; b += kPlanThreads) count[b] = 0;
  const int64_t begin = a.chunk * blockIdx.x, end = begin + a.chunk < a.N ? begin + a.chunk : a.N;
  int32_t e[kPlanSteps];
  for (int64_t c0 = begin; c0 < end; c0 += kPlanUnit) {
#pragma unroll
    for (int i = 0; i < kPlanSteps; ++i) {
      const int64_t c = c0 + i * kPlanThreads + threadIdx.x;
      e[i] = c < end ? a.experts[c] : -1;
    }
    if (c0 == begin) __syncthreads();
#pragma unroll
    for (int i = 0; i < kPlanSteps; ++i)
      if (c0 + i * kPlanThreads + threadIdx.x < end) atomicAdd(&count[plan_bin(e[i], a.E)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < plan_hist_row(a.E); b += kPlanThreads)
    a.hist[(int64_t)blockIdx.x * plan_hist_row(a.E) + b] = b <= a.E ? count[b] : 0;
}

// A wave turns the counts of n bins into where each begins; `out` (or NULL) gets the counts of the first n - 1.
__device__ __forceinline__ void plan_begins(int32_t* count, int n, int32_t* out) {
  const int lane = threadIdx.x & 63, per = (n + 63) / 64, b0 = lane * per;
  int sum = 0;
  for (int b = b0; b < b0 + per; ++b) sum += b < n ? count[b] : 0;
  int begin = wave_scan32(sum) - sum;
  for (int b = b0; b < b0 + per && b < n; ++b) {
    const int32_t v = count[b];
    if (out != nullptr && b < n - 1) out[b] = v;
    count[b] = begin;
    begin += v;
  }
}

__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(PlanArgs a) {
  // at[w * bins + b]: first the choices of wave w in bin b, then where its next one goes
  __shared__ int32_t at[kPlanWaves * (kMaxGroups + 1)];
  __shared__ int32_t total[kMaxGroups + 1], before[kMaxGroups + 1], own[kMaxGroups + 1];
  __shared__ int32_t sorted_row[kPlanUnit], sorted_choice[kPlanUnit];
  __shared__ float sorted_prob[kPlanUnit];
  const int bins = a.E + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // a wave's part of the chunk, kPlanSteps times 64 choices at a time; all of it stays in registers where that is the part
  const int64_t part = a.chunk / kPlanWaves, begin = a.chunk * blockIdx.x + part * wave;
  const int64_t end = begin + part < a.N ? begin + part : a.N;
  int32_t bin[kPlanSteps];
  auto load = [&](int64_t c0) {
#pragma unroll
    for (int i = 0; i < kPlanSteps; ++i) {
      const int64_t c = c0 + 64 * i + lane;
      bin[i] = c < end ? plan_bin(a.experts[c], a.E) : bins;  // (a bin of their own for the lanes past the end)
    }
  };
  load(begin);
  for (int i = threadIdx.x; i < kPlanWaves * bins; i += kPlanThreads) at[i] = 0;
  for (int b = threadIdx.x; b < bins; b += kPlanThreads) total[b] = before[b] = 0;
  __syncthreads();
  if (a.hist != nullptr) {
    // the chunks' counts: every 16th a wave's, 4 bins a lane, 8 loads in flight
    const int row = plan_hist_row(a.E);
    for (int b = 4 * lane; b < row; b += 256) {
      v4i all = {0, 0, 0, 0}, mine = {0, 0, 0, 0};
      for (int c0 = wave; c0 < a.chunks; c0 += 8 * kPlanWaves) {
        v4i n[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int c = c0 + u * kPlanWaves;
          n[u] = c < a.chunks ? *(const v4i*)(a.hist + (int64_t)c * row + b) : v4i{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          all += n[u];
          if (c0 + u * kPlanWaves < (int)blockIdx.x) mine += n[u];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (b + i < bins) {
          atomicAdd(&total[b + i], all[i]);  // (whole numbers: the order does not matter)
          atomicAdd(&before[b + i], mine[i]);
        }
      }
    }
  }
  for (int64_t c0 = begin; c0 < end; c0 += 64 * kPlanSteps) {
    if (c0 != begin) load(c0);
#pragma unroll
    for (int i = 0; i < kPlanSteps; ++i)
      if (bin[i] < bins) atomicAdd(&at[wave * bins + bin[i]], 1);
  }
  __syncthreads();
  // a bin's counts of the 16 waves, before each
  for (int b = threadIdx.x; b < bins; b += kPlanThreads) {
    int32_t n[kPlanWaves], sum = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) n[w] = at[w * bins + b];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      at[w * bins + b] = sum;
      sum += n[w];
    }
    if (a.hist == nullptr) total[b] = sum;
    own[b] = sum;
  }
  __syncthreads();
  // where the bins begin, in the rows and in the chunk
  if (wave == 0) plan_begins(total, bins, blockIdx.x == 0 ? a.splits : nullptr);
  if (wave == 1) plan_begins(own, bins, nullptr);
  __syncthreads();
  int32_t* next = at + wave * bins;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const int bits = 32 - __builtin_clz(bins);
  // a chunk of one unit is put in order in LDS first, so that an expert's run leaves as whole lines (4 bytes each to where
  // they go: 20 us for 1048576 choices where this took 16)
  const bool whole = a.chunk == kPlanUnit;
  for (int64_t c0 = begin; c0 < end; c0 += 64 * kPlanSteps) {
    if (!whole) load(c0);
#pragma unroll
    for (int i = 0; i < kPlanSteps; ++i) {
      const int64_t c = c0 + 64 * i + lane;
      const int b = bin[i];
      // the lanes of the same bin: for each of its bits those that have it as this lane has
      uint32_t lo = ~0u, hi = ~0u;
      for (int bit = 0; bit < bits; ++bit) {
        const int has = __builtin_amdgcn_sbfe(b, bit, 1);  // 0 or -1
        const uint64_t m = __ballot(has != 0);
        lo &= ~((uint32_t)m ^ (uint32_t)has);
        hi &= ~((uint32_t)(m >> 32) ^ (uint32_t)has);
      }
      const uint64_t same = (uint64_t)hi << 32 | lo;
      const int rank = __popcll(same & below);
      if (b < bins) {
        const int32_t mine = next[b] + rank, row = total[b] + before[b] + mine;
        __builtin_amdgcn_wave_barrier();
        if (rank == 0) next[b] = mine + __popcll(same);  // (a wave's LDS accesses are done in order)
        const bool dropped = b == a.E;
        a.rows[c] = dropped ? -1 : row;
        const float p = a.row_probs != nullptr && !dropped ? a.probs[c] : 0.0f;
        const int32_t choice = dropped ? -1 : (int32_t)c;
        if (whole) {
          const int to = own[b] + mine;
          sorted_row[to] = row;
          sorted_choice[to] = choice;
          sorted_prob[to] = p;
        } else {
          a.choices[row] = choice;
          if (a.row_probs != nullptr) a.row_probs[row] = p;
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
  if (!whole) return;
  __syncthreads();
  const int64_t left = a.N - a.chunk * blockIdx.x;
  const int n = left < kPlanUnit ? (int)left : (int)kPlanUnit;
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int32_t row = sorted_row[i];
    a.choices[row] = sorted_choice[i];
    if (a.row_probs != nullptr) a.row_probs[row] = sorted_prob[i];
  }
}

__global__ __launch_bounds__(kPlanThreads) void plan_empty_kernel(int32_t* splits, int E) {
  if ((int)threadIdx.x < E) splits[threadIdx.x] = 0;
}

int launch_dispatch_plan(const int32_t* experts, const float* probs, int64_t N, int E, int32_t* splits, int32_t* rows,
                         int32_t* choices, float* row_probs, void* workspace, hipStream_t stream) {
  const int64_t chunks = plan_chunks(N);
  if (chunks == 0) {
    hipLaunchKernelGGL(plan_empty_kernel, dim3(1), dim3(kPlanThreads), 0, stream, splits, E);
    return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
  }
  const PlanArgs a{experts, probs, N, E, plan_chunk(N), (int)chunks, chunks > 1 ? (int32_t*)workspace : nullptr,
                   splits, rows, choices, row_probs};
  if (chunks > 1) hipLaunchKernelGGL(plan_count_kernel, dim3((unsigned)chunks), dim3(kPlanThreads), 0, stream, a);
  hipLaunchKernelGGL(plan_place_kernel, dim3((unsigned)chunks), dim3(kPlanThreads), 0, stream, a);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

// ---------------------------------------------------------------------------------------------
// rows out and back
// ---------------------------------------------------------------------------------------------

struct MoveArgs {
  int64_t T, C, cap;
  int K;
  const int32_t* rows;
  const float* weights;
  const void *in, *add;
  void* out;
  const void* y;
  float* dweights;
  bool past;  // the output goes past the caches
};
// Outputs that no cache holds until they are read go past it (16384 tokens' sums of 4 rows of 4096 bf16 149 -> 141 us, their
// gradient 229 -> 224); smaller ones are left for what reads them next.
static bool move_past(int64_t rows, int64_t cols, bool f32) { return rows * cols * (f32 ? 4 : 2) >= int64_t(64) << 20; }

// A launch has fewer than 2^32 threads.
constexpr int64_t kMostThreads = (int64_t(1) << 32) - 1;

// Threads over (token, chunk of 8 columns): a workgroup takes 128 chunks of one token, or several whole tokens where
// their rows are shorter; `shift`: log2 of the threads that a token takes in a workgroup.  (Workgroups of 64 / 128 / 256 /
// 512 threads: sums of 4 rows of 4096 bf16 139 / 137 / 141 / 140 us, of 2050 fp32 135 / 135 / 171 / 133, rows out 113 /
// 113 / 117 / 122.)
constexpr int kMoveShift = 7, kMoveThreads = 1 << kMoveShift;
struct MoveShape {
  int shift;
  int64_t segments, blocks;
};
static MoveShape move_shape(int64_t T, int64_t C) {
  const int64_t chunks = (C + 7) / 8;
  int shift = 0;
  while (shift < kMoveShift && (int64_t(1) << shift) < chunks) ++shift;
  const int64_t seg = (chunks + (int64_t(1) << shift) - 1) >> shift, per = kMoveThreads >> shift;
  return {shift, seg, (T + per - 1) / per * seg};
}
__device__ __forceinline__ bool move_place(const MoveArgs& a, int shift, int64_t segments, int64_t& t, int64_t& c) {
  const int64_t seg = (int64_t)blockIdx.x % segments, set = (int64_t)blockIdx.x / segments;
  t = set * (kMoveThreads >> shift) + (threadIdx.x >> shift);
  c = 8 * (seg * kMoveThreads + (threadIdx.x & ((1 << shift) - 1)));
  return t < a.T && c < a.C;
}

// 8 elements as they were loaded, bit for bit.
__device__ __forceinline__ void copy8(float* p, int n, const Raw8<float>& v, bool past) {
  if (n >= 8) {
    if (past) stream8(p, v.t);
    else __builtin_memcpy(p, v.t, sizeof(v.t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v.t[i];
  }
}
__device__ __forceinline__ void copy8(uint16_t* p, int n, const Raw8<uint16_t>& v, bool past) {
  if (n >= 8) {
    uint16_t t[8];
    __builtin_memcpy(t, v.w, sizeof(t));
    if (past) stream8(p, t);
    else __builtin_memcpy(p, t, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(v.w[i >> 1] >> (16 * (i & 1)));
  }
}

template <class T>
__global__ __launch_bounds__(kMoveThreads) void dispatch_kernel(MoveArgs a, int shift, int64_t segments) {
  int64_t t, c;
  if (!move_place(a, shift, segments, t, c)) return;
  const int n = a.C - c < 8 ? (int)(a.C - c) : 8;
  Raw8<T> v;
  v.load((const T*)a.in + t * a.C + c, n);
  for (int j = 0; j < a.K; ++j) {
    const int64_t r = a.rows[t * a.K + j];
    if (r < 0 || r >= a.cap) continue;
    T* out = (T*)a.out + r * a.C + c;
    if (a.weights == nullptr) {
      copy8(out, n, v, a.past);
      continue;
    }
    float o[8];
    const float w = a.weights[t * a.K + j];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i] * w;
    store8(out, n, o, a.past);
  }
}

// The rows of KB of a token's choices from j0 on (-1: none), and their weights.
template <int KB>
struct TokenRows {
  int32_t r[KB];
  float w[KB];
  __device__ __forceinline__ TokenRows(const MoveArgs& a, int64_t t, int j0) {
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      const bool in = j0 + j < a.K;
      r[j] = in ? a.rows[t * a.K + j0 + j] : -1;
      w[j] = in && a.weights != nullptr ? a.weights[t * a.K + j0 + j] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < KB; ++j) r[j] = r[j] >= 0 && r[j] < a.cap ? r[j] : -1;
  }
};

// KB rows are in flight at a time.
template <class T, int KB>
__global__ __launch_bounds__(kMoveThreads) void combine_kernel(MoveArgs a, int shift, int64_t segments) {
  int64_t t, c;
  if (!move_place(a, shift, segments, t, c)) return;
  const int n = a.C - c < 8 ? (int)(a.C - c) : 8;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  for (int j0 = 0; j0 < a.K; j0 += KB) {
    const TokenRows<KB> rows(a, t, j0);
    Raw8<T> v[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j)
      if (rows.r[j] >= 0) v[j].load((const T*)a.in + rows.r[j] * a.C + c, n);
#pragma unroll
    for (int j = 0; j < KB; ++j)
      if (rows.r[j] >= 0)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(rows.w[j], v[j][i], sum[i]);
  }
  if (a.add != nullptr) {
    float v[8];
    load8((const T*)a.add + t * a.C + c, n, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += v[i];
  }
  store8((T*)a.out + t * a.C + c, n, sum, a.past);
}

// A token per wave (W == 1) or per workgroup of W waves, KB of its choices at a time; Y: with the dot products, O: with the
// rows' gradients.
template <class T, int W, int KB, bool Y, bool O>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void combine_grad_kernel(MoveArgs a) {
  __shared__ float sums[W][KB];
  const int lane = threadIdx.x & 63, wave = W == 1 ? 0 : threadIdx.x >> 6;
  const int64_t first = W == 1 ? (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) : blockIdx.x;
  const int64_t step = (int64_t)gridDim.x * (W == 1 ? 4 : 1);
  for (int64_t t = first; t < a.T; t += step) {
    for (int j0 = 0; j0 < a.K; j0 += KB) {
      const T* dout = (const T*)a.in + t * a.C;
      const TokenRows<KB> rows(a, t, j0);
      float dot[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) dot[j] = 0.0f;
      for (int64_t c = 8 * (wave * 64 + lane); c < a.C; c += 512 * W) {
        const int n = a.C - c < 8 ? (int)(a.C - c) : 8;
        Raw8<T> d, y[Y ? KB : 1];
        d.load(dout + c, n);
        // (every row of the set is asked for before the first is used, and before any gradient is stored: dy may be y)
        if constexpr (Y) {
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (rows.r[j] >= 0) y[j].load((const T*)a.y + rows.r[j] * a.C + c, n);
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          if (rows.r[j] < 0) continue;
          if constexpr (Y) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[j] = __builtin_fmaf(d[i], y[j][i], dot[j]);
          }
          if constexpr (O) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = d[i] * rows.w[j];
            store8((T*)a.out + rows.r[j] * a.C + c, n, o, a.past);
          }
        }
      }
      if constexpr (!Y) continue;
#pragma unroll
      for (int j = 0; j < KB; ++j) dot[j] = wave_sum(dot[j]);
      if constexpr (W == 1) {
        if (lane == 63)
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (j0 + j < a.K) a.dweights[t * a.K + j0 + j] = dot[j];
      } else {
        if (lane == 63)
#pragma unroll
          for (int j = 0; j < KB; ++j) sums[wave][j] = dot[j];
        __syncthreads();
        if ((int)threadIdx.x < KB && j0 + (int)threadIdx.x < a.K) {
          float s = 0.0f;
          for (int w = 0; w < W; ++w) s += sums[w][threadIdx.x];
          a.dweights[t * a.K + j0 + threadIdx.x] = s;
        }
        __syncthreads();
      }
    }
  }
}

// f with how many of top_k choices are taken at a time, all of up to 4, sets of 8 above (4 of fp32, to stay within registers),
// and an element.
template <class F>
static void for_top_k(int K, bool f32, F f) {
  if (f32) {
    if (K <= 2) f(std::integral_constant<int, 2>(), float());
    else f(std::integral_constant<int, 4>(), float());
  } else {
    if (K <= 2) f(std::integral_constant<int, 2>(), uint16_t());
    else if (K <= 4) f(std::integral_constant<int, 4>(), uint16_t());
    else f(std::integral_constant<int, 8>(), uint16_t());
  }
}

int launch_dispatch(const void* x, bool f32, int64_t T, int64_t C, const int32_t* rows, int K, const float* weights,
                    void* out, int64_t cap, hipStream_t stream) {
  const MoveShape s = move_shape(T, C);
  if (s.blocks > kMostThreads / kMoveThreads) return BSFP8_ERR_SHAPE;
  const MoveArgs a{T, C, cap, K, rows, weights, x, nullptr, out, nullptr, nullptr, move_past(cap, C, f32)};
  const dim3 grid((unsigned)s.blocks), block(kMoveThreads);
  if (f32) hipLaunchKernelGGL(dispatch_kernel<float>, grid, block, 0, stream, a, s.shift, s.segments);
  else hipLaunchKernelGGL(dispatch_kernel<uint16_t>, grid, block, 0, stream, a, s.shift, s.segments);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

int launch_combine(const void* y, bool f32, int64_t cap, int64_t C, const int32_t* rows, int64_t T, int K,
                   const float* weights, const void* add, void* out, hipStream_t stream) {
  const MoveShape s = move_shape(T, C);
  if (s.blocks > kMostThreads / kMoveThreads) return BSFP8_ERR_SHAPE;
  const MoveArgs a{T, C, cap, K, rows, weights, y, add, out, nullptr, nullptr, move_past(T, C, f32)};
  const dim3 grid((unsigned)s.blocks), block(kMoveThreads);
  for_top_k(K, f32, [&](auto kb, auto element) {
    hipLaunchKernelGGL((combine_kernel<decltype(element), decltype(kb)::value>), grid, block, 0, stream, a, s.shift,
                       s.segments);
  });
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

int launch_combine_grad(const void* dout, bool f32, int64_t T, int64_t C, const void* y, int64_t cap,
                        const int32_t* rows, int K, const float* weights, void* dy, float* dweights,
                        hipStream_t stream) {
  const MoveArgs a{T, C, cap, K, rows, weights, dout, nullptr, dy, y, dweights, move_past(cap, C, f32)};
  // A token's row is a workgroup's, with a wave for each KB of it up to 8, or a wave's: few tokens in flight at a time, whose
  // rows are read and written as a whole (waves a token 1 / 2 / 4 / 8: 16384 x 4 rows of 4096 bf16 246 / 236 / 227 / 223 us,
  // of 2050 101 / 94 / 92 / 118, 32768 x 4 of 1024 114 / 111 / 120 / 188, 65536 x 4 of 512 112 / 122 / 189 / 327; 16384 x 4
  // of 2048 fp32 277 / 256 / 241 / 225, of 1024 137 / 125 / 119 / 134, 65536 x 4 of 256 123 / 157 / 232 / 363).  Up to an
  // eighth more goes without waves of its own.
  auto launch = [&](auto w, auto kb, auto element, auto y, auto o) {
    constexpr int W = decltype(w)::value, KB = decltype(kb)::value, THREADS = W == 1 ? 256 : 64 * W;
    constexpr bool Y = decltype(y)::value, O = decltype(o)::value;
    const int64_t blocks = W == 1 ? (T + 3) / 4 : T, most = kMostThreads / THREADS;
    const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(THREADS);
    hipLaunchKernelGGL((combine_grad_kernel<decltype(element), W, KB, Y, O>), grid, block, 0, stream, a);
  };
  auto go = [&](auto kb, auto element, auto y, auto o) {
    const int64_t bytes = C * (int64_t)sizeof(element);
    if (bytes <= 1152) launch(std::integral_constant<int, 1>(), kb, element, y, o);
    else if (bytes <= 2304) launch(std::integral_constant<int, 2>(), kb, element, y, o);
    else if (bytes <= 4608) launch(std::integral_constant<int, 4>(), kb, element, y, o);
    else launch(std::integral_constant<int, 8>(), kb, element, y, o);
  };
  const std::integral_constant<bool, true> yes;
  const std::integral_constant<bool, false> no;
  for_top_k(K, f32, [&](auto kb, auto element) {
    if (dweights != nullptr && dy != nullptr) go(kb, element, yes, yes);
    else if (dweights != nullptr) go(kb, element, yes, no);
    else go(kb, element, no, yes);
  });
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
