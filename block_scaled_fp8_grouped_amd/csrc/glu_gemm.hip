// The gated feed-forward projection of an expert layer in one kernel, and its gradient (gfx950;
// formulas in include/bsfp8.h):
//
//  forward   (a | b) = x W1_e^T over both projections at once, y = p silu(a) b, kept in bf16 / fp32
//            and / or quantized to MXFP8 along both axes from its fp32 values
//  gradient  dh = dy W2_e (W2 quantized colwise, as the dgrad GEMM takes it), then da, db and the
//            probabilities' gradient from the (a | b) that the forward kept
//
// Bound by the bf16 MFMA on large inputs: the operands stay e4m3 in HBM and LDS, are widened to
// bf16 with their block scale folded in (exact) and accumulated in fp32, as in the plain grouped
// GEMMs.  What the fusion saves is a bf16 round trip of the product through HBM and a launch.
// Measured (32 experts, 65536 tokens, hidden 4096, ffn 2048, all of the layer's outputs): forward 1.97 ms =
// 1120 TFLOP/s, gradient 1.18 ms = 930 TFLOP/s; the forward's main loop alone runs at 1450 TFLOP/s (from two values of
// hidden), the rest is each tile's start and epilogue.  Under that load the chip holds 1.6 to 1.8 of its
// 2.4 GHz: other schedules of the same instructions in the 256 x 256 tiles (deeper rings, half the step, LDS reads ahead,
// two workgroups of 256 x 128) end within 3% of each other; waves of 128 x 128 (a third fewer conversions and LDS reads,
// but one wave per SIMD) are 8% slower.
//
// Tiles of 256 x 256 (large forwards) or 128 x 128 (tokens x rows of the weight), waves of 128 x 64 or 64 x 64, K steps of 128 or 64
// bytes in a ring of two or three LDS stages filled by LDS DMA, 16-byte chunks XOR-swizzled; the E8M0 bytes come
// by DMA too and go into the conversions as they are.  A step's barrier stands before its last MFMAs: behind it the
// stage is free, the loads of the step a ring ahead go into it and the next step's first fragments are read, both
// beside those MFMAs.
//
// In the forward the weight rows of a tile are half of each projection's, interleaved 32 by 32: a wave's column
// fragments are a and b of the same 32 outputs, so a lane holds both halves of its elements in registers and the
// activation needs no exchange; a run of 32 LDS rows has one scalar base, so the interleave costs nothing.
//
// Epilogue: a wave owns its block from its accumulators to memory, 32 rows at a time through its own
// piece of LDS (no barrier): rows of 8 columns per lane for the row-major outputs, whole 32-token
// columns per lane for the colwise ones.
//
// One workgroup per tile, fixed order, no atomics: the same bits every time.  Rows past a group's
// live rows read as zeros and are not stored; the colwise pad lanes get the zeros that those rows
// count as.
#include <type_traits>

#include "glu_epilogue.hpp"
#include "tile_addr.hpp"
#include "tile_sched.hpp"

namespace bsfp8 {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

struct GluArgs {
  const uint8_t *a_q, *a_s;  // tokens, rowwise: [R][K], [K/32][R]
  const uint8_t *b_q, *b_s;  // forward: W1 rowwise; gradient: W2 colwise
  int64_t R, K, F;
  int64_t b_ld, b_estride, bs_estride, bs_bstride;  // bytes: B row, B group; scale group, scale block row
  const int32_t* splits;
  int E;
  int tiles_n;
  int64_t tiles;
  const float* probs;
  uint16_t* ab;      // forward: kept product, or NULL; gradient: read
  GluOut out;        // forward [R][F]; gradient [R][2F]
  float* dpart;      // gradient: [tiles_n][R] parts of dprobs (dprobs itself with one tile column), or NULL
  uint32_t* status;
};

// The LDS DMAs are issued in assembly and waited for by count (glu_wait): issued through the builtins, the
// compiler cannot tell a DMA into one stage from the reads of another and waits for all of them.
// 16 bytes per lane to LDS address lds + 16 * lane; a lane whose offset lies past the resource's range
// stores zeros.  M0 holds the wave-uniform LDS address (one wait state before its use).
__device__ __forceinline__ void glu_dma16(v4i rsrc, uint32_t lds, uint32_t voff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(voff), "s"(rsrc), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void glu_dma16(const void* g, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(g), "{m0}"(lds) : "memory");
}
// Words of a raw buffer resource over `bytes` bytes at `base` (wave-uniform).
__device__ __forceinline__ v4i glu_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)a), __builtin_amdgcn_readfirstlane((int)((a >> 32) & 0xffff)),
             __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// All of this wave's DMAs but the newest N have landed and its LDS reads have returned; then the barrier.
template <int N>
__device__ __forceinline__ void glu_wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// An E8M0 byte as the scale operand of the widening conversions, which use its exponent field alone (0 stands
// for 2^-127 there too: checked on the GPU for every byte and code).
__device__ __forceinline__ float glu_e8m0(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight e4m3 codes -> eight bf16 values times `scale` (exact).
__device__ __forceinline__ v8bf glu_widen8(int d0, int d1, float scale) {
  const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)d0, scale, false);
  const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)d0, scale, true);
  const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)d1, scale, false);
  const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)d1, scale, true);
  return v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Chunk c (16 bytes) of an LDS row of BK bytes sits at c ^ glu_swz(r): the 16 lanes that a 16-byte LDS read
// serves at once (0-3, 12-15, 20-27 and the rest of each 32) see every bank once.
template <int BK>
__device__ __forceinline__ int glu_swz(int row) {
  return BK == 128 ? swz(row) : (row >> 2) & 3;
}
// Source offset of DMA lane `lane` of the 1 KB of LDS rows that begin at `row0`: row-major rows of ld bytes.
template <int BK>
__device__ __forceinline__ uint32_t glu_dma_offset(int row0, int lane, uint32_t ld) {
  constexpr int C = BK / 16;
  const int row = row0 + lane / C;
  return (uint32_t)row * ld + 16u * (uint32_t)((lane % C) ^ glu_swz<BK>(row));
}

// Tiles of BM x BN, K steps of BK bytes, waves of BM / 2 x WN, NS stages of LDS.
template <bool GRAD, int BM_, int BN_, int WN_, int BK_, int NS_>
struct GluShape {
  static constexpr int BM = BM_, BN = BN_, BK = BK_, NS = NS_, WM = BM / 2, WN = WN_, BLKS = BK / 32;
  static constexpr int WAVES_N = BN / WN, NW = 2 * WAVES_N, NT = 64 * NW;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int COLS = GRAD ? BN : BN / 2;  // output columns (of one half) per tile
  // a stage: A rows, B rows, then the E8M0 bytes as the scale DMAs leave them: AL lanes of 16 bytes per block
  // of A (from the 16-byte boundary before its first row), then BL per block of B
  static constexpr int AL = BM / 16 + 1, BL = BN / 16;
  static constexpr int SC_INS = (BLKS * (AL + BL) + 63) / 64;  // scale DMAs per step; wave w < SC_INS issues one
  static constexpr int B_OFF = BM * BK, SC_OFF = (BM + BN) * BK, STAGE = SC_OFF + SC_INS * 1024;
  static constexpr int SB_OFF = SC_OFF + BLKS * AL * 16;
  static constexpr int A_INS = BM * BK / 1024 / NW, B_INS = BN * BK / 1024 / NW;
  // epilogue: each wave's 32 rows of fp32, the row pitch shifting the rows 4 apart (one register's two
  // half-waves) by half of the 64 banks
  static constexpr int PITCH = GRAD ? 72 : 40;
  static constexpr int AB_PITCH = 72;  // forward: the kept product's 32 rows of 64 bf16, behind them
  static constexpr int EP = 32 * PITCH * 4 + (GRAD ? 0 : 32 * AB_PITCH * 2);
  static constexpr int INS_ROWS = 1024 / BK, RUNS = B_INS * INS_ROWS / 32;  // runs of 32 weight rows per wave
  static_assert(NT >= BM && RUNS * 32 == B_INS * INS_ROWS, "the probabilities' loads, the weight's");
  static_assert(SC_INS <= NW, "scale loads");
  static_assert(NW * EP + (BN / 64 + 1) * BM * 4 <= NS * STAGE && (int)sizeof(GroupScanSmem<NT>) <= NS * STAGE, "LDS reuse");
  static_assert(NS * STAGE <= 160 * 1024, "LDS budget");
};

// Inclusive sum over a wave, with data-parallel lane moves.
__device__ __forceinline__ int glu_wave_scan(int v) {
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

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ int64_t glu_uniform(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// The tile's group, as group_scan gives it (tiles of BM rows).  Up to 64 groups in a buffer of less than 2^24
// rows (sums below 2^31) every wave scans the sizes by itself: no LDS, no barrier, a third of the time, which
// counts where a workgroup is alone on its CU.
template <int NT>
__device__ __forceinline__ uint32_t glu_place(const GluArgs& args, int BM, int64_t mt, GroupScanSmem<NT>& sm,
                                              GroupInfo& gi) {
  if (args.E > 64 || args.R >= (1 << 24)) {
    const uint32_t flags = group_scan<NT>(args.splits, args.E, args.R, BM, mt, 0, sm, gi);
    gi.e = __builtin_amdgcn_readfirstlane(gi.e);
    gi.k = glu_uniform(gi.k);
    gi.off = glu_uniform(gi.off);
    gi.kp = glu_uniform(gi.kp);
    gi.p = glu_uniform(gi.p);
    gi.tile = glu_uniform(gi.tile);
    return __builtin_amdgcn_readfirstlane((int)flags);
  }
  const int lane = threadIdx.x & 63;
  const int v = lane < args.E ? args.splits[lane] : 0;
  const bool negative = __ballot(v < 0) != 0;
  const bool large = __ballot((int64_t)v > args.R) != 0;
  const int k = v < 0 || (int64_t)v > args.R ? 0 : v, kp = (k + 127) & ~127, tl = (k + BM - 1) / BM;
  const int sk = glu_wave_scan(k), skp = glu_wave_scan(kp), stl = glu_wave_scan(tl);
  gi.e = -1;
  uint32_t flags = negative ? BSFP8_STATUS_NEGATIVE_SPLIT : 0u;
  if (large || (int64_t)__builtin_amdgcn_readlane(sk, 63) > args.R) flags |= BSFP8_STATUS_EXCEEDS_CAPACITY;
  if (flags) return flags;
  const uint64_t own = __ballot(mt >= stl - tl && mt < stl);
  if (own == 0) return 0;
  const int e = __builtin_ctzll(own);
  gi.e = e;
  gi.k = __builtin_amdgcn_readlane(k, e);
  gi.off = __builtin_amdgcn_readlane(sk - k, e);
  gi.kp = __builtin_amdgcn_readlane(kp, e);
  gi.p = __builtin_amdgcn_readlane(skp - kp, e);
  gi.tile = __builtin_amdgcn_readlane(stl - tl, e);
  return 0;
}

template <bool GRAD, int BM, int BN, int WN, int BK, int NS>
__global__ __launch_bounds__(128 * BN / WN, NS == 3 ? 3 : 2) void glu_gemm_kernel(GluArgs args) {
  using S = GluShape<GRAD, BM, BN, WN, BK, NS>;
  constexpr int NT = S::NT, FM = S::FM, FN = S::FN, BLKS = S::BLKS;
  __shared__ __attribute__((aligned(16))) uint8_t smem[NS * S::STAGE];
  GroupScanSmem<NT>& gsm = *(GroupScanSmem<NT>*)smem;  // done before the first DMA (a barrier below)

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, l32 = lane & 31;
  const int wm = wave & 1, wn = wave >> 1;

  const int64_t L = xcd_logical(blockIdx.x);
  if (L >= args.tiles) return;
  int64_t mt;
  int tn;
  fprop_tile(L, args.tiles_n, &mt, &tn);
  GroupInfo gi{};
  const uint32_t flags = glu_place<NT>(args, BM, mt, gsm, gi);
  report_status(args.status, flags);
  if (gi.e < 0) return;
  const int64_t row0 = (mt - gi.tile) * BM;  // the tile's first row within the group (< gi.k)
  const int64_t col0 = (int64_t)tn * S::COLS;
  const int64_t F = args.F, K = args.K;
  const int a_last = (int)(gi.k - row0 < BM ? gi.k - row0 : BM) - 1;      // last live tile row
  const int b_last = (int)(F - col0 < S::COLS ? F - col0 : S::COLS) - 1;  // last live column of a half
  // this thread's row of the probabilities, to LDS behind the main loop
  float my_prob = 0.0f;
  if (tid < BM && tid <= a_last) my_prob = args.probs != nullptr ? args.probs[gi.off + row0 + tid] : 1.0f;

  // ---------------- loads of one K step ----------------
  // B: LDS rows in runs of 32; forward: run k is rows 32 (k / 2) .. of projection k % 2
  const uint8_t* a_base = args.a_q + (gi.off + row0) * K;
  const uint8_t* b_base = args.b_q + gi.e * args.b_estride + col0 * args.b_ld;
  // (the live rows of the tile only: below 2^30 bytes, so an offset from 2^31 up is past them)
  const v4i a_rs = glu_rsrc(a_base, (uint32_t)(a_last + 1) * (uint32_t)K);
  v4i b_rs[S::RUNS];
#pragma unroll
  for (int k = 0; k < S::RUNS; ++k)
    b_rs[k] = glu_rsrc(b_base + (GRAD ? 0 : ((wave * S::RUNS + k) & 1) * F * args.b_ld),
                       (uint32_t)(b_last + 1) * (uint32_t)args.b_ld);
  const uint32_t smem_lds =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem);
  uint32_t a_off[S::A_INS], b_off[S::B_INS];
#pragma unroll
  for (int u = 0; u < S::A_INS; ++u) a_off[u] = glu_dma_offset<BK>((wave * S::A_INS + u) * S::INS_ROWS, lane, (uint32_t)K);
#pragma unroll
  for (int u = 0; u < S::B_INS; ++u) {
    const int row = (wave * S::B_INS + u) * S::INS_ROWS, run = wave * S::RUNS + u * S::INS_ROWS / 32;
    b_off[u] = glu_dma_offset<BK>(row, lane, (uint32_t)args.b_ld);
    if constexpr (!GRAD) b_off[u] -= (uint32_t)((run - (run >> 1)) * 32) * (uint32_t)args.b_ld;
  }
  // Scales, 16 bytes per lane.  A: a group's rows begin anywhere, so the lanes read the aligned 16 bytes that
  // hold them (the first at or after the buffer's own aligned start, the last the one that holds the last
  // live row's).  B: 16 LDS rows, which lie in one run of 32 columns.  Lanes with nothing to load repeat a
  // live address.
  constexpr int AL = S::AL, BL = S::BL;
  const int sc_lane = wave * 64 + lane;
  const bool sc_is_a = sc_lane < BLKS * AL;
  const int sc_at = sc_is_a ? sc_lane : (sc_lane - BLKS * AL) % (BLKS * BL);
  const int sc_blk = sc_is_a ? sc_at / AL : sc_at / BL, sc_chunk = sc_is_a ? sc_at % AL : sc_at % BL;
  const uint8_t* a_sc = args.a_s + gi.off + row0;
  const uint8_t* b_sc;
  {
    const int r = GRAD ? 16 * sc_chunk : (sc_chunk >> 2) * 32 + 16 * (sc_chunk & 1);
    b_sc = args.b_s + gi.e * args.bs_estride + (GRAD ? 0 : ((sc_chunk >> 1) & 1) * F) + col0 +
           (r <= b_last ? r : b_last & ~15);
  }
  const int nblk = (int)(K / 32), nk = (int)((K + BK - 1) / BK);
  // step kk into `stage` (kk % NS), parts [p0, p1): 0 the scales, then A_INS + B_INS DMAs.  A step past the last
  // stores zeros (offsets past every resource's range, as the host bounds 256 rows by 2^31 bytes), so that the
  // counts stay the same.
  constexpr int NP = S::A_INS + S::B_INS + 1;
  auto issue = [&](int kk, int stage, int p0, int p1) {
    const uint32_t k0 = kk < nk ? (uint32_t)kk * BK : 0x80000000u;
    const uint32_t base = smem_lds + (uint32_t)stage * S::STAGE;
    if (p0 == 0 && p1 > 0 && wave < S::SC_INS) {
      const int kb = BLKS * kk + sc_blk, kc = kb < nblk ? kb : nblk - 1;
      const uint8_t* src;
      if (sc_is_a) {
        const uintptr_t first = (uintptr_t)(a_sc + (int64_t)kc * args.R), last = (first + a_last) & ~(uintptr_t)15;
        const uintptr_t at = (first & ~(uintptr_t)15) + 16 * sc_chunk;
        src = (const uint8_t*)(at < last ? at : last);
      } else {
        src = b_sc + (int64_t)kc * args.bs_bstride;
      }
      glu_dma16(src, base + S::SC_OFF + wave * 1024);
    }
#pragma unroll
    for (int u = 0; u < S::A_INS; ++u) {
      if (1 + u < p0 || 1 + u >= p1) continue;
      glu_dma16(a_rs, base + (wave * S::A_INS + u) * 1024, a_off[u] + k0);
    }
#pragma unroll
    for (int u = 0; u < S::B_INS; ++u) {
      if (1 + S::A_INS + u < p0 || 1 + S::A_INS + u >= p1) continue;
      glu_dma16(b_rs[u * S::INS_ROWS / 32], base + S::B_OFF + (wave * S::B_INS + u) * 1024, b_off[u] + k0);
    }
  };
  // waits until all but the newest `steps` steps' loads have landed, in every wave
  auto wait = [&](auto steps) {
    constexpr int N = decltype(steps)::value;
    if (N == 0 || wave < S::SC_INS) glu_wait_barrier<N * NP>();
    else glu_wait_barrier<N*(NP - 1)>();
  };

  v16f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // The fragments of one scale block (32 bytes of K) of a step and their scales: of two such sets one is read from
  // LDS while the other is worked on.
  struct Block {
    v4i a[FM], b[FN];
    float as[FM], bs[FN];
  };
  constexpr int NF = FM + FN, NM = FM * FN;
  auto read = [&](Block& q, int kk, int stage, int blk, int f0, int f1) {  // of the FM + FN fragments [f0, f1)
    const uint8_t* cur = smem + stage * S::STAGE;
    // where the block's A scales begin in the stage
    const int sh = S::SC_OFF + blk * AL * 16 + (int)((uintptr_t)(a_sc + (int64_t)(BLKS * kk + blk) * args.R) & 15);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (i < f0 || i >= f1) continue;
      const int row = wm * S::WM + i * 32 + l32;
      q.a[i] = *(const v4i*)(cur + row * BK + (((2 * blk + h) ^ glu_swz<BK>(row)) << 4));
      q.as[i] = glu_e8m0(cur[sh + row]);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if (FM + j < f0 || FM + j >= f1) continue;
      const int row = wn * S::WN + j * 32 + l32;
      q.b[j] = *(const v4i*)(cur + S::B_OFF + row * BK + (((2 * blk + h) ^ glu_swz<BK>(row)) << 4));
      q.bs[j] = glu_e8m0(cur[S::SB_OFF + blk * BN + row]);
    }
  };
  // Half a block, 16 bytes of K per half wave, as the MFMAs take it.
  struct Half {
    v8bf a[FM], b[FN];
  };
  auto widen = [&](Half& w, const Block& q, int t, int f) {
    if (f < FM) w.a[f] = glu_widen8(q.a[f][2 * t], q.a[f][2 * t + 1], q.as[f]);
    else w.b[f - FM] = glu_widen8(q.b[f - FM][2 * t], q.b[f - FM][2 * t + 1], q.bs[f - FM]);
  };
  auto mfma = [&](const Half& w, int u) {
    acc[u / FN][u % FN] =
        __builtin_amdgcn_mfma_f32_32x32x16_bf16(w.a[u / FN], w.b[u % FN], acc[u / FN][u % FN], 0, 0, 0);
  };
  Block q[2];

  __syncthreads();  // the group scan's LDS is free
#pragma unroll
  for (int kk = 0; kk < NS; ++kk) issue(kk, kk, 0, NP);
  wait(std::integral_constant<int, NS - 1>());

  if constexpr (BM == 128) {
    // Few waves per SIMD: the schedule is the wave's own.  Behind each MFMA of a half go its share of the next half's
    // conversions (32 cycles for 32) and of the LDS reads and the DMAs, and the stages are unrolled, so that their
    // addresses are constants.  A tile alone on its CU: a step of 128 takes 1.05 us, with the halves one after
    // another and the DMAs sent together 1.25; K = 4128, 128 / 256 tiles of the gradient 45 / 47 us (50 / 52).
    Half w[2];
    auto half = [&](const Half& now, Half& next, const Block& from, int t, auto other) {
#pragma unroll
      for (int u = 0; u < NM; ++u) {
        mfma(now, u);
#pragma unroll
        for (int f = u * NF / NM; f < (u + 1) * NF / NM; ++f) widen(next, from, t, f);
        other(u);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // One K step.  A block is read two blocks ahead, where its set of registers has been widened.  Behind the first
    // half of the last block but one the next step's loads have landed and this one's reads have returned, in every
    // wave: its stage is free, and the loads of the step NS ahead go out over the three halves that are left.
    auto step = [&](int kk, auto stage_) {
      constexpr int stage = decltype(stage_)::value, after = (stage + 1) % NS;
      auto send = [&](int v) { issue(kk + NS, stage, v * NP / (3 * NM), (v + 1) * NP / (3 * NM)); };
#pragma unroll
      for (int blk = 0; blk < BLKS; ++blk) {
        half(w[0], w[1], q[blk & 1], 1, [&](int u) {
          if (blk == BLKS - 1) send(NM + u);
        });
        if (blk == BLKS - 2) wait(std::integral_constant<int, NS - 2>());
        half(w[1], w[0], q[(blk + 1) & 1], 0, [&](int u) {
          const int f0 = u * NF / NM, f1 = (u + 1) * NF / NM;
          if (blk + 2 < BLKS) read(q[blk & 1], kk, stage, blk + 2, f0, f1);
          else read(q[blk & 1], kk + 1, after, blk + 2 - BLKS, f0, f1);
          if (blk >= BLKS - 2) send((blk == BLKS - 1 ? 2 * NM : 0) + u);
        });
      }
    };
    read(q[0], 0, 0, 0, 0, NF);
    read(q[1], 0, 0, 1, 0, NF);
#pragma unroll
    for (int f = 0; f < NF; ++f) widen(w[0], q[0], 0, f);
    const int whole = nblk / BLKS, rest = nblk % BLKS;
    int kk = 0;
    for (; kk + NS <= whole; kk += NS) {
      step(kk, std::integral_constant<int, 0>());
      step(kk + 1, std::integral_constant<int, 1>());
      if constexpr (NS == 3) step(kk + 2, std::integral_constant<int, 2>());
    }
    if (kk < whole) step(kk++, std::integral_constant<int, 0>());
    if constexpr (NS == 3)
      if (kk < whole) step(kk++, std::integral_constant<int, 1>());
    // the blocks of a last step that K does not fill
#pragma unroll
    for (int blk = 0; blk < BLKS - 1; ++blk) {
      if (blk >= rest) break;
      half(w[0], w[1], q[blk & 1], 1, [](int) {});
      half(w[1], w[0], q[(blk + 1) & 1], 0, [&](int u) {
        if (blk + 2 < BLKS) read(q[blk & 1], whole, whole % NS, blk + 2, u * NF / NM, (u + 1) * NF / NM);
      });
    }
  } else {
    // Two waves per SIMD cover for each other, and there are no registers for a half ahead: one block's LDS reads go
    // out beside the MFMAs of the block before.
    auto multiply = [&](const Block& from, auto between) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        v8bf aw[FM], bw[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) aw[i] = glu_widen8(from.a[i][2 * t], from.a[i][2 * t + 1], from.as[i]);
#pragma unroll
        for (int j = 0; j < FN; ++j) bw[j] = glu_widen8(from.b[j][2 * t], from.b[j][2 * t + 1], from.bs[j]);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(aw[i], bw[j], acc[i][j], 0, 0, 0);
        between(t);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto nothing = [](int) {};
    // One K step; q[0] holds its first block.  Before its last block's MFMAs all its reads have returned and the
    // next step's loads have landed: behind that barrier its stage is free, the loads of the step NS ahead go
    // into it, and the next step's first block is read, both beside those MFMAs.  Blocks past K (a last step that
    // K does not fill) are not multiplied.
    auto step = [&](int kk) {
#pragma unroll
      for (int blk = 0; blk + 1 < BLKS; ++blk) {
        read(q[(blk + 1) & 1], kk, kk % NS, blk + 1, 0, NF);
        __builtin_amdgcn_sched_barrier(0);
        if (blk == 0 || BLKS * kk + blk < nblk) multiply(q[blk & 1], nothing);
      }
      wait(std::integral_constant<int, NS - 2>());
      read(q[0], kk + 1, (kk + 1) % NS, 0, 0, NF);
      __builtin_amdgcn_sched_barrier(0);
      if (BLKS * kk + BLKS - 1 < nblk)
        multiply(q[(BLKS - 1) & 1], [&](int t) { issue(kk + NS, kk % NS, t * NP / 2, (t + 1) * NP / 2); });
      else
        issue(kk + NS, kk % NS, 0, NP);
    };
    read(q[0], 0, 0, 0, 0, NF);
    for (int kk = 0; kk < nk; ++kk) step(kk);
  }
  glu_wait_barrier<0>();  // the zeros past the last step have landed: LDS is free

  // ---------------- epilogue ----------------
  // register r of fragment (i, j): row 32 i + 8 (r / 4) + 4 h + r % 4, column 32 j + l32 of the block
  float* tile = (float*)(smem + wave * S::EP);
  float* probs = (float*)(smem + S::NW * S::EP);
  if (tid < BM) probs[tid] = my_prob;
  __syncthreads();
  constexpr int PITCH = S::PITCH;
  if constexpr (!GRAD) {
    uint16_t* ab_tile = (uint16_t*)(tile + 32 * PITCH);
    const GluTileOut o = glu_tile_out(args.out, args.R, F, gi, row0, col0);
    uint16_t* ab = args.ab == nullptr ? nullptr : args.ab + (gi.off + row0) * 2 * F + col0;
#pragma unroll
    for (int pair = 0; pair < FN / 2; ++pair) {
      const int cw = wn * (S::WN / 2) + 32 * pair;  // the pair's first column within the tile
      const bool cols = cw <= b_last;  // its 32 columns all exist, or none
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int rb = wm * S::WM + i * 32;
        const v16f &a = acc[i][2 * pair], &b = acc[i][2 * pair + 1];
        float v[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v4f p = *(const v4f*)&probs[rb + 8 * q + 4 * h];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[4 * q + k] = swiglu(a[4 * q + k], b[4 * q + k], p[k]);
        }
        if (rb + 31 > a_last) {  // dead rows, whose scales may have been anything, count as zeros
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] = rb + 8 * (r >> 2) + 4 * h + (r & 3) <= a_last ? v[r] : 0.0f;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) tile[(8 * (r >> 2) + 4 * h + (r & 3)) * PITCH + l32] = v[r];
        if (args.ab != nullptr) {
#pragma unroll
          for (int r = 0; r < 16; r += 2) {
            const uint32_t wa = __builtin_bit_cast(uint32_t, v2bf{(__bf16)a[r], (__bf16)a[r + 1]});
            const uint32_t wb = __builtin_bit_cast(uint32_t, v2bf{(__bf16)b[r], (__bf16)b[r + 1]});
            uint16_t* t = ab_tile + (8 * (r >> 2) + 4 * h + (r & 3)) * S::AB_PITCH + l32;
            t[0] = (uint16_t)wa;
            t[32] = (uint16_t)wb;
            t[S::AB_PITCH] = (uint16_t)(wa >> 16);
            t[S::AB_PITCH + 32] = (uint16_t)(wb >> 16);
          }
        }
        wave_lds_order();
        if (args.ab != nullptr) {
#pragma unroll
          for (int pass = 0; pass < 4; ++pass) {  // 8 lanes per row: 4 of a, 4 of b
            const int r = pass * 8 + (lane >> 3), c = 8 * (lane & 7);
            const v8s w = *(const v8s*)(ab_tile + r * S::AB_PITCH + c);
            if (cols && rb + r <= a_last)
              *(v8s*)(ab + ((uint32_t)(rb + r) * (uint32_t)(2 * F) + (uint32_t)cw +
                            (c < 32 ? (uint32_t)c : (uint32_t)F + (uint32_t)c - 32u))) = w;
          }
        }
        if (args.out.col_q != nullptr && row0 + rb < gi.kp) {
          float c[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) c[k] = tile[k * PITCH + l32];
          put_col32(o, rb, cw + l32, cols && h == 0, c);
        }
        if (args.out.y != nullptr || args.out.row_q != nullptr) {
#pragma unroll
          for (int pass = 0; pass < 2; ++pass) {
            const int r = pass * 16 + (lane >> 2), ch = 8 * (lane & 3);
            float w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = tile[r * PITCH + ch + k];
            put_row8(o, rb + r, cw + ch, cols && rb + r <= a_last, w);
          }
        }
        wave_lds_order();
      }
    }
  } else {
    const GluTileOut oa = glu_tile_out(args.out, args.R, 2 * F, gi, row0, col0);
    const GluTileOut ob = glu_tile_out(args.out, args.R, 2 * F, gi, row0, F + col0);
    const uint16_t* ab = args.ab + (gi.off + row0) * 2 * F + col0;
#pragma unroll
    for (int part = 0; part < S::WN / 64; ++part) {
      const int cw = wn * S::WN + 64 * part;
      float* dp_sum = probs + (1 + cw / 64) * BM;  // these 64 columns' part of dprobs, per row
      const int ch = 8 * (lane & 7);
      const bool cols = cw + ch <= b_last;
      // a and b of 32 rows, 8 columns of 4 rows per lane; the next 32 rows' are fetched once these are used
      v8s av[4], bv[4];
      auto fetch = [&](int i) {
#pragma unroll
        for (int pass = 0; pass < 4; ++pass) {
          const int r = wm * S::WM + i * 32 + pass * 8 + (lane >> 3);
          av[pass] = bv[pass] = v8s{0, 0, 0, 0, 0, 0, 0, 0};
          if (cols && r <= a_last) {
            const uint16_t* p = ab + ((uint32_t)r * (uint32_t)(2 * F) + (uint32_t)(cw + ch));
            av[pass] = *(const v8s*)p;
            bv[pass] = *(const v8s*)(p + F);
          }
        }
      };
      fetch(0);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int rb = wm * S::WM + i * 32;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            tile[(8 * (r >> 2) + 4 * h + (r & 3)) * PITCH + j * 32 + l32] = acc[i][2 * part + j][r];
        if (rb + 31 > a_last) {  // dead rows, whose scales may have been anything, count as zeros
          wave_lds_order();
          for (int r = a_last + 1 > rb ? a_last + 1 - rb : 0; r < 32; ++r) tile[r * PITCH + lane] = 0.0f;
        }
        wave_lds_order();
        float db[4][8];
#pragma unroll
        for (int pass = 0; pass < 4; ++pass) {
          const int r = pass * 8 + (lane >> 3);
          const float p = probs[rb + r];
          const bool live = cols && rb + r <= a_last;
          float da[8], dp = 0.0f;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            swiglu_grad(to_f32(av[pass][k]), to_f32(bv[pass][k]), p, tile[r * PITCH + ch + k], da[k],
                        db[pass][k], dp);
          put_row8(oa, rb + r, cw + ch, live, da);
          put_row8(ob, rb + r, cw + ch, live, db[pass]);
          dp += __shfl_xor(dp, 1, 64);
          dp += __shfl_xor(dp, 2, 64);
          dp += __shfl_xor(dp, 4, 64);
          if ((lane & 7) == 0) dp_sum[rb + r] = dp;
#pragma unroll
          for (int k = 0; k < 8; ++k) tile[r * PITCH + ch + k] = da[k];
          __builtin_amdgcn_sched_barrier(0);  // (the rows' temporaries end here: registers)
        }
        if (i + 1 < FM) fetch(i + 1);
        if (args.out.col_q != nullptr && row0 + rb < gi.kp) {
          float c[32];
          const bool live = cw + lane <= b_last;
          wave_lds_order();
#pragma unroll
          for (int k = 0; k < 32; ++k) c[k] = tile[k * PITCH + lane];
          put_col32(oa, rb, cw + lane, live, c);
          wave_lds_order();
#pragma unroll
          for (int pass = 0; pass < 4; ++pass)
#pragma unroll
            for (int k = 0; k < 8; ++k) tile[(pass * 8 + (lane >> 3)) * PITCH + ch + k] = db[pass][k];
          wave_lds_order();
#pragma unroll
          for (int k = 0; k < 32; ++k) c[k] = tile[k * PITCH + lane];
          put_col32(ob, rb, cw + lane, live, c);
        }
        wave_lds_order();
      }
    }
    if (args.dpart != nullptr) {
      __syncthreads();
      const float* s = probs + BM;
      if (tid <= a_last) {
        float d = s[tid];
#pragma unroll
        for (int w = 1; w < BN / 64; ++w) d += s[w * BM + tid];
        args.dpart[(int64_t)tn * args.R + gi.off + row0 + tid] = d;
      }
    }
  }
}

// ------------------------------------------------------------------------------------------
// Few rows per expert (serving)
// ------------------------------------------------------------------------------------------
//
// Bound by HBM: every live expert's weight is read once for a handful of rows, so what counts is the
// bytes in flight.  Tile: 32 tokens x 64 weight rows (forward: 32 of each projection).  The 4 waves of
// a workgroup share the K extent, wave w taking the steps w, w + 4, ..., and their sums are added in
// order at the end: no barrier and no LDS until then, each wave keeps two steps of weights (16 KB) in
// flight in registers.  16 x 16 x 32 MFMAs; lane (row, q) of a fragment loads the whole scale block q of
// its row (two 16-byte loads), so it needs one scale byte per step.  The order of K within an MFMA is
// that of the lanes, the same for both operands.  8 tokens at 8 of 32 experts, hidden 7168, ffn 2048: 41 us with
// the 242 MB of weights in the last-level cache, 49 us = 4.9 TB/s from HBM (256 x 256 tiles, which
// keep half of the chip busy: 149).
constexpr int kRowsBM = 32, kRowsBN = 64, kRowsNW = 4, kRowsPitch = 68;

template <bool GRAD>
__global__ __launch_bounds__(256, 2) void glu_rows_kernel(GluArgs args) {
  constexpr int BM = kRowsBM, BN = kRowsBN, NW = kRowsNW, NT = 64 * NW, P = kRowsPitch;
  constexpr int COLS = GRAD ? BN : BN / 2;
  __shared__ GroupScanSmem<NT> gsm;
  __shared__ __attribute__((aligned(16))) float part[NW][BM][P];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, l16 = lane & 15;
  const int64_t L = xcd_logical(blockIdx.x);
  if (L >= args.tiles) return;
  int64_t mt;
  int tn;
  fprop_tile(L, args.tiles_n, &mt, &tn);
  GroupInfo gi{};
  const uint32_t flags = glu_place<NT>(args, BM, mt, gsm, gi);
  report_status(args.status, flags);
  if (gi.e < 0) return;
  const int64_t row0 = (mt - gi.tile) * BM, col0 = (int64_t)tn * COLS;
  const int64_t F = args.F, K = args.K;
  const int a_last = (int)(gi.k - row0 < BM ? gi.k - row0 : BM) - 1;
  const int b_last = (int)(F - col0 < COLS ? F - col0 : COLS) - 1;

  // Fragments: tokens 16 i + l16; weight rows 16 j + l16 of the tile's 64 (forward: j < 2 of a, j >= 2 of b).  All
  // loads go through buffer resources that end with the last live row: what lies past it, or past K, reads as
  // zeros (a scale of 0 stands for 2^-127).
  const int nblk = (int)(K / 32), nk = (nblk + 3) / 4;
  const __amdgpu_buffer_rsrc_t a_rs = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(args.a_q + (gi.off + row0) * K), (short)0, (int)((a_last + 1) * K), 0x00020000);
  const int64_t b_half = GRAD ? 32 : F;  // weight rows from fragment 0 to fragment 2
  const uint8_t* b_base = args.b_q + gi.e * args.b_estride + col0 * args.b_ld;
  __amdgpu_buffer_rsrc_t b_rs[2];
  int b_rows[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    b_rows[k] = GRAD ? b_last + 1 - 32 * k : 32;
    b_rows[k] = b_rows[k] < 0 ? 0 : b_rows[k] > 32 ? 32 : b_rows[k];
    b_rs[k] = __builtin_amdgcn_make_buffer_rsrc((void*)(b_base + k * b_half * args.b_ld), (short)0,
                                                (int)(b_rows[k] * args.b_ld), 0x00020000);
  }
  uint32_t a_off[2], b_off[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a_off[i] = (uint32_t)(16 * i + l16) * (uint32_t)K + 32 * q;
    b_off[i] = (uint32_t)(16 * i + l16) * (uint32_t)args.b_ld + 32 * q;
  }
  const uint32_t as_off = (uint32_t)q * (uint32_t)args.R + l16, bs_off = (uint32_t)q * (uint32_t)args.bs_bstride + l16;
  const uint8_t* a_sc = args.a_s + gi.off + row0;
  const uint8_t* b_sc = args.b_s + gi.e * args.bs_estride + col0;

  struct Frag {
    v4i a[2][2], b[4][2];
    uint8_t as[2], bs[4];
  };
  auto load = [&](Frag& f, int kk) {
    const int left = nblk - 4 * kk;  // blocks from this step on; may be negative
    const uint32_t k0 = q < left ? (uint32_t)kk * 128u : 0x80000000u;
    // the block rows of this step's scales, to their last live entry
    auto scales = [&](const uint8_t* base, int64_t stride, int live) {
      const int m = left < 4 ? left : 4;
      return __builtin_amdgcn_make_buffer_rsrc((void*)(base + 4 * (left > 0 ? kk : 0) * stride), (short)0,
                                               m > 0 && live > 0 ? (int)((m - 1) * stride + live) : 0, 0x00020000);
    };
    const __amdgpu_buffer_rsrc_t as = scales(a_sc, args.R, a_last + 1);
    const __amdgpu_buffer_rsrc_t bs[2] = {scales(b_sc, args.bs_bstride, b_rows[0]),
                                          scales(b_sc + b_half, args.bs_bstride, b_rows[1])};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f.b[j][0] = __builtin_amdgcn_raw_buffer_load_b128(b_rs[j >> 1], (int)(b_off[j & 1] + k0), 0, 0);
      f.b[j][1] = __builtin_amdgcn_raw_buffer_load_b128(b_rs[j >> 1], (int)(b_off[j & 1] + k0 + 16), 0, 0);
      f.bs[j] = __builtin_amdgcn_raw_buffer_load_b8(bs[j >> 1], (int)bs_off + (j & 1) * 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f.a[i][0] = __builtin_amdgcn_raw_buffer_load_b128(a_rs, (int)(a_off[i] + k0), 0, 0);
      f.a[i][1] = __builtin_amdgcn_raw_buffer_load_b128(a_rs, (int)(a_off[i] + k0 + 16), 0, 0);
      f.as[i] = __builtin_amdgcn_raw_buffer_load_b8(as, (int)as_off + i * 16, 0, 0);
    }
  };
  v4f acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  auto multiply = [&](const Frag& f) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      v8bf aw[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        aw[i] = glu_widen8(f.a[i][t >> 1][2 * (t & 1)], f.a[i][t >> 1][2 * (t & 1) + 1], glu_e8m0(f.as[i]));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v8bf bw = glu_widen8(f.b[j][t >> 1][2 * (t & 1)], f.b[j][t >> 1][2 * (t & 1) + 1], glu_e8m0(f.bs[j]));
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(aw[i], bw, acc[i][j], 0, 0, 0);
      }
    }
  };
  // three buffers: two steps' loads are in flight while one is multiplied (steps past the end load zeros)
  Frag f0, f1, f2;
  const int steps = (nk - wave + NW - 1) / NW;  // of this wave; may be 0
  load(f0, wave);
  load(f1, wave + NW);
  for (int s = 0; s < steps; s += 3) {
    // (the fences keep the loads in front of the products)
    load(f2, wave + NW * (s + 2));
    __builtin_amdgcn_sched_barrier(0);
    multiply(f0);
    load(f0, wave + NW * (s + 3));
    __builtin_amdgcn_sched_barrier(0);
    multiply(f1);
    load(f1, wave + NW * (s + 4));
    __builtin_amdgcn_sched_barrier(0);
    multiply(f2);
  }

  // register r of fragment (i, j): token 16 i + 4 q + r, weight row 16 j + l16
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][16 * i + 4 * q + r][16 * j + l16] = acc[i][j][r];
  __syncthreads();
  const int row = tid >> 3, ch = 8 * (tid & 7);  // 8 of the tile's 64 sums per thread
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = part[0][row][ch + k];
#pragma unroll
  for (int w = 1; w < NW; ++w)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += part[w][row][ch + k];
  const int64_t at = gi.off + row0 + row;
  const bool live_row = row <= a_last;
  const float p = !live_row ? 0.0f : args.probs != nullptr ? args.probs[at] : 1.0f;
  if constexpr (!GRAD) {
    // lanes 0 .. 3 of a row hold a, 4 .. 7 b
    if (args.ab != nullptr && live_row) {
      v8s w;
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = (short)f32_to_bf16(v[k]);
      *(v8s*)(args.ab + at * 2 * F + (ch < 32 ? 0 : F - 32) + col0 + ch) = w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float b = __shfl_xor(v[k], 4, 64);
      v[k] = live_row ? swiglu(v[k], b, p) : 0.0f;  // in the lanes that hold a
    }
    const GluTileOut o = glu_tile_out(args.out, args.R, F, gi, row0, col0);
    put_row8(o, row, ch, live_row && ch < 32, v);
    if (args.out.col_q != nullptr) {
      __syncthreads();  // every thread has read its sums
      if (ch < 32)
#pragma unroll
        for (int k = 0; k < 8; ++k) part[0][row][ch + k] = v[k];
      __syncthreads();
      if (wave == 0) {
        float c[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) c[k] = part[0][k][lane & 31];
        put_col32(o, 0, lane, lane < 32, c);
      }
    }
  } else {
    v8s av = {0, 0, 0, 0, 0, 0, 0, 0}, bv = av;
    const bool live = live_row && ch <= b_last;
    if (live) {
      const uint16_t* ab = args.ab + at * 2 * F + col0 + ch;
      av = *(const v8s*)ab;
      bv = *(const v8s*)(ab + F);
    }
    float da[8], db[8], dp = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) swiglu_grad(to_f32(av[k]), to_f32(bv[k]), p, live ? v[k] : 0.0f, da[k], db[k], dp);
    const GluTileOut oa = glu_tile_out(args.out, args.R, 2 * F, gi, row0, col0);
    const GluTileOut ob = glu_tile_out(args.out, args.R, 2 * F, gi, row0, F + col0);
    put_row8(oa, row, ch, live, da);
    put_row8(ob, row, ch, live, db);
    dp += __shfl_xor(dp, 1, 64);
    dp += __shfl_xor(dp, 2, 64);
    dp += __shfl_xor(dp, 4, 64);
    if (args.dpart != nullptr && (lane & 7) == 0 && live_row) args.dpart[(int64_t)tn * args.R + at] = dp;
    if (args.out.col_q != nullptr) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        part[0][row][ch + k] = da[k];
        part[1][row][ch + k] = db[k];
      }
      __syncthreads();
      if (wave < 2) {
        float c[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) c[k] = part[wave][k][lane];
        put_col32(wave == 0 ? oa : ob, 0, lane, lane <= b_last, c);
      }
    }
  }
  // the group's last tile also writes the pad lanes of the 32-row blocks that have no tile
  if (args.out.col_q != nullptr && row0 + BM >= gi.k) {
    constexpr int HALVES = GRAD ? 2 : 1;
    const int64_t N = HALVES * F;
    const int64_t first = row0 + BM, blocks = (gi.kp - first) / 32;  // at most 3
    for (int64_t x = tid; x < blocks * HALVES * COLS; x += NT) {
      const int c = (int)(x % COLS), half = (int)(x / COLS % HALVES);
      const int64_t t = first + 32 * (x / (COLS * HALVES)), col = half * F + col0 + c;
      if (c > b_last) continue;
      uint8_t* dst = args.out.col_q + col_elem(N, gi.p, gi.kp, col, t);
      *(v4i*)dst = v4i{0, 0, 0, 0};
      *(v4i*)(dst + 16) = v4i{0, 0, 0, 0};
      args.out.col_s[col_e8m0(N, gi.p, t / 32, col)] = 0;
    }
  }
}

// dprobs[row] = sum of the tile columns' parts, in order; rows past the last group's are not touched.
__global__ __launch_bounds__(256) void glu_dprobs_kernel(const float* __restrict__ part, int tiles_n, int64_t R,
                                                         const int32_t* __restrict__ splits, int E, float* dprobs) {
  __shared__ int64_t total[4];
  __shared__ int bad;
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  int64_t t = 0;
  for (int e = threadIdx.x; e < E; e += 256) {
    const int k = splits[e];
    if (k < 0) bad = 1;
    t += k;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) t += __shfl_xor(t, d, 64);
  if ((threadIdx.x & 63) == 0) total[threadIdx.x >> 6] = t;
  __syncthreads();
  t = total[0] + total[1] + total[2] + total[3];
  if (bad || t > R || row >= t) return;
  float s = 0.0f;
  for (int n = 0; n < tiles_n; ++n) s += part[(int64_t)n * R + row];
  dprobs[row] = s;
}

// ------------------------------------------------------------------------------------------
// Launchers
// ------------------------------------------------------------------------------------------

// Tile of a launch, by the rows of tiles that it is likely to have (groups end half a tile early on average: R / BM
// + E / 2).  Measured over 2 to 32 experts, hidden 2048 and 4096, ffn 512 to 2048, 8 to 2048 rows per expert
// (unequal ones), forward / gradient:
//  - few rows per expert, or so few tiles that the few-rows kernel's fill the chip better: at most 12 rows per
//    expert (8 experts of 8, 4096 x 2048: 30 / 30 us, 128 x 128 tiles 41 / 52) or 512 tiles (48 rows, 2048 x 1024: 21 /
//    20 us, 26 / 34; from 640 tiles on it loses, 39 / 34 to 25 / 34)
//  - the gradient: 128 x 128, K steps of 128, two workgroups per CU.  Steps of 64 and three workgroups take 0 to 11% longer
//    (8 experts, 4128 x 1024, 6500 rows: 93 us to 86; 16384 rows: 196 to 192; 16 experts of 512 rows, 2048 x 1024, are the
//    one shape that they suit: 79 to 81), 256 x 256 tiles 1 to 40% (16384 rows of 8 experts, 4096 x 2048: 392 to 328; 65536
//    rows: 8 experts of 2048 x 2048 797 to 747, 32 of 4096 x 2048 1235 to 1220, 16 of 7168 x 2048 1890 to 1876)
//  - the forward, up to two tiles per CU: the same (8 experts of 128 rows, 2048 x 1024 and 4096 x 2048: 26 and 63 us, steps
//    of 64 27 and 67)
//  - the forward, 128 x 128, more tiles: steps of 64, three workgroups per CU and loads two steps ahead where all tiles are
//    on the chip at once (768; 4099 rows of 8 experts at hidden 2048, 4128, 7168 and ffn 1024: 61, 120, 170 us, steps of 128
//    63, 120, 172) or K is short (16384 rows, 2048 x 1024, 8 and 32 experts: 179 and 187, steps of 128 181 and 192); else
//    steps of 128, whose barriers are half as many (6500 rows of 8 experts, 4128 and 7168 x 1024: 149 and 222, steps of 64
//    162 and 235; 16384 rows, 4128 x 1024: 318 to 336)
//  - the forward, 256 x 256 from 4096 tiles on (65536 rows: 8 experts of 2048 x 2048 1117 us, 32 of 4096 x 2048 2012, 16 of
//    7168 x 2048 3264; the better 128 x 128 tiles 1144, 2068, 3334.  Below: 49152 rows of 32 experts, 2048 x 2048, 3328
//    tiles, 909 to 893, 20480 rows, 4096 x 2048, 1536 tiles, 727 to 710)
// (operands from HBM, in sets taken in turn; random codes, which draw more power than a layer's)
struct GluTile {
  int bm, bn, bk;
};

// (K is not asked for where the gradient's workspace is sized)
static GluTile glu_tile(bool grad, int64_t R, int64_t F, int E, int64_t K) {
  auto tiles = [&](int bm, int bn) {
    const int64_t cols = grad ? bn : bn / 2;
    return (R / bm + (E + 1) / 2) * ((F + cols - 1) / cols);
  };
  // (the few-rows kernel addresses four block rows of scales with 32-bit offsets)
  if (R < (1 << 24) && 2 * F * E < (1 << 28) && (R <= 12 * (int64_t)E || tiles(kRowsBM, kRowsBN) <= 512))
    return {kRowsBM, kRowsBN, 0};
  if (grad) return {128, 128, 128};
  if (tiles(256, 256) >= 4096) return {256, 256, 128};
  const int64_t n = tiles(128, 128);
  return {128, 128, n > 512 && (n <= 768 || K <= 2048) ? 64 : 128};
}

// Columns of one half per tile, and the tiles of a row of them.
static int64_t glu_tiles_n(bool grad, GluTile t, int64_t F) {
  const int64_t c = grad ? t.bn : t.bn / 2;
  return (F + c - 1) / c;
}

size_t glu_grad_workspace_bytes(int64_t R, int64_t F, int E) {
  const int64_t n = glu_tiles_n(true, glu_tile(true, R, F, E, 0), F);
  return n > 1 ? (size_t)(n * R * 4) : 0;
}

// The grid of a launch: rows of tiles that any valid sizes can need (at most one per row), in whole runs.
static int glu_grid(GluArgs& a, bool grad, GluTile t, dim3* grid) {
  a.tiles_n = (int)glu_tiles_n(grad, t, a.F);
  const int64_t gm = fprop_run_mtiles(a.tiles_n);
  int64_t mt = (a.R + (int64_t)(t.bm - 1) * a.E) / t.bm;
  if (mt > a.R) mt = a.R;
  a.tiles = (mt + gm - 1) / gm * gm * a.tiles_n;
  if (xcd_launch_size(a.tiles) > 0x7fffffff) return BSFP8_ERR_SHAPE;
  *grid = dim3((unsigned)xcd_launch_size(a.tiles));
  return BSFP8_OK;
}

template <bool GRAD, int BM, int BN, int WN, int BK, int NS>
static void launch_glu_tile(const GluArgs& a, dim3 grid, hipStream_t stream) {
  hipLaunchKernelGGL((glu_gemm_kernel<GRAD, BM, BN, WN, BK, NS>), grid, dim3(128 * BN / WN), 0, stream, a);
}

template <bool GRAD>
static int launch_glu(GluArgs& a, hipStream_t stream) {
  const GluTile t = glu_tile(GRAD, a.R, a.F, a.E, a.K);
  dim3 grid;
  const int rc = glu_grid(a, GRAD, t, &grid);
  if (rc != BSFP8_OK) return rc;
  if (t.bm == kRowsBM) hipLaunchKernelGGL((glu_rows_kernel<GRAD>), grid, dim3(64 * kRowsNW), 0, stream, a);
  else if (GRAD || (t.bn == 128 && t.bk == 128)) launch_glu_tile<GRAD, 128, 128, 64, 128, 2>(a, grid, stream);
  else if (t.bn == 256) launch_glu_tile<false, 256, 256, 64, 128, 2>(a, grid, stream);
  else launch_glu_tile<false, 128, 128, 64, 64, 3>(a, grid, stream);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

int launch_grouped_gemm_swiglu(const uint8_t* x_q, const uint8_t* x_s, int64_t R, int64_t hidden, const uint8_t* w_q,
                               const uint8_t* w_s, int64_t F, const float* probs, const int32_t* splits, int E,
                               void* ab, void* y, int y_f32, uint8_t* row_q, uint8_t* row_s, uint8_t* col_q,
                               uint8_t* col_s, uint32_t* status, hipStream_t stream) {
  GluArgs a{};
  a.a_q = x_q;
  a.a_s = x_s;
  a.b_q = w_q;
  a.b_s = w_s;
  a.R = R;
  a.K = hidden;
  a.F = F;
  a.b_ld = hidden;  // W1 rowwise [E * 2F][hidden], scales [hidden / 32][E * 2F]
  a.b_estride = 2 * F * hidden;
  a.bs_estride = 2 * F;
  a.bs_bstride = (int64_t)E * 2 * F;
  a.splits = splits;
  a.E = E;
  a.probs = probs;
  a.ab = (uint16_t*)ab;
  a.out = GluOut{y, y_f32, row_q, row_s, col_q, col_s};
  a.status = status;
  return launch_glu<false>(a, stream);
}

int launch_grouped_gemm_swiglu_grad(const uint8_t* dy_q, const uint8_t* dy_s, int64_t R, int64_t hidden,
                                    const uint8_t* w_q, const uint8_t* w_s, int64_t F, const void* ab,
                                    const float* probs, const int32_t* splits, int E, void* dab, uint8_t* row_q,
                                    uint8_t* row_s, uint8_t* col_q, uint8_t* col_s, float* dprobs, float* workspace,
                                    uint32_t* status, hipStream_t stream) {
  GluArgs a{};
  const int64_t hp = col_padded_rows(hidden);  // W2 colwise: expert e's F channels of hp codes each
  a.a_q = dy_q;
  a.a_s = dy_s;
  a.b_q = w_q;
  a.b_s = w_s;
  a.R = R;
  a.K = hidden;
  a.F = F;
  a.b_ld = hp;
  a.b_estride = col_group_bytes(F, hp, 1);
  a.bs_estride = col_e8m0_group(F, hp);
  a.bs_bstride = col_e8m0_block_stride(F);
  a.splits = splits;
  a.E = E;
  a.probs = probs;
  a.ab = (uint16_t*)const_cast<void*>(ab);
  a.out = GluOut{dab, 0, row_q, row_s, col_q, col_s};
  a.status = status;
  const bool parts = dprobs != nullptr && glu_tiles_n(true, glu_tile(true, R, F, E, hidden), F) > 1;
  a.dpart = parts ? workspace : dprobs;
  const int rc = launch_glu<true>(a, stream);
  if (rc != BSFP8_OK || !parts) return rc;
  hipLaunchKernelGGL(glu_dprobs_kernel, dim3((unsigned)((R + 255) / 256)), dim3(256), 0, stream, workspace,
                     a.tiles_n, R, splits, E, dprobs);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
