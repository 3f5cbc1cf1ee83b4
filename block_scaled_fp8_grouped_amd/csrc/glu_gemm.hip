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
//
// Tile: 256 tokens x 256 rows of the weight, K step 128, 8 waves of 128 x 64, double-buffered LDS
// filled by LDS DMA, XOR-swizzled 16-byte chunks.  In the forward the 256 weight rows are 128 rows of
// each projection, interleaved 32 by 32: a wave's two column fragments are a and b of the same 32
// outputs, so a lane holds both halves of its elements in registers and the activation needs no
// exchange.  Wave w fetches LDS rows 32 w .. 32 w + 31, which are 32 rows of one projection (w & 1),
// so the interleave costs one scalar base per wave.
//
// Epilogue: a wave owns its block from its accumulators to memory, 32 rows at a time through its own
// piece of LDS (no barrier): rows of 8 columns per lane for the row-major outputs, whole 32-token
// columns per lane for the colwise ones.
//
// One workgroup per tile, fixed order, no atomics: the same bits every time.  Rows past a group's
// live rows read as zeros and are not stored; the colwise pad lanes get the zeros that those rows
// compute.
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

__device__ __forceinline__ void glu_dma16(__amdgpu_buffer_rsrc_t rs, uint8_t* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)lds, 16, voff, 0, 0, 0);
}

// fp32 value 2^(byte - 127) of an E8M0 byte (byte 0: the subnormal 2^-127).
__device__ __forceinline__ float glu_e8m0(uint32_t byte) { return __uint_as_float(max(byte << 23, 0x00400000u)); }

// Eight e4m3 codes -> eight bf16 values times `scale` (exact).
__device__ __forceinline__ v8bf glu_widen8(int d0, int d1, float scale) {
  const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)d0, scale, false);
  const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)d0, scale, true);
  const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)d1, scale, false);
  const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)d1, scale, true);
  return v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

constexpr int kGluBM = 256, kGluBN = 256;

template <bool GRAD>
struct GluShape {
  static constexpr int BM = kGluBM, BN = kGluBN, BK = 128, WM = 128, WN = 64, NW = 8, NT = 512;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int COLS = GRAD ? BN : BN / 2;  // output columns (of one half) per tile
  static constexpr int B_OFF = BM * BK, SA_OFF = (BM + BN) * BK, SB_OFF = SA_OFF + 16 * BM;
  static constexpr int STAGE = SB_OFF + 16 * BN;
  static constexpr int A_INS = BM / 8 / NW, B_INS = BN / 8 / NW;
  // epilogue: each wave's 32 rows of fp32, the row pitch shifting the rows 4 apart (one register's two
  // half-waves) by half of the 64 banks
  static constexpr int PITCH = GRAD ? 72 : 40;
  static constexpr int EP = 32 * PITCH * 4;
  static constexpr int SMEM = 2 * STAGE > NW * EP + 4 * BM * 4 ? 2 * STAGE : NW * EP + 4 * BM * 4;
  static_assert(SMEM + BM * 4 + (int)sizeof(GroupScanSmem<NT>) <= 160 * 1024, "LDS budget");
};

template <bool GRAD, bool KTAIL>
__global__ __launch_bounds__(512) void glu_gemm_kernel(GluArgs args) {
  using S = GluShape<GRAD>;
  constexpr int BM = S::BM, BN = S::BN, BK = S::BK, NT = S::NT, FM = S::FM, FN = S::FN;
  __shared__ GroupScanSmem<NT> gsm;
  __shared__ float probs[BM];
  __shared__ __attribute__((aligned(16))) uint8_t smem[S::SMEM];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, l32 = lane & 31;
  const int wm = wave & 1, wn = wave >> 1;

  const int64_t L = xcd_logical(blockIdx.x);
  if (L >= args.tiles) return;
  int64_t mt;
  int tn;
  fprop_tile(L, args.tiles_n, &mt, &tn);
  GroupInfo gi;
  const uint32_t flags = group_scan<NT>(args.splits, args.E, args.R, BM, mt, 0, gsm, gi);
  report_status(args.status, flags);
  if (gi.e < 0) return;
  const int64_t row0 = (mt - gi.tile) * BM;  // the tile's first row within the group (< gi.k)
  const int64_t col0 = (int64_t)tn * S::COLS;
  const int64_t F = args.F, K = args.K;
  const int a_last = (int)(gi.k - row0 < BM ? gi.k - row0 : BM) - 1;      // last live tile row
  const int b_last = (int)(F - col0 < S::COLS ? F - col0 : S::COLS) - 1;  // last live column of a half
  if (tid < BM)
    probs[tid] = tid > a_last ? 0.0f : args.probs != nullptr ? args.probs[gi.off + row0 + tid] : 1.0f;

  // ---------------- loads of one K step ----------------
  // B: LDS rows 32 w .. of wave w; forward: rows 32 (w / 2) .. of projection w % 2
  const int64_t half = GRAD ? 0 : (int64_t)(wave & 1) * F;
  const uint32_t b_shift = GRAD ? 0 : (uint32_t)(wave * 32 - (wave >> 1) * 32);  // LDS row minus source row
  const uint8_t* a_base = args.a_q + (gi.off + row0) * K;
  const uint8_t* b_base = args.b_q + gi.e * args.b_estride + (half + col0) * args.b_ld;
  const __amdgpu_buffer_rsrc_t a_rs =
      __builtin_amdgcn_make_buffer_rsrc((void*)a_base, (short)0, (int)tile_range(gi.k - row0, K), 0x00020000);
  const __amdgpu_buffer_rsrc_t b_rs =
      __builtin_amdgcn_make_buffer_rsrc((void*)b_base, (short)0, (int)tile_range(F - col0, args.b_ld), 0x00020000);
  uint32_t a_off[S::A_INS], b_off[S::B_INS];
#pragma unroll
  for (int u = 0; u < S::A_INS; ++u) a_off[u] = tile_dma_voffset(wave * S::A_INS + u, lane, (uint32_t)K, 0);
#pragma unroll
  for (int u = 0; u < S::B_INS; ++u)
    b_off[u] = tile_dma_voffset(wave * S::B_INS + u, lane, (uint32_t)args.b_ld, 0) - b_shift * (uint32_t)args.b_ld;
  // scales: threads of waves 2 b, 2 b + 1 take block b's A bytes (two rows each; a group's rows begin
  // anywhere), waves 4 + b its B bytes (4 LDS rows per lane, which lie in one run of 32 columns)
  const int sa_blk = wave >> 1, sa_row = 2 * ((wave & 1) * 64 + lane);
  const uint8_t* a_sc = args.a_s + gi.off + row0;
  int sb_row;  // this lane's first B scale: column of its projection, pulled back to a live one
  int64_t sb_half = 0;
  if constexpr (GRAD) {
    sb_row = scale_dma_row(0, lane, b_last);
  } else {
    sb_row = scale_dma_row(0, (lane >> 4) * 8 + (lane & 7), b_last);
    sb_half = ((lane >> 3) & 1) * F;
  }
  const uint8_t* b_sc = args.b_s + gi.e * args.bs_estride + sb_half + col0 + sb_row;
  uint8_t sa[2];
  uint32_t sb = 0;
  const int nk = (int)((K + BK - 1) / BK);
  // parts [p0, p1): 0 the scales, then A_INS + B_INS DMAs
  auto issue = [&](int kk, uint8_t* base, int p0, int p1) {
    const uint32_t k0 = (uint32_t)kk * BK;
    if (p0 == 0) {
      const int64_t kb = (int64_t)kk * 4 + sa_blk;
      if (!KTAIL || kb * 32 < K) {
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc((void*)(a_sc + kb * args.R), (short)0, a_last + 1, 0x00020000);
        sa[0] = __builtin_amdgcn_raw_buffer_load_b8(rs, sa_row, 0, 0);
        sa[1] = __builtin_amdgcn_raw_buffer_load_b8(rs, sa_row + 1, 0, 0);
      } else {
        sa[0] = sa[1] = 0x7f;  // past K: unit scales over zero data
      }
      if (wave >= 4) {
        const int64_t bb = (int64_t)kk * 4 + (wave - 4);
        sb = !KTAIL || bb * 32 < K ? *(const uint32_t*)(b_sc + bb * args.bs_bstride) : 0x7f7f7f7fu;
      }
    }
#pragma unroll
    for (int u = 0; u < S::A_INS; ++u) {
      if (1 + u < p0 || 1 + u >= p1) continue;
      glu_dma16(a_rs, base + (wave * S::A_INS + u) * 1024, a_off[u] + k0);
    }
#pragma unroll
    for (int u = 0; u < S::B_INS; ++u) {
      if (1 + S::A_INS + u < p0 || 1 + S::A_INS + u >= p1) continue;
      glu_dma16(b_rs, base + S::B_OFF + (wave * S::B_INS + u) * 1024, b_off[u] + k0);
    }
  };
  auto settle = [&](uint8_t* base) {  // this step's scales to the stage, as fp32
    float* fa = (float*)(base + S::SA_OFF) + sa_blk * BM + sa_row;
    fa[0] = glu_e8m0(sa[0]);
    fa[1] = glu_e8m0(sa[1]);
    if (wave >= 4)
      *(v4f*)((float*)(base + S::SB_OFF) + (wave - 4) * BN + 4 * lane) =
          v4f{glu_e8m0(sb & 0xffu), glu_e8m0((sb >> 8) & 0xffu), glu_e8m0((sb >> 16) & 0xffu), glu_e8m0(sb >> 24)};
  };
  auto wait_dma = [&]() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };

  v16f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  auto step = [&](bool tail, int kk, const uint8_t* __restrict__ cur, uint8_t* __restrict__ nxt) {
    const int64_t k0 = (int64_t)kk * BK;
    auto chunk = [&](const uint8_t* p, int c) {
      const v4i v = *(const v4i*)p;
      return !KTAIL || !tail || k0 + 16 * c < K ? v : v4i{0, 0, 0, 0};
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      v8i af[FM], bf[FN];
      float as[FM][2], bs[FN][2];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int row = wm * S::WM + i * 32 + l32;
        const v4i lo = chunk(cur + row * BK + (((4 * s + h) ^ swz(row)) << 4), 4 * s + h);
        const v4i hi = chunk(cur + row * BK + (((4 * s + 2 + h) ^ swz(row)) << 4), 4 * s + 2 + h);
        af[i] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        as[i][0] = ((const float*)(cur + S::SA_OFF))[(2 * s) * BM + row];
        as[i][1] = ((const float*)(cur + S::SA_OFF))[(2 * s + 1) * BM + row];
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int row = wn * S::WN + j * 32 + l32;
        const v4i lo = chunk(cur + S::B_OFF + row * BK + (((4 * s + h) ^ swz(row)) << 4), 4 * s + h);
        const v4i hi = chunk(cur + S::B_OFF + row * BK + (((4 * s + 2 + h) ^ swz(row)) << 4), 4 * s + 2 + h);
        bf[j] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        bs[j][0] = ((const float*)(cur + S::SB_OFF))[(2 * s) * BN + row];
        bs[j][1] = ((const float*)(cur + S::SB_OFF))[(2 * s + 1) * BN + row];
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        v8bf aw[FM], bw[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) aw[i] = glu_widen8(af[i][2 * t], af[i][2 * t + 1], as[i][t >> 1]);
#pragma unroll
        for (int j = 0; j < FN; ++j) bw[j] = glu_widen8(bf[j][2 * t], bf[j][2 * t + 1], bs[j][t >> 1]);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(aw[i], bw[j], acc[i][j], 0, 0, 0);
        // the next step's loads go out behind this half's reads, spread over its MFMA groups
        if (s == 0 && kk + 1 < nk) {
          constexpr int NP = S::A_INS + S::B_INS + 1;
          issue(kk + 1, nxt, t * NP / 4, (t + 1) * NP / 4);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };

  issue(0, smem, 0, 1 << 20);
  wait_dma();
  settle(smem);
  __syncthreads();
  const int nfull = KTAIL ? nk - 1 : nk;
  for (int kk = 0; kk < nfull; ++kk) {
    uint8_t* cur = smem + (kk & 1) * S::STAGE;
    uint8_t* nxt = smem + ((kk & 1) ^ 1) * S::STAGE;
    step(false, kk, cur, nxt);
    if (kk + 1 < nk) {
      wait_dma();
      settle(nxt);
    }
    __syncthreads();
  }
  if constexpr (KTAIL) {  // the step that runs past K (its loads were issued by the one before)
    step(true, nfull, smem + (nfull & 1) * S::STAGE, smem + ((nfull & 1) ^ 1) * S::STAGE);
    __syncthreads();
  }

  // ---------------- epilogue ----------------
  // register r of fragment (i, j): row 32 i + 8 (r / 4) + 4 h + r % 4, column 32 j + l32 of the block
  float* tile = (float*)(smem + wave * S::EP);
  constexpr int PITCH = S::PITCH;
  if constexpr (!GRAD) {
    const int cw = wn * 32;  // the wave's first column within the tile
    const int64_t col = col0 + cw;
    const bool cols = cw <= b_last;  // its 32 columns all exist, or none
    const int64_t N2 = 2 * F;
    // the kept product: a buffer resource over the block's live rows, its halves F columns apart
    const int left = a_last + 1 - wm * S::WM;
    const int vrows = left < 0 ? 0 : left > S::WM ? S::WM : left;
    const __amdgpu_buffer_rsrc_t ab_rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(args.ab + (gi.off + row0 + wm * S::WM) * N2 + col), (short)0,
        args.ab != nullptr && vrows > 0 && cols ? (int)(((int64_t)(vrows - 1) * N2 + F + 32) * 2) : 0, 0x00020000);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int rb = wm * S::WM + i * 32;
      float v[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v4f p = *(const v4f*)&probs[rb + 8 * q + 4 * h];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 4 * q + k;
          v[r] = swiglu(acc[i][0][r], acc[i][1][r], p[k]);
          if (args.ab != nullptr) {
            const uint32_t at = ((uint32_t)(i * 32 + 8 * q + 4 * h + k) * (uint32_t)N2 + (uint32_t)l32) * 2;
            __builtin_amdgcn_raw_buffer_store_b16((short)f32_to_bf16(acc[i][0][r]), ab_rs, (int)at, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b16((short)f32_to_bf16(acc[i][1][r]), ab_rs, (int)(at + 2 * (uint32_t)F), 0, 0);
          }
          tile[(8 * q + 4 * h + k) * PITCH + l32] = v[r];
        }
      }
      wave_lds_order();
      if (args.out.col_q != nullptr && row0 + rb < gi.kp) {
        float c[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) c[k] = tile[k * PITCH + l32];
        put_col32(args.out, F, gi, row0 + rb, col + l32, cols && h == 0, c);
      }
      if (args.out.y != nullptr || args.out.row_q != nullptr) {
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
          const int r = pass * 16 + (lane >> 2), ch = 8 * (lane & 3);
          float w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = tile[r * PITCH + ch + k];
          put_row8(args.out, args.R, F, gi.off + row0 + rb + r, col + ch, cols && rb + r <= a_last, w);
        }
      }
      wave_lds_order();
    }
  } else {
    const int cw = wn * 64;
    float* dp_sum = (float*)(smem + S::NW * S::EP) + wn * BM;  // this wave's column part of dprobs, per row
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int rb = wm * S::WM + i * 32;
      const int ch = 8 * (lane & 7);
      const bool cols = cw + ch <= b_last;
      v8s av[4], bv[4];
#pragma unroll
      for (int pass = 0; pass < 4; ++pass) {
        const int r = rb + pass * 8 + (lane >> 3);
        av[pass] = bv[pass] = v8s{0, 0, 0, 0, 0, 0, 0, 0};
        if (cols && r <= a_last) {
          const uint16_t* p = args.ab + (gi.off + row0 + r) * 2 * F + col0 + cw + ch;
          av[pass] = *(const v8s*)p;
          bv[pass] = *(const v8s*)(p + F);
        }
      }
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) tile[(8 * (r >> 2) + 4 * h + (r & 3)) * PITCH + j * 32 + l32] = acc[i][j][r];
      wave_lds_order();
      float db[4][8];
#pragma unroll
      for (int pass = 0; pass < 4; ++pass) {
        const int r = pass * 8 + (lane >> 3);
        const float p = probs[rb + r];
        float da[8], dp = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          swiglu_grad(to_f32(av[pass][k]), to_f32(bv[pass][k]), p, tile[r * PITCH + ch + k], da[k], db[pass][k], dp);
        const bool live = cols && rb + r <= a_last;
        const int64_t row = gi.off + row0 + rb + r, col = col0 + cw + ch;
        put_row8(args.out, args.R, 2 * F, row, col, live, da);
        put_row8(args.out, args.R, 2 * F, row, F + col, live, db[pass]);
        dp += __shfl_xor(dp, 1, 64);
        dp += __shfl_xor(dp, 2, 64);
        dp += __shfl_xor(dp, 4, 64);
        if ((lane & 7) == 0) dp_sum[rb + r] = dp;
#pragma unroll
        for (int k = 0; k < 8; ++k) tile[r * PITCH + ch + k] = da[k];
      }
      if (args.out.col_q != nullptr && row0 + rb < gi.kp) {
        float c[32];
        const bool live = cw + lane <= b_last;
        wave_lds_order();
#pragma unroll
        for (int k = 0; k < 32; ++k) c[k] = tile[k * PITCH + lane];
        put_col32(args.out, 2 * F, gi, row0 + rb, col0 + cw + lane, live, c);
        wave_lds_order();
#pragma unroll
        for (int pass = 0; pass < 4; ++pass)
#pragma unroll
          for (int k = 0; k < 8; ++k) tile[(pass * 8 + (lane >> 3)) * PITCH + ch + k] = db[pass][k];
        wave_lds_order();
#pragma unroll
        for (int k = 0; k < 32; ++k) c[k] = tile[k * PITCH + lane];
        put_col32(args.out, 2 * F, gi, row0 + rb, F + col0 + cw + lane, live, c);
      }
      wave_lds_order();
    }
    if (args.dpart != nullptr) {
      __syncthreads();
      const float* s = (const float*)(smem + S::NW * S::EP);
      if (tid <= a_last) args.dpart[(int64_t)tn * args.R + gi.off + row0 + tid] = ((s[tid] + s[BM + tid]) + s[2 * BM + tid]) + s[3 * BM + tid];
    }
  }
}

// dprobs[row] = sum of the tile columns' parts, in order; rows past the last group's are not touched.
__global__ __launch_bounds__(256) void glu_dprobs_kernel(const float* __restrict__ part, int tiles_n, int64_t R,
                                                         const int32_t* __restrict__ splits, int E, float* dprobs) {
  __shared__ GroupScanSmem<256> gsm;
  GroupInfo gi;
  // the group of rows [256 b, 256 b + 256) laid end to end: tiles of one row
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const uint32_t flags = group_scan<256>(splits, E, R, 0, 0, E - 1, gsm, gi);
  if (flags || gi.e < 0 || row >= gi.off + gi.k) return;
  float s = 0.0f;
  for (int n = 0; n < tiles_n; ++n) s += part[(int64_t)n * R + row];
  dprobs[row] = s;
}

// ------------------------------------------------------------------------------------------
// Launchers
// ------------------------------------------------------------------------------------------

static int64_t glu_tiles_n(bool grad, int64_t F) {
  const int64_t c = grad ? GluShape<true>::COLS : GluShape<false>::COLS;
  return (F + c - 1) / c;
}

size_t glu_grad_workspace_bytes(int64_t R, int64_t F, int) {
  const int64_t n = glu_tiles_n(true, F);
  return n > 1 ? (size_t)(n * R * 4) : 0;
}

template <bool GRAD>
static int launch_glu(GluArgs& a, hipStream_t stream) {
  a.tiles_n = (int)glu_tiles_n(GRAD, a.F);
  const int64_t gm = fprop_run_mtiles(a.tiles_n);
  const int64_t mt = (a.R + (int64_t)(kGluBM - 1) * a.E) / kGluBM;
  a.tiles = (mt + gm - 1) / gm * gm * a.tiles_n;
  if (xcd_launch_size(a.tiles) > 0x7fffffff) return BSFP8_ERR_SHAPE;
  const dim3 grid((unsigned)xcd_launch_size(a.tiles)), block(512);
  if (a.K % 128 != 0) hipLaunchKernelGGL((glu_gemm_kernel<GRAD, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((glu_gemm_kernel<GRAD, false>), grid, block, 0, stream, a);
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
  const bool parts = dprobs != nullptr && glu_tiles_n(true, F) > 1;
  a.dpart = parts ? workspace : dprobs;
  const int rc = launch_glu<true>(a, stream);
  if (rc != BSFP8_OK || !parts) return rc;
  hipLaunchKernelGGL(glu_dprobs_kernel, dim3((unsigned)((R + 255) / 256)), dim3(256), 0, stream, workspace,
                     (int)glu_tiles_n(true, F), R, splits, E, dprobs);
  return hipGetLastError() == hipSuccess ? BSFP8_OK : BSFP8_ERR_LAUNCH;
}

}  // namespace bsfp8
