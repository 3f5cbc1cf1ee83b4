// Launch shapes of the router's and the plan's kernels, shared by the launchers and the workspace queries.
#pragma once

#include <stdint.h>

namespace bsfp8 {

// Router: lanes per token (a row of 16 where 16 values a lane hold all experts, a wave above) and the workgroups of 4
// waves, each walking every gridDim-th set of tokens: at most 8 per CU, as many as partial sums of the scores (131072
// tokens, 128 experts: 44 us then, with 4 per CU 47).  The gradient asks for its next tokens ahead and takes 4 per CU (33 us,
// with 8 per CU 35).
inline int route_lanes(int experts) { return experts <= 256 ? 16 : 64; }
inline int64_t route_blocks(int64_t tokens, int experts, bool grad = false) {
  const int64_t per = 256 / route_lanes(experts), need = (tokens + per - 1) / per, most = grad ? 1024 : 2048;
  return need < most ? need : most;
}

// Plan: choices are sorted in chunks of whole 4096s, at most 512 of them, one workgroup each.
constexpr int64_t kPlanUnit = 4096;
inline int64_t plan_chunk(int64_t choices) {
  const int64_t units = (choices + kPlanUnit - 1) / kPlanUnit;
  return (units + 511) / 512 * kPlanUnit;
}
inline int64_t plan_chunks(int64_t choices) {
  return choices == 0 ? 0 : (choices + plan_chunk(choices) - 1) / plan_chunk(choices);
}

// Counts of a chunk in the workspace: one per expert and one of the dropped choices, in whole vectors of 4.
#if defined(__HIPCC__)
__host__ __device__
#endif
constexpr int plan_hist_row(int experts) { return (experts + 4) / 4 * 4; }

}  // namespace bsfp8
