// Host-side decomposition of the norm / gate / residual step: rows of d_model
// values over workgroups, and the layout of the backward pass's workspace.
// Pure host code: no HIP calls.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "plan.h"

namespace bimamba {
namespace adaln {

constexpr int64_t kVec = 8;           // values per thread and vector load
constexpr int64_t kMaxWidth = 8192;   // widest row: 16 wavefronts, one vector per lane
constexpr int64_t kScaleCols = 128;   // columns that share a scale of the 8-bit output: 16 lanes
constexpr int64_t kFwdGroups = 2048;  // workgroups the forward pass aims at (8 per CU)
constexpr int kSums = 4;              // column sums of the backward pass: dgamma, dbeta, dgate, dpost_weight

// Wavefronts per row, one vector per lane.  A row of up to 512 values stays in one wavefront, and its sums need no
// barrier.
inline int waves_for(int64_t d) {
  int w = 1;
  while (w * 64 * kVec < d) w *= 2;
  return w;
}

// Workgroups of the backward pass that 256 CUs hold at once: its 132 to 157 registers allow 3 wavefronts per SIMD, so 12 per
// CU.  One round of them: 8 x 8192 rows of 2048 in 320 + 11 us (kernel and partial sums) at 768, 373 + 15 us at 1024 (a
// third of a round is left over), 335 + 8 us at 512.
inline int64_t bwd_resident(int waves) {
  const int per_wg = waves == 1 ? 4 : waves;
  return 256 * (per_wg >= 8 ? 1 : 12 / per_wg);
}

// Rows a workgroup holds at once.
inline int row_groups(int waves) { return waves == 1 ? 4 : 1; }

struct Plan {
  int waves;
  int64_t rows_per_wg;  // consecutive rows of one batch element
  int64_t chunks;       // workgroups per batch element
  size_t part_bytes;    // backward: partial column sums [batch][chunk][row group][kSums][d] fp32
};

// per_batch: workgroups per batch element at most.
inline Plan make_plan(int64_t batch, int64_t seqlen, int64_t d, int64_t per_batch) {
  Plan p{};
  p.waves = waves_for(d);
  const int64_t g = row_groups(p.waves);
  int64_t rows = (seqlen + per_batch - 1) / per_batch;
  rows = (rows + g - 1) / g * g;
  p.rows_per_wg = rows;
  p.chunks = (seqlen + rows - 1) / rows;
  p.part_bytes = align256(static_cast<size_t>(batch) * p.chunks * g * kSums * d * sizeof(float));
  return p;
}

inline Plan fwd_plan(int64_t batch, int64_t seqlen, int64_t d) {
  return make_plan(batch, seqlen, d, (kFwdGroups + batch - 1) / batch);
}

// Rounded down, so that the launch stays in its one round: rounded up, two workgroups past 256 walk their rows alone at the
// end (3 x 8192 rows of 4096: 455 against 261 us; 7 x 8192 of 2048: 402 against 292).  One per sequence above half of the
// resident number too: 512 x 128 of 2048 427 against 470 us, 129 x 256 of 4096 637 against 643.
inline Plan bwd_plan(int64_t batch, int64_t seqlen, int64_t d) {
  const int64_t fit = bwd_resident(waves_for(d)) / batch;
  return make_plan(batch, seqlen, d, fit > 1 ? fit : 1);
}

}  // namespace adaln
}  // namespace bimamba
