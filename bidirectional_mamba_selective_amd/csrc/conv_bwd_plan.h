// Host-side decomposition of the short convolution's backward pass and the
// layout of its workspace.  Pure host code: no HIP calls.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "plan.h"

namespace bimamba {
namespace conv {

constexpr int64_t kBwdBlk = 8;     // tokens per window step
constexpr int64_t kBwdChans = 128; // channels per wavefront, two per lane
constexpr int64_t kBwdWaves = 4;   // wavefronts per workgroup: consecutive tiles of the same channels
constexpr int64_t kBwdTargetWaves = 8192;
constexpr int64_t kBwdTileMax = 256;
constexpr int kBwdSums = 10;       // dw_f[4], db_f, dw_r[4], db_r

struct BwdPlan {
  int64_t tile;    // tokens per wavefront (multiple of kBwdBlk)
  int64_t groups;  // workgroups along the tokens of one sequence
  int64_t cblocks; // workgroups along the channels
  size_t total;    // partial sums [batch][group][kBwdSums][channels] fp32
};

// Longer tiles re-read fewer halo rows (6 of u and 3 of each gradient per tile) and leave fewer partial sums; shorter
// ones fill the chip.  A tile's rows with their halo must fit one buffer resource (2^31 - 1 bytes).
inline BwdPlan make_conv_bwd_plan(int64_t batch, int64_t L, int64_t C) {
  BwdPlan p{};
  p.cblocks = (C + kBwdChans - 1) / kBwdChans;
  const int64_t columns = batch * p.cblocks;
  const int64_t want = (kBwdTargetWaves + columns - 1) / columns;  // tiles per sequence
  int64_t tile = (L + want - 1) / want;
  tile = (tile + kBwdBlk - 1) / kBwdBlk * kBwdBlk;
  if (tile > kBwdTileMax) tile = kBwdTileMax;
  const int64_t fits = INT32_MAX / (C * 4) - 16;  // fp32 rows
  if (tile > fits) tile = fits / kBwdBlk * kBwdBlk;
  p.tile = tile;
  p.groups = (L + tile * kBwdWaves - 1) / (tile * kBwdWaves);
  p.total = align256(static_cast<size_t>(batch) * p.groups * kBwdSums * C * sizeof(float));
  return p;
}

}  // namespace conv
}  // namespace bimamba
