// Host-side decomposition of the scan's backward pass and the layout of its
// caller-provided workspace.  Pure host code: no HIP calls.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "plan.h"

namespace bimamba {

// Wavefronts of the main backward kernel that a 256-CU part holds at once: two per SIMD.
constexpr int64_t kBwdResidentWaves = 2048;

struct BwdPlan {
  int64_t batch, seqlen, d_inner, d_state;
  int64_t chunk;   // tokens per chunk (multiple of kSub)
  int64_t nchunk;  // chunks per sequence
  int64_t nsub;    // tiles per full chunk (chunk / kSub)
  int64_t ntile;   // kSub-token tiles per sequence (chunks start on tile boundaries)
  // workspace offsets in bytes (each 256-byte aligned): per chunk and state the summaries of the four chains
  // (overwritten by their carries) and the decay; per tile and state the two boundary states; per tile the
  // suffix sum of delta; the transposed A; the B/C table; the partial sums of dB and dC, of dA, and of dD and
  // the bias gradient
  size_t off_sf, off_sp, off_sr, off_sg, off_p, off_rr, off_rg, off_sig, off_a2t, off_bct, off_pbc, off_pa, off_pv;
  size_t total;
};

// Chunks per sequence for row_waves = batch * d_inner / 64 wavefronts per chunk: as many as stay resident together.  One
// more would leave a second round of a few wavefronts, each walking a whole chunk on an idle chip (bf16, both directions,
// N 16, rounded down against up: 5 x 2048 x 4096 896 against 1150 us, 8 x 1024 x 3840 672 against 874, 1 x 8192 x 3840 659
// against 663).  Above half of the resident number that would be one chunk, a wavefront per sequence, and two rounds of
// half the length are no longer than it: 20 x 512 x 4096 1121 against 1166 us, 31 x 512 x 4096 1358 either way.
inline int64_t bwd_chunks(int64_t row_waves) {
  const int64_t fit = kBwdResidentWaves / row_waves;
  return fit >= 2 ? fit : row_waves < kBwdResidentWaves ? 2 : 1;
}

inline BwdPlan make_bwd_plan(int64_t batch, int64_t seqlen, int64_t d_inner, int64_t d_state) {
  BwdPlan p{};
  p.batch = batch;
  p.seqlen = seqlen;
  p.d_inner = d_inner;
  p.d_state = d_state;
  const int64_t row_waves = batch * (d_inner / kLanes);
  const int64_t want_chunks = bwd_chunks(row_waves);
  int64_t chunk = (seqlen + want_chunks - 1) / want_chunks;
  chunk = ((chunk + kSub - 1) / kSub) * kSub;
  p.chunk = chunk;
  p.nchunk = (seqlen + chunk - 1) / chunk;
  p.nsub = chunk / kSub;
  p.ntile = (seqlen + kSub - 1) / kSub;
  const size_t row = static_cast<size_t>(d_inner) * sizeof(float);
  const size_t state = static_cast<size_t>(batch) * p.nchunk * d_state * row;
  const size_t bound = static_cast<size_t>(batch) * p.ntile * d_state * row;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  p.off_sf = take(state);
  p.off_sp = take(state);
  p.off_sr = take(state);
  p.off_sg = take(state);
  p.off_p = take(state);
  p.off_rr = take(bound);
  p.off_rg = take(bound);
  p.off_sig = take(static_cast<size_t>(batch) * p.ntile * row);
  p.off_a2t = take(static_cast<size_t>(d_state) * row);
  p.off_bct = take(static_cast<size_t>(batch) * p.ntile * d_state * 2 * kSub * sizeof(float));
  p.off_pbc = take(static_cast<size_t>(batch) * p.ntile * (d_inner / kLanes) * d_state * 2 * kSub * sizeof(float));
  p.off_pa = take(state);
  p.off_pv = take(static_cast<size_t>(batch) * p.nchunk * 2 * row);
  p.total = off;
  return p;
}

}  // namespace bimamba
