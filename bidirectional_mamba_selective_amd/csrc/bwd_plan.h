// Host-side decomposition of the scan's backward pass and the layout of its
// caller-provided workspace.  Pure host code: no HIP calls.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "plan.h"

namespace bimamba {

// Wavefronts the chunking aims to give the main backward kernel: two per SIMD of a 256-CU part, all of them resident.
constexpr int64_t kBwdTargetWaves = 2048;

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

inline BwdPlan make_bwd_plan(int64_t batch, int64_t seqlen, int64_t d_inner, int64_t d_state) {
  BwdPlan p{};
  p.batch = batch;
  p.seqlen = seqlen;
  p.d_inner = d_inner;
  p.d_state = d_state;
  const int64_t row_waves = batch * (d_inner / kLanes);
  const int64_t want_chunks = (kBwdTargetWaves + row_waves - 1) / row_waves;
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
