// Host-side decomposition of the gated delta rule: chunks of tokens, the operands that the walk over them reads, and the
// layout of the workspace.  Pure host code: no HIP calls.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "plan.h"

namespace bimamba {
namespace delta {

constexpr int64_t kC = 64;            // tokens per chunk
// Tokens up to which the forward pass goes token by token, without a workspace: 16, and 24 where the states hold 2^22
// values.  By chunks a call takes as long for 1 token as for 64 (token by token | by chunks, us; batch x heads of
// 128 x 128 unless given):
//    8 tokens:  32: 11.6 | 14.9   512: 24.5 | 54.5
//   16 tokens:  32: 19.4 | 14.9   128: 21.0 | 22.8   256: 23.3 | 33.4   512: 37.0 | 55.3   of 64 x 64: 32: 15.0 | 13.6
//   24 tokens: 128: 28.6 | 23.2   256: 31.0 | 33.8   512: 49.6 | 56.1   of 64 x 64: 256: 22.1 | 18.2, 1024: 33.8 | 41.0
//   28 tokens: 256: 34.8 | 34.2   512: 55.5 | 56.6   1024: 95.1 | 98.2
// With few heads chunks are the faster way from 12 tokens on, by up to 4.5 us at 16: a decoding block of 16 tokens gets by
// without a workspace whatever its heads.
constexpr int64_t kStepTokens = 16, kStepTokensWide = 24, kStepWide = int64_t{1} << 22;

inline bool token_by_token(int64_t batch, int64_t seqlen, int64_t heads, int64_t dk, int64_t dv) {
  return seqlen <= (batch * heads * dk * dv >= kStepWide ? kStepTokensWide : kStepTokens);
}

constexpr size_t kFragBytes = 1024;   // one matrix operand of 16 x 32 bf16 values, 16 bytes a lane
constexpr int64_t kTriFrags = 6;      // operands that a triangular 64 x 64 matrix has (of 8; the others are zero)
constexpr int64_t kGateFloats = 320;  // per (head, chunk): five rows of 64, see k_delta_prep

// What the preparing kernel leaves for one (batch element, head, chunk), in bytes from the start of its record.
struct Layout {
  size_t gates, t, tt, a, at, bytes;  // forward: t, a; backward: t, tt, at
  size_t key_bytes;                   // per (batch element, key head, chunk): K^T, backward also Q^T
};

inline Layout make_layout(int64_t dk, bool grad) {
  Layout l{};
  size_t off = kGateFloats * 4;
  l.t = off, off += kTriFrags * 3 * kFragBytes;
  if (grad) {
    l.tt = off, off += kTriFrags * 3 * kFragBytes;
    l.at = off, off += kTriFrags * 3 * kFragBytes;
  } else {
    l.a = off, off += kTriFrags * 3 * kFragBytes;
  }
  l.bytes = align256(off);
  l.key_bytes = static_cast<size_t>(dk / 16) * 2 * kFragBytes * (grad ? 2 : 1);
  return l;
}

// Columns of a value head that one workgroup of a walk takes, in tiles of 16.  While 16 each give every compute unit at most
// one workgroup a step is latency, and narrower is faster (32 heads of 128 columns, 4096 tokens: forward 188 us with 16,
// 205 with 32; backward 722 and 786); beyond that what a step reads is shared by more columns (64 heads: 4096 tokens
// forward 355 us with 16, 273 with 32; 2048 backward 720 and 607; 128 heads 700 and 525, 1400 and 1156).
inline int walk_tiles(int64_t heads, int64_t dv) {
  return heads * (dv / 16) <= 256 ? 1 : 2;
}

struct Plan {
  int64_t nchunk;  // ceil(seqlen / kC)
  int64_t seg;     // chunks prepared at a time (forward); nchunk (backward)
  int tiles;
  size_t head_off, key_off, carry_off, s_off, ds_off, u_off, dr_off, part_off, total;
};

// Forward: the operands of `seg` chunks of every head at a time, so that they are read from the last-level cache (256 MiB)
// rather than from memory; the states between two segments.  Segments of 32, 64, 96, 128 and 160 MiB: 65536 tokens of 32
// heads of 128 x 128 in 3.07, 2.78, 2.65, 2.71 and 2.99 ms, 16384 tokens in 781, 714, 673, 699 and 749 us, 4 x 8192
// tokens in 1.10, 1.17, 1.05, 1.10 and 1.14 ms.
constexpr size_t kSegBytes = size_t{96} << 20;

inline Plan make_fwd_plan(int64_t batch, int64_t seqlen, int64_t hk, int64_t heads, int64_t dk, int64_t dv) {
  Plan p{};
  p.nchunk = (seqlen + kC - 1) / kC;
  p.tiles = walk_tiles(batch * heads, dv);
  if (token_by_token(batch, seqlen, heads, dk, dv)) return p;
  const Layout l = make_layout(dk, false);
  const size_t per_chunk = static_cast<size_t>(batch) * (heads * l.bytes + hk * l.key_bytes);
  int64_t seg = static_cast<int64_t>(kSegBytes / per_chunk);
  seg = seg < 8 ? 8 : seg;
  // segments of equal length
  const int64_t n = (p.nchunk + seg - 1) / seg;
  p.seg = (p.nchunk + n - 1) / n;
  p.head_off = 0;
  size_t off = static_cast<size_t>(batch) * heads * p.seg * l.bytes;
  p.key_off = off, off += align256(static_cast<size_t>(batch) * hk * p.seg * l.key_bytes);
  p.carry_off = off;
  if (p.seg < p.nchunk) off += align256(static_cast<size_t>(batch) * heads * dk * dv * 4);
  p.total = off;
  return p;
}

// Backward: the operands, both states (entering from the left, gradient entering from the right), U and the gradient of
// its right-hand side for every chunk, and the chunks' partial sums of the gradients of A and dt_bias.
inline Plan make_bwd_plan(int64_t batch, int64_t seqlen, int64_t hk, int64_t heads, int64_t dk, int64_t dv) {
  Plan p{};
  p.nchunk = (seqlen + kC - 1) / kC;
  p.seg = p.nchunk;
  p.tiles = walk_tiles(batch * heads, dv);
  const Layout l = make_layout(dk, true);
  const size_t hc = static_cast<size_t>(batch) * heads * p.nchunk;
  p.head_off = 0;
  size_t off = hc * l.bytes;
  p.key_off = off, off += align256(static_cast<size_t>(batch) * hk * p.nchunk * l.key_bytes);
  p.s_off = off, off += hc * dk * dv * 4;
  p.ds_off = off, off += hc * dk * dv * 4;
  p.u_off = off, off += hc * kC * dv * 4;
  p.dr_off = off, off += hc * kC * dv * 4;
  p.part_off = off, off += align256(hc * 8);
  p.total = off;
  return p;
}

}  // namespace delta
}  // namespace bimamba
