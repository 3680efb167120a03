// Internal interface between the C-ABI layer and the kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bwd_plan.h"
#include "conv_bwd_plan.h"
#include "delta_plan.h"
#include "plan.h"
#include "ssd_plan.h"

namespace bimamba {

enum : uint32_t { kNoGate = 1u, kFwdOnly = 2u, kRevOnly = 4u };

struct ScanArgs {
  const void* x;
  const void* dt;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* dt_bias;
  void* out;
  const float* h_in;  // forward state entering the sequence (NULL = zeros)
  float* h_out;       // forward state after the last token (NULL = not written)
  int io_dtype;       // 0 = fp32, 1 = bf16
  uint32_t flags;
};

// Three-kernel chunked scan (summary -> carry -> output) for any length.
// stage < 0 launches all three; 0, 1, 2 launch one of them.
hipError_t launch_chunked(const ScanArgs& a, const Plan& p, void* workspace, hipStream_t stream, int stage = -1);

// Size of the library's fixed device scratch array (csrc/scratch.hip), which holds the workspace of
// the allocation-free entry point.
constexpr size_t kScratchBytes = size_t{256} << 20;

// Address of the scratch array on the current device (looked up once per device).
hipError_t scratch_address(void** out);

// Single-kernel block step for block_len <= kBlockFusedMax: one workgroup per
// (16 channels, batch element), one lane per (channel, state) recurrence; no workspace.
hipError_t launch_block_fused(const ScanArgs& a, int64_t batch, int64_t block_len, int64_t d_inner,
                              int64_t d_state, hipStream_t stream);

// Backward pass of the scan: gradients of every input of ScanArgs for the gradient dout of out.
struct ScanBwdArgs {
  const void* dout;
  const void* x;
  const void* dt;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* dt_bias;
  void* dx;
  void* ddt;
  float* dA;
  void* dB;
  void* dC;
  float* dD;        // null = not written
  void* dz;         // null without the gate
  float* ddt_bias;  // null = not written
  int io_dtype;
  uint32_t flags;
};

hipError_t launch_scan_bwd(const ScanBwdArgs& a, const BwdPlan& p, void* workspace, hipStream_t stream);

namespace adaln {

// The norm / gate / residual step between two blocks; null pointers as in the C ABI.
struct AdalnArgs {
  const void* x;  // forward only
  const void* branch;
  const float* post_weight;
  const float* gate;
  const float* gamma;
  const float* beta;  // forward only
  void* h;            // written by the forward pass, read by the backward pass
  void* out;          // forward only
  int64_t batch, seqlen, d_model, mod_rows;
  float eps;
  int rms;
  int io_dtype;
  float* scales = nullptr;  // forward only: given, out is e4m3 with these scales
};

struct AdalnGrads {
  const void* dout;
  const void* dres;
  void* dx;
  void* dbranch;
  float* dpost_weight;
  float* dgate;
  float* dgamma;
  float* dbeta;
};

hipError_t launch_adaln_fwd(const AdalnArgs& a, hipStream_t stream);
hipError_t launch_adaln_bwd(const AdalnArgs& a, const AdalnGrads& g, void* workspace, hipStream_t stream);

}  // namespace adaln

namespace delta {

// The gated delta rule, one direction; null pointers as in the C ABI.
struct DeltaArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* dt;
  const float* A;
  const void* b;
  const float* dt_bias;
  const float* h_in;
  float* h_out;
  void* out;
  int64_t batch, seqlen, hk, heads, dk, dv;
  float scale;
  int rev;
};

struct DeltaGrads {
  const void* dout;
  const float* dh_out;  // null: 0
  void* dq;
  void* dk;
  void* dv;
  void* ddt;
  float* dA;
  void* db;
  float* ddt_bias;  // null: not written
  float* dh_in;     // null: not written
};

// Forward: token by token (no workspace) where token_by_token says so, by chunks otherwise.
hipError_t launch_delta_step(const DeltaArgs& a, hipStream_t stream);
hipError_t launch_delta_fwd(const DeltaArgs& a, const Plan& p, void* workspace, hipStream_t stream);
hipError_t launch_delta_bwd(const DeltaArgs& a, const DeltaGrads& g, const Plan& p, void* workspace,
                            hipStream_t stream);

// Its parts over chunks [chunk0, chunk0 + chunks): the chunks' operands, and the walk over them; `save` keeps for the
// backward pass what it meets and computes no output.
hipError_t launch_delta_prep(const DeltaArgs& a, const Plan& p, int64_t chunk0, int64_t chunks, bool grad,
                             void* workspace, hipStream_t stream);
hipError_t launch_delta_walk(const DeltaArgs& a, const Plan& p, int64_t chunk0, int64_t chunks, bool save,
                             const float* state_in, float* state_out, void* workspace, hipStream_t stream);

}  // namespace delta

namespace proj {

// Product of e4m3 rows x [m, k] and weights w [n, k] with block scales; out [m, n].
struct ProjArgs {
  const void* x;
  const float* xs;
  const void* w;
  const float* ws;
  void* out;
  int64_t m, n, k;
  int out_dtype;
};

hipError_t launch_proj(const ProjArgs& a, hipStream_t stream);

}  // namespace proj

namespace conv {

// Short causal / anti-causal depthwise convolution (width 4) with optional SiLU.
struct ConvArgs {
  const void* u;
  const float* w_f;
  const float* b_f;
  const float* w_r;
  const float* b_r;
  const void* cache_in;  // block decoding: the 3 tokens before the block (null = zeros)
  void* cache_out;       // block decoding: receives the last 3 tokens (null = not written)
  void* out_f;           // null = forward direction not computed
  void* out_r;           // null = reverse direction not computed
  int act;
};

// Its backward pass; a null dout_f or dout_r leaves that direction out.
struct ConvBwdArgs {
  const void* dout_f;
  const void* dout_r;
  const void* u;
  const float* w_f;
  const float* b_f;
  const float* w_r;
  const float* b_r;
  void* du;
  float* dw_f;  // null with their direction
  float* db_f;  // null = not written
  float* dw_r;
  float* db_r;
  int act;
};

hipError_t launch_conv_bwd(const ConvBwdArgs& a, const BwdPlan& p, int64_t batch, int64_t L, int64_t C, int io_dtype,
                           void* workspace, hipStream_t stream);

hipError_t launch_conv(const ConvArgs& a, int64_t batch, int64_t L, int64_t C, int io_dtype, hipStream_t stream);

}  // namespace conv

namespace ssd {

// Mamba-2 (SSD) scan: bf16 x, dt, B, C, z, out; fp32 A, D, dt_bias per head.
struct SsdArgs {
  const void* x;
  const void* dt;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* dt_bias;
  void* out;
  uint32_t flags;
  const float* h_in;  // block decoding: forward state entering the sequence (null = zeros)
  float* h_out;       // block decoding: receives the forward state after it (null = not written)
};

// Staged chunked scan: stage 0 tiles B and C, 1 chunk summaries, 2 carry,
// 3 output; stage < 0 launches all four.  h_in / h_out enter and leave
// through the carry stage.
hipError_t launch_ssd(const SsdArgs& a, const SsdPlan& p, void* workspace, hipStream_t stream, int stage = -1);

// One direction of a Mamba-2 layer (dir 1 forward, 2 reverse) on a projection stream of xs elements per token
// holding x, B and C as channels [0, H*P), [H*P, H*P+N), [H*P+N, H*P+2N) (in.x is the stream; in.B, in.C,
// in.h_in and in.h_out are not used), with the short convolution of taps cw [xs, 4] and bias cb applied to
// the stream first when cw is not null: causal for dir 1, anti-causal for dir 2.
hipError_t launch_ssd_one_dir(const SsdArgs& in, const float* cw, const float* cb, int64_t xs, const SsdPlan& p,
                              void* workspace, int dir, hipStream_t stream);

// One block-cache decoding step of at most kQ tokens in a single kernel (no workspace).
hipError_t launch_ssd_block(const SsdArgs& a, int64_t batch, int64_t block_len, int64_t nheads, hipStream_t stream);

}  // namespace ssd

}  // namespace bimamba
