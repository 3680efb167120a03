// Backward pass of the bidirectional selective scan, for gfx950.
//
// Forward (csrc/scan_kernels.hip), per channel d and state n, over tokens t:
//   delta = softplus(dt + dt_bias), a = exp(delta A[n]), u = delta x
//   f_t = a_t f_{t-1} + u_t B_t[n]        r_t = a_t r_{t+1} + u_t B_t[n]
//   y_t = sum_n C_t[n] (f_t + r_t) + k D x_t     (k = the directions kept)
//   out_t = y_t silu(z_t)
// With g = d(loss)/d(out), dy = g silu(z) and dz = g y silu'(z), the adjoint of
// each state runs against its direction:
//   forward states:  gf_t = C_t dy_t + G_{t+1},   G_t = a_t gf_t
//   reverse states:  gr_t = C_t dy_t + p_{t-1},   p_t = a_t gr_t
// and with w_t = G_t f_{t-1} + p_t r_{t+1} (the gradient of log a_t)
//   dB_t[n] = sum_d u (gf + gr)     dC_t[n] = sum_d dy (f + r)
//   du = sum_n B (gf + gr)          ddelta = x du + sum_n A[n] w
//   dx = delta du + k D dy          ddt = ddelta sigmoid(dt + dt_bias)
//   dA[n] = sum_t delta w           dD = sum_t k x dy       d(bias) = sum_t ddt
// w is formed from a_t f_{t-1} rather than as gf_t (f_t - u_t B_t), which would
// cancel where a_t is small.  Nothing of the forward call is kept: every state
// is recomputed from the inputs.
//
// The four recurrences f, p (left to right) and r, G (right to left) have the
// same diagonal transition, so they share the two-level scheme of the forward
// pass: lane = channel, a wavefront walks one chunk of one sequence in tiles of
// kSub tokens held in registers.
//   k_bwd_stage    B and C as an fp32 table per tile and state (read later with
//                  wave-uniform loads into SGPRs), A log2(e) transposed.
//   k_bwd_summary  walks each chunk right to left: r and G continue from tile
//                  to tile and are stored at every tile boundary; f and p run
//                  from zero inside a tile and are composed into the chunk's.
//   k_bwd_carry    composes the chunk maps of all four chains, in place.
//   k_bwd_main     walks each chunk left to right with f and p carried and r, G
//                  entering each tile from its boundary: every gradient above.
//   k_bwd_reduce   adds the partial sums in a fixed order (no atomics).
// dB and dC are sums over the channels, which lie across the lanes: a state's 32
// terms per lane go through LDS, one row per token, and are added in fp32 by two
// lanes a row while the next state is under way.
//
// What bounds it, at 8192 tokens x 4096 channels x 16 states, bf16, both directions (0.67 ms a call; its tensors alone
// would stream in 0.09 ms): vector issue.  k_bwd_main, 415 us, runs 28 operations per (token, channel, state) and
// k_bwd_summary, 210 us, 12; at the 2.3 clocks that independent operations take that is 0.4 ms.  The rest: scalar
// operands back to back (3.5 clocks), exponentials (7), and the loads at a tile's two ends, which two wavefronts per SIMD
// do not cover.  k_bwd_carry 14 us, k_bwd_reduce 14 us and k_bwd_stage 5 us are streams of the workspace.  These are
// medians of 200 calls once the clock has settled (two cards differ by 3 %).  The figures from here on are of 20 calls
// before that, where the kept kernels take 467 and 233 us; the next five stood beside kept forms of 552 to 490.
// Measured and not kept for k_bwd_main: tiles of 12 tokens at 3 wavefronts per SIMD 552 us and of 8 at 4
// 671 (a tile's boundary states are read and written that much more often); lane swaps and DPP adds for the sums over
// channels 550; the same sums on the matrix cores, exact in 4 x 4 blocks, 603; the next tile brought to LDS or to
// registers during the current one 586 and 490; B and C loaded a state ahead into a second set of SGPRs 518.
// The wavefronts of a SIMD take turns: the exponentials (in k_bwd_main the right-to-left walk and a tile's two ends too)
// run at a raised wave priority, so that one wavefront's slow operations and dependent steps fall into the other's
// independent ones: 493 -> 467 us, 247 -> 233 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bwd_plan.h"
#include "device_math.h"
#include "launch.h"

namespace bimamba {
namespace bwd {
namespace {

constexpr int SUB = static_cast<int>(kSub);
constexpr int NM = 16;  // states per channel at most
constexpr int NS = 8;   // states per wavefront of the summary pass
constexpr int kRsrcWord3 = 0x00020000;  // gfx9 buffer descriptor, untyped 32-bit data format

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, size_t bytes) {
  const int n = bytes > 0x7fffffffull ? 0x7fffffff : static_cast<int>(bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), n, kRsrcWord3);
}

// non-temporal: the nt bit of the buffer instruction's cache-policy field, for data touched once
constexpr int kStream = 2;

template <int CP = 0>
__device__ __forceinline__ float ld_buf(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, const float*) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, CP));
}
template <int CP = 0>
__device__ __forceinline__ float ld_buf(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, const bf16_t*) {
  const unsigned short h = __builtin_amdgcn_raw_buffer_load_b16(r, voff, soff, CP);
  return __uint_as_float(static_cast<uint32_t>(h) << 16);
}
template <int CP = 0>
__device__ __forceinline__ void st_buf(float v, __amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, const float*) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, voff, soff, CP);
}
// round to nearest even
template <int CP = 0>
__device__ __forceinline__ void st_buf(float v, __amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff,
                                       const bf16_t*) {
  __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, static_cast<__bf16>(v)), r, voff, soff, CP);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

// v[k] = row k of this lane's column of a tile; rows past the resource's end read as 0.  The row goes into the VGPR
// offset: the range check covers that one (an SGPR offset is subtracted from the range, which must not underflow).
template <typename T>
__device__ __forceinline__ void load_col(const T* base, size_t bytes, uint32_t voff, uint32_t row_bytes,
                                         float (&v)[SUB]) {
  const __amdgpu_buffer_rsrc_t r = make_rsrc(base, bytes);
#pragma unroll
  for (int k = 0; k < SUB; ++k) v[k] = ld_buf(r, voff + static_cast<uint32_t>(k) * row_bytes, 0, base);
}

// Rows past the resource's end are dropped.
template <typename T>
__device__ __forceinline__ void store_col(const float (&v)[SUB], T* base, size_t bytes, uint32_t voff,
                                          uint32_t row_bytes) {
  const __amdgpu_buffer_rsrc_t r = make_rsrc(base, bytes);
#pragma unroll
  for (int k = 0; k < SUB; ++k) st_buf<kStream>(v[k], r, voff + static_cast<uint32_t>(k) * row_bytes, 0, base);
}

// wave-uniform loads through a constant-address-space pointer become scalar loads into SGPRs
typedef const float __attribute__((address_space(4))) sfloat;
__device__ __forceinline__ const sfloat* scalar_ptr(const float* p) { return (const sfloat*)p; }

__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}

template <typename T>
__device__ __forceinline__ float ld_elem(const T* p) { return to_f32(*p); }

// ---------------------------------------------------------------------------
// k_bwd_stage: bct[((b * ntile + g) * N + n) * 2 kSub + {k, kSub + k}] = {B, C}[b, g kSub + k, n] in fp32, zero past
// the sequence end; then A2T[n][d] = A[d, n] log2(e).
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(256) void k_bwd_stage(const T* __restrict__ Bm, const T* __restrict__ Cm,
                                                   const float* __restrict__ A, float* __restrict__ bct,
                                                   float* __restrict__ A2T, int L, int D, int N, int ntile,
                                                   size_t total_bc, size_t total) {
  const size_t idx = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= total) return;
  if (idx >= total_bc) {
    const size_t i = idx - total_bc;
    const size_t n = i / D, d = i % D;
    A2T[i] = A[d * N + n] * kLog2e;
    return;
  }
  const int k = static_cast<int>(idx % SUB);
  const size_t rest = idx / SUB;
  const int n = static_cast<int>(rest % N);
  const size_t bg = rest / N;
  const int g = static_cast<int>(bg % ntile);
  const size_t b = bg / ntile;
  const int t = g * SUB + k;
  float bv = 0.0f, cv = 0.0f;
  if (t < L) {
    const size_t src = (b * L + t) * N + n;
    bv = ld_elem(Bm + src);
    cv = ld_elem(Cm + src);
  }
  float* dst = bct + rest * 2 * SUB;
  dst[k] = bv;
  dst[SUB + k] = cv;
}

template <typename T>
struct Args {
  const T* x;
  const T* dt;
  const T* z;     // null without the gate
  const T* dout;
  const float* D;        // or null
  const float* dt_bias;  // or null
  T* dx;
  T* ddt;
  T* dz;
  const float* bct;
  const float* A2T;
  float* Sf;  // per chunk: end state of f from zero, then (after the carry) the state entering from the left
  float* Sp;
  float* Sr;  // per chunk: start state of r from zero, then the state entering from the right
  float* Sg;
  float* P;
  float* Rr;  // per tile: r entering it from the right, started from zero at the chunk end
  float* Rg;
  float* sig;  // per tile: sum of delta from its right edge to the chunk end
  float* pbc;
  float* pA;
  float* pv;
  int L, Dn, N, chunk, nchunk, nsub, ntile;
};

// The tile's delta and dy; tokens past nvalid get delta = 0 (their transition is 1 and their input 0) and dy = 0.
template <typename T, bool GATE>
__device__ __forceinline__ void tile_inputs(const Args<T>& a, size_t tile, size_t bytes, uint32_t voff,
                                            uint32_t row_bytes, float bias, int nvalid, float (&dl)[SUB],
                                            float (&u)[SUB], float (&dy)[SUB]) {
  float xr[SUB], dr[SUB], gr[SUB];
  load_col(a.dt + tile, bytes, voff, row_bytes, dr);
  load_col(a.x + tile, bytes, voff, row_bytes, xr);
  load_col(a.dout + tile, bytes, voff, row_bytes, gr);
  if (GATE) {
    float zr[SUB];
    load_col(a.z + tile, bytes, voff, row_bytes, zr);
#pragma unroll
    for (int k = 0; k < SUB; ++k) dy[k] = gr[k] * silu_f32(zr[k]);
  } else {
#pragma unroll
    for (int k = 0; k < SUB; ++k) dy[k] = gr[k];
  }
  if (nvalid == SUB) {
#pragma unroll
    for (int k = 0; k < SUB; ++k) dl[k] = softplus_f32(dr[k] + bias);
  } else {
#pragma unroll
    for (int k = 0; k < SUB; ++k) dl[k] = k < nvalid ? softplus_f32(dr[k] + bias) : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < SUB; ++k) u[k] = dl[k] * xr[k];
}

// ---------------------------------------------------------------------------
// k_bwd_summary: grid (D / 64 * ceil(N / NS), nchunk, batch), one wavefront.  DS: bit 0 = the forward layer (f, G), bit
// 1 = the reverse layer (r, p).  A wavefront takes NS = 8 of the states: its four chains are in LDS, 1 KiB a state, and
// with all 16 a CU held 10 wavefronts and took 312 us instead of 248 (6 and 4 states: 293, 283).  Per tile it forms
// delta, u and dy once more, but the waits of its short state steps are covered by 4 wavefronts per SIMD.
// ---------------------------------------------------------------------------
template <typename T, int DS, bool GATE>
__global__ __launch_bounds__(64, 4) void k_bwd_summary(Args<T> a) {
  __shared__ float sF[(DS & 1) ? NS : 1][64];  // f of the chunk so far, decayed to the chunk end
  __shared__ float sG[(DS & 1) ? NS : 1][64];  // running G
  __shared__ float sP[(DS & 2) ? NS : 1][64];
  __shared__ float sR[(DS & 2) ? NS : 1][64];
  const int lane = threadIdx.x;
  const int D = a.Dn, N = a.N;
  const size_t col0 = static_cast<size_t>(blockIdx.x % (D / 64)) * 64;
  const int n0 = static_cast<int>(blockIdx.x / (D / 64)) * NS;  // this wavefront's states are n0 + s
  const int ns = min(NS, N - n0);
  const int c = blockIdx.y;
  const size_t b = blockIdx.z;
  const int t0 = c * a.chunk;
  const int te = min(a.L, t0 + a.chunk);
  const size_t row = b * a.L;
  const size_t cbase = b * a.nchunk + c;
  const float bias = a.dt_bias ? a.dt_bias[col0 + lane] : 0.0f;
  const uint32_t voff = static_cast<uint32_t>(lane) * static_cast<uint32_t>(sizeof(T));
  const uint32_t row_bytes = static_cast<uint32_t>(D) * static_cast<uint32_t>(sizeof(T));
  const size_t state_bytes = (static_cast<size_t>(N) * D - col0) * 4;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A2T + col0, state_bytes);
  const uint32_t voff4 = static_cast<uint32_t>(lane) * 4u;
  const uint32_t nstride = static_cast<uint32_t>(D) * 4u;
  for (int n = 0; n < ns; ++n) {
    if (DS & 1) sF[n][lane] = sG[n][lane] = 0.0f;
    if (DS & 2) sP[n][lane] = sR[n][lane] = 0.0f;
  }
  float sigma = 0.0f;  // sum of delta from the current tile's right edge to the chunk end
  const int ntile_c = (te - t0 + SUB - 1) / SUB;
  for (int j = ntile_c - 1; j >= 0; --j) {
    const int ts = t0 + j * SUB;
    const int nvalid = min(SUB, te - ts);
    const size_t tile = (row + ts) * D + col0;
    const size_t gt = b * a.ntile + static_cast<size_t>(c) * a.nsub + j;  // the tile's index
    float dl[SUB], u[SUB], dy[SUB];
    tile_inputs<T, GATE>(a, tile, static_cast<size_t>(nvalid) * row_bytes, voff, row_bytes, bias, nvalid, dl, u, dy);
    float tile_sum = 0.0f;
#pragma unroll
    for (int k = 0; k < SUB; ++k) tile_sum += dl[k];
    const float* bt = a.bct + gt * N * 2 * SUB;
    const size_t prev = gt - (j > 0 ? 1 : 0);  // the boundary left of this tile is the next one's right edge
    const size_t keep = j > 0 ? state_bytes : 0;
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.Rr + prev * N * D + col0, (DS & 2) ? keep : 0);
    const __amdgpu_buffer_rsrc_t wg = make_rsrc(a.Rg + prev * N * D + col0, (DS & 1) ? keep : 0);
    float a2_next = ld_buf(ra, voff4, static_cast<uint32_t>(n0) * nstride, a.A2T);
#pragma unroll 1
    for (int n = 0; n < ns; ++n) {
      const float a2 = a2_next;
      a2_next = ld_buf(ra, voff4, static_cast<uint32_t>(n0 + min(n + 1, ns - 1)) * nstride, a.A2T);
      __builtin_amdgcn_s_setprio(1);
      const sfloat* bn = scalar_ptr(bt + static_cast<size_t>(n0 + n) * 2 * SUB);
      float av[SUB], bb[SUB];
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        av[k] = fast_exp2(dl[k] * a2);
        bb[k] = u[k] * bn[k];
      }
      __builtin_amdgcn_s_setprio(0);
      float f = 0.0f, p = 0.0f;
      float r = (DS & 2) ? sR[(DS & 2) ? n : 0][lane] : 0.0f;
      float g = (DS & 1) ? sG[(DS & 1) ? n : 0][lane] : 0.0f;
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        const int q = SUB - 1 - k;
        if (DS & 1) {
          f = fmaf(av[k], f, bb[k]);
          g = av[q] * fmaf(bn[SUB + q], dy[q], g);
        }
        if (DS & 2) {
          p = av[k] * fmaf(bn[SUB + k], dy[k], p);
          r = fmaf(av[q], r, bb[q]);
        }
      }
      const float dec = fast_exp2(a2 * sigma);
      const uint32_t off = voff4 + static_cast<uint32_t>(n0 + n) * nstride;
      if (DS & 1) {
        sF[(DS & 1) ? n : 0][lane] = fmaf(dec, f, sF[(DS & 1) ? n : 0][lane]);
        sG[(DS & 1) ? n : 0][lane] = g;
        st_buf<kStream>(g, wg, off, 0, a.Rg);
      }
      if (DS & 2) {
        sP[(DS & 2) ? n : 0][lane] = fmaf(dec, p, sP[(DS & 2) ? n : 0][lane]);
        sR[(DS & 2) ? n : 0][lane] = r;
        st_buf<kStream>(r, wr, off, 0, a.Rr);
      }
    }
    sigma += tile_sum;
    if (j > 0 && n0 == 0) a.sig[prev * D + col0 + lane] = sigma;
  }
  for (int n = 0; n < ns; ++n) {
    const size_t o = (cbase * N + n0 + n) * D + col0 + lane;
    if (DS & 1) {
      a.Sf[o] = sF[(DS & 1) ? n : 0][lane];
      a.Sg[o] = sG[(DS & 1) ? n : 0][lane];
    }
    if (DS & 2) {
      a.Sp[o] = sP[(DS & 2) ? n : 0][lane];
      a.Sr[o] = sR[(DS & 2) ? n : 0][lane];
    }
    a.P[o] = fast_exp2(a.A2T[static_cast<size_t>(n0 + n) * D + col0 + lane] * sigma);
  }
}

// ---------------------------------------------------------------------------
// k_bwd_carry: one thread per (b, n, d) and walk direction (blockIdx.y = 0: f and p, left to right; 1: r and G, right
// to left); replaces each chunk's summary by the state that enters it.  The inputs of kBatch chunks are loaded
// before they are composed, so the loop pays one memory latency per batch.
// ---------------------------------------------------------------------------
template <int DS>
__global__ __launch_bounds__(256) void k_bwd_carry(float* __restrict__ Sf, float* __restrict__ Sp,
                                                   float* __restrict__ Sr, float* __restrict__ Sg,
                                                   const float* __restrict__ P, size_t total, int nchunk, int N,
                                                   int D) {
  constexpr int kBatch = 16;
  const size_t idx = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= total) return;
  const size_t nd = static_cast<size_t>(N) * D;  // states per chunk
  const size_t base = idx / nd * nchunk * nd + idx % nd;
  const bool right = blockIdx.y != 0;
  // the two chains of this walk: the forward layer's and the reverse layer's
  float* __restrict__ s1 = right ? Sg : Sf;
  float* __restrict__ s2 = right ? Sr : Sp;
  float c1 = 0.0f, c2 = 0.0f;
  for (int c0 = 0; c0 < nchunk; c0 += kBatch) {
    float pv[kBatch], v1[kBatch], v2[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int ci = min(c0 + i, nchunk - 1);
      const size_t o = base + static_cast<size_t>(right ? nchunk - 1 - ci : ci) * nd;
      pv[i] = P[o];
      if (DS & 1) v1[i] = s1[o];
      if (DS & 2) v2[i] = s2[o];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (c0 + i < nchunk) {
        const size_t o = base + static_cast<size_t>(right ? nchunk - 1 - c0 - i : c0 + i) * nd;
        if (DS & 1) {
          s1[o] = c1;
          c1 = fmaf(pv[i], c1, v1[i]);
        }
        if (DS & 2) {
          s2[o] = c2;
          c2 = fmaf(pv[i], c2, v2[i]);
        }
      }
    }
  }
}

template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// Sum over the 64 lanes of 2 SUB = 32 rows of LDS values: lane l takes half l % 2 of row l / 2, 16 bytes at a time, its
// first chunk turned by the row so that any 16 lanes in a row read 16 different groups of banks.
struct RowParts {
  f32x4 q[8];
};

__device__ __forceinline__ RowParts read_rows(const float (*rows)[64], int lane) {
  static_assert(SUB == 16, "two lanes a row");
  const int j = lane >> 1;
  const f32x4* row = reinterpret_cast<const f32x4*>(&rows[j][(lane & 1) * 32]);
  RowParts p;
#pragma unroll
  for (int i = 0; i < 8; ++i) p.q[i] = row[(i + j) & 7];
  return p;
}

__device__ __forceinline__ float total(const RowParts& p) {
  const f32x4 s = ((p.q[0] + p.q[1]) + (p.q[2] + p.q[3])) + ((p.q[4] + p.q[5]) + (p.q[6] + p.q[7]));
  return add_dpp<0xB1>((s[0] + s[1]) + (s[2] + s[3]));  // quad_perm [1,0,3,2]: the row's other half
}

// ---------------------------------------------------------------------------
// k_bwd_main: grid (D / 64, nchunk, batch), one wavefront.
// ---------------------------------------------------------------------------
template <typename T, int DS, bool GATE>
__global__ __launch_bounds__(64, 2) void k_bwd_main(Args<T> a) {
  __shared__ float sF[(DS & 1) ? NM : 1][64];
  __shared__ float sP[(DS & 2) ? NM : 1][64];
  __shared__ float sA[NM][64];  // dA of the chunk so far
  __shared__ __align__(16) float sV[2 * SUB][64];  // a state's terms of dB and dC, one row per token
  const int lane = threadIdx.x;
  const int D = a.Dn, N = a.N;
  const size_t col0 = static_cast<size_t>(blockIdx.x) * 64;
  const int c = blockIdx.y;
  const size_t b = blockIdx.z;
  const int t0 = c * a.chunk;
  const int te = min(a.L, t0 + a.chunk);
  const size_t row = b * a.L;
  const size_t cbase = b * a.nchunk + c;
  const float bias = a.dt_bias ? a.dt_bias[col0 + lane] : 0.0f;
  constexpr float ndir = DS == 3 ? 2.0f : 1.0f;
  const float skip = a.D ? ndir * a.D[col0 + lane] : 0.0f;
  const uint32_t voff = static_cast<uint32_t>(lane) * static_cast<uint32_t>(sizeof(T));
  const uint32_t row_bytes = static_cast<uint32_t>(D) * static_cast<uint32_t>(sizeof(T));
  const size_t state_bytes = (static_cast<size_t>(N) * D - col0) * 4;
  const uint32_t voff4 = static_cast<uint32_t>(lane) * 4u;
  const uint32_t nstride = static_cast<uint32_t>(D) * 4u;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A2T + col0, state_bytes);
  const __amdgpu_buffer_rsrc_t rcr = make_rsrc(a.Sr + cbase * N * D + col0, state_bytes);
  const __amdgpu_buffer_rsrc_t rcg = make_rsrc(a.Sg + cbase * N * D + col0, state_bytes);
  for (int n = 0; n < N; ++n) {
    const size_t o = (cbase * N + n) * D + col0 + lane;
    if (DS & 1) sF[(DS & 1) ? n : 0][lane] = a.Sf[o];
    if (DS & 2) sP[(DS & 2) ? n : 0][lane] = a.Sp[o];
    sA[n][lane] = 0.0f;
  }
  float sumD = 0.0f, sumBias = 0.0f;
  const int ntile_c = (te - t0 + SUB - 1) / SUB;
  for (int j = 0; j < ntile_c; ++j) {
    const int ts = t0 + j * SUB;
    const int nvalid = min(SUB, te - ts);
    const size_t tile = (row + ts) * D + col0;
    const size_t bytes = static_cast<size_t>(nvalid) * row_bytes;
    const size_t gt = b * a.ntile + static_cast<size_t>(c) * a.nsub + j;
    const bool edge = j == ntile_c - 1;  // r and G enter the chunk's last tile as the chunk's carries
    float dl[SUB], u[SUB], dy[SUB];
    tile_inputs<T, GATE>(a, tile, bytes, voff, row_bytes, bias, nvalid, dl, u, dy);
    const float sj = edge ? 0.0f : a.sig[gt * D + col0 + lane];
    const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.Rr + gt * N * D + col0, edge ? 0 : state_bytes);
    const __amdgpu_buffer_rsrc_t rg = make_rsrc(a.Rg + gt * N * D + col0, edge ? 0 : state_bytes);
    const float* bt = a.bct + gt * N * 2 * SUB;
    float* pbc = a.pbc + (gt * gridDim.x + blockIdx.x) * N * 2 * SUB;
    float y[SUB], du[SUB], dd[SUB];
#pragma unroll
    for (int k = 0; k < SUB; ++k) y[k] = du[k] = dd[k] = 0.0f;

    float a2_next = ld_buf(ra, voff4, 0, a.A2T);
    float rj_next = 0.0f, cr_next = 0.0f, gj_next = 0.0f, cg_next = 0.0f;
    if (DS & 2) {
      rj_next = ld_buf<kStream>(rr, voff4, 0, a.Rr);
      cr_next = ld_buf(rcr, voff4, 0, a.Sr);
    }
    if (DS & 1) {
      gj_next = ld_buf<kStream>(rg, voff4, 0, a.Rg);
      cg_next = ld_buf(rcg, voff4, 0, a.Sg);
    }
#pragma unroll 1
    for (int n = 0; n < N; ++n) {
      const float a2 = a2_next;
      const uint32_t s1 = static_cast<uint32_t>(min(n + 1, N - 1)) * nstride;
      a2_next = ld_buf(ra, voff4, s1, a.A2T);
      const sfloat* bn = scalar_ptr(bt + static_cast<size_t>(n) * 2 * SUB);
      __builtin_amdgcn_s_setprio(1);  // back to 0 after the right-to-left walk
      // the previous state's terms: read here, added after the right-to-left walk, so that their way through LDS costs
      // no wait (state 0 reads what the tile before left and drops it)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const RowParts parts = read_rows(sV, lane);
      __builtin_amdgcn_sched_barrier(0);
      // the chunk end's resource is empty: the boundary state reads as 0 and the decay is 1
      const float q = fast_exp2(a2 * sj);
      float r = 0.0f, g = 0.0f;
      if (DS & 2) {
        r = fmaf(q, cr_next, rj_next);
        rj_next = ld_buf<kStream>(rr, voff4 + s1, 0, a.Rr);
        cr_next = ld_buf(rcr, voff4, s1, a.Sr);
      }
      if (DS & 1) {
        g = fmaf(q, cg_next, gj_next);
        gj_next = ld_buf<kStream>(rg, voff4 + s1, 0, a.Rg);
        cg_next = ld_buf(rcg, voff4, s1, a.Sg);
      }
      float av[SUB], bb[SUB];
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        av[k] = fast_exp2(dl[k] * a2);
        bb[k] = u[k] * bn[k];
      }
      // right to left: r before each token (for w) and after it, gf, G
      float rv[SUB + 1], gf[SUB];
      rv[SUB] = r;
#pragma unroll
      for (int k = SUB - 1; k >= 0; --k) {
        if (DS & 2) {
          r = fmaf(av[k], r, bb[k]);
          rv[k] = r;
        }
        if (DS & 1) {
          gf[k] = fmaf(bn[SUB + k], dy[k], g);
          g = av[k] * gf[k];
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      {
        const float s = total(parts);
        if (n > 0 && (lane & 1) == 0) pbc[(n - 1) * 2 * SUB + (lane >> 1)] = s;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      __builtin_amdgcn_s_setprio(0);
      // left to right: f and p, and everything formed from the four states of a token
      float f = (DS & 1) ? sF[(DS & 1) ? n : 0][lane] : 0.0f;
      float p = (DS & 2) ? sP[(DS & 2) ? n : 0][lane] : 0.0f;
      float dA = sA[n][lane], dA1 = 0.0f;  // even and odd tokens: half the dependent chain
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        float w, gs, hs;
        if (DS & 1) {
          w = (av[k] * gf[k]) * f;
          gs = gf[k];
          f = fmaf(av[k], f, bb[k]);
          hs = f;
        }
        if (DS & 2) {
          const float gr = fmaf(bn[SUB + k], dy[k], p);
          p = av[k] * gr;
          w = (DS & 1) ? fmaf(p, rv[k + 1], w) : p * rv[k + 1];
          gs = (DS & 1) ? gs + gr : gr;
          hs = (DS & 1) ? hs + rv[k] : rv[k];
        }
        dd[k] = fmaf(a2, w, dd[k]);
        if (k & 1) dA1 = fmaf(dl[k], w, dA1);
        else dA = fmaf(dl[k], w, dA);
        du[k] = fmaf(bn[k], gs, du[k]);
        if (GATE) y[k] = fmaf(bn[SUB + k], hs, y[k]);
        sV[k][lane] = u[k] * gs;
        sV[SUB + k][lane] = dy[k] * hs;
      }
      if (DS & 1) sF[(DS & 1) ? n : 0][lane] = f;
      if (DS & 2) sP[(DS & 2) ? n : 0][lane] = p;
      sA[n][lane] = dA + dA1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const float last = total(read_rows(sV, lane));
    if ((lane & 1) == 0) pbc[(N - 1) * 2 * SUB + (lane >> 1)] = last;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_s_setprio(1);  // through the next tile's start
    // the gradients of the token's own inputs
    float xr[SUB], dr[SUB];
    load_col(a.x + tile, bytes, voff, row_bytes, xr);
    load_col(a.dt + tile, bytes, voff, row_bytes, dr);
#pragma unroll
    for (int k = 0; k < SUB; ++k) {
      const float ddelta = fmaf(xr[k], du[k], dd[k] * kLn2);
      dr[k] = ddelta * sigmoid_f32(dr[k] + bias);
      if (k < nvalid) {
        sumBias += dr[k];
        sumD = fmaf(xr[k], dy[k], sumD);
      }
      du[k] = fmaf(dl[k], du[k], skip * dy[k]);
    }
    store_col(dr, a.ddt + tile, bytes, voff, row_bytes);
    store_col(du, a.dx + tile, bytes, voff, row_bytes);
    __builtin_amdgcn_sched_barrier(0);
    if (GATE) {
      float zr[SUB], gr[SUB];
      load_col(a.z + tile, bytes, voff, row_bytes, zr);
      load_col(a.dout + tile, bytes, voff, row_bytes, gr);
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        const float s = sigmoid_f32(zr[k]);
        zr[k] = gr[k] * fmaf(skip, xr[k], y[k]) * (s * fmaf(zr[k], 1.0f - s, 1.0f));
      }
      store_col(zr, a.dz + tile, bytes, voff, row_bytes);
    }
  }
  for (int n = 0; n < N; ++n) a.pA[(cbase * N + n) * D + col0 + lane] = sA[n][lane];
  a.pv[(cbase * 2) * D + col0 + lane] = ndir * sumD;
  a.pv[(cbase * 2 + 1) * D + col0 + lane] = sumBias;
}

__device__ __forceinline__ void st_elem(float v, float* p) { *p = v; }
__device__ __forceinline__ void st_elem(float v, bf16_t* p) { from_f32(v, p); }

// ---------------------------------------------------------------------------
// k_bwd_reduce, 256 threads.  The first nbc workgroups: dB and dC, one thread per (tile, state, token of B or C), summed
// over the channel groups.  The rest: 64 channels of one row of (dA[0..N-1], dD, d(bias)), summed over the batch and the
// chunks by four wavefronts that meet in LDS.
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(256) void k_bwd_reduce(const float* __restrict__ pbc, const float* __restrict__ pA,
                                                    const float* __restrict__ pv, T* __restrict__ dB,
                                                    T* __restrict__ dC, float* __restrict__ dA,
                                                    float* __restrict__ dD, float* __restrict__ dbias, int L, int D,
                                                    int N, int ntile, size_t nrow, size_t nbc, size_t total_bc) {
  const int W = D / 64;
  if (blockIdx.x < nbc) {
    const size_t idx = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
    if (idx >= total_bc) return;
    const size_t per = static_cast<size_t>(N) * 2 * SUB;
    const size_t gt = idx / per, i = idx % per;
    const float* src = pbc + gt * W * per + i;
    float s = 0.0f;
#pragma unroll 8
    for (int w = 0; w < W; ++w) s += src[static_cast<size_t>(w) * per];
    const int n = static_cast<int>(i / (2 * SUB)), k = static_cast<int>(i % (2 * SUB));
    const size_t b = gt / ntile;
    const int t = static_cast<int>(gt % ntile) * SUB + k % SUB;
    if (t < L) st_elem(s, (k < SUB ? dB : dC) + (b * L + t) * N + n);
    return;
  }
  __shared__ float part[4][64];
  const size_t o = blockIdx.x - nbc;
  const int r = static_cast<int>(o / W);
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const size_t d = (o % W) * 64 + lane;
  const float* src = r < N ? pA + static_cast<size_t>(r) * D + d : pv + static_cast<size_t>(r - N) * D + d;
  const size_t stride = static_cast<size_t>(r < N ? N : 2) * D;
  float s = 0.0f;
#pragma unroll 8
  for (size_t i = wv; i < nrow; i += 4) s += src[i * stride];
  part[wv][lane] = s;
  __syncthreads();
  if (wv != 0) return;
  s = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
  if (r < N) dA[d * N + r] = s;
  else if (r == N && dD) dD[d] = s;
  else if (r == N + 1 && dbias) dbias[d] = s;
}

template <typename T, int DS, bool GATE>
hipError_t launch_passes(const Args<T>& a, const BwdPlan& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.Dn / 64), static_cast<unsigned>(a.nchunk), static_cast<unsigned>(p.batch));
  const dim3 sgrid(grid.x * static_cast<unsigned>((a.N + NS - 1) / NS), grid.y, grid.z);
  hipLaunchKernelGGL((k_bwd_summary<T, DS, GATE>), sgrid, dim3(64), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t nth = static_cast<size_t>(p.batch) * a.N * a.Dn;
  hipLaunchKernelGGL((k_bwd_carry<DS>), dim3(static_cast<unsigned>((nth + 255) / 256), 2), dim3(256), 0, stream, a.Sf,
                     a.Sp, a.Sr, a.Sg, a.P, nth, a.nchunk, a.N, a.Dn);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_bwd_main<T, DS, GATE>), grid, dim3(64), 0, stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_typed(const ScanBwdArgs& in, const BwdPlan& p, void* ws, hipStream_t stream) {
  char* w = static_cast<char*>(ws);
  auto at = [&](size_t off) { return reinterpret_cast<float*>(w + off); };
  Args<T> a{};
  a.x = static_cast<const T*>(in.x);
  a.dt = static_cast<const T*>(in.dt);
  a.z = static_cast<const T*>(in.z);
  a.dout = static_cast<const T*>(in.dout);
  a.D = in.D;
  a.dt_bias = in.dt_bias;
  a.dx = static_cast<T*>(in.dx);
  a.ddt = static_cast<T*>(in.ddt);
  a.dz = static_cast<T*>(in.dz);
  a.bct = at(p.off_bct);
  a.A2T = at(p.off_a2t);
  a.Sf = at(p.off_sf);
  a.Sp = at(p.off_sp);
  a.Sr = at(p.off_sr);
  a.Sg = at(p.off_sg);
  a.P = at(p.off_p);
  a.Rr = at(p.off_rr);
  a.Rg = at(p.off_rg);
  a.sig = at(p.off_sig);
  a.pbc = at(p.off_pbc);
  a.pA = at(p.off_pa);
  a.pv = at(p.off_pv);
  a.L = static_cast<int>(p.seqlen);
  a.Dn = static_cast<int>(p.d_inner);
  a.N = static_cast<int>(p.d_state);
  a.chunk = static_cast<int>(p.chunk);
  a.nchunk = static_cast<int>(p.nchunk);
  a.nsub = static_cast<int>(p.nsub);
  a.ntile = static_cast<int>(p.ntile);
  const size_t nbc = static_cast<size_t>(p.batch) * p.ntile * p.d_state * SUB;
  const size_t nst = nbc + static_cast<size_t>(p.d_state) * p.d_inner;
  hipLaunchKernelGGL((k_bwd_stage<T>), dim3(static_cast<unsigned>((nst + 255) / 256)), dim3(256), 0, stream,
                     static_cast<const T*>(in.B), static_cast<const T*>(in.C), in.A, at(p.off_bct), at(p.off_a2t), a.L,
                     a.Dn, a.N, a.ntile, nbc, nst);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool gate = (in.flags & kNoGate) == 0;
  if (in.flags & kFwdOnly) {
    e = gate ? launch_passes<T, 1, true>(a, p, stream) : launch_passes<T, 1, false>(a, p, stream);
  } else if (in.flags & kRevOnly) {
    e = gate ? launch_passes<T, 2, true>(a, p, stream) : launch_passes<T, 2, false>(a, p, stream);
  } else {
    e = gate ? launch_passes<T, 3, true>(a, p, stream) : launch_passes<T, 3, false>(a, p, stream);
  }
  if (e != hipSuccess) return e;
  const size_t total_bc = 2 * nbc, gbc = (total_bc + 255) / 256;
  const size_t gpar = static_cast<size_t>(p.d_state + 2) * (p.d_inner / 64);
  hipLaunchKernelGGL((k_bwd_reduce<T>), dim3(static_cast<unsigned>(gbc + gpar)), dim3(256), 0, stream, a.pbc, a.pA,
                     a.pv, static_cast<T*>(in.dB), static_cast<T*>(in.dC), in.dA, in.dD, in.ddt_bias, a.L, a.Dn, a.N,
                     a.ntile, static_cast<size_t>(p.batch) * p.nchunk, gbc, total_bc);
  return hipGetLastError();
}

}  // namespace
}  // namespace bwd

hipError_t launch_scan_bwd(const ScanBwdArgs& a, const BwdPlan& p, void* workspace, hipStream_t stream) {
  if (a.io_dtype == 1) return bwd::launch_typed<bf16_t>(a, p, workspace, stream);
  return bwd::launch_typed<float>(a, p, workspace, stream);
}

}  // namespace bimamba
