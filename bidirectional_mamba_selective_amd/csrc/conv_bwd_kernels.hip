// Backward pass of the short causal / anti-causal convolution, for gfx950.
//
// Forward (csrc/conv_kernels.hip), per channel, w_f and w_r of width 4:
//   p_f[t] = b_f + sum_k w_f[k] u[t - 3 + k]     p_r[t] = b_r + sum_k w_r[k] u[t + 3 - k]
//   out_f = silu(p_f), out_r = silu(p_r)          (u = 0 outside the sequence)
// Backward, from the gradients of out_f and out_r, with dp = dout silu'(p):
//   du[t]   = sum_k w_f[k] dp_f[t + 3 - k] + sum_k w_r[k] dp_r[t - 3 + k]
//   dw_f[k] = sum_t dp_f[t] u[t - 3 + k], db_f = sum_t dp_f[t];  dw_r, db_r likewise
//
// One read of u and of the two gradients, one write of du: an HBM stream with
// about 50 operations per (token, channel), four of them exponentials and
// reciprocals.  32768 x 4096 bf16: 229 us a call (kernel 221 and 228 on two cards,
// the sum of the partial sums 6), against 215 us for its bytes at the rate of a
// large copy.  254 us while the wavefront's number was a vector value, which made
// each access a loop over resources; 4-token steps 235 us; a register limit for 4
// wavefronts per SIMD 241.
// A lane owns two channels and walks a tile of
// tokens in steps of 8.  At step t0 it holds u[t0 .. t0 + 10]; from those 11
// rows it forms dp_f of tokens t0 + 3 .. t0 + 10 and dp_r of t0 .. t0 + 7, the
// two new ends of the windows that du[t0 .. t0 + 7] needs, so nothing but a
// tile's first three values is computed twice.  The next step's rows are loaded
// while the current one is computed.  dw and db stay in registers along the tile,
// four tiles meet in LDS, and a second kernel adds the workgroups' partial sums
// in a fixed order (no atomics).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "conv_bwd_plan.h"
#include "device_math.h"
#include "launch.h"

namespace bimamba {
namespace conv {
namespace {

constexpr int BLK = static_cast<int>(kBwdBlk);
constexpr int WAVES = static_cast<int>(kBwdWaves);
constexpr int kRsrcWord3 = 0x00020000;  // gfx9 buffer descriptor, untyped 32-bit data format
constexpr int kStream = 2;              // non-temporal

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two channels of a row, undecoded while the load is in flight.
template <typename T>
struct Pair;

template <>
struct Pair<float> {
  u32x2 v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    v = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
  }
  __device__ __forceinline__ void get(float (&o)[2]) const {
    o[0] = __uint_as_float(v.x);
    o[1] = __uint_as_float(v.y);
  }
  static __device__ __forceinline__ void store(const float (&o)[2], __amdgpu_buffer_rsrc_t r, uint32_t off) {
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(o[0]), __float_as_uint(o[1])}, r, off, 0, kStream);
  }
};

template <>
struct Pair<bf16_t> {
  uint32_t v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    v = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  }
  __device__ __forceinline__ void get(float (&o)[2]) const {
    o[0] = __uint_as_float(v << 16);
    o[1] = __uint_as_float(v & 0xffff0000u);
  }
  // round to nearest even
  static __device__ __forceinline__ void store(const float (&o)[2], __amdgpu_buffer_rsrc_t r, uint32_t off) {
    const f32x2 f = {o[0], o[1]};
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2)), r, off, 0,
                                          kStream);
  }
};

template <typename T>
struct BwdArgs {
  const T* u;
  const T* go_f;  // gradients of out_f, out_r; null: direction not computed
  const T* go_r;
  const float* w_f;
  const float* b_f;
  const float* w_r;
  const float* b_r;
  T* du;
  float* part;
  int64_t L, C, tile, cblocks;
};

// d silu(p) / dp times g
template <bool ACT>
__device__ __forceinline__ float act_grad(float g, float p) {
  if (!ACT) return g;
  const float s = __builtin_amdgcn_rcpf(1.0f + fast_exp2(-p * kLog2e));
  return g * (s * fmaf(p, 1.0f - s, 1.0f));
}

// DIRS: bit 0 = causal, bit 1 = anti-causal.
template <typename T, bool ACT, int DIRS>
__global__ __launch_bounds__(WAVES * 64) void k_conv_bwd(BwdArgs<T> a) {
  constexpr bool F = (DIRS & 1) != 0, R = (DIRS & 2) != 0;
  __shared__ float red[WAVES][kBwdSums][2][64];
  // the wavefront's number as a scalar: its tile's buffer resources must be uniform, or every access becomes a loop
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int64_t group = static_cast<int64_t>(blockIdx.x) / a.cblocks;
  const int64_t c0 = ((static_cast<int64_t>(blockIdx.x) - group * a.cblocks) * 64 + lane) * 2;
  const int64_t b = blockIdx.y;
  const bool on = c0 < a.C;  // channels come in fours, so both of a lane's are there or neither
  const int64_t T0 = (group * WAVES + wv) * a.tile;
  float acc[kBwdSums][2];
#pragma unroll
  for (int i = 0; i < kBwdSums; ++i) acc[i][0] = acc[i][1] = 0.0f;

  if (on && T0 < a.L) {
    float wf[4][2], wr[4][2], bf[2], br[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        wf[k][i] = F ? a.w_f[(c0 + i) * 4 + k] : 0.0f;
        wr[k][i] = R ? a.w_r[(c0 + i) * 4 + k] : 0.0f;
      }
      bf[i] = F && a.b_f ? a.b_f[c0 + i] : 0.0f;
      br[i] = R && a.b_r ? a.b_r[c0 + i] : 0.0f;
    }
    // Resources start 3 rows before the tile (at the sequence start for the first tile) and end with the sequence or
    // the tile's halo.  Rows outside it read as 0: the row goes into the VGPR offset, which the range check covers, and
    // a row before the sequence is an offset below 0, i.e. past any range.
    const uint32_t row_bytes = static_cast<uint32_t>(a.C) * static_cast<uint32_t>(sizeof(T));
    const int64_t rb = T0 >= 3 ? T0 - 3 : 0;
    const int64_t rows = min(a.L - rb, a.tile + 16);
    const int64_t at = (b * a.L + rb) * a.C;
    const int bytes = static_cast<int>(static_cast<uint32_t>(rows) * row_bytes);
    auto rsrc = [&](const T* p) {
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), static_cast<short>(0), bytes, kRsrcWord3);
    };
    const __amdgpu_buffer_rsrc_t ru = rsrc(a.u + at), rd = rsrc(a.du + at);
    const __amdgpu_buffer_rsrc_t rf = rsrc(F ? a.go_f + at : a.u), rr = rsrc(R ? a.go_r + at : a.u);
    const uint32_t lane_off = static_cast<uint32_t>(c0) * static_cast<uint32_t>(sizeof(T));
    // offset of row T0 + t
    auto off = [&](int t) { return lane_off + static_cast<uint32_t>(static_cast<int>(T0 - rb) + t) * row_bytes; };

    // u[t0 .. t0 + 10], dp_f[t0 .. t0 + 10], dp_r[t0 - 3 .. t0 + 7]
    float u[BLK + 3][2], pf[BLK + 3][2], pr[BLK + 3][2];
    auto causal = [&](const float (*v)[2], int i) {  // p_f of the token of v[3]
      float p = bf[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) p = fmaf(wf[k][i], v[k][i], p);
      return p;
    };
    auto anti = [&](const float (*v)[2], int i) {  // p_r of the token of v[0]
      float p = br[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) p = fmaf(wr[k][i], v[3 - k][i], p);
      return p;
    };
    {
      Pair<T> qu[6], qf[3], qr[3];
#pragma unroll
      for (int m = 0; m < 6; ++m) qu[m].load(ru, off(m - 3));
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        if (F) qf[m].load(rf, off(m));
        if (R) qr[m].load(rr, off(m - 3));
      }
      float h[6][2];
#pragma unroll
      for (int m = 0; m < 6; ++m) qu[m].get(h[m]);
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        float g[2];
        if (F) {
          qf[m].get(g);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            pf[m][i] = act_grad<ACT>(g[i], causal(&h[m], i));
            // these tokens' sums belong to the tile before, except where there is none
            if (T0 == 0) {
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[k][i] = fmaf(pf[m][i], h[m + k][i], acc[k][i]);
              acc[4][i] += pf[m][i];
            }
          }
        }
        if (R) {
          qr[m].get(g);
#pragma unroll
          for (int i = 0; i < 2; ++i) pr[m][i] = act_grad<ACT>(g[i], anti(&h[m], i));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) u[m][i] = h[3 + m][i];
      }
    }
    Pair<T> nu[BLK], nf[BLK], nr[BLK];
    auto fetch = [&](int t0) {
#pragma unroll
      for (int m = 0; m < BLK; ++m) {
        nu[m].load(ru, off(t0 + 3 + m));
        if (F) nf[m].load(rf, off(t0 + 3 + m));
        if (R) nr[m].load(rr, off(t0 + m));
      }
    };
    fetch(0);
    const int nt = static_cast<int>(min(a.tile, a.L - T0));
    for (int t0 = 0; t0 < nt; t0 += BLK) {
      float gf[BLK][2], gr[BLK][2];
#pragma unroll
      for (int m = 0; m < BLK; ++m) {
        nu[m].get(u[3 + m]);
        if (F) nf[m].get(gf[m]);
        if (R) nr[m].get(gr[m]);
      }
      if (t0 + BLK < nt) fetch(t0 + BLK);
#pragma unroll
      for (int m = 0; m < BLK; ++m) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (F) {
            // token t0 + 3 + m; the next tile's three first tokens are taken here, with zeros past the sequence end
            const float d = act_grad<ACT>(gf[m][i], causal(&u[m], i));
            pf[3 + m][i] = d;
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k][i] = fmaf(d, u[m + k][i], acc[k][i]);
            acc[4][i] += d;
          }
          if (R) {
            const float d = act_grad<ACT>(gr[m][i], anti(&u[m], i));  // token t0 + m
            pr[3 + m][i] = d;
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[5 + k][i] = fmaf(d, u[m + 3 - k][i], acc[5 + k][i]);
            acc[9][i] += d;
          }
        }
      }
#pragma unroll
      for (int m = 0; m < BLK; ++m) {
        float o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float s = 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (F) s = fmaf(wf[k][i], pf[m + 3 - k][i], s);
            if (R) s = fmaf(wr[k][i], pr[m + k][i], s);
          }
          o[i] = s;
        }
        if (t0 + m < nt) Pair<T>::store(o, rd, off(t0 + m));
      }
#pragma unroll
      for (int m = 0; m < 3; ++m) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          u[m][i] = u[BLK + m][i];
          pf[m][i] = pf[BLK + m][i];
          pr[m][i] = pr[BLK + m][i];
        }
      }
    }
  }
#pragma unroll
  for (int s = 0; s < kBwdSums; ++s) {
    red[wv][s][0][lane] = acc[s][0];
    red[wv][s][1][lane] = acc[s][1];
  }
  __syncthreads();
  const int64_t ngroup = static_cast<int64_t>(gridDim.x) / a.cblocks;
  float* part = a.part + (b * ngroup + group) * kBwdSums * a.C;
  for (int i = threadIdx.x; i < kBwdSums * 128; i += WAVES * 64) {
    const int s = i / 128, ch = i % 128;
    const int64_t c = c0 - 2 * lane + ch;
    if (c >= a.C) continue;
    float t = red[0][s][ch & 1][ch >> 1];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) t += red[w][s][ch & 1][ch >> 1];
    part[s * a.C + c] = t;
  }
}

struct BwdReduceArgs {
  const float* part;
  float* dw_f;
  float* db_f;
  float* dw_r;
  float* db_r;
  int64_t C, rows;
};

// 64 channels of one sum per workgroup; 16 wavefronts take every sixteenth partial sum and meet in LDS.
__global__ __launch_bounds__(1024) void k_conv_bwd_reduce(BwdReduceArgs a) {
  __shared__ float red[16][64];
  const int s = blockIdx.y, k = s % 5;
  float* dst = s < 5 ? (k < 4 ? a.dw_f : a.db_f) : (k < 4 ? a.dw_r : a.db_r);
  if (!dst) return;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  float t = 0.0f;
  if (c < a.C) {
    const float* p = a.part + s * a.C + c;
#pragma unroll 8
    for (int64_t i = wv; i < a.rows; i += 16) t += p[i * kBwdSums * a.C];
  }
  red[wv][lane] = t;
  __syncthreads();
  if (wv != 0 || c >= a.C) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) t += red[w][lane];
  if (k < 4) dst[c * 4 + k] = t;
  else dst[c] = t;
}

template <typename T, bool ACT>
hipError_t launch_typed(const ConvBwdArgs& in, const BwdPlan& p, int64_t batch, int64_t L, int64_t C, void* ws,
                        hipStream_t stream) {
  const BwdArgs<T> a{static_cast<const T*>(in.u), static_cast<const T*>(in.dout_f), static_cast<const T*>(in.dout_r),
                     in.w_f, in.b_f, in.w_r, in.b_r, static_cast<T*>(in.du), static_cast<float*>(ws), L, C, p.tile,
                     p.cblocks};
  const dim3 grid(static_cast<unsigned>(p.groups * p.cblocks), static_cast<unsigned>(batch)), block(WAVES * 64);
  if (in.dout_f && in.dout_r) hipLaunchKernelGGL((k_conv_bwd<T, ACT, 3>), grid, block, 0, stream, a);
  else if (in.dout_f) hipLaunchKernelGGL((k_conv_bwd<T, ACT, 1>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((k_conv_bwd<T, ACT, 2>), grid, block, 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const BwdReduceArgs r{static_cast<const float*>(ws), in.dw_f, in.db_f, in.dw_r, in.db_r, C, batch * p.groups};
  hipLaunchKernelGGL(k_conv_bwd_reduce, dim3(static_cast<unsigned>((C + 63) / 64), kBwdSums), dim3(1024), 0, stream, r);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_bwd(const ConvBwdArgs& a, const BwdPlan& p, int64_t batch, int64_t L, int64_t C, int io_dtype,
                           void* ws, hipStream_t stream) {
  if (io_dtype == 1)
    return a.act ? launch_typed<bf16_t, true>(a, p, batch, L, C, ws, stream)
                 : launch_typed<bf16_t, false>(a, p, batch, L, C, ws, stream);
  return a.act ? launch_typed<float, true>(a, p, batch, L, C, ws, stream)
               : launch_typed<float, false>(a, p, batch, L, C, ws, stream);
}

}  // namespace conv
}  // namespace bimamba
