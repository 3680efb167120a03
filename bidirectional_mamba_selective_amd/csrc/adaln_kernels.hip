// The step between two blocks of the denoiser, forward and backward, for
// gfx950: the branch's post-norm, its gate and residual sum, and the modulated
// norm in front of the next block.
//
//   m' = m * q * w,  q = 1 / sqrt(mean(m^2) + eps)     (w given; else m' = m)
//   h  = x + g * m'
//   out = gamma * (h - mu) * r + beta,  r = 1 / sqrt(var(h) + eps)
// ("DiffuMamba: High-Throughput Diffusion LMs with Mamba Backbone", arXiv v4,
// Appendix A.1 eq. (10): AdaLN; eq. (11)-(12): the residual sum around each
// mixer.)  gamma, beta, g belong to a sequence (or to all of them), w to all
// rows.  Backward, from the gradients dout of out and dres of h, with
// xhat = (h - mu) r, e = dout gamma, mh = m q, f = g dh w:
//   dh = dres + r (e - mean(e) - xhat mean(e xhat))      dx = dh
//   dm = q (f - mh mean(f mh))          (w given; else dm = g dh)
//   dgamma = sum dout xhat, dbeta = sum dout, dg = sum dh m', dw = sum g dh mh
// q, mu and r are taken again from m and h: nothing else of the forward pass is
// kept.  The variance is summed from the centred values (a second pass over
// registers), so a large mean costs no accuracy.
//
// Both directions read each tensor once and write each result once; what bounds
// them is HBM: 8 x 8192 rows of 2048 in bf16 take 216 us forward (1.07 GB, 5.0 TB/s)
// and 330 us backward (1.61 GB, 4.9 TB/s), the rate of a large copy.  A few rows are
// bound by the launch (32 rows: 3.2 us on the device).  A row sits in registers,
// 8 values a lane, across one to sixteen wavefronts; a workgroup walks consecutive
// rows of one sequence, so gamma, beta, g and w are
// loaded once per workgroup, and the next row's loads are in flight while the
// current row is summed.  The column sums of the backward pass stay in registers
// along that walk; each workgroup writes its partial sums once, and a second
// kernel adds them in a fixed order (no atomics).
//
// With an 8-bit result (FP8) 16 lanes hold a block of 128 columns: its largest magnitude is a maximum over those lanes,
// the values are divided by the scale in registers and rounded to e4m3, and lane 0 of the 16 writes
// the scale.  The pass stays one read and one write: 8 x 8192 rows of 2048 in 190 us (943 MB, 5.0 TB/s; a large copy
// reaches 5.06).  The divisions cost 1 % of it, the compiler's would 3 %; the product with 1 / scale, which would cost
// nothing, rounds twice and puts values next to a border on its other side.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "adaln_plan.h"
#include "device_math.h"
#include "launch.h"

namespace bimamba {
namespace adaln {
namespace {

constexpr int V = static_cast<int>(kVec);

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 consecutive values, kept undecoded while the load is in flight.  Activations pass through once: non-temporal.
template <typename T>
struct Raw;

template <>
struct Raw<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
    b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
  static __device__ __forceinline__ void put(const float* v, float* p) {
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(p));
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4*>(p) + 1);
  }
};

template <>
struct Raw<bf16_t> {
  u32x4 a;
  __device__ __forceinline__ void load(const bf16_t* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  }
  __device__ __forceinline__ void clear() { a = u32x4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
  // round to nearest even, two values per v_cvt_pk_bf16_f32
  static __device__ __forceinline__ void put(const float* v, bf16_t* p) {
    const f32x8 f = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, __builtin_convertvector(f, bf16x8)),
                                reinterpret_cast<u32x4*>(p));
  }
};

template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// Sum over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0xB1>(v);   // quad_perm [1,0,3,2]
  v = add_dpp<0x4E>(v);   // quad_perm [2,3,0,1]
  v = add_dpp<0x141>(v);  // row_half_mirror
  v = add_dpp<0x140>(v);  // row_mirror
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Sums over a row's wavefronts.  The buffers alternate, so one barrier per sum suffices: a buffer is written again
// only after the barrier of the sum between, which every wavefront reaches after its reads.
template <int WPR, int K>
struct RowSums {
  float buf[2][WPR][K];
};

template <int WPR, int K, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], RowSums<WPR, K>& sm, int& phase, int wave) {
  static_assert(N <= K, "more sums than the buffer holds");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (WPR > 1) {
    float(*b)[K] = sm.buf[phase & 1];
    ++phase;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) b[wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = b[0][i];
#pragma unroll
      for (int w = 1; w < WPR; ++w) s += b[w][i];
      v[i] = s;
    }
  }
}

// A thread's 8 columns; past the row's end it holds zeros and stores nothing.
struct Cols {
  int64_t at;
  bool on;
};

template <int WPR>
__device__ __forceinline__ Cols my_cols(int64_t d) {
  const int64_t at = static_cast<int64_t>(threadIdx.x % (WPR * 64)) * V;
  return Cols{at, at < d};
}

__device__ __forceinline__ void load_vec(const float* p, const Cols& c, float none, float (&v)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = none;
  if (p && c.on) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p + c.at);
    const f32x4 b = *reinterpret_cast<const f32x4*>(p + c.at + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  }
}

template <typename T>
__device__ __forceinline__ void load_row(const T* base, int64_t row, int64_t d, const Cols& c, Raw<T>& v) {
  if (c.on) v.load(base + row * d + c.at);
  else v.clear();
}

template <typename T>
__device__ __forceinline__ void put_row(const float (&v)[V], T* base, int64_t row, int64_t d, const Cols& c) {
  if (c.on) Raw<T>::put(v, base + row * d + c.at);
}

// columns past the row's end hold 0 and must stay out of centred sums
__device__ __forceinline__ void centre(float (&v)[V], const Cols& c, float mu) {
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = c.on ? v[e] - mu : 0.0f;
}

// 1 / sqrt(v) by the hardware's estimate, within 1 ulp (2^-23 relative) of the root
__device__ __forceinline__ float rsqrt_f32(float v) { return __builtin_amdgcn_rsqf(v); }

template <typename T>
struct FwdArgs {
  const T* x;
  const T* m;          // null: no branch
  const float* w;      // null: no post-norm
  const float* g;      // null: 1
  const float* gamma;  // null: 1
  const float* beta;   // null: 0
  T* h;                // null without a branch; may be x
  void* out;           // T, or 8 bits
  float* scales;       // 8 bits only: [row][d / kScaleCols]
  int64_t L, d, rows_per_wg, mod_stride;  // mod_stride: d, or 0 where one gamma, beta, g serves every sequence
  float inv_d, eps;
  int rms;
};

template <int CTRL>
__device__ __forceinline__ float max_dpp(float v) {
  return fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true)));
}

// 8 values of a row as e4m3 (round to nearest even), with one scale for the 128 columns that 16 lanes hold:
// scale = max(largest magnitude, 2^-100) / 448.  The magnitude's floor keeps the scale and its reciprocal normal numbers,
// so a block of zeros gives zeros.  Values are divided, correctly rounded: r is the rounded reciprocal, a first remainder
// brings the quotient within one step, and the second then rounds it as a division does (Markstein's theorem).  The
// maximum passes over a NaN; the value itself stays one.
__device__ __forceinline__ void put_fp8(const float (&v)[V], uint8_t* out, float* scales, int64_t row, int64_t d,
                                        const Cols& c) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int e = 1; e < V; ++e) m = fmaxf(m, fabsf(v[e]));
  m = max_dpp<0xB1>(m);   // quad_perm [1,0,3,2]
  m = max_dpp<0x4E>(m);   // quad_perm [2,3,0,1]
  m = max_dpp<0x141>(m);  // row_half_mirror
  m = max_dpp<0x140>(m);  // row_mirror
  const float s = fmaxf(m, 0x1p-100f) / 448.0f;
  // a power of two keeps the remainders normal numbers; a block with an infinity has r = 0: its finite values give 0
  const float up = s < 1.0f ? 0x1p64f : 1.0f, div = s * up, r = 1.0f / div, by = r > 0.0f ? div : 0.0f;
  float q[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float n = v[e] * up, q0 = n * r, q1 = fmaf(fmaf(-q0, by, n), r, q0);
    q[e] = fmaf(fmaf(-q1, by, n), r, q1);
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  if (!c.on) return;
  __builtin_nontemporal_store(u32x2{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)},
                              reinterpret_cast<u32x2*>(out + row * d + c.at));
  if ((threadIdx.x & 15) == 0) scales[row * (d / kScaleCols) + c.at / kScaleCols] = s;
}

template <typename T, int WPR, bool FP8>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void k_adaln_fwd(FwdArgs<T> a) {
  constexpr int G = WPR == 1 ? 4 : 1;
  __shared__ RowSums<WPR, 1> sm;
  int phase = 0;
  const int wave = static_cast<int>(threadIdx.x) / 64;
  const int grp = WPR == 1 ? wave : 0;
  const Cols c = my_cols<WPR>(a.d);
  const int64_t b = blockIdx.y;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.rows_per_wg;
  const int64_t r1 = min(a.L, r0 + a.rows_per_wg);
  const int64_t base = b * a.L;
  const bool branch = a.m != nullptr, post = a.w != nullptr;
  const int64_t mod = b * a.mod_stride;
  float w[V], g[V], gamma[V], beta[V];
  load_vec(a.w, c, 1.0f, w);
  load_vec(a.g ? a.g + mod : nullptr, c, 1.0f, g);
  load_vec(a.gamma ? a.gamma + mod : nullptr, c, 1.0f, gamma);
  load_vec(a.beta ? a.beta + mod : nullptr, c, 0.0f, beta);
#pragma unroll
  for (int i = 0; i < V; ++i) w[i] *= g[i];  // m' and its gate in one factor
  Raw<T> xn, mn;
  if (r0 + grp < r1) {
    load_row<T>(a.x, base + r0 + grp, a.d, c, xn);
    if (branch) load_row<T>(a.m, base + r0 + grp, a.d, c, mn);
  }
  for (int64_t r = r0 + grp; r < r1; r += G) {
    float h[V];
    xn.get(h);
    if (branch) {
      float m[V];
      mn.get(m);
      if (r + G < r1) {
        load_row<T>(a.x, base + r + G, a.d, c, xn);
        load_row<T>(a.m, base + r + G, a.d, c, mn);
      }
      float q[1] = {1.0f};
      if (post) {
        q[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) q[0] = fmaf(m[i], m[i], q[0]);
        row_sum(q, sm, phase, wave);
        q[0] = rsqrt_f32(fmaf(q[0], a.inv_d, a.eps));
      }
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = fmaf(m[i] * q[0], w[i], h[i]);
      put_row<T>(h, a.h, base + r, a.d, c);
    } else if (r + G < r1) {
      load_row<T>(a.x, base + r + G, a.d, c, xn);
    }
    // the norm takes h before its rounding to the I/O type
    if (!a.rms) {
      float mu[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i) mu[0] += h[i];
      row_sum(mu, sm, phase, wave);
      centre(h, c, mu[0] * a.inv_d);
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) s[0] = fmaf(h[i], h[i], s[0]);
    row_sum(s, sm, phase, wave);
    const float rs = rsqrt_f32(fmaf(s[0], a.inv_d, a.eps));
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = fmaf(h[i] * rs, gamma[i], beta[i]);
    if constexpr (FP8) put_fp8(h, static_cast<uint8_t*>(a.out), a.scales, base + r, a.d, c);
    else put_row<T>(h, static_cast<T*>(a.out), base + r, a.d, c);
  }
}

template <typename T>
struct BwdArgs {
  const T* dout;
  const T* dres;  // null: 0
  const T* h;
  const T* m;
  const float* w;
  const float* g;
  const float* gamma;
  T* dx;  // may be dres
  T* dm;
  float* part;  // [batch][chunk][group][kSums][d]
  int64_t L, d, rows_per_wg, mod_stride;
  float inv_d, eps;
  int rms;
};

template <typename T, int WPR>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void k_adaln_bwd(BwdArgs<T> a) {
  constexpr int G = WPR == 1 ? 4 : 1;
  __shared__ RowSums<WPR, 4> sm;
  int phase = 0;
  const int wave = static_cast<int>(threadIdx.x) / 64;
  const int grp = WPR == 1 ? wave : 0;
  const Cols c = my_cols<WPR>(a.d);
  const int64_t b = blockIdx.y;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.rows_per_wg;
  const int64_t r1 = min(a.L, r0 + a.rows_per_wg);
  const int64_t base = b * a.L;
  const bool branch = a.m != nullptr, post = a.w != nullptr, res = a.dres != nullptr;
  const int64_t mod = b * a.mod_stride;
  float w[V], g[V], gamma[V];
  load_vec(a.w, c, 1.0f, w);
  load_vec(a.g ? a.g + mod : nullptr, c, 1.0f, g);
  load_vec(a.gamma ? a.gamma + mod : nullptr, c, 1.0f, gamma);
  float sgam[V], sbet[V], sg[V], sw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sgam[i] = sbet[i] = sg[i] = sw[i] = 0.0f;
  Raw<T> on, rn, hn, mn;
  auto fetch = [&](int64_t r) {
    load_row<T>(a.h, base + r, a.d, c, hn);
    load_row<T>(a.dout, base + r, a.d, c, on);
    if (branch) load_row<T>(a.m, base + r, a.d, c, mn);
    if (res) load_row<T>(a.dres, base + r, a.d, c, rn);
  };
  // at 16 wavefronts a lane has 128 registers, which the next row's loads would exceed
  constexpr bool kAhead = WPR < 16;
  if (kAhead && r0 + grp < r1) fetch(r0 + grp);
  for (int64_t r = r0 + grp; r < r1; r += G) {
    if (!kAhead) fetch(r);
    float x[V], o[V], m[V], dh[V];
    hn.get(x);
    on.get(o);
#pragma unroll
    for (int i = 0; i < V; ++i) m[i] = dh[i] = 0.0f;
    if (branch) mn.get(m);
    if (res) rn.get(dh);
    if (kAhead && r + G < r1) fetch(r + G);
    // s: sum of squares of the (centred) h, of e, of e times the centred h
    float q = 1.0f, s[3] = {0.0f, 0.0f, 0.0f};
    if (!a.rms) {
      float t[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        t[0] += x[i];
        t[1] = fmaf(m[i], m[i], t[1]);
      }
      row_sum(t, sm, phase, wave);
      centre(x, c, t[0] * a.inv_d);
      q = t[1];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float e = o[i] * gamma[i];
        s[0] = fmaf(x[i], x[i], s[0]);
        s[1] += e;
        s[2] = fmaf(e, x[i], s[2]);
      }
      row_sum(s, sm, phase, wave);
    } else {
      float t[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        t[0] = fmaf(x[i], x[i], t[0]);
        t[1] = fmaf(m[i], m[i], t[1]);
        t[2] = fmaf(o[i] * gamma[i], x[i], t[2]);
      }
      row_sum(t, sm, phase, wave);
      s[0] = t[0];
      s[2] = t[2];
      q = t[1];
    }
    const float rs = rsqrt_f32(fmaf(s[0], a.inv_d, a.eps));
    const float c1 = s[1] * a.inv_d, c2 = s[2] * a.inv_d * rs;  // means of e and of e xhat
    q = post ? rsqrt_f32(fmaf(q, a.inv_d, a.eps)) : 1.0f;
    float u[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float xhat = x[i] * rs;
      sgam[i] = fmaf(o[i], xhat, sgam[i]);
      sbet[i] += o[i];
      dh[i] = fmaf(rs, fmaf(-xhat, c2, fmaf(o[i], gamma[i], -c1)), dh[i]);
      m[i] *= q;                      // mh
      o[i] = dh[i] * g[i];            // g dh
      sg[i] = fmaf(dh[i], m[i], sg[i]);  // without w: multiplied in at the end
      sw[i] = fmaf(o[i], m[i], sw[i]);
      o[i] *= w[i];                   // f
      u[0] = fmaf(o[i], m[i], u[0]);
    }
    put_row<T>(dh, a.dx, base + r, a.d, c);
    if (branch) {
      if (post) {
        row_sum(u, sm, phase, wave);
        const float c3 = u[0] * a.inv_d;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = q * fmaf(-m[i], c3, o[i]);
      }
      put_row<T>(o, a.dm, base + r, a.d, c);
    }
  }
  float* part = a.part + ((b * gridDim.x + blockIdx.x) * G + grp) * kSums * a.d;
  if (!c.on) return;
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    float* p = part + k * a.d + c.at;
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = k == 0 ? sgam[j] : k == 1 ? sbet[j] : k == 2 ? sg[j] * w[j] : sw[j];
  }
}

struct ReduceArgs {
  const float* part;
  float* dst[kSums];  // null: not wanted
  int64_t d, groups;  // partial sums per sequence
  int64_t batch;
  int mod_rows_one;   // dst[0..2] are one row for the whole batch
};

// 64 columns of one sum and one output row per workgroup; its 16 wavefronts take every sixteenth partial sum and meet in
// LDS.
__global__ __launch_bounds__(1024) void k_adaln_reduce(ReduceArgs a) {
  __shared__ float s[16][64];
  const int which = blockIdx.z;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const bool whole = which == 3 || a.mod_rows_one;  // one row, summed over the batch
  if (!a.dst[which] || (whole && blockIdx.y != 0)) return;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const int64_t n = whole ? a.groups * a.batch : a.groups;
  const int64_t first = whole ? 0 : blockIdx.y * a.groups;
  float t = 0.0f;
  if (col < a.d) {
    const float* p = a.part + (first * kSums + which) * a.d + col;
#pragma unroll 8
    for (int64_t i = wv; i < n; i += 16) t += p[i * kSums * a.d];
  }
  s[wv][lane] = t;
  __syncthreads();
  if (wv != 0 || col >= a.d) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) t += s[w][lane];
  a.dst[which][(whole ? 0 : blockIdx.y) * a.d + col] = t;
}

template <typename F>
void with_waves(int waves, F&& f) {
  switch (waves) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    default: return f(std::integral_constant<int, 16>{});
  }
}

template <typename T>
hipError_t fwd_typed(const AdalnArgs& in, const Plan& p, hipStream_t stream) {
  FwdArgs<T> a{static_cast<const T*>(in.x), static_cast<const T*>(in.branch), in.post_weight, in.gate, in.gamma, in.beta,
               static_cast<T*>(in.h), in.out, in.scales, in.seqlen, in.d_model, p.rows_per_wg,
               in.mod_rows == 1 ? 0 : in.d_model, 1.0f / static_cast<float>(in.d_model), in.eps, in.rms};
  const dim3 grid(static_cast<unsigned>(p.chunks), static_cast<unsigned>(in.batch));
  with_waves(p.waves, [&](auto w) {
    constexpr int W = decltype(w)::value;
    const dim3 block(W == 1 ? 256 : W * 64);
    if (in.scales) hipLaunchKernelGGL((k_adaln_fwd<T, W, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((k_adaln_fwd<T, W, false>), grid, block, 0, stream, a);
  });
  return hipGetLastError();
}

template <typename T>
hipError_t bwd_typed(const AdalnArgs& in, const AdalnGrads& g, const Plan& p, void* ws, hipStream_t stream) {
  BwdArgs<T> a{static_cast<const T*>(g.dout), static_cast<const T*>(g.dres), static_cast<const T*>(in.h),
               static_cast<const T*>(in.branch), in.post_weight, in.gate, in.gamma, static_cast<T*>(g.dx),
               static_cast<T*>(g.dbranch), static_cast<float*>(ws), in.seqlen, in.d_model, p.rows_per_wg,
               in.mod_rows == 1 ? 0 : in.d_model, 1.0f / static_cast<float>(in.d_model), in.eps, in.rms};
  const dim3 grid(static_cast<unsigned>(p.chunks), static_cast<unsigned>(in.batch));
  with_waves(p.waves, [&](auto w) {
    constexpr int W = decltype(w)::value;
    hipLaunchKernelGGL((k_adaln_bwd<T, W>), grid, dim3(W == 1 ? 256 : W * 64), 0, stream, a);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!g.dgamma && !g.dbeta && !g.dgate && !g.dpost_weight) return e;
  const ReduceArgs r{static_cast<const float*>(ws), {g.dgamma, g.dbeta, g.dgate, g.dpost_weight}, in.d_model,
                     p.chunks * row_groups(p.waves), in.batch, in.mod_rows == 1};
  hipLaunchKernelGGL(k_adaln_reduce, dim3(static_cast<unsigned>((in.d_model + 63) / 64),
                                          static_cast<unsigned>(in.mod_rows == 1 ? 1 : in.batch), kSums),
                     dim3(1024), 0, stream, r);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adaln_fwd(const AdalnArgs& a, hipStream_t stream) {
  const Plan p = fwd_plan(a.batch, a.seqlen, a.d_model);
  return a.io_dtype == 1 ? fwd_typed<bf16_t>(a, p, stream) : fwd_typed<float>(a, p, stream);
}

hipError_t launch_adaln_bwd(const AdalnArgs& a, const AdalnGrads& g, void* workspace, hipStream_t stream) {
  const Plan p = bwd_plan(a.batch, a.seqlen, a.d_model);
  return a.io_dtype == 1 ? bwd_typed<bf16_t>(a, g, p, workspace, stream)
                         : bwd_typed<float>(a, g, p, workspace, stream);
}

}  // namespace adaln
}  // namespace bimamba
