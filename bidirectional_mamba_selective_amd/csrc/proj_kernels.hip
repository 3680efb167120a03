// Product of 8-bit rows and 8-bit weights (OCP e4m3) with a scale for each row and 128 inputs, and for each 128 x 128
// weights, for gfx950:
//   out[m,n] = sum_j xs[m,j] ws[n/128,j] sum_{k in block j} x[m,k] w[n,k]
// The inner sums run on the matrix cores, the two scales are applied to each block's sum in fp32.
//
// bf16 results take a block of 128 inputs in one v_mfma_f32_16x16x128_f8f6f4.  Its adder drops low bits of small products
// beside large ones: sums of N(0, 1) operands come out 1.4e-5 off normwise (1.3e-5 of the terms' magnitudes at most on
// single ones; 1.5e-5 of the rms for 128 to 16384 inputs), the same as with the older 8-bit instructions.  Next to the
// result's own rounding, up to 2^-8, it moves the distance to the exact product in the fifth digit (1.65878e-3 and
// 1.65871e-3 from fp32 sums, 32 x 8056 x 1920), for twice the rate of bf16 operands.  fp32 results are to be better than
// that: there the operands are widened to bf16, which holds every e4m3 value, and take four v_mfma_f32_16x16x32_bf16, whose
// sums are fp32 ones (1e-7), at half the rate.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "launch.h"
#include "lds_barrier.h"

namespace bimamba {
namespace proj {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int BK = 128;  // inputs that share a scale

struct Args {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* out;
  int64_t m, n, k;
};

// A row's 128 inputs as an operand: lane l holds row l % 16 at 16-byte chunks l / 16 and 4 + l / 16 (both operands alike,
// so the order of the inputs within the block does not matter), and of the result column l % 16 (of the second operand's
// rows), rows 4 (l / 16) .. + 3 (of the first's).
template <bool WIDE>
struct Operand;

template <>
struct Operand<false> {
  i32x8 v;
  __device__ __forceinline__ void set(i32x4 a, i32x4 b) { v = i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }
};

template <>
struct Operand<true> {
  bf16x8 v[4];
  static __device__ __forceinline__ bf16x8 widen(int a, int b) {
    const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const bf16x2 q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const bf16x2 s = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return bf16x8{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
  }
  __device__ __forceinline__ void set(i32x4 a, i32x4 b) {
    v[0] = widen(a[0], a[1]), v[1] = widen(a[2], a[3]), v[2] = widen(b[0], b[1]), v[3] = widen(b[2], b[3]);
  }
};

__device__ __forceinline__ f32x4 block_sum(const Operand<false>& a, const Operand<false>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7f7f7f7f, 0,
                                                          0x7f7f7f7f);
}

__device__ __forceinline__ f32x4 block_sum(const Operand<true>& a, const Operand<true>& b) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

template <typename T>
__device__ __forceinline__ void store4(f32x4 v, T* p) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4*>(p) = v;
  else *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(v, bf16x4);
}

// Rows of 128 bytes in LDS, their 16-byte chunks permuted so that 16 lanes reading one chunk of 16 rows meet all banks.
__device__ __forceinline__ int chunk_at(int row, int c) { return row * BK + ((c ^ (row & 7)) << 4); }

// The operand of rows row + 16 i: lo and hi point at the two chunks of row (the permutation has a period of 8 rows).
template <bool WIDE>
__device__ __forceinline__ void read_operand(const uint8_t* lo, const uint8_t* hi, int i, Operand<WIDE>* o) {
  o->set(*reinterpret_cast<const i32x4*>(lo + 16 * BK * i), *reinterpret_cast<const i32x4*>(hi + 16 * BK * i));
}

// A tile's rows of k bytes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rows(const uint8_t* p, int64_t row0, int64_t rows, int64_t k,
                                                            int tile) {
  const int64_t n = min(rows - row0, static_cast<int64_t>(tile));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p + row0 * k), static_cast<short>(0),
                                           static_cast<int>(n * k), 0x00020000);
}

// Tiles of WM x WN wavefronts of 16 MI rows x 16 NI outputs (16 NI divides 128, so a wavefront's outputs share their
// scales).  Two LDS buffers and one barrier per step of 128 inputs: rows are loaded into registers two steps ahead and
// written to the other buffer one step ahead, in pieces that are spread over the step's products.  Measured at 16384 x
// 8192 x 4096, bf16 results: 565 to 600 us with the clock (1.85 to 1.95 PFLOP/s; the library's 8-bit product with a
// single scale reaches 2.49 on 8192^3); loads in one burst at the step's start 626, straight into LDS slower (later LDS
// reads wait for them), two row tiles read ahead 802 (spills).  What bounds it: after each barrier the matrix cores wait for
// the first operands from LDS, and 16 fp32 multiply-adds a product apply the scales.  fp32 results are bound by the
// widening to bf16, done again by each wavefront that reads an operand: 1001 x 1920 x 3840 in 28 us.
template <typename T, bool WIDE, int MI, int NI, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_proj(Args a, int tiles_m, int tiles_n) {
  constexpr int W = WM * WN, BM = 16 * MI * WM, BN = 16 * NI * WN, LX = BM / 8 / W, LW = BN / 8 / W;
  __shared__ __align__(16) uint8_t sx[2][BM * BK], sw[2][BN * BK];
  __shared__ float ss[2][64 * W];  // the rows' scales of the step (each thread brings one; those past BM are not used)
  static_assert(64 * W >= BM, "a thread per row");
  const int lane = threadIdx.x & 63, l16 = lane & 15, q4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroups go to the eight XCDs in turn: each XCD takes a run of tiles of its own, in columns of 8 tiles of rows, so
  // that rows and weights are reused in its L2
  const int total = tiles_m * tiles_n, run = (total + 7) / 8;
  const int id = static_cast<int>(blockIdx.x & 7) * run + static_cast<int>(blockIdx.x >> 3);
  if (static_cast<int>(blockIdx.x >> 3) >= run || id >= total) return;
  const int group = id / (8 * tiles_n), rows_here = min(8, tiles_m - 8 * group), in_group = id - group * 8 * tiles_n;
  const int64_t m0 = static_cast<int64_t>(8 * group + in_group % rows_here) * BM;
  const int64_t n0 = static_cast<int64_t>(in_group / rows_here) * BN;
  const int wm = wave % WM * 16 * MI, wn = wave / WM * 16 * NI;
  const int kb = static_cast<int>(a.k / BK);

  // thread t brings chunk t % 8 of rows t / 8 + 8 W i; rows past the end come from the last one and are not stored
  const int brow = threadIdx.x >> 3, bat = chunk_at(brow, threadIdx.x & 7);
  const __amdgpu_buffer_rsrc_t rx = tile_rows(a.x, m0, a.m, a.k, BM), rw = tile_rows(a.w, n0, a.n, a.k, BN);
  uint32_t ox[LX], ow[LW];
#pragma unroll
  for (int i = 0; i < LX; ++i)
    ox[i] = static_cast<uint32_t>(min(static_cast<int64_t>(brow + 8 * W * i), a.m - m0 - 1) * a.k) + (threadIdx.x & 7) * 16;
#pragma unroll
  for (int i = 0; i < LW; ++i)
    ow[i] = static_cast<uint32_t>(min(static_cast<int64_t>(brow + 8 * W * i), a.n - n0 - 1) * a.k) + (threadIdx.x & 7) * 16;
  const float* xs = a.xs + min(m0 + threadIdx.x, a.m - 1) * kb;
  const float* ws = a.ws + min((n0 + wn) / BK, (a.n - 1) / BK) * kb;

  // a step's rows in pieces: LX of x, LW of w
  constexpr int kPieces = LX + LW;
  i32x4 g[kPieces];
  float gs, gws;
  auto fetch = [&](int p, int j) {
    g[p] = __builtin_bit_cast(i32x4, p < LX ? __builtin_amdgcn_raw_buffer_load_b128(rx, ox[p < LX ? p : 0], j * BK, 0)
                                            : __builtin_amdgcn_raw_buffer_load_b128(rw, ow[p < LX ? 0 : p - LX], j * BK, 0));
  };
  auto fetch_scales = [&](int j) { gs = xs[j], gws = ws[j]; };
  auto put = [&](int p, int j) {
    *reinterpret_cast<i32x4*>((p < LX ? sx[j & 1] + 8 * W * BK * p : sw[j & 1] + 8 * W * BK * (p - LX)) + bat) = g[p];
  };

  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int xlo = chunk_at(wm + l16, q4), xhi = chunk_at(wm + l16, 4 + q4);
  const int wlo = chunk_at(wn + l16, q4), whi = chunk_at(wn + l16, 4 + q4);
  fetch_scales(0);
#pragma unroll
  for (int p = 0; p < kPieces; ++p) fetch(p, 0);
  float wsj = gws;
  ss[0][threadIdx.x] = gs;
#pragma unroll
  for (int p = 0; p < kPieces; ++p) put(p, 0);
  fetch_scales(min(1, kb - 1));
#pragma unroll
  for (int p = 0; p < kPieces; ++p) fetch(p, min(1, kb - 1));
  for (int j = 0; j < kb; ++j) {
    // no branch in the loop: the compiler would move the products across it
    const int ahead = min(j + 2, kb - 1);
    lds_barrier();
    const uint8_t *cx = sx[j & 1], *cw = sw[j & 1];
    Operand<WIDE> wf[NI], xf[2];
    read_operand(cx + xlo, cx + xhi, 0, &xf[0]);
#pragma unroll
    for (int n = 0; n < NI; ++n) read_operand(cw + wlo, cw + whi, n, &wf[n]);
    // a row tile's products are scaled, one by one, between those of the next; the pieces that came in during the last
    // step go into the other buffer, and those of the step after next are asked for, evenly over the step
    f32x4 t[NI];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i <= MI; ++i) {
      const float next = i < MI ? ss[j & 1][wm + 16 * i + l16] * wsj : 0.0f;
      if (i + 1 < MI) read_operand(cx + xlo, cx + xhi, i + 1, &xf[(i + 1) & 1]);
#pragma unroll
      for (int n = 0; n < NI; ++n) {
        if (i > 0) acc[i - 1][n] += t[n] * s;
        if (i < MI) t[n] = block_sum(wf[n], xf[i & 1]);
      }
      s = next;
#pragma unroll
      for (int p = kPieces * i / MI; p < kPieces * (i + 1) / MI && p < kPieces; ++p) {
        put(p, j + 1);
        fetch(p, ahead);
      }
    }
    ss[(j + 1) & 1][threadIdx.x] = gs;
    wsj = gws;
    fetch_scales(ahead);
  }
  T* out = static_cast<T*>(a.out);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t m = m0 + wm + 16 * i + l16;
#pragma unroll
    for (int n = 0; n < NI; ++n) {
      const int64_t col = n0 + wn + 16 * n + 4 * q4;
      if (m < a.m && col < a.n) store4<T>(acc[i][n], out + m * a.n + col);
    }
  }
}

// Few rows: the weights pass through once and bound the call.  A workgroup takes 16 outputs of all rows (16 MI of them); its
// eight wavefronts take every eighth block of inputs, straight into registers, and add their sums in LDS.  What bounds it
// beside the weights (16 rows x 4096 x 4096: 7.2 us, 2.3 TB/s) is reading the rows again for each 16 outputs, from the L2.
template <typename T, bool WIDE, int MI>
__global__ __launch_bounds__(512) void k_proj_rows(Args a) {
  constexpr int W = 8;
  __shared__ float sums[W][MI][256];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int kb = static_cast<int>(a.k / BK);
  const uint8_t* wrow = a.w + min(n0 + l16, a.n - 1) * a.k + q4 * 16;
  const float* ws = a.ws + n0 / BK * kb;
  const uint8_t* xrow[MI];
  const float* xs[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t m = min(static_cast<int64_t>(16 * i + l16), a.m - 1);
    xrow[i] = a.x + m * a.k + q4 * 16;
    xs[i] = a.xs + m * kb;
  }
  f32x4 acc[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int j = wave; j < kb; j += W) {
    Operand<WIDE> wf;
    wf.set(__builtin_nontemporal_load(reinterpret_cast<const i32x4*>(wrow + static_cast<int64_t>(j) * BK)),
           __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(wrow + static_cast<int64_t>(j) * BK + 64)));
    const float wsj = ws[j];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      Operand<WIDE> xf;
      xf.set(*reinterpret_cast<const i32x4*>(xrow[i] + static_cast<int64_t>(j) * BK),
             *reinterpret_cast<const i32x4*>(xrow[i] + static_cast<int64_t>(j) * BK + 64));
      acc[i] += block_sum(wf, xf) * (xs[i][j] * wsj);
    }
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) *reinterpret_cast<f32x4*>(&sums[wave][i][4 * lane]) = acc[i];
  __syncthreads();
  T* out = static_cast<T*>(a.out);
  for (int i = wave; i < MI; i += W) {
    f32x4 t = *reinterpret_cast<const f32x4*>(&sums[0][i][4 * lane]);
#pragma unroll
    for (int v = 1; v < W; ++v) t += *reinterpret_cast<const f32x4*>(&sums[v][i][4 * lane]);
    const int64_t m = 16 * i + l16, col = n0 + 4 * q4;
    if (m < a.m && col < a.n) store4<T>(t, out + m * a.n + col);
  }
}

template <typename T, bool WIDE, int MI, int NI, int WM, int WN>
void launch_tiles(const Args& a, hipStream_t stream) {
  constexpr int BM = 16 * MI * WM, BN = 16 * NI * WN;
  const int64_t tm = (a.m + BM - 1) / BM, tn = (a.n + BN - 1) / BN;
  const dim3 grid(static_cast<unsigned>((tm * tn + 7) / 8 * 8));
  hipLaunchKernelGGL((k_proj<T, WIDE, MI, NI, WM, WN>), grid, dim3(64 * WM * WN), 0, stream, a, static_cast<int>(tm),
                     static_cast<int>(tn));
}

template <typename T, bool WIDE, int MI>
void launch_rows(const Args& a, hipStream_t stream) {
  hipLaunchKernelGGL((k_proj_rows<T, WIDE, MI>), dim3(static_cast<unsigned>((a.n + 15) / 16)), dim3(512), 0, stream, a);
}

// Which kernel, by the groups of 16 rows times the outputs and by the tiles of each size (us a call, k = 4096 unless
// given; bf16 | fp32 results):
// - k_proj_rows reads every row again for each 16 outputs, tiles of 64 x 64 walk all of k one after the other.  Rows for
//   groups x n <= 8192 and 32 rows (fp32, whose tiles are slower: 16384 and 64), rows and tiles at
//     16 x 4096: 7.2, 14.2 | 7.2, 18.5       32 x 4096: 10.4, 14.1 | 10.2, 18.7     16 x 8192: 12.1, 14.7 | 12.2, 19.4
//     32 x 8192: 17.5, 14.9 | 17.2, 19.4     64 x 4096: 16.3, 14.5 | 16.4, 19.0     16 x 16384: 22.4, 15.7 | 22.5, 20.1
// - 128 x 128 from more than 192 of them, below that too few compute units have one; 64 x 64 and 128 x 128 at
//     768 x 4096 (192): 41.9, 42.2 | 48.8, 52.0       896 x 4096 (224): 50.4, 41.9 | 58.0, 53.4
//     768 x 4096, k = 1024: 11.7, 13.3 | 14.6, 17.3   896 x 4096: 14.1, 13.5 | 17.5, 17.8
// - 256 x 256 from more than 128 of them; 128 x 128 and 256 x 256 at
//     2048 x 4096 (128): 61.7, 62.8       2304 x 4096 (144): 88.5, 59.9       4096 x 4096 (256): 109.3, 70.6
//     2048 x 4096, k = 1024: 19.9, 24.4   2560 x 4096 (160): 29.9, 25.0       5120 x 4096 (320): 45.2, 44.8
//   The operands of fp32 results, widened, do not fit the registers of such a tile.
// All measured with 4096 outputs or more and k of 1024 and 4096; narrower outputs, whose last tiles are partly empty, and
// longer k follow the same rules unmeasured.
template <typename T, bool WIDE>
void launch_typed(const Args& a, hipStream_t stream) {
  const int64_t groups = (a.m + 15) / 16;
  if (a.m <= (WIDE ? 64 : 32) && groups * a.n <= (WIDE ? 16384 : 8192)) {
    if (groups == 1) return launch_rows<T, WIDE, 1>(a, stream);
    if (groups == 2) return launch_rows<T, WIDE, 2>(a, stream);
    if constexpr (WIDE) return launch_rows<T, WIDE, 4>(a, stream);
  }
  const int64_t t128 = (a.m + 127) / 128 * ((a.n + 127) / 128), t256 = (a.m + 255) / 256 * ((a.n + 255) / 256);
  if constexpr (!WIDE) {
    if (t256 > 128) return launch_tiles<T, WIDE, 8, 4, 2, 4>(a, stream);
  }
  if (t128 > 192) launch_tiles<T, WIDE, 4, 4, 2, 2>(a, stream);
  else launch_tiles<T, WIDE, 2, 2, 2, 2>(a, stream);
}

}  // namespace

hipError_t launch_proj(const ProjArgs& in, hipStream_t stream) {
  const Args a{static_cast<const uint8_t*>(in.x), in.xs, static_cast<const uint8_t*>(in.w), in.ws, in.out, in.m, in.n,
               in.k};
  if (in.out_dtype == 1) launch_typed<bf16_t, false>(a, stream);
  else launch_typed<float, true>(a, stream);
  return hipGetLastError();
}

}  // namespace proj
}  // namespace bimamba
