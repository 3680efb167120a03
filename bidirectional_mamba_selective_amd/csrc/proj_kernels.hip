// Product of 8-bit rows and 8-bit weights (OCP e4m3) with a scale for each row and 128 inputs, and for each 128 x 128
// weights, for gfx950:
//   out[m,n] = sum_j xs[m,j] ws[n/128,j] sum_{k in block j} x[m,k] w[n,k]
// The inner sums run on the matrix cores (v_mfma_f32_16x16x128_f8f6f4: a block of 128 inputs in one instruction, products
// of e4m3 values are exact, sums in fp32); the two scales are applied to each block's sum in fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "launch.h"

namespace bimamba {
namespace proj {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Args {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* out;
  int64_t m, n, k;
};

// Lane l holds row l % 16 of an operand at 16-byte chunks l / 16 and 4 + l / 16 of the block's 128 bytes (both operands
// alike, so the order of the inputs within the block does not matter), and of the result column l % 16 (of the second
// operand's rows), rows 4 (l / 16) .. + 3 (of the first's).
__device__ __forceinline__ f32x4 mfma128(i32x8 a, i32x8 b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7f7f7f7f, 0,
                                                          0x7f7f7f7f);
}

constexpr int BM = 128, BN = 128, BK = 128;

__device__ __forceinline__ int chunk_at(int row, int c) { return row * BK + ((c ^ (row & 7)) << 4); }

__device__ __forceinline__ i32x8 operand(const uint8_t* s, int row, int q4) {
  const i32x4 a = *reinterpret_cast<const i32x4*>(s + chunk_at(row, q4));
  const i32x4 b = *reinterpret_cast<const i32x4*>(s + chunk_at(row, 4 + q4));
  return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

template <typename T>
__device__ __forceinline__ void store4(f32x4 v, T* p) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<f32x4*>(p) = v;
  } else {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(v, bf16x4);
  }
}

// 128 rows x 128 outputs per workgroup, 64 x 64 per wavefront.
template <typename T>
__global__ __launch_bounds__(256) void k_proj(Args a) {
  __shared__ __align__(16) uint8_t sx[2][BM * BK], sw[2][BN * BK];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q4 = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * BM, n0 = static_cast<int64_t>(blockIdx.y) * BN;
  const int64_t kb = a.k / BK;
  const int wm = (w & 1) * 64, wn = (w >> 1) * 64;
  i32x4 rx[4], rw[4];
  auto fetch = [&](int64_t j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = tid + 256 * i, row = c >> 3;
      const int64_t m = m0 + row < a.m ? m0 + row : a.m - 1, n = n0 + row < a.n ? n0 + row : a.n - 1;
      rx[i] = *reinterpret_cast<const i32x4*>(a.x + m * a.k + j * BK + (c & 7) * 16);
      rw[i] = *reinterpret_cast<const i32x4*>(a.w + n * a.k + j * BK + (c & 7) * 16);
    }
  };
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float* xs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + wm + 16 * i + l16;
    xs[i] = a.xs + (m < a.m ? m : a.m - 1) * kb;
  }
  const float* ws = a.ws + blockIdx.y * kb;
  fetch(0);
  for (int64_t j = 0; j < kb; ++j) {
    uint8_t* bx = sx[j & 1];
    uint8_t* bw = sw[j & 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = tid + 256 * i;
      *reinterpret_cast<i32x4*>(bx + chunk_at(c >> 3, c & 7)) = rx[i];
      *reinterpret_cast<i32x4*>(bw + chunk_at(c >> 3, c & 7)) = rw[i];
    }
    __syncthreads();
    if (j + 1 < kb) fetch(j + 1);
    i32x8 wf[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wf[i] = operand(bw, wn + 16 * i + l16, q4);
    const float s = ws[j];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const i32x8 xf = operand(bx, wm + 16 * i + l16, q4);
      const float c = xs[i][j] * s;
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[i][n] += mfma128(wf[n], xf) * c;
    }
  }
  T* out = static_cast<T*>(a.out);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + wm + 16 * i + l16;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int64_t col = n0 + wn + 16 * n + 4 * q4;
      if (m < a.m && col < a.n) store4<T>(acc[i][n], out + m * a.n + col);
    }
  }
}

}  // namespace

hipError_t launch_proj(const ProjArgs& in, hipStream_t stream) {
  const Args a{static_cast<const uint8_t*>(in.x), in.xs, static_cast<const uint8_t*>(in.w), in.ws, in.out, in.m, in.n,
               in.k};
  const dim3 grid(static_cast<unsigned>((in.m + BM - 1) / BM), static_cast<unsigned>((in.n + BN - 1) / BN));
  if (in.out_dtype == 1) hipLaunchKernelGGL((k_proj<bf16_t>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((k_proj<float>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace proj
}  // namespace bimamba
