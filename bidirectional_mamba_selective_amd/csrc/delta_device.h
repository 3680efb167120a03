// Device helpers of the gated delta rule's kernels: matrix operands, fp32 values as sums of bf16 parts, LDS tiles.
// gfx950 only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "delta_plan.h"
#include "device_math.h"

namespace bimamba {
namespace delta {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// D += A B, 16 x 16 x 32.  Lane l holds row (A) or column (B) l % 16 of its operand at k = 8 (l / 16) .. + 7, and of the
// result column l % 16, rows 4 (l / 16) .. + 3.
__device__ __forceinline__ f32x4 mfma(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The same in fp32, 16 x 16 x 4: one value a lane, row or column l % 16, k = l / 16.
__device__ __forceinline__ f32x4 mfma_f32(float a, float b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }
__device__ __forceinline__ bf16x8 zero8() { return __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u}); }

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// An fp32 value as a sum of bf16 parts, each the rounding of what the ones before leave: two parts carry it to 2^-17
// relative, three to its last bit (where the parts stay normal numbers).
template <int PARTS>
__device__ __forceinline__ void split4(f32x4 v, u32x2 (&p)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const bf16x4 r = __builtin_convertvector(v, bf16x4);
    p[i] = __builtin_bit_cast(u32x2, r);
    if (i + 1 < PARTS) v -= __builtin_convertvector(r, f32x4);
  }
}

template <int PARTS>
__device__ __forceinline__ void split8(f32x8 v, bf16x8 (&p)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    p[i] = __builtin_convertvector(v, bf16x8);
    if (i + 1 < PARTS) v -= __builtin_convertvector(p[i], f32x8);
  }
}

// LDS tiles of rows of W bf16 values (W 64 or 128) in 16-byte chunks, each row's chunks permuted so that 16 lanes that
// read one chunk of 16 rows meet different banks.  Index in values.
template <int W>
__device__ __forceinline__ int at(int row, int col) {
  const int c = col >> 3;
  if constexpr (W == 128) return row * 128 + ((c ^ (row & 15)) << 3) + (col & 7);
  else return row * 64 + ((c ^ ((row >> 1) & 7)) << 3) + (col & 7);
}

template <int W>
__device__ __forceinline__ bf16x8 read8(const uint16_t* s, int row, int col) {
  return *reinterpret_cast<const bf16x8*>(s + at<W>(row, col));
}

template <int W>
__device__ __forceinline__ void write4(uint16_t* s, int row, int col, u32x2 v) {
  *reinterpret_cast<u32x2*>(s + at<W>(row, col)) = v;
}

// Where the operands of a triangular 64 x 64 matrix lie in a record.  lower: rows 16 w, k 32 s, entries with k <= row;
// upper: entries with k >= row.
__device__ __forceinline__ int lower_at(int w, int s) { return w < 2 ? w : 2 * w - 2 + s; }
__device__ __forceinline__ int upper_at(int w, int s) { return w < 2 ? 2 * w + s : w + 2; }
__device__ __forceinline__ bool lower_has(int w, int s) { return s <= (w >> 1); }
__device__ __forceinline__ bool upper_has(int w, int s) { return s >= (w >> 1); }

__device__ __forceinline__ bf16x8 load_frag(const unsigned char* base, int frag, int lane) {
  return *reinterpret_cast<const bf16x8*>(base + static_cast<size_t>(frag) * kFragBytes + lane * 16);
}

__device__ __forceinline__ void store_frag(unsigned char* base, int frag, int lane, bf16x8 v) {
  *reinterpret_cast<bf16x8*>(base + static_cast<size_t>(frag) * kFragBytes + lane * 16) = v;
}

// (sum of X's parts) (sum of Y's parts), leaving out products below 2^-24 of the whole.
template <int PX, int PY>
__device__ __forceinline__ f32x4 mfma_parts(const bf16x8 (&x)[PX], const bf16x8 (&y)[PY], f32x4 c) {
  constexpr int last = (PX > PY ? PX : PY) - 1;
#pragma unroll
  for (int i = PX - 1; i >= 0; --i)
#pragma unroll
    for (int j = PY - 1; j >= 0; --j)
      if (i + j <= last) c = mfma(x[i], y[j], c);
  return c;
}

__device__ __forceinline__ float ex(float v) { return fast_exp2(v * kLog2e); }

__device__ __forceinline__ float sigmoid_f32(float v) { return __builtin_amdgcn_rcpf(1.0f + ex(-v)); }

// What a call works on; the sequence's tokens in the order in which the direction meets them: place p is token
// p (forward) or L - 1 - p (reverse).
struct Shape {
  int64_t L, hk, heads;
  int rev;
  __device__ __forceinline__ int64_t token(int64_t p) const { return rev ? L - 1 - p : p; }
};

}  // namespace delta
}  // namespace bimamba
