// Device helpers of the gated delta rule's kernels: matrix operands, fp32 values as sums of bf16 parts, LDS tiles.
// gfx950 only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "delta_plan.h"
#include "device_math.h"
#include "lds_barrier.h"

namespace bimamba {
namespace delta {

constexpr int C = static_cast<int>(kC);

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
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
// Two values as one part, which they lose: the rounded pair, first in the low half.
__device__ __forceinline__ uint32_t take_part(float& a, float& b, bool more) {
  const uint32_t p = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
  if (more) {
    a -= __uint_as_float(p << 16);
    b -= __uint_as_float(p & 0xffff0000u);
  }
  return p;
}

template <int PARTS>
__device__ __forceinline__ void split4(f32x4 v, u32x2 (&p)[PARTS]) {
  float a = v[0], b = v[1], c = v[2], d = v[3];
#pragma unroll
  for (int i = 0; i < PARTS; ++i) p[i] = u32x2{take_part(a, b, i + 1 < PARTS), take_part(c, d, i + 1 < PARTS)};
}

template <int PARTS>
__device__ __forceinline__ void split8(f32x8 v, bf16x8 (&p)[PARTS]) {
  u32x2 lo[PARTS], hi[PARTS];
  split4(f32x4{v[0], v[1], v[2], v[3]}, lo);
  split4(f32x4{v[4], v[5], v[6], v[7]}, hi);
#pragma unroll
  for (int i = 0; i < PARTS; ++i) p[i] = __builtin_bit_cast(bf16x8, u32x4{lo[i][0], lo[i][1], hi[i][0], hi[i][1]});
}

// A wavefront's rows of the state, column tile nt, as operands of three parts.
template <int ST, int NT, typename T>
__device__ __forceinline__ void split_own(const f32x4 (&S)[ST][NT], int nt, T (&p)[3]) {
  u32x2 x[ST][3];
#pragma unroll
  for (int st = 0; st < ST; ++st) split4(S[st][nt], x[st]);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if constexpr (ST == 1) p[i] = __builtin_bit_cast(T, x[0][i]);
    else p[i] = __builtin_bit_cast(T, u32x4{x[0][i][0], x[0][i][1], x[1][i][0], x[1][i][1]});
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

// D += A B with the terms that a wavefront's own result rows make up: lane l holds 4 (16 x 16 x 16) or 8 (16 x 16 x 32)
// consecutive ones from 4 (l / 16) or 8 (l / 16).
__device__ __forceinline__ f32x4 mfma_own(const bf16x8& a, const bf16x8& b, const f32x4& c) { return mfma(a, b, c); }
__device__ __forceinline__ f32x4 mfma_own(const bf16x4& a, const bf16x4& b, const f32x4& c) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a), __builtin_bit_cast(s16x4, b), c, 0, 0, 0);
}

template <int ST>
struct Own;  // the operand of a wavefront's ST tiles of state rows
template <>
struct Own<1> {
  typedef bf16x4 type;
};
template <>
struct Own<2> {
  typedef bf16x8 type;
};

// Rows of the state: a wavefront owns 16 ST consecutive ones as ST result tiles, whose rows are numbered so that a lane's
// 4 ST values are consecutive rows (and make up an operand of the next product without leaving the lane): row m of tile t
// of wavefront w is state row
template <int ST>
__device__ __forceinline__ int state_row(int w, int t, int m) {
  return 16 * ST * w + 4 * ST * (m >> 2) + 4 * t + (m & 3);
}

// Where the operands of a triangular 64 x 64 matrix lie in a record.  lower: rows 16 w, k 32 s, entries with k <= row;
// upper: entries with k >= row.
__device__ __forceinline__ int lower_at(int w, int s) { return w < 2 ? w : 2 * w - 2 + s; }
__device__ __forceinline__ int upper_at(int w, int s) { return w < 2 ? 2 * w + s : w + 2; }
__device__ __forceinline__ bool lower_has(int w, int s) { return s <= (w >> 1); }
__device__ __forceinline__ bool upper_has(int w, int s) { return s >= (w >> 1); }

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

// What a call works on.  Chunks are runs of 64 tokens from the sequence's start in both directions; the reverse one meets
// them from the last to the first, and their tokens from the last to the first.  In the last run the places past the
// sequence's end are empty (for the reverse direction the first ones that it meets): q = k = v = 0, no decay, beta = 0,
// a token that changes nothing.
struct Shape {
  int64_t L, hk, heads;
  int rev;
  // the run that is met as the i-th of n, and the token of its i-th place
  __device__ __forceinline__ int run(int i, int n) const { return rev ? n - 1 - i : i; }
  __device__ __forceinline__ int place(int i) const { return rev ? C - 1 - i : i; }
};

// The rows of a run of 64 tokens in a tensor [batch, L, nh, D] of bf16, one head, as a buffer: rows past the sequence's end
// read zeros and drop stores, and a lane's offset is the same for every run.  base: the sequence's first row; pitch:
// bytes from one token's row to the next; width: bytes of a row that are used.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t run_rows(const void* base, const Shape& sh, int pitch, int width,
                                                           int run) {
  const int left = static_cast<int>(sh.L) - run * C, n = left < C ? left : C;
  return __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char*>(static_cast<const char*>(base) + static_cast<int64_t>(run) * (C * pitch)),
      static_cast<short>(0), (n - 1) * pitch + width, 0x00020000);
}

__device__ __forceinline__ bf16x8 row_load8(__amdgpu_buffer_rsrc_t t, int offset) {
  return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(t, offset, 0, 0));
}

__device__ __forceinline__ bf16x4 row_load4(__amdgpu_buffer_rsrc_t t, int offset) {
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_raw_buffer_load_b64(t, offset, 0, 0));
}

__device__ __forceinline__ void row_load(__amdgpu_buffer_rsrc_t t, int offset, bf16x8* v) { *v = row_load8(t, offset); }
__device__ __forceinline__ void row_load(__amdgpu_buffer_rsrc_t t, int offset, bf16x4* v) { *v = row_load4(t, offset); }

__device__ __forceinline__ uint16_t row_load1(__amdgpu_buffer_rsrc_t t, int offset) {
  return __builtin_amdgcn_raw_buffer_load_b16(t, offset, 0, 0);
}

__device__ __forceinline__ void row_store1(__amdgpu_buffer_rsrc_t t, int offset, float v) {
  bf16_t o;
  from_f32(v, &o);
  __builtin_amdgcn_raw_buffer_store_b16(o.bits, t, offset, 0, 0);
}

// A record of operands, the same way.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t record(const unsigned char* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char*>(p), static_cast<short>(0),
                                           static_cast<int>(bytes), 0x00020000);
}

// The frag-th operand from byte off (the same for all lanes) of a record; four share one scalar offset.
__device__ __forceinline__ bf16x8 record_frag(__amdgpu_buffer_rsrc_t r, int off, int frag, int lane16) {
  constexpr int kB = static_cast<int>(kFragBytes);
  return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(r, lane16 + frag % 4 * kB,
                                                                          off + frag / 4 * (4 * kB), 0));
}

// (x[0] + x[1] + x[2]) (y[0] + y[1] + y[2]) in three sums that do not wait for one another.
__device__ __forceinline__ void mfma_three(const bf16x8 (&x)[3], const bf16x8 (&y)[3], f32x4 (&c)[3]) {
  c[0] = mfma(x[0], y[2], c[0]);
  c[1] = mfma(x[1], y[1], c[1]);
  c[2] = mfma(x[2], y[0], c[2]);
  c[1] = mfma(x[0], y[1], c[1]);
  c[2] = mfma(x[1], y[0], c[2]);
  c[0] = mfma(x[0], y[0], c[0]);
}

// x (y[0] + y[1] + y[2]), likewise.
__device__ __forceinline__ void mfma_three(const bf16x8& x, const bf16x8 (&y)[3], f32x4 (&c)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) c[i] = mfma(x, y[i], c[i]);
}

__device__ __forceinline__ f32x4 sum3(const f32x4 (&c)[3]) { return c[0] + (c[1] + c[2]); }

}  // namespace delta
}  // namespace bimamba
