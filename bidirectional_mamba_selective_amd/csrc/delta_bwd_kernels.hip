// Backward pass of the gated delta rule (delta_kernels.hip has the forward pass and its symbols) for gfx950.  With dO the
// gradient of O, dS that of the state after a chunk, R = V - diag(e^g) K S and all of it per chunk of 64 tokens:
//   dU = A^T dO + diag(e^(g_C - g)) K dS,   dR = T^T dU = dV
//   dS_before = e^(g_C) dS + scale (diag(e^g) Q)^T dO - (diag(e^g) K)^T dR
//   D1_ij = scale e^(g_i - g_j) dO_i.U_j (j <= i),   D2_ij = -e^(g_i - g_j) dR_i.U_j (j < i)
//   dQ = scale diag(e^g) dO S^T + D1 K
//   dK = -diag(e^g) dR S^T + D2 K + diag(e^(g_C - g)) U dS^T + D1^T Q + D2^T K
//   db_i = (1 - beta_i) / beta_i dR_i.U_i        (both factors carry a beta_i)
// A token's log decay multiplies every term that reaches across it, so its gradient is the sum of just those terms (no
// sums that cancel): with P_ij = D1_ij q_i.k_j + D2_ij k_i.k_j, s_i = scale e^(g_i) dO_i.S^T q_i - e^(g_i) dR_i.S^T k_i,
// e_j = e^(g_C - g_j) U_j.dS^T k_j,
//   dg_t = sum_{j < t <= i} P_ij + sum_{i >= t} s_i + sum_{j < t} e_j + e^(g_C) <S, dS>
//
// The chunks' operands and states come from the forward kernels, which run again; k_delta_rwalk goes over the chunks from
// the last to the first as k_delta_walk goes the other way; k_delta_grads then takes all chunks at once, a workgroup per
// chunk and key head, so that the gradients of shared keys and queries are summed in registers in a fixed order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "delta_device.h"
#include "launch.h"

namespace bimamba {
namespace delta {
namespace {

struct RWalkArgs {
  const uint16_t* dout;
  const uint16_t* k;
  uint16_t* dv_out;
  const unsigned char* heads;
  const unsigned char* keys;
  const float* dh_out;  // null: zeros
  float* dh_in;         // null: not written
  float* dstates;       // dS after each chunk, [batch][head][chunk][dk][dv]
  float* drs;           // dR, [batch][head][chunk][64][dv]
  Shape sh;
  Layout lay;
  int64_t batch, dv, chunks;
  float scale;
};

// Heads over XCDs as in the forward walk: the workgroups of one head share an L2.
__device__ __forceinline__ bool place(int64_t slices, int64_t rows, int64_t* row, int64_t* slice) {
  const int64_t x = blockIdx.x & 7, i = blockIdx.x >> 3;
  *row = i / slices * 8 + x;
  *slice = i % slices;
  return *row < rows;
}

// One workgroup: 16 NT columns of the state's gradient.  Four wavefronts carry it as those of the forward walk carry the
// state (K dS, T^T dU, K^T dR).  What does not depend on it (A^T dO and Q^T dO) is made by four more, a chunk ahead,
// between the same barriers, and waits in LDS.  Bound as the forward walk is, by the chain of a chunk (3.4 us at 32 heads
// of 128 x 128: 128 chunks in 438 us), with the states' gradients and dR (96 KB a chunk and head) stored on the way.
template <int DK, int NT>
__global__ __launch_bounds__(512, 2) void k_delta_rwalk(RWalkArgs a) {
  constexpr int ST = DK / 64, NS = 16 * NT, kB = static_cast<int>(kFragBytes);
  typedef typename Own<ST>::type own_t;
  __shared__ __align__(16) float sP[NT][4][4][256], sX[2][NT][4][ST + 1][256];
  __shared__ __align__(16) uint16_t sD[NS * C], sE[3][NS * C], sR[3][NS * C], sU[3][NS * C];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q4 = lane >> 4, lane16 = lane * 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3;
  int64_t bh, slice;
  if (!place(a.dv / NS, a.batch * a.sh.heads, &bh, &slice)) return;
  const int64_t b = bh / a.sh.heads, h = bh % a.sh.heads, kh = h / (a.sh.heads / a.sh.hk);
  const int n0 = static_cast<int>(slice) * NS, dv = static_cast<int>(a.dv), chunks = static_cast<int>(a.chunks);
  const unsigned char* rec = a.heads + bh * a.chunks * a.lay.bytes;
  const unsigned char* key = a.keys + (b * a.sh.hk + kh) * a.chunks * a.lay.key_bytes;
  const int rec_bytes = static_cast<int>(a.lay.bytes), key_bytes = static_cast<int>(a.lay.key_bytes);
  const int key_pitch = static_cast<int>(a.sh.hk) * DK * 2, val_pitch = static_cast<int>(a.sh.heads) * dv * 2;
  int val_row[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) val_row[r] = a.sh.place(16 * w + 4 * q4 + r) * val_pitch + 2 * l16;
  auto gates4 = [&](__amdgpu_buffer_rsrc_t r, int row) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, 16 * q4, 4 * C * row + 64 * w, 0));
  };
  auto head_record = [&](int ci) { return record(rec + static_cast<int64_t>(ci) * rec_bytes, a.lay.bytes); };
  auto load_tri = [&](int ci, size_t off, bf16x8(&f)[2][3]) {
    const __amdgpu_buffer_rsrc_t r = head_record(ci);
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (upper_has(w, s))
#pragma unroll
        for (int i = 0; i < 3; ++i) f[s][i] = record_frag(r, static_cast<int>(off) + upper_at(w, s) * 3 * kB, i, lane16);
  };
  // tile rows of K^T (which 0) or Q^T (1)
  auto load_keys = [&](int ci, int which, bf16x8(&f)[ST][2]) {
    const __amdgpu_buffer_rsrc_t r = record(key + static_cast<int64_t>(ci) * key_bytes, a.lay.key_bytes);
#pragma unroll
    for (int st = 0; st < ST; ++st)
#pragma unroll
      for (int s = 0; s < 2; ++s) f[st][s] = record_frag(r, (which * (DK / 8) + ST * w * 2) * kB, 2 * st + s, lane16);
  };

  if (wave >= 4) {
    const uint16_t* o0 = a.dout + (b * a.sh.L * a.sh.heads + h) * dv + n0;
    bf16x8 af[2][3], qtf[ST][2];
    uint16_t vv[NT][4];
    f32x4 eg;
    auto load = [&](int ci) {
      const __amdgpu_buffer_rsrc_t o = run_rows(o0, a.sh, val_pitch, 2 * NS, a.sh.run(ci, chunks));
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) vv[nt][r] = row_load1(o, val_row[r] + 32 * nt);
      eg = gates4(head_record(ci), 0);
      load_tri(ci, a.lay.at, af);
      load_keys(ci, 1, qtf);
    };
    auto put = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const u32x2 raw = {vv[nt][0] | static_cast<uint32_t>(vv[nt][1]) << 16,
                           vv[nt][2] | static_cast<uint32_t>(vv[nt][3]) << 16};
        write4<C>(sD, 16 * nt + l16, 16 * w + 4 * q4, raw);
        u32x2 p[3];
        split4(f32x4{bf(vv[nt][0]), bf(vv[nt][1]), bf(vv[nt][2]), bf(vv[nt][3])} * (eg * a.scale), p);
#pragma unroll
        for (int i = 0; i < 3; ++i) write4<C>(sE[i], 16 * nt + l16, 16 * w + 4 * q4, p[i]);
      }
    };
    auto products = [&](int ci) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f32x4 x[3] = {zero4(), zero4(), zero4()}, y[ST][3];
#pragma unroll
        for (int st = 0; st < ST; ++st) y[st][0] = y[st][1] = y[st][2] = zero4();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bf16x8 d = read8<C>(sD, 16 * nt + l16, 32 * s + 8 * q4);
          bf16x8 e[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) e[i] = read8<C>(sE[i], 16 * nt + l16, 32 * s + 8 * q4);
          if (upper_has(w, s))
#pragma unroll
            for (int i = 0; i < 3; ++i) x[i] = mfma(af[s][i], d, x[i]);
#pragma unroll
          for (int st = 0; st < ST; ++st) mfma_three(qtf[st][s], e, y[st]);
        }
        *reinterpret_cast<f32x4*>(&sX[ci & 1][nt][w][ST][4 * lane]) = sum3(x);
#pragma unroll
        for (int st = 0; st < ST; ++st) *reinterpret_cast<f32x4*>(&sX[ci & 1][nt][w][st][4 * lane]) = sum3(y[st]);
      }
    };
    load(chunks - 1);
    put();
    lds_barrier();
    products(chunks - 1);
    if (chunks > 1) load(chunks - 2);
    lds_barrier();
    for (int ci = chunks - 1; ci >= 0; --ci) {
      if (ci > 0) put();
      lds_barrier();
      if (ci > 0) products(ci - 1);
      if (ci > 1) load(ci - 2);
      lds_barrier();
      lds_barrier();
    }
    return;
  }

  const uint16_t* k0 = a.k + (b * a.sh.L * a.sh.hk + kh) * DK + 16 * ST * w;
  uint16_t* dv0 = a.dv_out + (b * a.sh.L * a.sh.heads + h) * dv + n0;
  const int64_t state0 = (bh * DK + state_row<ST>(w, 0, 4 * q4)) * dv + n0 + l16;
  f32x4 S[ST][NT];
#pragma unroll
  for (int st = 0; st < ST; ++st)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[st][nt][r] = a.dh_out ? a.dh_out[state0 + (4 * st + r) * dv + 16 * nt] : 0.0f;

  own_t kf[4];
  bf16x8 tf[2][3], ktf[ST][2];
  f32x4 eg, keep;
  float last;
  int key_row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) key_row[i] = a.sh.place(16 * i + l16) * key_pitch + 8 * ST * q4;
  auto load_k = [&](int ci) {
    const __amdgpu_buffer_rsrc_t k = run_rows(k0, a.sh, key_pitch, 32 * ST, a.sh.run(ci, chunks));
#pragma unroll
    for (int i = 0; i < 4; ++i) row_load(k, key_row[i], &kf[i]);
  };
  auto load_gates = [&](int ci) {
    const __amdgpu_buffer_rsrc_t r = head_record(ci);
    eg = gates4(r, 0);
    keep = gates4(r, 1);
    last = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, 4 * (C - 1), 0, 0));
  };
  load_k(chunks - 1), load_tri(chunks - 1, a.lay.tt, tf), load_gates(chunks - 1), load_keys(chunks - 1, 0, ktf);
  lds_barrier();
  lds_barrier();

  for (int ci = chunks - 1; ci >= 0; --ci) {
    const int next = ci > 0 ? ci - 1 : 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      own_t own[3];
      split_own<ST, NT>(S, nt, own);
      f32x4 P[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) P[i] = zero4();
#pragma unroll
      for (int j = 2; j >= 0; --j)
#pragma unroll
        for (int i = 0; i < 4; ++i) P[i] = mfma_own(kf[i], own[j], P[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4*>(&sP[nt][w][i][4 * lane]) = P[i];
      float* to = a.dstates + ((bh * a.chunks + ci) * DK + state_row<ST>(w, 0, 4 * q4)) * dv + n0 + 16 * nt + l16;
#pragma unroll
      for (int st = 0; st < ST; ++st)
#pragma unroll
        for (int r = 0; r < 4; ++r) to[(4 * st + r) * dv] = S[st][nt][r];
    }
    load_k(next);
    lds_barrier();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const f32x4*>(&sP[nt][i][w][4 * lane]);
      const f32x4 x = *reinterpret_cast<const f32x4*>(&sX[ci & 1][nt][w][ST][4 * lane]);
      u32x2 y[3];
      split4(((p[0] + p[1]) + (p[2] + p[3])) * keep + x, y);
#pragma unroll
      for (int i = 0; i < 3; ++i) write4<C>(sR[i], 16 * nt + l16, 16 * w + 4 * q4, y[i]);
    }
    lds_barrier();
    f32x4 R[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 u[3] = {zero4(), zero4(), zero4()};
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (upper_has(w, s)) {
          bf16x8 y[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) y[i] = read8<C>(sR[i], 16 * nt + l16, 32 * s + 8 * q4);
          mfma_three(tf[s], y, u);
        }
      R[nt] = sum3(u);
      u32x2 p[3];
      split4(-eg * R[nt], p);
#pragma unroll
      for (int i = 0; i < 3; ++i) write4<C>(sU[i], 16 * nt + l16, 16 * w + 4 * q4, p[i]);
    }
    load_tri(next, a.lay.tt, tf);
    const float decay = last;
    load_gates(next);
    lds_barrier();
    const __amdgpu_buffer_rsrc_t out = run_rows(dv0, a.sh, val_pitch, 2 * NS, a.sh.run(ci, chunks));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 add[ST][3];
#pragma unroll
      for (int st = 0; st < ST; ++st) {
        add[st][0] = *reinterpret_cast<const f32x4*>(&sX[ci & 1][nt][w][st][4 * lane]);
        add[st][1] = add[st][2] = zero4();
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x8 y[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) y[i] = read8<C>(sU[i], 16 * nt + l16, 32 * s + 8 * q4);
#pragma unroll
        for (int st = 0; st < ST; ++st) mfma_three(ktf[st][s], y, add[st]);
      }
#pragma unroll
      for (int st = 0; st < ST; ++st) S[st][nt] = S[st][nt] * decay + sum3(add[st]);
      float* to = a.drs + ((bh * a.chunks + ci) * C + 16 * w + 4 * q4) * dv + n0 + 16 * nt + l16;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        to[r * dv] = R[nt][r];
        row_store1(out, val_row[r] + 32 * nt, R[nt][r]);
      }
    }
    load_keys(next, 0, ktf);
  }
  if (a.dh_in) {
#pragma unroll
    for (int st = 0; st < ST; ++st)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) a.dh_in[state0 + (4 * st + r) * dv + 16 * nt] = S[st][nt][r];
  }
}

struct GradArgs {
  const uint16_t* dout;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* dt;
  const uint16_t* b;
  const float* A;
  const float* dt_bias;
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* ddt;
  uint16_t* db;
  const unsigned char* heads;
  const unsigned char* keys;
  const float* states;
  const float* dstates;
  const float* us;
  const float* drs;
  float* part;  // [batch][head][chunk][2]: the chunk's sums for dA and ddt_bias
  Shape sh;
  Layout lay;
  int64_t chunks;
  float scale;
};

// n fp32 values as a buffer, and 8 of them at byte offset + step.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t floats(const float* p, int n) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p), static_cast<short>(0), n * 4, 0x00020000);
}

__device__ __forceinline__ f32x8 load_f32x8(__amdgpu_buffer_rsrc_t r, int offset, int step) {
  const f32x4 a = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, offset, step, 0));
  const f32x4 b = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, offset + 16, step, 0));
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// Sum over the 16 lanes of a row.
__device__ __forceinline__ float sum16(float v) {
  v = add_dpp<0xB1>(v);
  v = add_dpp<0x4E>(v);
  v = add_dpp<0x141>(v);
  return add_dpp<0x140>(v);
}

// Sum over lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float sum_rows(float v) {
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Sum over lanes 0 .. l, by shifts within rows of 16 lanes and broadcasts from row to row.
__device__ __forceinline__ float prefix_sum(float v) {
  v = add_dpp<0x111>(v);  // row_shr:1, 2, 4, 8
  v = add_dpp<0x112>(v);
  v = add_dpp<0x114>(v);
  v = add_dpp<0x118>(v);
  // the last lane of rows 0 and 2 to the rows after them, then lane 31 to rows 2 and 3
  v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x142, 0xa, 0xf, true));
  v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x143, 0xc, 0xf, true));
  return v;
}

// 32 columns of the states, of U and of dR as operands in LDS: rows of 64 bytes, their 16-byte chunks permuted so that 8 lanes
// reading one chunk of 8 rows meet all banks.  Index in values.
__device__ __forceinline__ int slice_at(int row, int chunk) { return row * 32 + ((chunk ^ ((row >> 1) & 3)) << 3); }

template <int DK>
struct Slices {
  uint16_t s[3][DK * 32], ds[3][DK * 32], u[3][C * 32], r[3][C * 32];
};

struct Scores {
  uint16_t d1[3][C * C], d1t[3][C * C], d2[3][C * C], d2t[3][C * C];
};

__device__ __forceinline__ void put_slice(uint16_t* to, int size, int at, f32x8 v) {
  bf16x8 p[3];
  split8(v, p);
#pragma unroll
  for (int i = 0; i < 3; ++i) *reinterpret_cast<bf16x8*>(to + i * size + at) = p[i];
}

__device__ __forceinline__ void get_slice(const uint16_t* from, int size, int at, bf16x8 (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) p[i] = *reinterpret_cast<const bf16x8*>(from + i * size + at);
}

// Eight wavefronts: wavefront w + 4 c takes the chunk's tokens 16 w .. + 15 and, of the tokens or columns that it meets
// them with, the tiles of parity c.  The contractions over the value head's columns go 32 columns at a time: every value of
// the states, U and dR is loaded once, a slice ahead, and split once into the three parts that all wavefronts read from
// LDS.  All of these, and D1 and D2 as operands of the products within the chunk, keep their three parts.  Bound by the
// vector instructions that split values and the waits between slices at one workgroup a compute unit, which is what the
// LDS holds (151 KB with keys of 128, 135 with 64; the registers, some 250 a lane, allow no second one either): 128
// chunks of 32 heads of 128 x 128 in 584 us, of which the 0.8 GB of states, U and dR take 160.
template <int DK, int DV>
__global__ __launch_bounds__(512, 2) void k_delta_grads(GradArgs a) {
  constexpr int KS = DK / 32, ST = DK / 64, VS = DV / 32, KT = DK / 32, kRow = DK + 8, kPitch = C + 1;
  constexpr int kShared = sizeof(Slices<DK>) > sizeof(Scores) ? sizeof(Slices<DK>) : sizeof(Scores);
  __shared__ __align__(16) unsigned char shared[kShared];  // the slices, then the scores
  __shared__ __align__(16) uint16_t sQ[C * kRow], sK[C * kRow];
  __shared__ float sP[C * kPitch];
  __shared__ __align__(16) float sHi[C], sLo[C], sEg[C], sKeep[C];
  __shared__ float sS0[2][C], sS1[2][C], sDb[C], sAcc[8][C], sDot[8];
  Slices<DK>& sl = *reinterpret_cast<Slices<DK>*>(shared);
  Scores& sc = *reinterpret_cast<Scores*>(shared);
  const int lane = threadIdx.x & 63, l16 = lane & 15, q4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3, c = wave >> 2;
  const int64_t ci = blockIdx.x, kh = blockIdx.y, b = blockIdx.z, L = a.sh.L, share = a.sh.heads / a.sh.hk;
  const int run = a.sh.run(static_cast<int>(ci), static_cast<int>(a.chunks));
  const int64_t t0 = static_cast<int64_t>(run) * C;
  const unsigned char* key = a.keys + ((b * a.sh.hk + kh) * a.chunks + ci) * a.lay.key_bytes;

  const int64_t my_t = t0 + a.sh.place(16 * w + l16), my_row = b * L + (my_t < L ? my_t : L - 1);
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    bf16x8 v = *reinterpret_cast<const bf16x8*>((c ? a.q : a.k) + (my_row * a.sh.hk + kh) * DK + 32 * s + 8 * q4);
    if (my_t >= L) v = zero8();
    *reinterpret_cast<bf16x8*>((c ? sQ : sK) + (16 * w + l16) * kRow + 32 * s + 8 * q4) = v;
  }
  f32x4 dq[KT], dk[KT];
#pragma unroll
  for (int i = 0; i < KT; ++i) dq[i] = dk[i] = zero4();

  for (int64_t g = 0; g < share; ++g) {
    const int64_t h = kh * share + g, bh = b * a.sh.heads + h, hc = bh * a.chunks + ci;
    const float* gates = reinterpret_cast<const float*>(a.heads + hc * a.lay.bytes);
    lds_barrier();  // the previous head's readers of what is written here
    if (wave == 0) sEg[lane] = gates[lane], sKeep[lane] = gates[C + lane];
    // what the last step takes: this lane's token
    const bool real = t0 + a.sh.place(lane) < L;
    const int64_t t_own = (b * L + (real ? t0 + a.sh.place(lane) : L - 1)) * a.sh.heads + h;
    uint16_t own_dt = 0, own_b = 0;
    float own_beta = 0.0f;
    if (wave == 0) own_dt = a.dt[t_own], own_b = a.b[t_own], own_beta = gates[4 * C + lane];
    if (wave == 1) sHi[lane] = gates[2 * C + lane], sLo[lane] = gates[3 * C + lane];
    f32x4 d1[2], d2[2], t1[KT], t2[KT], t3[KT];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < KT; ++i) t1[i] = t2[i] = t3[i] = zero4();
    d1[0] = d1[1] = d2[0] = d2[1] = zero4();
    const int val_pitch = static_cast<int>(a.sh.heads) * DV * 2;
    const __amdgpu_buffer_rsrc_t go = run_rows(a.dout + (b * L * a.sh.heads + h) * DV, a.sh, val_pitch, DV * 2, run);
    const __amdgpu_buffer_rsrc_t gs = floats(a.states + hc * DK * DV, DK * DV), gd = floats(a.dstates + hc * DK * DV, DK * DV);
    // half of the workgroup brings U, the other dR
    const __amdgpu_buffer_rsrc_t gur = floats((c ? a.drs : a.us) + hc * C * DV, C * DV);
    const int orow = a.sh.place(16 * w + l16) * val_pitch + 16 * q4;
    const int row = threadIdx.x >> 2, chunk = threadIdx.x & 3;  // of the states (DK 64: the first 256 threads')
    const bool states = DK == 128 || c == 0;
    const int at_state = (row * DV + 8 * chunk) * 4, at_ur = ((row & 63) * DV + 8 * chunk) * 4;
    f32x8 st, ds, ur;
    bf16x8 od[1], on;
    auto fetch = [&](int s) {
      if (states) st = load_f32x8(gs, at_state, 128 * s), ds = load_f32x8(gd, at_state, 128 * s);
      ur = load_f32x8(gur, at_ur, 128 * s);
      on = row_load8(go, orow + 64 * s);
    };
    fetch(0);
#pragma unroll 1
    for (int s = 0; s < VS; ++s) {
      if (states) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = fmaf(st[e], ds[e], dot);
        put_slice(sl.s[0], DK * 32, slice_at(row, chunk), st);
        put_slice(sl.ds[0], DK * 32, slice_at(row, chunk), ds);
      }
      put_slice(c ? sl.r[0] : sl.u[0], C * 32, slice_at(row & 63, chunk), ur);
      od[0] = on;
      fetch(s + 1 < VS ? s + 1 : s);
      lds_barrier();
      bf16x8 rd[3], ud[3];
      get_slice(sl.r[0], C * 32, slice_at(16 * w + l16, q4), rd);
      get_slice(sl.u[0], C * 32, slice_at(16 * w + l16, q4), ud);
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        const int at_row = slice_at(state_row<ST>((2 * i + c) / ST, (2 * i + c) % ST, l16), q4);
        bf16x8 y[3];
        get_slice(sl.s[0], DK * 32, at_row, y);
        t1[i] = mfma_parts(od, y, t1[i]);
        t2[i] = mfma_parts(rd, y, t2[i]);
        get_slice(sl.ds[0], DK * 32, at_row, y);
        t3[i] = mfma_parts(ud, y, t3[i]);
      }
#pragma unroll
      for (int jj = 0; jj < 2; ++jj)
        if (2 * jj + c <= w) {
          bf16x8 y[3];
          get_slice(sl.u[0], C * 32, slice_at(16 * (2 * jj + c) + l16, q4), y);
          d1[jj] = mfma_parts(od, y, d1[jj]);
          d2[jj] = mfma_parts(rd, y, d2[jj]);
        }
      lds_barrier();
    }
    const f32x4 eg = *reinterpret_cast<const f32x4*>(sEg + 16 * w + 4 * q4);
    const f32x4 keep = *reinterpret_cast<const f32x4*>(sKeep + 16 * w + 4 * q4);

#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      const int j = 2 * jj + c;
      f32x4 pr = zero4();
      if (j <= w) {
        f32x4 qk = zero4(), kk = zero4();
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const bf16x8 o = *reinterpret_cast<const bf16x8*>(sK + (16 * j + l16) * kRow + 32 * s + 8 * q4);
          const bf16x8 kw = *reinterpret_cast<const bf16x8*>(sK + (16 * w + l16) * kRow + 32 * s + 8 * q4);
          const bf16x8 qw = *reinterpret_cast<const bf16x8*>(sQ + (16 * w + l16) * kRow + 32 * s + 8 * q4);
          qk = mfma(qw, o, qk);
          kk = mfma(kw, o, kk);
        }
        const int col = 16 * j + l16;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * w + 4 * q4 + r;
          const float d = col <= row ? ex((sHi[row] - sHi[col]) + (sLo[row] - sLo[col])) : 0.0f;
          d1[jj][r] = col <= row ? d1[jj][r] * d * a.scale : 0.0f;
          if (col == row) sDb[row] = d2[jj][r];  // dR_i.U_i
          d2[jj][r] = col < row ? -d2[jj][r] * d : 0.0f;
          pr[r] = col < row ? fmaf(d1[jj][r], qk[r], d2[jj][r] * kk[r]) : 0.0f;
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) sP[(16 * w + 4 * q4 + r) * kPitch + 16 * j + l16] = pr[r];
      u32x2 p1[3], p2[3];
      split4(d1[jj], p1);
      split4(d2[jj], p2);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        write4<C>(sc.d1t[i], 16 * j + l16, 16 * w + 4 * q4, p1[i]);
        write4<C>(sc.d2t[i], 16 * j + l16, 16 * w + 4 * q4, p2[i]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          sc.d1[i][at<C>(16 * w + 4 * q4 + r, 16 * j + l16)] = static_cast<uint16_t>(p1[i][r >> 1] >> (16 * (r & 1)));
          sc.d2[i][at<C>(16 * w + 4 * q4 + r, 16 * j + l16)] = static_cast<uint16_t>(p2[i][r >> 1] >> (16 * (r & 1)));
        }
      }
    }
    f32x4 s0 = zero4(), s1 = zero4();
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      const int tile = 2 * i + c;
      t1[i] *= eg * a.scale;
      t2[i] *= -eg;
      t3[i] *= keep;
      dq[i] += t1[i];
      dk[i] += t2[i] + t3[i];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int e = (16 * w + 4 * q4 + r) * kRow + state_row<ST>(tile / ST, tile % ST, l16);
        const float kv = bf(sK[e]);
        s0[r] = fmaf(bf(sQ[e]), t1[i][r], fmaf(kv, t2[i][r], s0[r]));
        s1[r] = fmaf(kv, t3[i][r], s1[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float v0 = sum16(s0[r]), v1 = sum16(s1[r]);
      if (l16 == 0) sS0[c][16 * w + 4 * q4 + r] = v0, sS1[c][16 * w + 4 * q4 + r] = v1;
    }
    dot = sum_rows(sum16(dot));
    if (lane == 0) sDot[wave] = dot;
    lds_barrier();

    // products within the chunk
    constexpr int kB = static_cast<int>(kFragBytes);
    const __amdgpu_buffer_rsrc_t keys = record(key, a.lay.key_bytes);
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      bf16x8 d1[3], d2[3], d1t[3], d2t[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        d1[i] = read8<C>(sc.d1[i], 16 * w + l16, 32 * s + 8 * q4);
        d2[i] = read8<C>(sc.d2[i], 16 * w + l16, 32 * s + 8 * q4);
        d1t[i] = read8<C>(sc.d1t[i], 16 * w + l16, 32 * s + 8 * q4);
        d2t[i] = read8<C>(sc.d2t[i], 16 * w + l16, 32 * s + 8 * q4);
      }
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        const bf16x8 kt[1] = {record_frag(keys, 2 * c * kB, 4 * i + s, 16 * lane)};
        if (lower_has(w, s)) {
          dq[i] = mfma_parts(d1, kt, dq[i]);
          dk[i] = mfma_parts(d2, kt, dk[i]);
        }
        if (upper_has(w, s)) {
          const bf16x8 qt[1] = {record_frag(keys, (DK / 8 + 2 * c) * kB, 4 * i + s, 16 * lane)};
          dk[i] = mfma_parts(d1t, qt, dk[i]);
          dk[i] = mfma_parts(d2t, kt, dk[i]);
        }
      }
    }
    // sum of P_ij over j < t <= i: prefix sums along 8 rows of each wavefront, added for the rows from t on
    {
      float acc = 0.0f;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int i = 8 * wave + r;
        const float before = prefix_sum(lane > 0 ? sP[i * kPitch + lane - 1] : 0.0f);
        acc += i >= lane ? before : 0.0f;
      }
      sAcc[wave][lane] = acc;
    }
    lds_barrier();
    if (wave == 0) {
      // sums of s over i >= t (as prefix sums of the reversed row) and of e over j < t
      const float from = prefix_sum(sS0[0][C - 1 - lane] + sS0[1][C - 1 - lane]);
      const float before = prefix_sum(lane > 0 ? sS1[0][lane - 1] + sS1[1][lane - 1] : 0.0f);
      float dg = __shfl(from, C - 1 - lane) + before, all = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) dg += sAcc[i][lane], all += sDot[i];
      dg = fmaf(sEg[C - 1], all, dg);
      float pa = 0.0f, pb = 0.0f;
      if (real) {
        const float x = bf(own_dt) + (a.dt_bias ? a.dt_bias[h] : 0.0f);
        const float ddt = dg * a.A[h] * sigmoid_f32(x);
        // (0 where nothing crosses the token: its step may be infinite there)
        pa = dg == 0.0f ? 0.0f : dg * softplus_f32(x);
        pb = ddt;
        bf16_t o;
        from_f32(ddt, &o);
        a.ddt[t_own] = o.bits;
        // (0 below 2^-60, where the product of two factors of beta leaves the range)
        from_f32(own_beta > 0x1p-60f ? sDb[lane] / own_beta * sigmoid_f32(-bf(own_b)) : 0.0f, &o);
        a.db[t_own] = o.bits;
      }
      pa = sum_rows(sum16(pa));
      pb = sum_rows(sum16(pb));
      if (lane == 0) a.part[2 * hc] = pa, a.part[2 * hc + 1] = pb;
    }
  }
#pragma unroll
  for (int i = 0; i < KT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t t = t0 + a.sh.place(16 * w + 4 * q4 + r);
      if (t < L) {
        const int tile = 2 * i + c;
        const int64_t to = ((b * L + t) * a.sh.hk + kh) * DK + state_row<ST>(tile / ST, tile % ST, l16);
        bf16_t o;
        from_f32(dq[i][r], &o);
        a.dq[to] = o.bits;
        from_f32(dk[i][r], &o);
        a.dk[to] = o.bits;
      }
    }
}

// dA and ddt_bias of one head: its chunks' sums over all batch elements, in a fixed order.
__global__ __launch_bounds__(256) void k_delta_reduce(const float* part, float* dA, float* ddt_bias, int64_t batch,
                                                      int64_t heads, int64_t chunks) {
  __shared__ float s[2][4];
  const int64_t h = blockIdx.x;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  float x = 0.0f, y = 0.0f;
  for (int64_t b = 0; b < batch; ++b) {
    const float* p = part + (b * heads + h) * chunks * 2;
    for (int64_t c = threadIdx.x; c < chunks; c += 256) x += p[2 * c], y += p[2 * c + 1];
  }
  x = sum_rows(sum16(x));
  y = sum_rows(sum16(y));
  if (lane == 0) s[0][w] = x, s[1][w] = y;
  lds_barrier();
  if (threadIdx.x != 0) return;
  dA[h] = (s[0][0] + s[0][1]) + (s[0][2] + s[0][3]);
  if (ddt_bias) ddt_bias[h] = (s[1][0] + s[1][1]) + (s[1][2] + s[1][3]);
}

template <int DK>
void launch_rwalk(const RWalkArgs& a, int tiles, hipStream_t stream) {
  const int64_t rows = (a.batch * a.sh.heads + 7) / 8 * 8;
  const dim3 grid(static_cast<unsigned>(rows * (a.dv / (16 * tiles))));
  if (tiles == 1) hipLaunchKernelGGL((k_delta_rwalk<DK, 1>), grid, dim3(512), 0, stream, a);
  else hipLaunchKernelGGL((k_delta_rwalk<DK, 2>), grid, dim3(512), 0, stream, a);
}

template <int DK>
void launch_grads(const GradArgs& a, int64_t dv, dim3 grid, hipStream_t stream) {
  if (dv == 64) hipLaunchKernelGGL((k_delta_grads<DK, 64>), grid, dim3(512), 0, stream, a);
  else hipLaunchKernelGGL((k_delta_grads<DK, 128>), grid, dim3(512), 0, stream, a);
}

}  // namespace

hipError_t launch_delta_bwd(const DeltaArgs& in, const DeltaGrads& g, const Plan& p, void* ws, hipStream_t stream) {
  unsigned char* base = static_cast<unsigned char*>(ws);
  const Layout lay = make_layout(in.dk, true);
  const Shape sh{in.seqlen, in.hk, in.heads, in.rev};
  float* states = reinterpret_cast<float*>(base + p.s_off);
  float* dstates = reinterpret_cast<float*>(base + p.ds_off);
  float* us = reinterpret_cast<float*>(base + p.u_off);
  float* drs = reinterpret_cast<float*>(base + p.dr_off);
  float* part = reinterpret_cast<float*>(base + p.part_off);
  hipError_t e = launch_delta_prep(in, p, 0, p.nchunk, true, ws, stream);
  if (e != hipSuccess) return e;
  e = launch_delta_walk(in, p, 0, p.nchunk, true, in.h_in, nullptr, ws, stream);
  if (e != hipSuccess) return e;
  const uint16_t* dout = static_cast<const uint16_t*>(g.dout);
  const uint16_t* k = static_cast<const uint16_t*>(in.k);
  const RWalkArgs r{dout, k, static_cast<uint16_t*>(g.dv), base + p.head_off, base + p.key_off, g.dh_out, g.dh_in,
                    dstates, drs, sh, lay, in.batch, in.dv, p.nchunk, in.scale};
  if (in.dk == 64) launch_rwalk<64>(r, p.tiles, stream);
  else launch_rwalk<128>(r, p.tiles, stream);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const GradArgs a{dout, static_cast<const uint16_t*>(in.q), k, static_cast<const uint16_t*>(in.dt),
                   static_cast<const uint16_t*>(in.b), in.A, in.dt_bias, static_cast<uint16_t*>(g.dq),
                   static_cast<uint16_t*>(g.dk), static_cast<uint16_t*>(g.ddt), static_cast<uint16_t*>(g.db),
                   base + p.head_off, base + p.key_off, states, dstates, us, drs, part, sh, lay, p.nchunk, in.scale};
  const dim3 grid(static_cast<unsigned>(p.nchunk), static_cast<unsigned>(in.hk), static_cast<unsigned>(in.batch));
  if (in.dk == 64) launch_grads<64>(a, in.dv, grid, stream);
  else launch_grads<128>(a, in.dv, grid, stream);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_delta_reduce, dim3(static_cast<unsigned>(in.heads)), dim3(256), 0, stream, part, g.dA,
                     g.ddt_bias, in.batch, in.heads, p.nchunk);
  return hipGetLastError();
}

}  // namespace delta
}  // namespace bimamba
