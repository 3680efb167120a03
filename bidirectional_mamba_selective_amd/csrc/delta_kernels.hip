// The gated delta rule for gfx950: a recurrent mixer whose state is a dk x dv matrix per head,
//   delta = softplus(dt + dt_bias), a = exp(delta A), beta = sigmoid(b)
//   S_t = a_t S_{t-1} + beta_t k_t (v_t - (a_t S_{t-1})^T k_t)^T,     o_t = scale S_t^T q_t
// over chunks of 64 tokens.  With g the logarithms of the decays summed from the chunk's start, S the state that enters,
// N_ij = beta_i e^(g_i - g_j) k_i.k_j (j < i) and A_ij = scale e^(g_i - g_j) q_i.k_j (j <= i), the corrections u_t that
// the tokens add to the state solve a unit lower triangular system:
//   U = T (V - diag(e^g) K S),  T = (I + N)^-1 diag(beta)
//   O = scale diag(e^g) Q S + A U,     S' = e^(g_C) S + K^T diag(e^(g_C - g)) U
// Every decay is exp of a difference g_i - g_j <= 0, never a quotient, so strong decays neither overflow nor divide by
// zero.
//
// k_delta_prep forms T, A, the decays and K^T of all chunks at once; k_delta_walk then goes over the chunks with the state
// in fp32 registers, a workgroup per head and 16 or 32 columns of it (the columns of S, U, V and O are independent).
// Products run on the matrix cores with bf16 operands and fp32 sums.  q, k and v are bf16 already; S, U, T and A are taken
// as three bf16 parts (24 bits): a state keeps fp32 accuracy over any number of chunks, and out's terms have it when
// their sum is rounded.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "delta_device.h"
#include "launch.h"

namespace bimamba {
namespace delta {
namespace {

constexpr int kPitch = C + 1;  // fp32 rows in LDS

struct PrepArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* dt;
  const uint16_t* b;
  const float* A;
  const float* dt_bias;
  unsigned char* heads;  // records of Layout::bytes, [batch][head][seg]
  unsigned char* keys;   // K^T (and Q^T), [batch][key head][seg]
  Shape sh;
  Layout lay;
  int64_t chunk0, seg;  // the segment's first chunk in the direction's order, records per head
  int chunks;           // of the whole sequence
  float scale;
};

__device__ __forceinline__ void put_tile(float* s, int row0, int col0, int l16, int q4, f32x4 v) {
#pragma unroll
  for (int r = 0; r < 4; ++r) s[(row0 + 4 * q4 + r) * kPitch + col0 + l16] = v[r];
}

// sum over K of X[row0 + ., k0 + .] Y[k1 + ., col0 + .], 16 x 16 results, KT x 16 terms, from fp32 rows in LDS.
template <int KT>
__device__ __forceinline__ f32x4 tile_product(const float* x, int row0, int k0, const float* y, int k1, int col0,
                                              int l16, int q4) {
  f32x4 acc = zero4();
#pragma unroll
  for (int s = 0; s < 4 * KT; ++s)
    acc = mfma_f32(x[(row0 + l16) * kPitch + k0 + 4 * s + q4], y[(k1 + 4 * s + q4) * kPitch + col0 + l16], acc);
  return acc;
}

// One workgroup per (chunk, head, batch element); all chunks are independent.  N and A are two products of the chunk's
// rows; (I + N)^-1 is built from its four 16 x 16 diagonal blocks, inverted by substitution, and products of blocks, in
// fp32 matrix instructions.  Bound by the latency of that chain of small products and the LDS between them: 57 chunks of
// 32 heads of 128 x 128 take 40 us, 99 MB written to the last-level cache, a quarter of the call.  The record's gates:
// e^g, e^(g_C - g), g as two floats whose sum carries it to 2^-48 (differences of g stay exact to fp32 however far the
// chunk has decayed), beta; 64 of each.
template <int DK, bool GRAD>
__global__ __launch_bounds__(256) void k_delta_prep(PrepArgs a) {
  constexpr int KS = DK / 32, ST = DK / 64;
  constexpr int kRow = DK + 8;
  // K's rows (then Q's, for their transposes), then N; A, then T: 34 KB, so that a compute unit holds four workgroups
  // (68 KB, with arrays of their own, took a fifth longer)
  constexpr int kRows = C * kRow * 2 > C * kPitch * 4 ? C * kRow * 2 : C * kPitch * 4;
  __shared__ __align__(16) unsigned char sKN[kRows];
  __shared__ float sT[C * kPitch];
  __shared__ float sHi[C], sLo[C], sBeta[C];
  uint16_t* sK = reinterpret_cast<uint16_t*>(sKN);
  float* sN = reinterpret_cast<float*>(sKN);
  float* sA = sT;
  const int lane = threadIdx.x & 63, l16 = lane & 15, q4 = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t ci = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int64_t share = a.sh.heads / a.sh.hk, kh = h / share, L = a.sh.L;
  const int64_t t0 = static_cast<int64_t>(a.sh.run(static_cast<int>(a.chunk0 + ci), a.chunks)) * C;
  unsigned char* rec = a.heads + ((b * a.sh.heads + h) * a.seg + ci) * a.lay.bytes;
  float* gates = reinterpret_cast<float*>(rec);

  if (w == 0) {
    const int64_t t = t0 + a.sh.place(lane);
    float g = 0.0f, beta = 0.0f;
    if (t < L) {
      const int64_t i = (b * L + t) * a.sh.heads + h;
      g = softplus_f32(bf(a.dt[i]) + (a.dt_bias ? a.dt_bias[h] : 0.0f)) * a.A[h];
      // e^-256 is 0 in fp32 as any stronger decay is; sums of the logarithms stay finite
      if (g < -256.0f) g = -256.0f;
      beta = sigmoid_f32(bf(a.b[i]));
    }
    double sum = g;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const double end = __shfl(sum, 63);
    const float hi = static_cast<float>(sum);
    const float lo = static_cast<float>(sum - static_cast<double>(hi));
    sHi[lane] = hi, sLo[lane] = lo, sBeta[lane] = beta;
    gates[lane] = ex(hi);
    gates[C + lane] = ex(static_cast<float>(end - sum));
    gates[2 * C + lane] = hi;
    gates[3 * C + lane] = lo;
    gates[4 * C + lane] = beta;
  }
  bf16x8 kf[KS], qf[KS];
  {
    const int64_t t = t0 + a.sh.place(16 * w + l16);
    const int64_t row = ((b * L + (t < L ? t : L - 1)) * a.sh.hk + kh) * DK;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      kf[s] = *reinterpret_cast<const bf16x8*>(a.k + row + 32 * s + 8 * q4);
      qf[s] = *reinterpret_cast<const bf16x8*>(a.q + row + 32 * s + 8 * q4);
      if (t >= L) kf[s] = qf[s] = zero8();
      *reinterpret_cast<bf16x8*>(sK + (16 * w + l16) * kRow + 32 * s + 8 * q4) = kf[s];
    }
  }
  lds_barrier();

  // scores of this wavefront's 16 rows against the tokens up to them
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kk[j] = qk[j] = zero4();
    if (j <= w) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const bf16x8 o = *reinterpret_cast<const bf16x8*>(sK + (16 * j + l16) * kRow + 32 * s + 8 * q4);
        kk[j] = mfma(kf[s], o, kk[j]);
        qk[j] = mfma(qf[s], o, qk[j]);
      }
      const int col = 16 * j + l16;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * q4 + r;
        const float d = col <= row ? ex((sHi[row] - sHi[col]) + (sLo[row] - sLo[col])) : 0.0f;
        kk[j][r] = col < row ? kk[j][r] * d * sBeta[row] : 0.0f;
        qk[j][r] = col <= row ? qk[j][r] * d * a.scale : 0.0f;
      }
    }
  }
  // K^T and Q^T once for the heads that share them
  if (h % share == 0) {
    unsigned char* key = a.keys + ((b * a.sh.hk + kh) * a.seg + ci) * a.lay.key_bytes;
#pragma unroll
    for (int which = 0; which < (GRAD ? 2 : 1); ++which) {
      if (which == 1) {
        lds_barrier();
#pragma unroll
        for (int s = 0; s < KS; ++s)
          *reinterpret_cast<bf16x8*>(sK + (16 * w + l16) * kRow + 32 * s + 8 * q4) = qf[s];
        lds_barrier();
      }
      for (int f = w; f < DK / 8; f += 4) {  // tile f / 2 of the state's rows, tokens 32 (f % 2)
        const int col = state_row<ST>(f / (2 * ST), f / 2 % ST, l16);
        union {
          uint16_t u[8];
          bf16x8 v;
        } x;
#pragma unroll
        for (int e = 0; e < 8; ++e) x.u[e] = sK[(32 * (f & 1) + 8 * q4 + e) * kRow + col];
        store_frag(key, which * (DK / 8) + f, lane, x.v);
      }
    }
  }
  lds_barrier();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j <= w) {
      put_tile(sN, 16 * w, 16 * j, l16, q4, kk[j]);
      put_tile(sA, 16 * w, 16 * j, l16, q4, qk[j]);
    }
  lds_barrier();
  // A's operands, before T takes its place
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int row = 16 * w + l16;
    f32x8 m;
    if constexpr (GRAD) {
      if (upper_has(w, s)) {  // of its transpose
        bf16x8 p[3];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int col = 32 * s + 8 * q4 + e;
          m[e] = col >= row ? sA[col * kPitch + row] : 0.0f;
        }
        split8(m, p);
#pragma unroll
        for (int i = 0; i < 3; ++i) store_frag(rec + a.lay.at, upper_at(w, s) * 3 + i, lane, p[i]);
      }
    } else {
      if (lower_has(w, s)) {
        bf16x8 p[3];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int col = 32 * s + 8 * q4 + e;
          m[e] = col <= row ? sA[row * kPitch + col] : 0.0f;
        }
        split8(m, p);
#pragma unroll
        for (int i = 0; i < 3; ++i) store_frag(rec + a.lay.a, lower_at(w, s) * 3 + i, lane, p[i]);
      }
    }
  }
  lds_barrier();

  // (I + N)^-1: the four 16 x 16 blocks on the diagonal by substitution, a column per lane, then blocks joined two by
  // two, [[x, 0], [n, y]]^-1 = [[x', 0], [-y' n x', y']], as stable as the substitution.  What is above the diagonal of
  // sT is scratch.
  if (w == 0) {
    const int o = 16 * q4;
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == l16 ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) v = fmaf(-sN[(o + i) * kPitch + o + j], t[j], v);
      t[i] = v;
      sT[(o + i) * kPitch + o + l16] = v;
    }
  }
  lds_barrier();
  if (w < 2) put_tile(sT, 32 * w, 32 * w + 16, l16, q4, tile_product<1>(sN, 32 * w + 16, 32 * w, sT, 32 * w, 32 * w, l16, q4));
  lds_barrier();
  if (w < 2)
    put_tile(sT, 32 * w + 16, 32 * w, l16, q4,
             -tile_product<1>(sT, 32 * w + 16, 32 * w + 16, sT, 32 * w, 32 * w + 16, l16, q4));
  lds_barrier();
  // the upper right block of each half is scratch until now and zero from here on, for the products over 32 terms
  if (w < 2) put_tile(sT, 32 * w, 32 * w + 16, l16, q4, zero4());
  lds_barrier();
  {
    const int wr = 16 * (w >> 1), wc = 16 * (w & 1);
    const f32x4 x = tile_product<2>(sN, 32 + wr, 0, sT, 0, wc, l16, q4);
    put_tile(sT, wr, 32 + wc, l16, q4, x);
    lds_barrier();
    const f32x4 y = tile_product<2>(sT, 32 + wr, 32, sT, 0, 32 + wc, l16, q4);
    put_tile(sT, 32 + wr, wc, l16, q4, -y);
  }
  lds_barrier();

  // T's operands
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int row = 16 * w + l16;
    f32x8 t;
    bf16x8 p[3];
    if (lower_has(w, s)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int col = 32 * s + 8 * q4 + e;
        t[e] = col <= row ? sT[row * kPitch + col] * sBeta[col] : 0.0f;
      }
      split8(t, p);
#pragma unroll
      for (int i = 0; i < 3; ++i) store_frag(rec + a.lay.t, lower_at(w, s) * 3 + i, lane, p[i]);
    }
    if (GRAD && upper_has(w, s)) {  // of its transpose
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int col = 32 * s + 8 * q4 + e;
        t[e] = col >= row ? sT[col * kPitch + row] * sBeta[row] : 0.0f;
      }
      split8(t, p);
#pragma unroll
      for (int i = 0; i < 3; ++i) store_frag(rec + a.lay.tt, upper_at(w, s) * 3 + i, lane, p[i]);
    }
  }
}

struct WalkArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  const unsigned char* heads;
  const unsigned char* keys;
  const float* state_in;  // null: zeros
  float* state_out;       // null: not kept
  float* states;          // backward: the state entering each chunk, [batch][head][chunk][dk][dv]
  float* us;              // backward: U, [batch][head][chunk][64][dv]
  Shape sh;
  Layout lay;
  int64_t batch, dv, seg;
  int first, chunks, all;  // the segment's first chunk, its chunks, those of the whole sequence
  float scale;
};

// Workgroups of one head on one XCD, so that what they share is fetched into its L2 once: consecutive workgroups go to
// the eight XCDs in turn, so head 8 i + x takes the places x, x + 8, ... of the i-th run of 8 x slices workgroups.
__device__ __forceinline__ bool place(int64_t slices, int64_t rows, int64_t* row, int64_t* slice) {
  const int64_t x = blockIdx.x & 7, i = blockIdx.x >> 3;
  *row = i / slices * 8 + x;
  *slice = i % slices;
  return *row < rows;
}

// One workgroup: 16 NT columns of one head's state over `chunks` chunks.  Four wavefronts carry the state, a quarter of its
// rows each; three products follow from one another with one barrier before each:
//   K S: every wavefront takes its own rows of S, which its registers hold in operand order, for all 64 tokens; the four
//        partial sums meet in LDS, where wavefront w takes the sum for its tokens 16 w .. + 15
//   T R: through LDS, rows 16 w .. + 15 of U
//   K^T U: through LDS, the wavefront's rows of S
// What bounds it is the latency of one chunk's chain, which no other chunk can shorten: three LDS round trips of 140 to 185
// cycles, three barriers, the products between them and the three-part splits; 2.0 us a chunk at 32 heads of 128 x 128
// (57 chunks in 115 us; 65536 tokens, with k_delta_prep, in 2.67 ms, where the inputs' bytes take 0.43).  16 columns
// a workgroup put one on every compute unit at 32 heads.  The whole chain in the registers of one wavefront, without
// barriers, took 166 us where this took 130: its vector instructions, no longer spread over four SIMDs, then set the
// pace.
// Four more take the products that only the output needs (Q S, A U) between the same barriers, where the main ones leave
// the matrix cores free: one part of S behind the first barrier, two behind the second (all three behind the first: 2.96
// ms), the query rows asked for a chunk ahead (2.78 ms otherwise).  Without an output (SAVE) there are none.  The next
// chunk's other operands are loaded into the registers of the current chunk's as soon as these have been used.
template <int DK, int NT, bool SAVE>
__global__ __launch_bounds__(SAVE ? 256 : 512, SAVE ? 1 : 2) void k_delta_walk(WalkArgs a) {
  constexpr int KS = DK / 32, ST = DK / 64, NS = 16 * NT, kB = static_cast<int>(kFragBytes);
  typedef typename Own<ST>::type own_t;
  __shared__ __align__(16) float sP[NT][4][4][256];
  __shared__ __align__(16) uint16_t sS[3][NS * DK], sR[3][NS * C], sU[3][NS * C], sV[3][NS * C];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q4 = lane >> 4, lane16 = lane * 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3;
  int64_t bh, slice;
  if (!place(a.dv / NS, a.batch * a.sh.heads, &bh, &slice)) return;
  const int64_t b = bh / a.sh.heads, h = bh % a.sh.heads, kh = h / (a.sh.heads / a.sh.hk);
  const int n0 = static_cast<int>(slice) * NS, dv = static_cast<int>(a.dv);
  const int chunks = a.chunks;
  const unsigned char* rec = a.heads + bh * a.seg * a.lay.bytes;
  const int rec_bytes = static_cast<int>(a.lay.bytes);
  const int key_pitch = static_cast<int>(a.sh.hk) * DK * 2, val_pitch = static_cast<int>(a.sh.heads) * dv * 2;
  int val_row[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) val_row[r] = a.sh.place(16 * w + 4 * q4 + r) * val_pitch + 2 * l16;
  auto gates4 = [&](__amdgpu_buffer_rsrc_t r, int row) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, 16 * q4, 4 * C * row + 64 * w, 0));
  };

  if (!SAVE && wave >= 4) {
    const uint16_t* q0 = a.q + (b * a.sh.L * a.sh.hk + kh) * DK;
    uint16_t* out0 = a.out + (b * a.sh.L * a.sh.heads + h) * dv + n0;
    const int key_row = a.sh.place(16 * w + l16) * key_pitch + 16 * q4;
    bf16x8 qf[KS], qn[KS], af[2][3];
    f32x4 eg;
    auto load_q = [&](int ci) {
      const __amdgpu_buffer_rsrc_t q = run_rows(q0, a.sh, key_pitch, DK * 2, a.sh.run(a.first + ci, a.all));
#pragma unroll
      for (int s = 0; s < KS; ++s) qn[s] = row_load8(q, key_row + 64 * s);
    };
    auto load_eg = [&]() { eg = gates4(record(rec, a.lay.bytes), 0); };
    auto load_a = [&]() {
      const __amdgpu_buffer_rsrc_t r = record(rec, a.lay.bytes);
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (lower_has(w, s))
#pragma unroll
          for (int i = 0; i < 3; ++i)
            af[s][i] = record_frag(r, static_cast<int>(a.lay.a) + lower_at(w, s) * 3 * kB, i, lane16);
    };
    load_q(0), load_eg(), load_a();
    for (int ci = 0; ci < chunks; ++ci) {
      const int next = ci + 1 < chunks ? ci + 1 : ci;
#pragma unroll
      for (int s = 0; s < KS; ++s) qf[s] = qn[s];
      load_q(next);
      lds_barrier();
      // sS holds until the chunk's last barrier
      f32x4 o[NT][3];
      auto read_state = [&](int i) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[nt][i] = zero4();
#pragma unroll
          for (int s = 0; s < KS; ++s)
            o[nt][i] = mfma(qf[s], read8<DK>(sS[i], 16 * nt + l16, 32 * s + 8 * q4), o[nt][i]);
        }
      };
      read_state(0);
      lds_barrier();
      read_state(1), read_state(2);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[nt][0] = sum3(o[nt]) * (eg * a.scale);
      if (next > ci) rec += rec_bytes;
      load_eg();
      lds_barrier();
      const __amdgpu_buffer_rsrc_t out = run_rows(out0, a.sh, val_pitch, 2 * NS, a.sh.run(a.first + ci, a.all));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        o[nt][1] = o[nt][2] = zero4();
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (lower_has(w, s)) {
            bf16x8 y[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) y[i] = read8<C>(sV[i], 16 * nt + l16, 32 * s + 8 * q4);
            mfma_three(af[s], y, o[nt]);
          }
        o[nt][0] = sum3(o[nt]);
      }
      load_a();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) row_store1(out, val_row[r] + 32 * nt, o[nt][0][r]);
    }
    return;
  }

  const uint16_t* k0 = a.k + (b * a.sh.L * a.sh.hk + kh) * DK + 16 * ST * w;
  const uint16_t* v0 = a.v + (b * a.sh.L * a.sh.heads + h) * dv + n0;
  const unsigned char* key = a.keys + (b * a.sh.hk + kh) * a.seg * a.lay.key_bytes;
  const int key_bytes = static_cast<int>(a.lay.key_bytes);
  // this lane's rows of the state: state_row(w, st, 4 q4 + r) = the first one + 4 st + r
  const int64_t state0 = (bh * DK + state_row<ST>(w, 0, 4 * q4)) * dv + n0 + l16;
  f32x4 S[ST][NT];
#pragma unroll
  for (int st = 0; st < ST; ++st)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[st][nt][r] = a.state_in ? a.state_in[state0 + (4 * st + r) * dv + 16 * nt] : 0.0f;

  own_t kf[4];
  bf16x8 tf[2][3], ktf[ST][2];
  uint16_t vv[NT][4];
  f32x4 eg, keep;
  float last;
  int key_row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) key_row[i] = a.sh.place(16 * i + l16) * key_pitch + 8 * ST * q4;
  auto load_rows = [&](int ci) {
    const __amdgpu_buffer_rsrc_t k = run_rows(k0, a.sh, key_pitch, 32 * ST, a.sh.run(a.first + ci, a.all));
#pragma unroll
    for (int i = 0; i < 4; ++i) row_load(k, key_row[i], &kf[i]);
  };
  auto load_v = [&](int ci) {
    const __amdgpu_buffer_rsrc_t v = run_rows(v0, a.sh, val_pitch, 2 * NS, a.sh.run(a.first + ci, a.all));
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) vv[nt][r] = row_load1(v, val_row[r] + 32 * nt);
  };
  auto load_t = [&]() {
    const __amdgpu_buffer_rsrc_t r = record(rec, a.lay.bytes);
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (lower_has(w, s))
#pragma unroll
        for (int i = 0; i < 3; ++i)
          tf[s][i] = record_frag(r, static_cast<int>(a.lay.t) + lower_at(w, s) * 3 * kB, i, lane16);
  };
  auto load_eg = [&]() { eg = gates4(record(rec, a.lay.bytes), 0); };
  auto load_keep = [&]() {
    const __amdgpu_buffer_rsrc_t r = record(rec, a.lay.bytes);
    keep = gates4(r, 1);
    last = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, 4 * (C - 1), 0, 0));
  };
  auto load_kt = [&]() {
    const __amdgpu_buffer_rsrc_t r = record(key, a.lay.key_bytes);
#pragma unroll
    for (int st = 0; st < ST; ++st)
#pragma unroll
      for (int s = 0; s < 2; ++s) ktf[st][s] = record_frag(r, ST * w * 2 * kB, 2 * st + s, lane16);
  };
  load_rows(0), load_eg(), load_v(0), load_t(), load_keep(), load_kt();

  for (int ci = 0; ci < chunks; ++ci) {
    const int next = ci + 1 < chunks ? ci + 1 : ci;
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
      if constexpr (SAVE) {
        float* to = a.states + ((bh * a.seg + ci) * DK + state_row<ST>(w, 0, 4 * q4)) * dv + n0 + 16 * nt + l16;
#pragma unroll
        for (int st = 0; st < ST; ++st)
#pragma unroll
          for (int r = 0; r < 4; ++r) to[(4 * st + r) * dv] = S[st][nt][r];
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          *reinterpret_cast<own_t*>(sS[i] + at<DK>(16 * nt + l16, state_row<ST>(w, 0, 4 * q4))) = own[i];
      }
    }
    load_rows(next);
    lds_barrier();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const f32x4*>(&sP[nt][i][w][4 * lane]);
      const f32x4 ks = (p[0] + p[1]) + (p[2] + p[3]);
      f32x4 R;
#pragma unroll
      for (int r = 0; r < 4; ++r) R[r] = fmaf(-eg[r], ks[r], bf(vv[nt][r]));
      u32x2 x[3];
      split4(R, x);
#pragma unroll
      for (int i = 0; i < 3; ++i) write4<C>(sR[i], 16 * nt + l16, 16 * w + 4 * q4, x[i]);
    }
    if (next > ci) rec += rec_bytes, key += key_bytes;
    load_eg(), load_v(next);
    lds_barrier();
    f32x4 U[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 u[3] = {zero4(), zero4(), zero4()};
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (lower_has(w, s)) {
          bf16x8 y[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) y[i] = read8<C>(sR[i], 16 * nt + l16, 32 * s + 8 * q4);
          mfma_three(tf[s], y, u);
        }
      U[nt] = sum3(u);
    }
    load_t();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      u32x2 p[3];
      split4(U[nt] * keep, p);
#pragma unroll
      for (int i = 0; i < 3; ++i) write4<C>(sU[i], 16 * nt + l16, 16 * w + 4 * q4, p[i]);
      if constexpr (SAVE) {
        float* to = a.us + ((bh * a.seg + ci) * C + 16 * w + 4 * q4) * dv + n0 + 16 * nt + l16;
#pragma unroll
        for (int r = 0; r < 4; ++r) to[r * dv] = U[nt][r];
      } else {
        u32x2 o[3];
        split4(U[nt], o);
#pragma unroll
        for (int i = 0; i < 3; ++i) write4<C>(sV[i], 16 * nt + l16, 16 * w + 4 * q4, o[i]);
      }
    }
    const float decay = last;
    load_keep();
    lds_barrier();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 add[ST][3];
#pragma unroll
      for (int st = 0; st < ST; ++st) add[st][0] = add[st][1] = add[st][2] = zero4();
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
    }
    load_kt();
  }
  if (a.state_out) {
#pragma unroll
    for (int st = 0; st < ST; ++st)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) a.state_out[state0 + (4 * st + r) * dv + 16 * nt] = S[st][nt][r];
  }
}

// A few tokens (token_by_token), one after the other, all in fp32: a wavefront per 32 columns of a head's state, which it
// holds in registers (8 lanes x 4 columns, an eighth of the rows each).  One token is bound by the states, each read and
// written once: 16 x 32 heads of 128 x 128 (67 MB) in 14.8 us from memory (16 such calls on states of their own in turn,
// 4.5 TB/s), 12.9 us where the last-level cache holds them; further tokens by the two sums over the rows that follow from
// one another (0.97 us a token at 32 heads).
struct StepArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* dt;
  const uint16_t* b;
  const float* A;
  const float* dt_bias;
  const float* state_in;
  float* state_out;
  uint16_t* out;
  Shape sh;
  int64_t rows, dv;  // rows: batch * heads
  float scale;
};

__device__ __forceinline__ int64_t step_token(const Shape& sh, int64_t p) { return sh.rev ? sh.L - 1 - p : p; }

// Sum over the lanes that hold the same columns (lane % 8), in each of them.
__device__ __forceinline__ float row_parts_sum(float v) {
  v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x128, 0xf, 0xf, true));  // row_ror:8
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

template <int DK>
__global__ __launch_bounds__(256) void k_delta_step(StepArgs a) {
  constexpr int R = DK / 8;  // rows per lane
  const int lane = threadIdx.x & 63, part = lane >> 3;
  const int64_t slices = a.dv / 32;
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= a.rows * slices) return;
  const int64_t bh = wave / slices, b = bh / a.sh.heads, h = bh % a.sh.heads, kh = h / (a.sh.heads / a.sh.hk);
  const int64_t n = wave % slices * 32 + (lane & 7) * 4;
  const int64_t L = a.sh.L;
  f32x4 S[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    S[i] = a.state_in ? *reinterpret_cast<const f32x4*>(a.state_in + (bh * DK + part * R + i) * a.dv + n) : zero4();
  const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  bf16x8 kn[R / 8], qn[R / 8];
  u32x2 vn;
  uint16_t dtn, bn;
  auto fetch = [&](int64_t p) {
    const int64_t t = b * L + step_token(a.sh, p);
#pragma unroll
    for (int i = 0; i < R / 8; ++i) {
      kn[i] = *reinterpret_cast<const bf16x8*>(a.k + (t * a.sh.hk + kh) * DK + part * R + 8 * i);
      qn[i] = *reinterpret_cast<const bf16x8*>(a.q + (t * a.sh.hk + kh) * DK + part * R + 8 * i);
    }
    vn = *reinterpret_cast<const u32x2*>(a.v + (t * a.sh.heads + h) * a.dv + n);
    dtn = a.dt[t * a.sh.heads + h];
    bn = a.b[t * a.sh.heads + h];
  };
  fetch(0);
  for (int64_t p = 0; p < L; ++p) {
    float k[R], q[R];
#pragma unroll
    for (int i = 0; i < R; ++i) k[i] = static_cast<float>(kn[i / 8][i % 8]), q[i] = static_cast<float>(qn[i / 8][i % 8]);
    const f32x4 v = __builtin_convertvector(__builtin_bit_cast(bf16x4, vn), f32x4);
    const float decay = ex(softplus_f32(bf(dtn) + bias) * A), beta = sigmoid_f32(bf(bn));
    if (p + 1 < L) fetch(p + 1);
    f32x4 d = zero4(), o = zero4();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      S[i] *= decay;
      d += k[i] * S[i];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = beta * (v[e] - row_parts_sum(d[e]));
#pragma unroll
    for (int i = 0; i < R; ++i) {
      S[i] += k[i] * d;
      o += q[i] * S[i];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = row_parts_sum(o[e]) * a.scale;
    if (part == 0)
      *reinterpret_cast<u32x2*>(a.out + ((b * L + step_token(a.sh, p)) * a.sh.heads + h) * a.dv + n) =
          __builtin_bit_cast(u32x2, __builtin_convertvector(o, bf16x4));
  }
  if (a.state_out) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      *reinterpret_cast<f32x4*>(a.state_out + (bh * DK + part * R + i) * a.dv + n) = S[i];
  }
}

template <int DK, bool SAVE>
void launch_walk(const WalkArgs& a, int tiles, hipStream_t stream) {
  const int64_t rows = (a.batch * a.sh.heads + 7) / 8 * 8;
  const dim3 grid(static_cast<unsigned>(rows * (a.dv / (16 * tiles))));
  if (tiles == 1) hipLaunchKernelGGL((k_delta_walk<DK, 1, SAVE>), grid, dim3(SAVE ? 256 : 512), 0, stream, a);
  else hipLaunchKernelGGL((k_delta_walk<DK, 2, SAVE>), grid, dim3(SAVE ? 256 : 512), 0, stream, a);
}

}  // namespace

hipError_t launch_delta_step(const DeltaArgs& in, hipStream_t stream) {
  const StepArgs a{static_cast<const uint16_t*>(in.q), static_cast<const uint16_t*>(in.k),
                   static_cast<const uint16_t*>(in.v), static_cast<const uint16_t*>(in.dt),
                   static_cast<const uint16_t*>(in.b), in.A, in.dt_bias, in.h_in, in.h_out,
                   static_cast<uint16_t*>(in.out), Shape{in.seqlen, in.hk, in.heads, in.rev}, in.batch * in.heads,
                   in.dv, in.scale};
  const dim3 grid(static_cast<unsigned>((a.rows * (in.dv / 32) + 3) / 4));
  if (in.dk == 64) hipLaunchKernelGGL((k_delta_step<64>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((k_delta_step<128>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_delta_prep(const DeltaArgs& in, const Plan& p, int64_t chunk0, int64_t chunks, bool grad, void* ws,
                             hipStream_t stream) {
  const Layout lay = make_layout(in.dk, grad);
  unsigned char* w = static_cast<unsigned char*>(ws);
  const PrepArgs a{static_cast<const uint16_t*>(in.q), static_cast<const uint16_t*>(in.k),
                   static_cast<const uint16_t*>(in.dt), static_cast<const uint16_t*>(in.b), in.A, in.dt_bias,
                   w + p.head_off, w + p.key_off, Shape{in.seqlen, in.hk, in.heads, in.rev}, lay, chunk0, p.seg,
                   static_cast<int>(p.nchunk), in.scale};
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(in.heads), static_cast<unsigned>(in.batch));
  if (in.dk == 64) {
    if (grad) hipLaunchKernelGGL((k_delta_prep<64, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_delta_prep<64, false>), grid, dim3(256), 0, stream, a);
  } else {
    if (grad) hipLaunchKernelGGL((k_delta_prep<128, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_delta_prep<128, false>), grid, dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_delta_walk(const DeltaArgs& in, const Plan& p, int64_t chunk0, int64_t chunks, bool save,
                             const float* state_in, float* state_out, void* ws, hipStream_t stream) {
  unsigned char* w = static_cast<unsigned char*>(ws);
  const WalkArgs a{static_cast<const uint16_t*>(in.q), static_cast<const uint16_t*>(in.k),
                   static_cast<const uint16_t*>(in.v), static_cast<uint16_t*>(in.out), w + p.head_off, w + p.key_off,
                   state_in, state_out, reinterpret_cast<float*>(w + p.s_off), reinterpret_cast<float*>(w + p.u_off),
                   Shape{in.seqlen, in.hk, in.heads, in.rev}, make_layout(in.dk, save), in.batch, in.dv, p.seg,
                   static_cast<int>(chunk0), static_cast<int>(chunks), static_cast<int>(p.nchunk), in.scale};
  if (in.dk == 64) {
    if (save) launch_walk<64, true>(a, p.tiles, stream);
    else launch_walk<64, false>(a, p.tiles, stream);
  } else {
    if (save) launch_walk<128, true>(a, p.tiles, stream);
    else launch_walk<128, false>(a, p.tiles, stream);
  }
  return hipGetLastError();
}

hipError_t launch_delta_fwd(const DeltaArgs& in, const Plan& p, void* ws, hipStream_t stream) {
  float* carry = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + p.carry_off);
  const float* from = in.h_in;
  for (int64_t c0 = 0; c0 < p.nchunk; c0 += p.seg) {
    const int64_t n = p.nchunk - c0 < p.seg ? p.nchunk - c0 : p.seg;
    float* to = c0 + n == p.nchunk ? in.h_out : carry;
    hipError_t e = launch_delta_prep(in, p, c0, n, false, ws, stream);
    if (e != hipSuccess) return e;
    e = launch_delta_walk(in, p, c0, n, false, from, to, ws, stream);
    if (e != hipSuccess) return e;
    from = carry;
  }
  return hipSuccess;
}

}  // namespace delta
}  // namespace bimamba
