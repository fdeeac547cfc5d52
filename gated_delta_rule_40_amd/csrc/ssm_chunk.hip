// ssm_chunk.hip -- the selective state space scan over prompts, in chunks of
// 64 tokens on the matrix cores.
//
// For a chunk entered with state S (N x P), with step sizes d_j and
// Gamma_i = sum_{j<=i} -exp(A_log) d_j (non-increasing):
//   y_i = e^Gamma_i S^T C_i + sum_{j<=i} (C_i . B_j) e^(Gamma_i - Gamma_j) d_j x_j + D x_i
//   S'  = e^Gamma_L S + sum_j B_j (e^(Gamma_L - Gamma_j) d_j x_j)^T
// Every exponent used is <= 0, for any step size.  Gamma is summed in 64 bits
// and kept as two floats, so that differences late in a strongly decaying
// chunk stay exact.
//
// A workgroup owns 16 columns per wave of the state of a group's heads (the
// r P columns of the r = H / G heads that share B and C lie side by side in x
// and y) and walks the chunks in order with the state in matrix accumulators.
// Per chunk:
//   1. B, C, x and the step sizes, requested one chunk ahead, go to LDS;
//   2. the waves share out the ten 16x16 tiles of G^T = B C^T on and below the
//      diagonal and write, for every head of the workgroup,
//      P_ij = G_ij e^(Gamma_i - Gamma_j) d_j to LDS;
//   3. each wave, for its columns: y^T = e^Gamma S^T C^T + x^T P^T + D x^T
//      and the state's update.
// The state's accumulators are the S^T operand as they stand, with the rows of
// C stored in the matching order; the transposed operands of B and x (bf16)
// come through the transposing LDS loads.
//
// Roundings (bf16 io): P and the S^T operand round to bf16 once each before
// their products, next to the output's own rounding of the same size.  The
// state itself is an fp32 result: the weighted x is taken in three bf16 pieces
// (2^-25 of it is lost), x and B are exact.  fp32 io runs on fp32 matrix
// instructions throughout.
//
// Few units (rows x groups x column blocks) cannot fill the GPU by
// themselves, so the chunks are then cut into segments: a first pass forms
// each segment's state from zero (step 3's update alone) and its decay,
// ssm_start_kernel adds them up to every segment's start, and the second pass
// walks the segments side by side.
#include <type_traits>

#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"

namespace gdr {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int L = 64;  // tokens per chunk

// Matrix operands of one io type, KS the width of a contraction step.  Lane l supplies row l % 16 with g = l / 16.
template <typename T>
struct Op;

template <>
struct Op<bf16> {
  static constexpr int KS = 32, PIECES = 3;
  using F = bf16x8_t;
  __device__ static __forceinline__ f32x4 mma(F a, F b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  __device__ static __forceinline__ F join(bf16x4_t a, bf16x4_t b) {
    return F{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  // Contraction over the state's rows in accumulator order: step s, lane group
  // g takes rows 32 s + 4 g + {0..3} and 32 s + 16 + 4 g + {0..3}.
  __device__ static __forceinline__ F state(const f32x4* acc, int s) {
    F r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r[e] = static_cast<bf16>(acc[2 * s][e]);
      r[4 + e] = static_cast<bf16>(acc[2 * s + 1][e]);
    }
    return r;
  }
  __device__ static __forceinline__ F rows(const bf16* row, int s, int g) {
    return join(*reinterpret_cast<const bf16x4_t*>(row + 32 * s + 4 * g),
                *reinterpret_cast<const bf16x4_t*>(row + 32 * s + 16 + 4 * g));
  }
  // ... with the row stored in that order (store_ordered).
  __device__ static __forceinline__ F rows_ordered(const bf16* row, int s, int g) {
    return *reinterpret_cast<const F*>(row + 32 * s + 8 * g);
  }
  // Eight values from column c (a multiple of 8) of a row, to their places.
  __device__ static __forceinline__ void store_ordered(bf16* row, int c, uint4 v) {
    bf16* p = row + (c & ~31) + 4 * ((c & 31) / 16) + 2 * (c & 15);
    *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(p + 8) = make_uint2(v.z, v.w);
  }
  // Contraction over tokens, natural order: row operand and column operand.
  __device__ static __forceinline__ F tokens(const bf16* row, int s, int g) {
    return *reinterpret_cast<const F*>(row + 32 * s + 8 * g);
  }
  // Columns col0 + r of tokens 32 s + 8 g ... + 7: a transposing load takes 4
  // tokens x 16 columns for each lane group, its lane r addressing token r / 4
  // and columns 4 (r % 4), and hands lane r column r.
  __device__ static __forceinline__ F columns(const bf16* buf, int ld, int s, int g, int r,
                                              int col0) {
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
    const bf16* p = buf + (32 * s + 8 * g + r / 4) * ld + col0 + 4 * (r & 3);
    const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
    const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * ld));
    return join(__builtin_bit_cast(bf16x4_t, a), __builtin_bit_cast(bf16x4_t, b));
  }
  // x times per-token weights as pieces that add up to the product.
  __device__ static __forceinline__ void weigh(F x, const float* w, int s, int g,
                                               F (&out)[PIECES]) {
    const float4 w0 = *reinterpret_cast<const float4*>(w + 32 * s + 8 * g);
    const float4 w1 = *reinterpret_cast<const float4*>(w + 32 * s + 8 * g + 4);
    const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = static_cast<float>(x[i]) * ww[i];
#pragma unroll
      for (int q = 0; q < PIECES; ++q) {
        out[q][i] = static_cast<bf16>(v);
        v -= static_cast<float>(out[q][i]);
      }
    }
  }
  // Not finite: makes the sum NaN.
  __device__ static __forceinline__ float probe(F x, float sum) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(static_cast<float>(x[i]), 0.0f, sum);
    return sum;
  }
};

template <>
struct Op<float> {
  static constexpr int KS = 4, PIECES = 1;
  using F = float;
  __device__ static __forceinline__ f32x4 mma(F a, F b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
  }
  // Step s takes rows 16 (s / 4) + 4 g + s % 4.
  __device__ static __forceinline__ F state(const f32x4* acc, int s) { return acc[s / 4][s & 3]; }
  __device__ static __forceinline__ F rows(const float* row, int s, int g) {
    return row[16 * (s / 4) + 4 * g + (s & 3)];
  }
  __device__ static __forceinline__ F rows_ordered(const float* row, int s, int g) {
    return rows(row, s, g);
  }
  __device__ static __forceinline__ void store_ordered(float* row, int c, uint4 v) {
    *reinterpret_cast<uint4*>(row + c) = v;
  }
  __device__ static __forceinline__ F tokens(const float* row, int s, int g) {
    return row[4 * s + g];
  }
  __device__ static __forceinline__ F columns(const float* buf, int ld, int s, int g, int r,
                                              int col0) {
    return buf[(4 * s + g) * ld + col0 + r];
  }
  __device__ static __forceinline__ void weigh(F x, const float* w, int s, int g,
                                               F (&out)[PIECES]) {
    out[0] = x * w[4 * s + g];
  }
  __device__ static __forceinline__ float probe(F x, float sum) {
    return __builtin_fmaf(x, 0.0f, sum);
  }
};

// HB heads of the workgroup's 16 NW columns.
template <typename T, int N, int HB, int NW>
struct Shape {
  static constexpr int EV = 16 / static_cast<int>(sizeof(T));  // values per 16 bytes
  static constexpr int NP = N < Op<T>::KS ? Op<T>::KS : N;     // rows of the state, padded
  static constexpr int COLS = 16 * NW;
  static constexpr int NT = 64 * NW;
  static constexpr int LB = NP + EV;    // row pitches in LDS, 16-byte multiples
  static constexpr int LX = COLS + EV;
  static constexpr int LP = L + EV;
  static constexpr int BV = (L * (N / EV) + NT - 1) / NT;      // 16-byte loads per thread
  static constexpr int XV = (L * (COLS / EV) + NT - 1) / NT;
  T b[L][LB];
  T c[L][LB];
  T x[L][LX];
  T p[HB][L][LP];
  // Per head and token: Gamma log2(e) in two floats, d, e^Gamma, and
  // e^(Gamma_L - Gamma) d.
  float gh[HB][L], gl[HB][L], d[HB][L], eg[HB][L], w[HB][L];
};

// Workgroups that share B and C (neighbouring numbers) go to one XCD: hardware
// deals consecutive workgroups round the 8 XCDs.
__device__ __forceinline__ unsigned xcd_order(unsigned id, unsigned total) {
  const unsigned xcd = id & 7, k = id >> 3, per = total >> 3, rem = total & 7;
  return xcd * per + min(xcd, rem) + k;
}

// kStates: the first pass (segment states from zero).  ws: segment starts
// [B,H,segs,N,P], then segment log2 decays [B,H,segs].
template <typename T, int N, int HB, int NW, bool kStates>
__global__ __launch_bounds__(64 * NW) void ssm_chunk_kernel(SsmArgs a, int blocks, int segs,
                                                            int seg_chunks) {
  using Sh = Shape<T, N, HB, NW>;
  using O = Op<T>;
  using F = typename O::F;
  constexpr int KN = Sh::NP / O::KS, KL = L / O::KS, NTL = Sh::NP / 16, EV = Sh::EV;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Sh& sm = *reinterpret_cast<Sh*>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;

  const int pass_segs = kStates ? segs - 1 : segs;
  unsigned id = xcd_order(blockIdx.x, gridDim.x);
  const int block = id % blocks;
  id /= blocks;
  const int grp = id % a.G;
  id /= a.G;
  const int seg = id % pass_segs;
  const int b = id / pass_segs;

  const int n = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
  const int first = seg * seg_chunks;
  const int end = min(first + seg_chunks, (n + L - 1) / L);
  const int rh = a.H / a.G;                // heads of the group
  const int width = rh * a.P;              // its columns
  const int col0 = block * Sh::COLS;       // of the workgroup, in the group
  const int hb0 = col0 / a.P;              // its first head, in the group
  const int wcol = col0 + 16 * wave;       // of the wave
  const bool on = wcol < width;
  const int hw = on ? wcol / a.P - hb0 : 0;  // the wave's head in the workgroup
  const int head = grp * rh + min(wcol / a.P, rh - 1);
  const int pcol = wcol % a.P;

  // Loads of one chunk, a chunk ahead.
  uint4 pb[Sh::BV], pc[kStates ? 1 : Sh::BV], px[Sh::XV];
  float pdt[(HB + NW - 1) / NW];
  const size_t brow = static_cast<size_t>(a.G) * N, xrow = static_cast<size_t>(a.H) * a.P;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto request = [&](int chunk) {
    const int t0 = chunk * L;
    const size_t base = static_cast<size_t>(b) * a.T + t0;
    const T* bp = static_cast<const T*>(a.b) + base * brow + grp * N;
    const T* cp = static_cast<const T*>(a.c) + base * brow + grp * N;
    const T* xp = static_cast<const T*>(a.x) + base * xrow + static_cast<size_t>(grp) * width + col0;
#pragma unroll
    for (int i = 0; i < Sh::BV; ++i) {
      const int u = tid + i * Sh::NT, row = u / (N / EV), cc = u % (N / EV) * EV;
      const bool in = row < L && t0 + row < n;
      pb[i] = in ? *reinterpret_cast<const uint4*>(bp + row * brow + cc) : zero;
      if constexpr (!kStates) pc[i] = in ? *reinterpret_cast<const uint4*>(cp + row * brow + cc) : zero;
    }
#pragma unroll
    for (int i = 0; i < Sh::XV; ++i) {
      const int u = tid + i * Sh::NT, row = u / (Sh::COLS / EV), cc = u % (Sh::COLS / EV) * EV;
      const bool in = row < L && t0 + row < n && col0 + cc < width;
      px[i] = in ? *reinterpret_cast<const uint4*>(xp + row * xrow + cc) : zero;
    }
#pragma unroll
    for (int i = 0; i < (HB + NW - 1) / NW; ++i) {
      const int h = hb0 + wave + i * NW;
      const bool in = wave + i * NW < HB && h < rh && t0 + lane < n;
      pdt[i] = in ? a.dt[(base + lane) * a.H + grp * rh + h] : 0.0f;
    }
  };

  // The state: rows 16 k + 4 g + e, column pcol + r.
  f32x4 S[NTL];
  const size_t unit = static_cast<size_t>(b) * a.H + head;
  float* starts = static_cast<float*>(a.ws);
  float* decays = starts + static_cast<size_t>(a.B) * a.H * segs * N * a.P;
  const float* from = nullptr;
  if (!kStates) {
    if (segs > 1) from = starts + (unit * segs + seg) * N * a.P;
    else if (a.state_in) from = a.state_in + unit * N * a.P;
  }
#pragma unroll
  for (int k = 0; k < NTL; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 16 * k + 4 * g + e;
      S[k][e] = from && on && row < N ? from[static_cast<size_t>(row) * a.P + pcol + r] : 0.0f;
    }

  if constexpr (Sh::NP > N) {  // the columns that the loads never write stay zeros
    for (int i = tid; i < L * Sh::NP; i += Sh::NT) {
      sm.b[i / Sh::NP][i % Sh::NP] = from_f32<T>(0.0f);
      sm.c[i / Sh::NP][i % Sh::NP] = from_f32<T>(0.0f);
    }
    __syncthreads();
  }

  float rate[(HB + NW - 1) / NW], db[(HB + NW - 1) / NW];
  const float dskip = !kStates && a.D && on ? a.D[head] : 0.0f;
#pragma unroll
  for (int i = 0; i < (HB + NW - 1) / NW; ++i) {
    const int h = min(hb0 + wave + i * NW, rh - 1);
    rate[i] = -expf(a.A_log[grp * rh + h]);
    db[i] = a.dt_bias ? a.dt_bias[grp * rh + h] : 0.0f;
  }
  double total = 0.0;  // log2 decay of the segment so far (first pass)

  if (first < end) request(first);
  for (int chunk = first; chunk < end; ++chunk) {
    const int t0 = chunk * L;
    // ---- 1. to LDS ----
#pragma unroll
    for (int i = 0; i < Sh::BV; ++i) {
      const int u = tid + i * Sh::NT, row = u / (N / EV), cc = u % (N / EV) * EV;
      if (row < L) {
        *reinterpret_cast<uint4*>(&sm.b[row][cc]) = pb[i];
        if constexpr (!kStates) O::store_ordered(sm.c[row], cc, pc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < Sh::XV; ++i) {
      const int u = tid + i * Sh::NT, row = u / (Sh::COLS / EV), cc = u % (Sh::COLS / EV) * EV;
      if (row < L) *reinterpret_cast<uint4*>(&sm.x[row][cc]) = px[i];
    }
#pragma unroll
    for (int i = 0; i < (HB + NW - 1) / NW; ++i) {
      const int hb = wave + i * NW;
      if (hb < HB) {
        const float d = t0 + lane < n ? softplusf(pdt[i] + db[i]) : 0.0f;
        double gam = static_cast<double>(rate[i]) * d * 1.4426950408889634;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
          const double up = __shfl_up(gam, o, 64);
          gam += lane >= o ? up : 0.0;
        }
        const double last = __shfl(gam, 63, 64);
        const float hi = static_cast<float>(gam);
        sm.gh[hb][lane] = hi;
        sm.gl[hb][lane] = static_cast<float>(gam - static_cast<double>(hi));
        sm.d[hb][lane] = d;
        sm.eg[hb][lane] = __builtin_amdgcn_exp2f(hi);
        sm.w[hb][lane] = __builtin_amdgcn_exp2f(static_cast<float>(last - gam)) * d;
      }
    }
    __syncthreads();
    if (chunk + 1 < end) request(chunk + 1);

    // ---- 2. P ----
    if constexpr (!kStates) {
      // Tiles (ti, tj), tj <= ti, dealt round the waves.
#pragma unroll 1
      for (int tile = wave; tile < 10; tile += NW) {
        const int ti = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3;
        const int tj = tile - ti * (ti + 1) / 2;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KN; ++s)
          acc = O::mma(O::rows(sm.b[16 * tj + r], s, g), O::rows_ordered(sm.c[16 * ti + r], s, g),
                       acc);
        const int i = 16 * ti + r, j = 16 * tj + 4 * g;
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
          const float4 h4 = *reinterpret_cast<const float4*>(&sm.gh[hb][j]);
          const float4 l4 = *reinterpret_cast<const float4*>(&sm.gl[hb][j]);
          const float4 d4 = *reinterpret_cast<const float4*>(&sm.d[hb][j]);
          const float hi = sm.gh[hb][i], lo = sm.gl[hb][i];
          const float jh[4] = {h4.x, h4.y, h4.z, h4.w}, jl[4] = {l4.x, l4.y, l4.z, l4.w};
          const float jd[4] = {d4.x, d4.y, d4.z, d4.w};
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = __builtin_amdgcn_exp2f((hi - jh[e]) + (lo - jl[e])) * jd[e];
            v[e] = j + e <= i ? acc[e] * f : 0.0f;
          }
          store4<T>(&sm.p[hb][i][j], v[0], v[1], v[2], v[3]);
          // The tile right of the diagonal that a step of 32 tokens also takes.
          if (O::KS > 16 && ti == tj && (ti & 1) == 0)
            store4<T>(&sm.p[hb][i][j + 16], 0.f, 0.f, 0.f, 0.f);
        }
      }
      __syncthreads();
    }

    // ---- 3. this wave's columns ----
    if (on) {
      F xf[KL];
      float sum = 0.0f;
#pragma unroll
      for (int s = 0; s < KL; ++s) {
        xf[s] = O::columns(&sm.x[0][0], Sh::LX, s, g, r, 16 * wave);
        if constexpr (!kStates) sum = O::probe(xf[s], sum);
      }
      if constexpr (!kStates) {
        // x that is not finite must not reach earlier tokens through the zeros
        // above the diagonal of P: such columns are summed one by one.
        const bool plain = !__any(sum != 0.0f);
        F sf[KN];
#pragma unroll
        for (int s = 0; s < KN; ++s) sf[s] = O::state(S, s);
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) {
          const int i = 16 * ti + r;
          f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < KN; ++s) y = O::mma(sf[s], O::rows_ordered(sm.c[i], s, g), y);
          y *= sm.eg[hw][i];
          if (plain) {
#pragma unroll
            for (int s = 0; s * O::KS < 16 * (ti + 1); ++s)
              y = O::mma(xf[s], O::tokens(sm.p[hw][i], s, g), y);
          } else {
            for (int j = 0; j <= i; ++j) {
              const float p = to_f32(sm.p[hw][i][j]);
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] += p * to_f32(sm.x[j][16 * wave + 4 * g + e]);
            }
          }
          float xv[4];
          load_row<T, 4>(&sm.x[i][16 * wave + 4 * g], xv);
          if (t0 + i < n)
            store4<T>(static_cast<T*>(a.y) + (static_cast<size_t>(b) * a.T + t0 + i) * xrow +
                          static_cast<size_t>(head) * a.P + pcol + 4 * g,
                      y[0] + dskip * xv[0], y[1] + dskip * xv[1], y[2] + dskip * xv[2],
                      y[3] + dskip * xv[3]);
        }
      }
      const float decay = sm.eg[hw][L - 1];
#pragma unroll
      for (int k = 0; k < NTL; ++k) S[k] *= decay;
#pragma unroll
      for (int s = 0; s < KL; ++s) {
        F wx[O::PIECES];
        O::weigh(xf[s], sm.w[hw], s, g, wx);
#pragma unroll
        for (int k = 0; k < NTL; ++k) {
          const F bt = O::columns(&sm.b[0][0], Sh::LB, s, g, r, 16 * k);
#pragma unroll
          for (int q = 0; q < O::PIECES; ++q) S[k] = O::mma(bt, wx[q], S[k]);
        }
      }
      if constexpr (kStates)
        total += static_cast<double>(sm.gh[hw][L - 1]) + sm.gl[hw][L - 1];
    }
    __syncthreads();
  }

  // ---- the state's way out ----
  if (!on) return;
  float* to = nullptr;
  if constexpr (kStates) {
    to = starts + (unit * segs + seg + 1) * N * a.P;
    if (lane == 0 && pcol == 0) decays[unit * segs + seg] = static_cast<float>(total);
  } else if (seg == segs - 1) {
    to = a.state_out + unit * N * a.P;
  }
  if (to) {
#pragma unroll
    for (int k = 0; k < NTL; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 16 * k + 4 * g + e;
        if (row < N) to[static_cast<size_t>(row) * a.P + pcol + r] = S[k][e];
      }
  }
}

// Segment starts: start_0 = state_in, start_k+1 = e^decay_k start_k + N_k, with
// N_k in the place of start_k+1 before.
__global__ __launch_bounds__(256) void ssm_start_kernel(SsmArgs a, int segs) {
  const size_t quads = static_cast<size_t>(a.N) * a.P / 4;
  const size_t at = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  const size_t unit = at / quads, q = at % quads;
  if (unit >= static_cast<size_t>(a.B) * a.H) return;
  float4* starts = static_cast<float4*>(a.ws) + unit * segs * quads + q;
  const float* decays =
      static_cast<float*>(a.ws) + static_cast<size_t>(a.B) * a.H * segs * quads * 4 + unit * segs;
  float4 s = a.state_in ? reinterpret_cast<const float4*>(a.state_in)[unit * quads + q]
                        : make_float4(0.f, 0.f, 0.f, 0.f);
  starts[0] = s;
  for (int k = 1; k < segs; ++k) {
    const float f = __builtin_amdgcn_exp2f(decays[k - 1]);
    const float4 m = starts[k * quads];
    s = make_float4(f * s.x + m.x, f * s.y + m.y, f * s.z + m.z, f * s.w + m.w);
    starts[k * quads] = s;
  }
}

struct Cut {
  int blocks;      // column blocks of a group
  int segs;        // segments of the sequence
  int seg_chunks;  // chunks of a segment
};

// Columns of a workgroup: 64, or 32 where the P tiles of four 16-wide heads in
// fp32 would not fit LDS.
int block_cols(int P, int io_bf16) { return !io_bf16 && P == 16 ? 32 : 64; }

Cut cut_of(int B, int T, int G, int H, int P, int io_bf16) {
  Cut c;
  const int width = H / G * P, cols = block_cols(P, io_bf16);
  c.blocks = (width + cols - 1) / cols;
  const int chunks = (T + L - 1) / L;
  const long long units = static_cast<long long>(B) * G * c.blocks;
  // Enough workgroups for two on every CU, segments of at least 4 chunks.
  long long segs = (512 + units - 1) / units;
  if (segs > chunks / 4) segs = chunks / 4;
  if (segs < 1) segs = 1;
  c.seg_chunks = static_cast<int>((chunks + segs - 1) / segs);
  c.segs = c.seg_chunks > 0 ? (chunks + c.seg_chunks - 1) / c.seg_chunks : 1;
  return c;
}

template <typename T, int N, int HB, int NW>
hipError_t launch_shape(const SsmArgs& a, const Cut& c, hipStream_t stream) {
  using Sh = Shape<T, N, HB, NW>;
  static_assert(sizeof(Sh) <= 160 * 1024, "LDS of a workgroup");
  const unsigned units = static_cast<unsigned>(a.B) * a.G * c.blocks;
  if (c.segs > 1) {
    hipLaunchKernelGGL((ssm_chunk_kernel<T, N, HB, NW, true>), dim3(units * (c.segs - 1)),
                       dim3(Sh::NT), sizeof(Sh), stream, a, c.blocks, c.segs, c.seg_chunks);
    const size_t quads = static_cast<size_t>(a.B) * a.H * a.N * a.P / 4;
    hipLaunchKernelGGL(ssm_start_kernel, dim3(static_cast<unsigned>((quads + 255) / 256)),
                       dim3(256), 0, stream, a, c.segs);
  }
  hipLaunchKernelGGL((ssm_chunk_kernel<T, N, HB, NW, false>), dim3(units * c.segs), dim3(Sh::NT),
                     sizeof(Sh), stream, a, c.blocks, c.segs, c.seg_chunks);
  return hipGetLastError();
}

template <typename T, int N>
hipError_t launch_n(const SsmArgs& a, const Cut& c, hipStream_t stream) {
  if (a.P >= 64) return launch_shape<T, N, 1, 4>(a, c, stream);
  if (a.P == 32) return launch_shape<T, N, 2, 4>(a, c, stream);
  if constexpr (sizeof(T) == 4) return launch_shape<T, N, 2, 2>(a, c, stream);
  else return launch_shape<T, N, 4, 4>(a, c, stream);
}

template <typename T>
hipError_t launch_t(const SsmArgs& a, const Cut& c, hipStream_t stream) {
  switch (a.N) {
    case 16: return launch_n<T, 16>(a, c, stream);
    case 32: return launch_n<T, 32>(a, c, stream);
    case 64: return launch_n<T, 64>(a, c, stream);
    case 128: return launch_n<T, 128>(a, c, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

size_t ssm_workspace_bytes(int B, int T, int G, int H, int N, int P, int io_bf16) {
  if (T <= ssm_walk_max_t()) return 0;
  const Cut c = cut_of(B, T, G, H, P, io_bf16);
  if (c.segs == 1) return 0;
  return static_cast<size_t>(B) * H * c.segs * (static_cast<size_t>(N) * P + 1) * sizeof(float);
}

hipError_t launch_ssm_chunked(const SsmArgs& a, int io_bf16, hipStream_t stream) {
  const Cut c = cut_of(a.B, a.T, a.G, a.H, a.P, io_bf16);
  return io_bf16 ? launch_t<bf16>(a, c, stream) : launch_t<float>(a, c, stream);
}

}  // namespace gdr
