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
// A workgroup owns 16 CT columns per wave of the state of a group's heads (the
// r P columns of the r = H / G heads that share B and C lie side by side in x
// and y) and walks the chunks in order with the state in matrix accumulators.
// Per chunk:
//   1. B, C, x and the step sizes, requested one chunk ahead, go to LDS;
//   2. the waves share out the ten 16x16 tiles of G^T = B C^T on and below the
//      diagonal and write, for every head of the workgroup,
//      P_ij = G_ij e^(Gamma_i - Gamma_j) d_j to LDS;
//   3. each wave, for its columns: y^T = e^Gamma S^T C^T + x^T P^T + D x^T
//      and the state's update.
// Every product leaves its tiles as the next one's operands: the state's
// accumulators are the S^T operand as they stand, with the rows of C stored in the
// matching order, and a tile of P goes through LDS lane for lane; the transposed
// operands of B and x (bf16) come through the transposing LDS loads, tokens in the
// order of P's tiles.
//
// Roundings (bf16 io): P and the S^T operand are taken in two bf16 pieces (2^-16
// of them is lost), so that the output's own rounding is the only one of its size;
// in one piece each it would be off by 2.0e-3 instead of 1.7e-3 of the norm, up to
// 19 roundings in single values, for 3% (4000 tokens 76.6 against 78.7 us) to 5%
// (long rows 315 against 331) less time.  The state itself is an fp32 result: the
// weighted x is taken in three bf16 pieces (2^-25 of it is lost), x and B are
// exact.  fp32 io runs on fp32 matrix instructions throughout.
//
// Few units (rows x groups x column blocks) cannot fill the GPU by
// themselves, so the chunks are then cut into segments: a first pass forms
// each segment's state from zero (step 3's update alone) and its decay,
// ssm_start_kernel adds them up to every segment's start, and the second pass
// walks the segments side by side.
//
// Bound by issue: per wave and chunk (two column tiles, N = 128) 1211 vector, 193
// matrix and 150 LDS instructions, the waves waiting 39% of their cycles.  4000
// tokens of 64 heads (N = 128, P = 64, 8 groups, bf16), by kernel: segment states
// 23.5 us, their starts 10.6, the walk 48.1.
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

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int L = 64;  // tokens per chunk
// Segments whose starts the walk adds up itself, against a launch that does: four
// rows of 2000 tokens (4 segments) 121 against 126 us, eight of 1000 (2 segments)
// 114 against 124; with 8 segments (two of 1500) 74.7 against 67.3.
constexpr int kFewSegs = 4;
// Whether ssm_start_kernel adds the starts up, into the workspace.  It has to
// where the state is updated in place, however few the segments: the walk's last
// segment writes state_out, and nothing orders that behind the other segments'
// reads of state_in in the same launch.
__host__ __device__ inline bool starts_joined(const SsmArgs& a, int segs) {
  return segs > kFewSegs || (segs > 1 && a.state_in == a.state_out);
}

// 16 bytes, or zeros.
__device__ __forceinline__ u32x4 load16_if(bool in, const void* p) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (in) v = *static_cast<const u32x4*>(p);
  return v;
}

// Matrix operands of one io type, KS the width of a contraction step.  Lane l
// supplies row l % 16 with g = l / 16.  Contractions over the state's rows and over
// tokens run in accumulator order: what a lane holds of a product is its operand of
// the next.
template <typename T>
struct Op;

template <>
struct Op<bf16> {
  static constexpr int KS = 32, PIECES = 3;
  static constexpr int HALVES = 2;  // of the state's and P's values
  using F = bf16x8_t;
  __device__ static __forceinline__ f32x4 mma(F a, F b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  __device__ static __forceinline__ F join(bf16x4_t a, bf16x4_t b) {
    return F{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  // Two values as bf16 words: cut off, and what is left rounded (2^-16 is lost).
  __device__ static __forceinline__ void halves(float x, float y, unsigned (&out)[HALVES]) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const unsigned ux = __builtin_bit_cast(unsigned, x), uy = __builtin_bit_cast(unsigned, y);
    out[0] = __builtin_amdgcn_perm(uy, ux, 0x07060302u);
    x -= __builtin_bit_cast(float, ux & 0xffff0000u);
    y -= __builtin_bit_cast(float, uy & 0xffff0000u);
    out[1] = __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x, y}), bf16x2_t));
  }
  // Step s, lane group g takes rows 32 s + 4 g + {0..3} and 32 s + 16 + 4 g + {0..3}.
  __device__ static __forceinline__ void state(const f32x4* acc, int s, F (&out)[HALVES]) {
    u32x4 w[HALVES];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4& t = acc[2 * s + i / 2];
      unsigned h[HALVES];
      halves(t[2 * (i & 1)], t[2 * (i & 1) + 1], h);
#pragma unroll
      for (int k = 0; k < HALVES; ++k) w[k][i] = h[k];
    }
#pragma unroll
    for (int k = 0; k < HALVES; ++k) out[k] = __builtin_bit_cast(F, w[k]);
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
  __device__ static __forceinline__ void store_ordered(bf16* row, int c, u32x4 v) {
    bf16* p = row + (c & ~31) + 4 * ((c & 31) / 16) + 2 * (c & 15);
    *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(p + 8) = make_uint2(v.z, v.w);
  }
  // Columns col0 + r of tokens 32 s + 4 g ... + 3 and 32 s + 16 + 4 g ... + 3: a
  // transposing load takes 4 tokens x 16 columns for each lane group, its lane r
  // addressing token r / 4 and columns 4 (r % 4), and hands lane r column r.
  // SHIFT: what every other eight rows lie further by.
  template <int SHIFT>
  __device__ static __forceinline__ F columns(const bf16* buf, int ld, int s, int g, int r,
                                              int col0) {
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
    const bf16* p = buf + (32 * s + 4 * g + r / 4) * ld + (g >> 1) * SHIFT + col0 + 4 * (r & 3);
    const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
    const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * ld));
    return join(__builtin_bit_cast(bf16x4_t, a), __builtin_bit_cast(bf16x4_t, b));
  }
  // x times per-token weights as pieces that add up to the product.
  __device__ static __forceinline__ void weigh(F x, const float* w, int s, int g,
                                               F (&out)[PIECES]) {
    const float4 w0 = *reinterpret_cast<const float4*>(w + 32 * s + 4 * g);
    const float4 w1 = *reinterpret_cast<const float4*>(w + 32 * s + 16 + 4 * g);
    const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float v0 = static_cast<float>(x[i]) * ww[i], v1 = static_cast<float>(x[i + 1]) * ww[i + 1];
#pragma unroll
      for (int q = 0; q < PIECES; ++q) {
        typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const bf16x2_t h = __builtin_convertvector((f32x2{v0, v1}), bf16x2_t);
        out[q][i] = h[0];
        out[q][i + 1] = h[1];
        const unsigned u = __builtin_bit_cast(unsigned, h);
        v0 -= __builtin_bit_cast(float, u << 16);
        v1 -= __builtin_bit_cast(float, u & 0xffff0000u);
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
  static constexpr int KS = 4, PIECES = 1, HALVES = 1;
  using F = float;
  __device__ static __forceinline__ f32x4 mma(F a, F b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
  }
  // Step s takes rows 16 (s / 4) + 4 g + s % 4.
  __device__ static __forceinline__ void state(const f32x4* acc, int s, F (&out)[HALVES]) {
    out[0] = acc[s / 4][s & 3];
  }
  __device__ static __forceinline__ F rows(const float* row, int s, int g) {
    return row[16 * (s / 4) + 4 * g + (s & 3)];
  }
  __device__ static __forceinline__ F rows_ordered(const float* row, int s, int g) {
    return rows(row, s, g);
  }
  __device__ static __forceinline__ void store_ordered(float* row, int c, u32x4 v) {
    *reinterpret_cast<u32x4*>(row + c) = v;
  }
  template <int SHIFT>
  __device__ static __forceinline__ F columns(const float* buf, int ld, int s, int g, int r,
                                              int col0) {
    return buf[(16 * (s / 4) + 4 * g + (s & 3)) * ld + (g >> 1) * SHIFT + col0 + r];
  }
  __device__ static __forceinline__ void weigh(F x, const float* w, int s, int g,
                                               F (&out)[PIECES]) {
    out[0] = x * w[16 * (s / 4) + 4 * g + (s & 3)];
  }
  __device__ static __forceinline__ float probe(F x, float sum) {
    return __builtin_fmaf(x, 0.0f, sum);
  }
};

// What a token of a head contributes by, Gamma in units of log2.
struct Rows {
  float gh[L], gl[L];  // Gamma as two floats
  float d[L];          // step size
  float w[L];          // e^(Gamma_L - Gamma) d
  float rf[L];         // e^(Gamma - Gamma_m), m the last token before its 16
  float cf[96];        // e^(Gamma_m - Gamma) d of the tokens up to m, for m = 15, 31, 47
  // Where the m of tile row ti (1, 2, 3) begin.
  __device__ static __forceinline__ int at(int ti) { return 8 * ti * (ti - 1); }
};

// P of a head, as the operands that the products take: tile (ti, tj) of 16x16 is
// written by one wave, lane for lane as it has it (rows i = r, columns 4 g + e), and
// read by others in the same way.  Two tiles of a row that one contraction step
// takes together lie side by side per lane.
template <typename T>
struct Tiles {
  static constexpr int HALVES = Op<T>::HALVES;
  T v[HALVES][10 * 256];
  // The four values of a lane of tile (ti, tj); pairs begin at even tj.
  __device__ static __forceinline__ int at(int ti, int tj, int lane) {
    const int first = ti * (ti + 1) / 2 + (tj & ~1);
    const bool pair = sizeof(T) == 2 && (tj | 1) <= ti;
    return pair ? first * 256 + lane * 8 + (tj & 1) * 4
                : (first + (tj & 1)) * 256 + lane * 4;
  }
  __device__ __forceinline__ void put(int ti, int tj, int lane, const float (&x)[4]) {
    const int k = at(ti, tj, lane);
    if constexpr (HALVES == 1) {
      *reinterpret_cast<float4*>(&v[0][k]) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
      unsigned a[HALVES], b[HALVES];
      Op<T>::halves(x[0], x[1], a);
      Op<T>::halves(x[2], x[3], b);
#pragma unroll
      for (int q = 0; q < HALVES; ++q)
        *reinterpret_cast<uint2*>(&v[q][k]) = make_uint2(a[q], b[q]);
    }
  }
  // The order in which the products of fp32 add up tokens.
  __device__ static __forceinline__ int order(int k) {
    return HALVES == 1 ? (k & ~15) + 4 * (k & 3) + (k >> 2 & 3) : k;
  }
  __device__ __forceinline__ float value(int k) const {
    float x = to_f32(v[0][k]);
#pragma unroll
    for (int q = 1; q < HALVES; ++q) x += to_f32(v[q][k]);
    return x;
  }
  // y^T += x^T P^T for tile row ti, x as columns of all tokens.
  template <int CT, int KL>
  __device__ __forceinline__ void multiply(int ti, int lane, const typename Op<T>::F (&x)[CT][KL],
                                           f32x4 (&y)[CT]) const {
    if constexpr (HALVES == 1) {
#pragma unroll
      for (int tj = 0; tj <= ti; ++tj) {
        const f32x4 p = *reinterpret_cast<const f32x4*>(&v[0][at(ti, tj, lane)]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) y[ct] = Op<T>::mma(x[ct][4 * tj + e], p[e], y[ct]);
      }
    } else {
#pragma unroll
      for (int tj = 0; tj <= ti; tj += 2)
#pragma unroll
        for (int q = 0; q < HALVES; ++q) {
          const T* from = &v[q][at(ti, tj, lane)];
          bf16x8_t p;
          if (tj < ti) {
            p = *reinterpret_cast<const bf16x8_t*>(from);
          } else {
            const bf16x4_t h = *reinterpret_cast<const bf16x4_t*>(from);
            p = Op<T>::join(h, bf16x4_t{});
          }
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) y[ct] = Op<T>::mma(x[ct][tj / 2], p, y[ct]);
        }
    }
  }
};

// A workgroup's LDS: NW waves of CT 16-column tiles, over HB heads.  The row
// pitches keep the 16-byte reads of 16 rows (C) and the transposing reads
// of 4 rows (B, x: 32 bytes a row, a pitch of 32 bytes more than a multiple of
// 256) on distinct banks; B is also read 8 bytes from each of 16 rows, for
// which every other eight rows lie 16 bytes further.
template <typename T, int N, int HB, int NW, int CT, bool kStates>
struct Shape {
  static constexpr int EV = 16 / static_cast<int>(sizeof(T));  // values per 16 bytes
  static constexpr int NP = N < Op<T>::KS ? Op<T>::KS : N;     // rows of the state, padded
  static constexpr int COLS = 16 * NW * CT;
  static constexpr int NT = 64 * NW;
  static constexpr int LB = NP + 2 * EV, LC = NP + EV, LX = COLS + (COLS % 128 ? 1 : 2) * EV;
  static constexpr int BV = (L * (N / EV) + NT - 1) / NT;  // 16-byte loads per thread
  static constexpr int XV = (L * (COLS / EV) + NT - 1) / NT;
  static_assert(HB <= NW, "a wave forms the rows of one head at a time");
  Rows rows[2][HB];
  T b[L][LB];
  T x[L][LX];
  T c[kStates ? 1 : L][LC];
  Tiles<T> p[kStates ? 1 : HB];
  float rate[HB], db[HB];  // decay_rate(A_log), dt_bias
  __device__ __forceinline__ T* brow(int row) { return b[row] + ((row >> 3) & 1) * EV; }
};

// Workgroups that share B and C (neighbouring numbers) go to one XCD: hardware
// deals consecutive workgroups round the 8 XCDs.
__device__ __forceinline__ unsigned xcd_order(unsigned id, unsigned total) {
  const unsigned xcd = id & 7, k = id >> 3, per = total >> 3, rem = total & 7;
  return xcd * per + min(xcd, rem) + k;
}

// The lane's 64-bit value from another lane of the wave by a DPP move (0 where
// there is none).
template <int kCtrl, int kRows>
__device__ __forceinline__ double dpp_from(double x) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
  const unsigned lo = __builtin_amdgcn_update_dpp(0u, static_cast<unsigned>(u), kCtrl, kRows, 0xf, false);
  const unsigned hi =
      __builtin_amdgcn_update_dpp(0u, static_cast<unsigned>(u >> 32), kCtrl, kRows, 0xf, false);
  return __builtin_bit_cast(double, static_cast<unsigned long long>(hi) << 32 | lo);
}

// Inclusive prefix sum over the wave: row shifts inside each 16 lanes, then
// the last lanes of rows 0 and 2 to rows 1 and 3, then lane 31 to the upper half.
__device__ __forceinline__ double wave_prefix_sum(double x) {
  x += dpp_from<0x111, 0xf>(x);  // row_shr:1
  x += dpp_from<0x112, 0xf>(x);
  x += dpp_from<0x114, 0xf>(x);
  x += dpp_from<0x118, 0xf>(x);
  x += dpp_from<0x142, 0xa>(x);  // row_bcast:15
  x += dpp_from<0x143, 0xc>(x);  // row_bcast:31
  return x;
}

// The rows of one head's chunk: lane = token, z = dt + dt_bias (d = 0 where the
// token is not there).
__device__ __forceinline__ void form_rows(Rows& o, int lane, bool there, float z, float rate) {
  const float d = there ? softplus_hw(z) : 0.0f;
  // Past 2^-1024 a token's decay is 0 times whatever fp32 holds; ending it there
  // keeps the sums finite, and exact to 2^-32 behind such a token.
  double g2 = static_cast<double>(rate) * d * 1.4426950408889634;
  g2 = g2 < -1024.0 ? -1024.0 : g2;  // NaN stays
  const double gam = wave_prefix_sum(g2);
  const float hi = static_cast<float>(gam);
  o.gh[lane] = hi;
  o.gl[lane] = static_cast<float>(gam - static_cast<double>(hi));
  o.d[lane] = d;
  o.w[lane] = __builtin_amdgcn_exp2f(static_cast<float>(__shfl(gam, 63, 64) - gam)) * d;
  double before = 0.0;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const double m = __shfl(gam, 16 * k + 15, 64);
    if (lane / 16 == k + 1) before = m;
    if (lane < 16 * k + 16)
      o.cf[Rows::at(k + 1) + lane] = __builtin_amdgcn_exp2f(static_cast<float>(m - gam)) * d;
  }
  o.rf[lane] = __builtin_amdgcn_exp2f(static_cast<float>(gam - before));
}

// kStates: the first pass (segment states from zero).  ws: segment starts
// [B,H,segs,N,P], then segment log2 decays [B,H,segs].
template <typename T, int N, int HB, int NW, int CT, bool kStates>
__global__ __launch_bounds__(64 * NW, 2) void ssm_chunk_kernel(SsmArgs a, int blocks, int segs,
                                                               int seg_chunks) {
  using Sh = Shape<T, N, HB, NW, CT, kStates>;
  using O = Op<T>;
  using F = typename O::F;
  constexpr int KN = Sh::NP / O::KS, KL = L / O::KS, NTL = Sh::NP / 16, EV = Sh::EV;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Sh& sm = *reinterpret_cast<Sh*>(smem);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // scalar: so is what follows from it
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
  // The wave's columns: all of one head (P is a multiple of 16 CT).
  const int lcol = 16 * CT * wave;         // in the workgroup
  const bool on = col0 + lcol < width;
  const int hw = on ? (col0 + lcol) / a.P - hb0 : 0;
  const int head = grp * rh + min((col0 + lcol) / a.P, rh - 1);
  const int pcol = (col0 + lcol) % a.P;

  // Loads of one chunk, a chunk ahead: thread tid takes 16 bytes of row row_b +
  // i * kStepB of B and C (and likewise x), through one 32-bit lane offset each
  // from bases that are the same for all lanes.
  constexpr int kRowB = N / EV, kRowX = Sh::COLS / EV;  // 16-byte pieces of a row
  constexpr int kStepB = Sh::NT / kRowB, kStepX = Sh::NT / kRowX;
  static_assert(Sh::NT % kRowB == 0 && Sh::NT % kRowX == 0, "whole rows per pass");
  u32x4 pb[Sh::BV], pc[kStates ? 1 : Sh::BV], px[Sh::XV];
  const size_t brow = static_cast<size_t>(a.G) * N, xrow = static_cast<size_t>(a.H) * a.P;
  const int row_b = tid / kRowB, cc_b = tid % kRowB * EV;
  const int row_x = tid / kRowX, cc_x = tid % kRowX * EV;
  const unsigned off_b = (row_b * static_cast<unsigned>(brow) + cc_b) * sizeof(T);
  const unsigned off_x = (row_x * static_cast<unsigned>(xrow) + cc_x) * sizeof(T);
  const bool in_x = col0 + cc_x < width;
  // Every thread has something to load from every whole chunk.
  const bool in_all = col0 + Sh::COLS <= width && L % kStepB == 0 && L % kStepX == 0;
  auto request = [&](int chunk) {
    const int left = n - chunk * L;  // tokens from here on
    const size_t base = static_cast<size_t>(b) * a.T + static_cast<size_t>(chunk) * L;
    const char* bp = reinterpret_cast<const char*>(static_cast<const T*>(a.b) + base * brow + grp * N);
    const char* cp = reinterpret_cast<const char*>(static_cast<const T*>(a.c) + base * brow + grp * N);
    const char* xp = reinterpret_cast<const char*>(static_cast<const T*>(a.x) + base * xrow +
                                                   static_cast<size_t>(grp) * width + col0);
    if (left >= L && in_all) {
#pragma unroll
      for (int i = 0; i < Sh::BV; ++i) {
        const size_t step = i * kStepB * brow * sizeof(T);
        pb[i] = *reinterpret_cast<const u32x4*>(bp + step + off_b);
        if constexpr (!kStates) pc[i] = *reinterpret_cast<const u32x4*>(cp + step + off_b);
      }
#pragma unroll
      for (int i = 0; i < Sh::XV; ++i)
        px[i] = *reinterpret_cast<const u32x4*>(xp + i * kStepX * xrow * sizeof(T) + off_x);
      return;
    }
#pragma unroll
    for (int i = 0; i < Sh::BV; ++i) {
      const int row = row_b + i * kStepB;
      const bool in = row < L && row < left;
      const size_t step = i * kStepB * brow * sizeof(T);
      pb[i] = load16_if(in, bp + step + off_b);
      if constexpr (!kStates) pc[i] = load16_if(in, cp + step + off_b);
    }
#pragma unroll
    for (int i = 0; i < Sh::XV; ++i) {
      const int row = row_x + i * kStepX;
      px[i] = load16_if(in_x && row < L && row < left,
                        xp + i * kStepX * xrow * sizeof(T) + off_x);
    }
  };

  // The state: rows 16 k + 4 g + e, column pcol + 16 ct + r.
  f32x4 S[CT][NTL];
  const size_t unit = static_cast<size_t>(b) * a.H + head;
  float* starts = static_cast<float*>(a.ws);
  float* decays = starts + static_cast<size_t>(a.B) * a.H * segs * N * a.P;
  // Where the walk starts: from the state before the first token, or the
  // segment's start; with few segments and a state that is not updated in place
  // that is added up here from the states of the segments before it, which saves
  // ssm_start_kernel's launch.
  const float* from = nullptr;
  const float* before = starts + unit * segs * N * a.P;  // segment k's state at k + 1
  int add = 0;
  if (!kStates) {
    if (starts_joined(a, segs)) {
      from = before + static_cast<size_t>(seg) * N * a.P;
    } else {
      if (a.state_in) from = a.state_in + unit * N * a.P;
      add = seg;
    }
  }
  // Element (16 k + 4 g + e, pcol + 16 ct + r) of a state; rows past N (the
  // padding) are never reached, as k stays below N / 16.
  constexpr int NK = N / 16;
  auto at = [&](int k, int e, int ct) {
    return static_cast<size_t>(16 * k + 4 * g + e) * a.P + pcol + 16 * ct + r;
  };
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int k = 0; k < NTL; ++k) S[ct][k] = f32x4{0.f, 0.f, 0.f, 0.f};
  // The branches lie around whole loads of a state, not around its elements.
  if (from && on) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[ct][k][e] = from[at(k, e, ct)];
  }
  if (on) {
#pragma unroll 1
    for (int s = 0; s < add; ++s) {
      const float f = __builtin_amdgcn_exp2f(decays[unit * segs + s]);
      const float* m = before + static_cast<size_t>(s + 1) * N * a.P;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[ct][k][e] = f * S[ct][k][e] + m[at(k, e, ct)];
    }
  }

  if constexpr (Sh::NP > N) {  // the columns that the loads never write stay zeros
    for (int i = tid; i < L * Sh::NP; i += Sh::NT) {
      sm.brow(i / Sh::NP)[i % Sh::NP] = from_f32<T>(0.0f);
      if constexpr (!kStates) sm.c[i / Sh::NP][i % Sh::NP] = from_f32<T>(0.0f);
    }
    __syncthreads();
  }

  for (int hb = tid; hb < HB; hb += Sh::NT) {
    const int h = grp * rh + min(hb0 + hb, rh - 1);
    sm.rate[hb] = decay_rate(a.A_log[h]);
    sm.db[hb] = a.dt_bias ? a.dt_bias[h] : 0.0f;
  }
  __syncthreads();
  // The waves take turns at forming the rows of the next chunk's heads: wave
  // (hb + HB chunk) mod NW forms head hb's.
  auto turn = [&](int chunk) { return (wave + NW - (HB * chunk) % NW) % NW; };
  float pdt = 0.0f;
  auto request_dt = [&](int chunk) {
    const int hb = turn(chunk), t = chunk * L + lane;
    pdt = hb < HB && hb0 + hb < rh && t < n
              ? a.dt[(static_cast<size_t>(b) * a.T + t) * a.H + grp * rh + hb0 + hb]
              : 0.0f;
  };
  auto rows_of = [&](int chunk) {
    const int hb = turn(chunk);
    if (hb < HB)
      form_rows(sm.rows[chunk & 1][hb], lane, chunk * L + lane < n, pdt + sm.db[hb], sm.rate[hb]);
  };
  const unsigned off_y =
      (r * static_cast<unsigned>(xrow) + head * a.P + pcol + 4 * g) * sizeof(T);
  const float dskip = !kStates && a.D && on ? a.D[head] : 0.0f;
  double total = 0.0;  // log2 decay of the segment so far (first pass)

  if (first < end) {
    request_dt(first);
    request(first);
    rows_of(first);
    if (first + 1 < end) request_dt(first + 1);
  }
#pragma unroll 1
  for (int chunk = first; chunk < end; ++chunk) {
    const int t0 = chunk * L;
    // ---- 1. to LDS ----
#pragma unroll
    for (int i = 0; i < Sh::BV; ++i) {
      const int row = row_b + i * kStepB;
      if (row < L) {
        *reinterpret_cast<u32x4*>(sm.brow(row) + cc_b) = pb[i];
        if constexpr (!kStates) O::store_ordered(sm.c[row], cc_b, pc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < Sh::XV; ++i) {
      const int row = row_x + i * kStepX;
      if (row < L) *reinterpret_cast<u32x4*>(&sm.x[row][cc_x]) = px[i];
    }
    __syncthreads();
    if (chunk + 1 < end) request(chunk + 1);
    const Rows* rows = sm.rows[chunk & 1];

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
          acc = O::mma(O::rows(sm.brow(16 * tj + r), s, g), O::rows_ordered(sm.c[16 * ti + r], s, g),
                       acc);
        const int i = 16 * ti + r, j = 16 * tj + 4 * g;
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
          const Rows& w = rows[hb];
          float v[4];
          if (ti > tj) {
            // e^(Gamma_i - Gamma_j) through the last token before tile row ti.
            const float4 f4 = *reinterpret_cast<const float4*>(&w.cf[Rows::at(ti) + j]);
            const float f = w.rf[i];
            v[0] = acc[0] * f * f4.x;
            v[1] = acc[1] * f * f4.y;
            v[2] = acc[2] * f * f4.z;
            v[3] = acc[3] * f * f4.w;
          } else {
            const float4 h4 = *reinterpret_cast<const float4*>(&w.gh[j]);
            const float4 l4 = *reinterpret_cast<const float4*>(&w.gl[j]);
            const float4 d4 = *reinterpret_cast<const float4*>(&w.d[j]);
            const float hi = w.gh[i], lo = w.gl[i];
            const float jh[4] = {h4.x, h4.y, h4.z, h4.w}, jl[4] = {l4.x, l4.y, l4.z, l4.w};
            const float jd[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float f = __builtin_amdgcn_exp2f((hi - jh[e]) + (lo - jl[e])) * jd[e];
              v[e] = j + e <= i ? acc[e] * f : 0.0f;
            }
          }
          sm.p[hb].put(ti, tj, lane, v);
        }
      }
      __syncthreads();
    }

    // ---- 3. this wave's columns ----
    // Ahead of the other workgroup's staging and P (3% of long rows).
    __builtin_amdgcn_s_setprio(1);
    if (on) {
      const Rows& w = rows[hw];
      f32x4 y[4][CT];  // of tile rows ti: first S^T C^T
      if constexpr (!kStates) {
#pragma unroll
        for (int ti = 0; ti < 4; ++ti)
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) y[ti][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KN; ++s) {
          F sf[CT][O::HALVES];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) O::state(S[ct], s, sf[ct]);
#pragma unroll
          for (int ti = 0; ti < 4; ++ti) {
            const F c = O::rows_ordered(sm.c[16 * ti + r], s, g);
#pragma unroll
            for (int q = 0; q < O::HALVES; ++q)
#pragma unroll
              for (int ct = 0; ct < CT; ++ct) y[ti][ct] = O::mma(sf[ct][q], c, y[ti][ct]);
          }
        }
      }
      F xf[CT][KL];
      float sum = 0.0f;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int s = 0; s < KL; ++s) {
          xf[ct][s] = O::template columns<0>(&sm.x[0][0], Sh::LX, s, g, r, lcol + 16 * ct);
          if constexpr (!kStates) sum = O::probe(xf[ct][s], sum);
        }
      if constexpr (!kStates) {
        // x that is not finite must not reach earlier tokens through the zeros
        // above the diagonal of P: such columns are summed one by one.
        const bool plain = !__any(sum != 0.0f);
        char* yp = reinterpret_cast<char*>(static_cast<T*>(a.y) +
                                           (static_cast<size_t>(b) * a.T + t0) * xrow);
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) {
          const int i = 16 * ti + r;
          const float eg = __builtin_amdgcn_exp2f(w.gh[i]);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) y[ti][ct] *= eg;
          if (plain) {
            sm.p[hw].multiply(ti, lane, xf, y[ti]);
          } else {
#pragma unroll 1
            for (int k = 0; k < 16 * (ti + 1); ++k) {
              const int j = Tiles<T>::order(k);
              if (j > i) continue;
              const float p =
                  sm.p[hw].value(Tiles<T>::at(ti, j / 16, r + 16 * (j / 4 % 4)) + j % 4);
#pragma unroll
              for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  y[ti][ct][e] += p * to_f32(sm.x[j][lcol + 16 * ct + 4 * g + e]);
            }
          }
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            float xv[4];
            load_row<T, 4>(&sm.x[i][lcol + 16 * ct + 4 * g], xv);
            if (t0 + i < n)
              store4<T>(reinterpret_cast<T*>(yp + 16 * ti * xrow * sizeof(T) + off_y) + 16 * ct,
                        y[ti][ct][0] + dskip * xv[0], y[ti][ct][1] + dskip * xv[1],
                        y[ti][ct][2] + dskip * xv[2], y[ti][ct][3] + dskip * xv[3]);
          }
        }
      }
      const float decay = __builtin_amdgcn_exp2f(w.gh[L - 1]);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int k = 0; k < NTL; ++k) S[ct][k] *= decay;
#pragma unroll
      for (int s = 0; s < KL; ++s) {
        F wx[CT][O::PIECES];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) O::weigh(xf[ct][s], w.w, s, g, wx[ct]);
#pragma unroll
        for (int k = 0; k < NTL; ++k) {
          const F bt = O::template columns<EV>(&sm.b[0][0], Sh::LB, s, g, r, 16 * k);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int q = 0; q < O::PIECES; ++q) S[ct][k] = O::mma(bt, wx[ct][q], S[ct][k]);
        }
      }
      if constexpr (kStates) total += static_cast<double>(w.gh[L - 1]) + w.gl[L - 1];
    }
    __builtin_amdgcn_s_setprio(0);
    if (chunk + 1 < end) {
      rows_of(chunk + 1);  // the other half of sm.rows
      if (chunk + 2 < end) request_dt(chunk + 2);
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
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) to[at(k, e, ct)] = S[ct][k][e];
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
  constexpr int kAhead = 8;  // loads in flight: no store of the loop is read by it
  for (int k0 = 1; k0 < segs; k0 += kAhead) {
    float4 m[kAhead];
    float f[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = min(k0 + i, segs - 1);
      m[i] = starts[k * quads];
      f[i] = decays[k - 1];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float e = __builtin_amdgcn_exp2f(f[i]);
      s = make_float4(e * s.x + m[i].x, e * s.y + m[i].y, e * s.z + m[i].z, e * s.w + m[i].w);
      if (k0 + i < segs) starts[(k0 + i) * quads] = s;
    }
  }
}

struct Cut {
  int cols;        // columns of a workgroup
  int blocks;      // column blocks of a group
  int segs;        // segments of the sequence
  int seg_chunks;  // chunks of a segment
};

// Columns of a workgroup.  128 (two tiles a wave): every operand of B, C and P
// that is read from LDS serves two products, and heads of 64 share G.  64 where
// the group has no more or a head is narrower than two tiles, and for fp32,
// whose operands fill LDS; 32 where the P tiles of four 16-wide heads in fp32
// would not fit.
int block_cols(int width, int P, int io_bf16) {
  if (!io_bf16) return P == 16 ? 32 : 64;
  return width > 64 && P >= 32 ? 128 : 64;
}

Cut cut_of(int B, int T, int G, int H, int P, int io_bf16) {
  Cut c;
  const int width = H / G * P;
  c.cols = block_cols(width, P, io_bf16);
  c.blocks = (width + c.cols - 1) / c.cols;
  const int chunks = (T + L - 1) / L;
  const long long units = static_cast<long long>(B) * G * c.blocks;
  // As many workgroups as the GPU holds at a time, two on each of 256 CUs, and
  // not one more (a second round for a few costs as much as for all); segments
  // of at least 2 chunks, and none below 6, where the first pass and its
  // launches cost more than they save.
  long long segs = 512 / units;
  if (segs > chunks / 2) segs = chunks / 2;
  if (segs < 1 || chunks < 6) segs = 1;
  c.seg_chunks = static_cast<int>((chunks + segs - 1) / segs);
  c.segs = c.seg_chunks > 0 ? (chunks + c.seg_chunks - 1) / c.seg_chunks : 1;
  return c;
}

template <typename T, int N, int HB, int NW, int CT>
hipError_t launch_shape(const SsmArgs& a, const Cut& c, hipStream_t stream) {
  using Full = Shape<T, N, HB, NW, CT, false>;
  using States = Shape<T, N, HB, NW, CT, true>;
  static_assert(sizeof(Full) <= 160 * 1024, "LDS of a workgroup");
  const unsigned units = static_cast<unsigned>(a.B) * a.G * c.blocks;
  if (c.segs > 1) {
    hipLaunchKernelGGL((ssm_chunk_kernel<T, N, HB, NW, CT, true>), dim3(units * (c.segs - 1)),
                       dim3(States::NT), sizeof(States), stream, a, c.blocks, c.segs,
                       c.seg_chunks);
    if (starts_joined(a, c.segs)) {
      const size_t quads = static_cast<size_t>(a.B) * a.H * a.N * a.P / 4;
      hipLaunchKernelGGL(ssm_start_kernel, dim3(static_cast<unsigned>((quads + 255) / 256)),
                         dim3(256), 0, stream, a, c.segs);
    }
  }
  hipLaunchKernelGGL((ssm_chunk_kernel<T, N, HB, NW, CT, false>), dim3(units * c.segs),
                     dim3(Full::NT), sizeof(Full), stream, a, c.blocks, c.segs, c.seg_chunks);
  return hipGetLastError();
}

template <typename T, int N>
hipError_t launch_n(const SsmArgs& a, const Cut& c, hipStream_t stream) {
  if constexpr (sizeof(T) == 4) {
    if (a.P >= 64) return launch_shape<T, N, 1, 4, 1>(a, c, stream);
    if (a.P == 32) return launch_shape<T, N, 2, 4, 1>(a, c, stream);
    return launch_shape<T, N, 2, 2, 1>(a, c, stream);
  } else {
    if (c.cols == 128) {
      if (a.P == 128) return launch_shape<T, N, 1, 4, 2>(a, c, stream);
      if (a.P == 64) return launch_shape<T, N, 2, 4, 2>(a, c, stream);
      return launch_shape<T, N, 4, 4, 2>(a, c, stream);
    }
    if (a.P >= 64) return launch_shape<T, N, 1, 4, 1>(a, c, stream);
    if (a.P == 32) return launch_shape<T, N, 2, 4, 1>(a, c, stream);
    return launch_shape<T, N, 4, 4, 1>(a, c, stream);
  }
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
