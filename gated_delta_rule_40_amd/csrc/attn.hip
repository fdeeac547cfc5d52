// attn.hip -- softmax attention of new tokens over the 8-bit cache for gfx950.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp2(z_j - m),
//   z_j = scale log2(e) q . k_j,  m the running maximum over j
//
// in one pass over the keys.  The query heads that share a kv head and the
// new tokens of a row form one list of query rows (row t * group + h'), cut
// into tiles of 16; a wave takes MT tiles and walks the keys 64 at a time.
//
// Both products run transposed on 16x16x32 bf16 matrix instructions,
//   S^T = K Q^T,  O^T = V^T P^T,
// with the operand order chosen so that nothing passes through LDS:
//   * a lane of S^T holds 4 consecutive keys of one query row.  Which key a
//     row of the K operand is, is free: row r of tile t takes key
//     16 (r / 4) + 4 t + r % 4, so that lane group g ends up with keys
//     16 g ... 16 g + 15 over the four tiles -- as the P^T operand of the
//     second product, which takes 8 keys a lane, wants them;
//   * a lane of the V^T operand then reads those 16 keys of one row of the
//     transposed value page, 16 bytes; a lane of the K operand reads D/4
//     consecutive bytes of a key (the contraction index is permuted alike in
//     Q).  All loads go from the pages straight to registers.
// e4m3 values are exact in bf16.  The key scales join the score scale, the
// value scales (powers of two) multiply p.  p itself is split into bf16
// pieces, two for bf16 io and three, like q, for fp32 io, so that its rounding
// stays far below the output's own (one piece would be a second rounding of that
// size: 1024 queries over up to 3500 keys 70.7 instead of 82.4 us, but off by
// 1.82e-3 of the norm where the output's rounding alone is 1.65e-3).
//
// Two kernels.  With few query rows (attn_few_kernel, the order above) the
// waves of a workgroup share the keys and join in LDS: bound by HBM, one byte a
// cached element.  With many (attn_rows_kernel) each wave takes its own rows,
// the workgroup's waves read the same keys, and a step's keys and values are
// converted once, with their scales, into LDS: bound by the matrix and
// exponential pipes.  Where that gives too few workgroups, the keys are also
// cut into splits over workgroups, whose partial sums attn_join_kernel joins.
#include <type_traits>

#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"
#include "kv_device.hpp"

namespace gdr {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
// Query rows of a workgroup of attn_rows_kernel.
template <int MT>
constexpr int kRowsBlock = 16 * MT * (kThreads / 64);
constexpr int kTile = 64;  // keys per step
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 8.0f;  // how far (log2) a reference may lag behind the maximum

// Eight e4m3 codes as bf16, times a power of two (exact).
__device__ __forceinline__ bf16x8_t codes_to_bf16(unsigned w0, unsigned w1, float scale = 1.0f) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ unsigned word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// 1.0 in bf16 where a code is NaN, else 0.
__device__ __forceinline__ bf16x8_t nan_codes(unsigned w0, unsigned w1) {
  bf16x8_t r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned c = ((i < 4 ? w0 : w1) >> (8 * (i & 3))) & 0x7fu;
    r[i] = static_cast<bf16>(c == 0x7fu ? 1.0f : 0.0f);
  }
  return r;
}
__device__ __forceinline__ unsigned without_nan(unsigned w) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (((w >> (8 * i)) & 0x7fu) == 0x7fu) w &= ~(0xffu << (8 * i));
  return w;
}

// x as PIECES bf16 values that add up to it.
template <int PIECES>
__device__ __forceinline__ void split(float x, bf16 (&out)[PIECES]) {
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    out[i] = static_cast<bf16>(x);
    x -= static_cast<float>(out[i]);
  }
}

// Eight p's as PIECES matrix operands.  All but the last piece are cut off rather
// than rounded (the upper halves of two words are one byte permutation): three
// pieces of eight bits hold a float whole, of two 2^-16 is lost.
template <int PIECES>
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, bf16x8_t (&out)[PIECES]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
  u32x4_t w[PIECES];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x = i < 2 ? a[2 * i] : b[2 * i - 4], y = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
#pragma unroll
    for (int k = 0; k + 1 < PIECES; ++k) {
      const unsigned ux = __builtin_bit_cast(unsigned, x), uy = __builtin_bit_cast(unsigned, y);
      w[k][i] = __builtin_amdgcn_perm(uy, ux, 0x07060302u);
      x -= __builtin_bit_cast(float, ux & 0xffff0000u);
      y -= __builtin_bit_cast(float, uy & 0xffff0000u);
    }
    w[PIECES - 1][i] =
        __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x, y}), bf16x2_t));
  }
#pragma unroll
  for (int k = 0; k < PIECES; ++k) out[k] = __builtin_bit_cast(bf16x8_t, w[k]);
}

// The keys that query rows row0 ... row0 + rows - 1 of batch row b attend to:
// the first one's and the last one's count (rows behind the end left out).
struct Span {
  int lo, hi;
};
__device__ __forceinline__ int key_limit(const KvArgs& a, int b, int t) {
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  const long long k = min(static_cast<long long>(a.pos[b]) + t + 1, cap);
  return a.n_pages > 0 && k > 0 ? static_cast<int>(k) : 0;
}
__device__ __forceinline__ int tokens_of(const KvArgs& a, int b) {
  return a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
}

// Steps of a split: at least kMinSteps, so that short rows use few splits.
constexpr int kMinSteps = 4;
constexpr int kMaxSplits = 64;
__device__ __forceinline__ int split_steps(int steps, int splits) {
  return max(kMinSteps, (steps + splits - 1) / splits);
}

// Partial sums of a query row: splits x D accumulators, then splits x (m, l).
struct Partial {
  float* acc;
  float* ml;
};
__device__ __forceinline__ Partial partial_of(const KvArgs& a, int splits, size_t row) {
  float* base = static_cast<float*>(a.ws);
  const size_t rows = static_cast<size_t>(a.B) * a.T * a.H_q;
  return {base + row * splits * a.D, base + rows * splits * a.D + row * splits * 2};
}

template <typename T, int D, int NW>
__global__ __launch_bounds__(64 * NW) void attn_few_kernel(KvArgs a, int row_blocks, int splits) {
  constexpr int QP = sizeof(T) == 4 ? 3 : 1;  // pieces of q
  constexpr int PP = sizeof(T) == 4 ? 3 : 2;  // pieces of p
  constexpr int KS = D / 32;                  // contraction steps of S^T
  constexpr int KW = D / 64;                  // 16-byte loads of a lane's key slice
  constexpr int DT = D / 16;                  // row tiles of O^T
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;

  // Workgroups of one (row, kv head) are B * H_kv apart.
  const int bh = blockIdx.x % (a.B * a.H_kv);
  const int rest = blockIdx.x / (a.B * a.H_kv);
  const int b = bh / a.H_kv, head = bh % a.H_kv;
  const int part = rest % splits;
  const int block = row_blocks - 1 - rest / splits;  // longest first
  const int group = a.H_q / a.H_kv;
  const int* table = a.block_table + static_cast<size_t>(b) * a.max_pages;
  const int page_shift = __builtin_ctz(a.page);
  // The page of a 16-key group of step s, or -1.
  auto page_of = [&](int s, int grp) {
    const int at = (s * kTile + 16 * grp) >> page_shift;
    const int id = at < a.max_pages ? table[at] : -1;
    return id >= 0 && id < a.n_pages ? id : -1;
  };
  const int ka = r >> 2;  // the group of this lane's keys in the K operand
  uint4 kr[4][KW], vr[DT];
  auto load_k = [&](int s, int id) {
    const int slot = (s * kTile + 16 * ka + (r & 3)) & (a.page - 1);
    const uint8_t* p = a.k_cache +
                       ((static_cast<size_t>(max(id, 0)) * a.H_kv + head) * a.page + slot) * D +
                       g * (D / 4);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int w = 0; w < KW; ++w)
        kr[t][w] = *reinterpret_cast<const uint4*>(p + 4 * t * D + 16 * w);
  };
  auto load_v = [&](int s, int id) {
    const int slot = (s * kTile + 16 * g) & (a.page - 1);
    const uint8_t* p = a.v_cache +
                       ((static_cast<size_t>(max(id, 0)) * a.H_kv + head) * D + r) * a.page + slot;
#pragma unroll
    for (int d = 0; d < DT; ++d)
      vr[d] = *reinterpret_cast<const uint4*>(p + static_cast<size_t>(16 * d) * a.page);
  };

  // Without splits a wave's first step does not depend on the row's length: its
  // pages are looked up and its loads issued while that is on its way (a step
  // past the end is not used).
  int step = wave;
  int idk = -1, idv = -1;
  if (splits == 1 && a.n_pages > 0) {
    idk = page_of(step, ka);
    idv = page_of(step, g);
    load_k(step, idk);
  }

  const int n = tokens_of(a, b);
  const int row0 = block * 16;
  if (row0 >= n * group) return;
  const int last = min(row0 + 16, n * group) - 1;
  const Span span{key_limit(a, b, row0 / group), key_limit(a, b, last / group)};

  const int steps = (span.hi + kTile - 1) / kTile;
  const int per = split_steps(steps, splits);
  const int s_end = min((part + 1) * per, steps);
  if (splits > 1) step = part * per + wave;
  if (splits > 1 && part * per >= steps && part > 0) return;  // not read by the join

  // This lane's query row: column r.
  bf16x8_t q[QP][KS];
  const bool on = row0 + r <= last;
  const int tok = on ? (row0 + r) / group : 0;
  const int lim = on ? key_limit(a, b, tok) : 0;
  const T* src = static_cast<const T*>(a.q) +
                 ((static_cast<size_t>(b) * a.T + tok) * a.H_q + head * group +
                  (on ? (row0 + r) % group : 0)) * D + g * (D / 4);
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    float x[8];
    load_row<T, 8>(src + 8 * s, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bf16 p[QP];
      split<QP>(x[i], p);
#pragma unroll
      for (int c = 0; c < QP; ++c) q[c][s][i] = p[c];
    }
  }

  f32x4 acc[DT];
  float mx = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (splits > 1 && step < s_end) {
    idk = page_of(step, ka);
    idv = page_of(step, g);
    load_k(step, idk);
  }
  for (; step < s_end; step += NW) {
    load_v(step, idv);
    const size_t ph = static_cast<size_t>(max(idv, 0)) * a.H_kv + head;
    const float ks = a.k_scale[ph] * (a.scale * kLog2e);
    float vs = a.v_scale[ph];
    const int next = step + NW;
    int idk2 = -1, idv2 = -1;
    if (next < s_end) {
      idk2 = page_of(next, ka);
      idv2 = page_of(next, g);
    }

    f32x4 z[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      z[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const bf16x8_t k =
            codes_to_bf16(word(kr[t][s / 2], 2 * (s & 1)), word(kr[t][s / 2], 2 * (s & 1) + 1));
#pragma unroll
        for (int c = 0; c < QP; ++c)
          z[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[c][s], z[t], 0, 0, 0);
      }
    }
    if (next < s_end) load_k(next, idk2);

    // Every key of the step is there and in sight of every row?
    const int key0 = step * kTile + 16 * g;
    const bool whole = (step + 1) * kTile <= span.lo && __all(idv >= 0);
    const bool group_on = idv >= 0 && key0 < span.hi;
    if (!whole && !group_on) vs = 0.0f;
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = z[t][e] * ks;
        if (!whole && !(group_on && key0 + 4 * t + e < lim)) x = -INFINITY;
        z[t][e] = x;
        top = fmaxf(top, x);
      }
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float now = fmaxf(mx, top);
    if (__any(now > mx)) {
      const float back = __builtin_amdgcn_exp2f(mx - (now == -INFINITY ? 0.0f : now));
      sum *= back;
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[d] *= back;
      mx = now;
    }
    const float ref = now == -INFINITY ? 0.0f : now;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = __builtin_amdgcn_exp2f(z[t][e] - ref);
        sum += p;
        z[t][e] = p * vs;
      }

    bool has_nan = false;
    if (!whole) {
      // Codes behind the last key, or of no page, count as zeros; NaN codes of
      // keys that only some rows see are taken out and added to those rows.
      const int keep = group_on ? min(span.hi - key0, 16) : 0;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        unsigned w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int bytes = min(max(keep - 4 * i, 0), 4);
          w[i] = bytes == 4 ? word(vr[d], i) : word(vr[d], i) & ((1u << (8 * bytes)) - 1);
          has_nan |= without_nan(w[i]) != w[i];
        }
        vr[d] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      has_nan = __any(has_nan);
    }

#pragma unroll
    for (int u = 0; u < 2; ++u) {
      bf16x8_t p[PP];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bf16 c[PP];
        split<PP>(z[2 * u + i / 4][i & 3], c);
#pragma unroll
        for (int k = 0; k < PP; ++k) p[k][i] = c[k];
      }
      if (has_nan) {
        // The keys in sight, whatever their p: it may be too small for its type.
        bf16x8_t see;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          see[i] = static_cast<bf16>(
              group_on && key0 + 4 * (2 * u + i / 4) + (i & 3) < lim ? 1.0f : 0.0f);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const bf16x8_t bad = nan_codes(word(vr[d], 2 * u), word(vr[d], 2 * u + 1));
          const f32x4 hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              bad, see, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (hit[e] > 0.0f) acc[d][e] = NAN;
          const unsigned c0 = without_nan(word(vr[d], 2 * u));
          const unsigned c1 = without_nan(word(vr[d], 2 * u + 1));
          vr[d] = u == 0 ? make_uint4(c0, c1, vr[d].z, vr[d].w) : make_uint4(vr[d].x, vr[d].y, c0, c1);
        }
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const unsigned w0 = word(vr[d], 2 * u), w1 = word(vr[d], 2 * u + 1);
        const bf16x8_t v = codes_to_bf16(w0, w1);
#pragma unroll
        for (int k = 0; k < PP; ++k)
          acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[k], acc[d], 0, 0, 0);
      }
    }
    idk = idk2;
    idv = idv2;
  }
  sum += __shfl_xor(sum, 16, 64);
  sum += __shfl_xor(sum, 32, 64);

  // Join the waves' sums: every wave leaves its own in LDS, then 16 threads
  // share a row.
  constexpr int LD = D + 4;
  __shared__ float acc_s[NW][16][LD], ml_s[NW][16][2];
#pragma unroll
  for (int d = 0; d < DT; ++d)
    *reinterpret_cast<f32x4*>(&acc_s[wave][r][16 * d + 4 * g]) = acc[d];
  if (g == 0) {
    ml_s[wave][r][0] = mx;
    ml_s[wave][r][1] = sum;
  }
  __syncthreads();
  // Threads past the first 256 have no part in it.
  const int row = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * (D / 16);
  if (row >= 16 || row0 + row > last) return;
  float top = -INFINITY, tot = 0.0f, out[D / 16] = {};
#pragma unroll
  for (int w = 0; w < NW; ++w) top = fmaxf(top, ml_s[w][row][0]);
  const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const float f = __builtin_amdgcn_exp2f(ml_s[w][row][0] - ref);
    tot += f * ml_s[w][row][1];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) out[i] += f * acc_s[w][row][c0 + i];
  }
  const int qrow = row0 + row;
  const size_t at =
      (static_cast<size_t>(b) * a.T + qrow / group) * a.H_q + head * group + qrow % group;
  if (splits > 1) {
    const Partial p = partial_of(a, splits, at);
#pragma unroll
    for (int i = 0; i < D / 16; i += 4)
      store4<float>(p.acc + part * D + c0 + i, out[i], out[i + 1], out[i + 2], out[i + 3]);
    if (c0 == 0) {
      p.ml[2 * part] = top;
      p.ml[2 * part + 1] = tot;
    }
    return;
  }
  const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;  // NaN stays
#pragma unroll
  for (int i = 0; i < D / 16; i += 4)
    store4<T>(static_cast<T*>(a.o) + at * D + c0 + i, out[i] * inv, out[i + 1] * inv,
              out[i + 2] * inv, out[i + 3] * inv);
}

// A step's keys and values in LDS, in bf16 with their scales: keys as rows of D
// channels; values as rows (channels) of 64 tokens, each 32 tokens in the order
// in which a lane group takes 8 of them (4 g ... and 16 + 4 g ...).  The pitches
// keep 16-byte reads of 16 rows on distinct banks.
template <int D>
struct Tile {
  bf16 k[kTile][D + 8];
  bf16 v[D][kTile + 8];
};

// MT tiles of 16 query rows a wave, four waves.
template <typename T, int D, int MT>
__global__ __launch_bounds__(kThreads, 2) void attn_rows_kernel(KvArgs a, int row_blocks,
                                                                int splits) {
  constexpr int QP = sizeof(T) == 4 ? 3 : 1;
  constexpr int PP = sizeof(T) == 4 ? 3 : 2;
  constexpr int KS = D / 32, DT = D / 16;
  constexpr int LW = D / 64;  // 16-byte loads of a thread, of keys and of values
  __shared__ __attribute__((aligned(16))) Tile<D> tiles[2];
  __shared__ __attribute__((aligned(16))) int groups_on[2][kThreads / 64];
  __shared__ unsigned long long nan_s[2][D];  // tokens of a step with NaN in a value channel
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;

  const int bh = blockIdx.x % (a.B * a.H_kv);
  const int rest = blockIdx.x / (a.B * a.H_kv);
  const int b = bh / a.H_kv, head = bh % a.H_kv;
  const int part = rest % splits;
  const int block = row_blocks - 1 - rest / splits;  // longest first
  const int group = a.H_q / a.H_kv;
  const int n = tokens_of(a, b);
  const int block0 = block * kRowsBlock<MT>;
  if (block0 >= n * group) return;
  const int block_last = min(block0 + kRowsBlock<MT>, n * group) - 1;
  const Span all{key_limit(a, b, block0 / group), key_limit(a, b, block_last / group)};
  const int steps = (all.hi + kTile - 1) / kTile;
  const int per = split_steps(steps, splits);
  const int s_end = min((part + 1) * per, steps);
  int step = part * per;
  if (step >= steps && part > 0) return;  // not read by the join

  // The wave's rows: one column of S^T a lane and tile.
  const int row0 = block0 + wave * 16 * MT;
  const int last = min(row0 + 16 * MT - 1, block_last);
  const Span span{row0 <= last ? key_limit(a, b, row0 / group) : 0,
                  row0 <= last ? key_limit(a, b, last / group) : 0};
  // exp2(c z - c m): c >= 0, the sign of the score scale goes to q; c = 0 would
  // lose masked keys' -inf.
  const float c = fmaxf(__builtin_fabsf(a.scale) * kLog2e, 1e-30f);
  const float sign = a.scale < 0.0f ? -1.0f : a.scale == a.scale ? 1.0f : a.scale;  // NaN stays
  int lim[MT];
  size_t orow[MT];
  bf16x8_t q[MT][QP][KS];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = row0 + 16 * m + r;
    const bool on = row <= last;
    const int t = on ? row / group : 0;
    lim[m] = on ? key_limit(a, b, t) : 0;
    orow[m] = (static_cast<size_t>(b) * a.T + t) * a.H_q + head * group + (on ? row % group : 0);
    const T* src = static_cast<const T*>(a.q) + orow[m] * D + 8 * g;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float x[8];
      load_row<T, 8>(src + 32 * s, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bf16 p[QP];
        split<QP>(sign * x[i], p);
#pragma unroll
        for (int k = 0; k < QP; ++k) q[m][k][s][i] = p[k];
      }
    }
  }

  // Staging: a wave loads 16 neighbouring keys of each step, all of one page, and
  // their values.  The page, its scales and the bases are scalar; lane offsets
  // do not change: 16 KW bytes of key lane / 4, and 16 tokens of channels lane,
  // lane + 64.
  const int* table = a.block_table + static_cast<size_t>(b) * a.max_pages;
  const int page_shift = __builtin_ctz(a.page);
  auto page_of = [&](int s) {
    const int at = (s * kTile + 16 * wave) >> page_shift;
    const int id = at < a.max_pages ? table[at] : -1;
    return __builtin_amdgcn_readfirstlane(id >= 0 && id < a.n_pages ? id : -1);
  };
  const int kt = 16 * wave + lane / 4, kc = lane % 4 * 16 * LW;
  const unsigned koff = lane / 4 * D + kc, voff = lane * a.page;
  u32x4 kr[LW], vr[LW];
  float ksc = 1.0f, vsc = 1.0f;
  int id_now = -1, id_next = -1;
  auto request = [&](int s) {
    id_now = id_next;
    const size_t ph = static_cast<size_t>(max(id_now, 0)) * a.H_kv + head;
    const int slot = (s * kTile + 16 * wave) & (a.page - 1);
    const uint8_t* kp = a.k_cache + (ph * a.page + slot) * D;
    const uint8_t* vp = a.v_cache + ph * D * a.page + slot;
    ksc = a.k_scale[ph];
    vsc = a.v_scale[ph];
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      kr[i] = *reinterpret_cast<const u32x4*>(kp + koff + 16 * i);
      vr[i] = *reinterpret_cast<const u32x4*>(vp + 64 * i * a.page + voff);
    }
  };

  f32x4 acc[MT][DT];
  float mx[MT], sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mx[m] = -INFINITY;
    sum[m] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  if (step < s_end) {
    id_next = page_of(step);
    request(step);
    if (step + 1 < s_end) id_next = page_of(step + 1);
  }
#pragma unroll 1
  for (; step < s_end; ++step) {
    Tile<D>& tile = tiles[step & 1];
    const bool block_whole = (step + 1) * kTile <= all.lo;
    bool odd = false;
    float vs = vsc;
    if (id_now < 0) {
      // No page: the loads took page 0, whose codes and scale may be anything,
      // and p = 0 would not take NaN out of the product.
      vs = 1.0f;
#pragma unroll
      for (int i = 0; i < LW; ++i) vr[i] = u32x4{0u, 0u, 0u, 0u};
    }
    if (!block_whole) {
      // A step that some rows see in part.  Codes behind the last key count as
      // zeros.  NaN must not reach the rows that do not see its key through
      // p = 0: it is taken out and noted, a bit for each token.
      const int keep = min(max(all.hi - step * kTile - 16 * wave, 0), 16);
      if (keep == 0) vs = 1.0f;
#pragma unroll
      for (int i = 0; i < LW; ++i) {
        unsigned at = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int bytes = min(max(keep - 4 * k, 0), 4);
          if (bytes < 4) vr[i][k] &= (1u << (8 * bytes)) - 1;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((vr[i][k] >> (8 * j) & 0x7fu) == 0x7fu) at |= 1u << (4 * k + j);
          vr[i][k] = without_nan(vr[i][k]);
        }
        reinterpret_cast<uint16_t*>(&nan_s[step & 1][lane + 64 * i])[wave] =
            static_cast<uint16_t>(at);
        odd |= at != 0;
      }
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      *reinterpret_cast<bf16x8_t*>(&tile.k[kt][kc + 16 * i]) = codes_to_bf16(kr[i][0], kr[i][1], ksc);
      *reinterpret_cast<bf16x8_t*>(&tile.k[kt][kc + 16 * i + 8]) =
          codes_to_bf16(kr[i][2], kr[i][3], ksc);
      const bf16x8_t v0 = codes_to_bf16(vr[i][0], vr[i][1], vs);
      const bf16x8_t v1 = codes_to_bf16(vr[i][2], vr[i][3], vs);
      bf16* vp = &tile.v[lane + 64 * i][32 * (wave / 2) + 4 * (wave & 1)];
      *reinterpret_cast<bf16x4_t*>(vp) = bf16x4_t{v0[0], v0[1], v0[2], v0[3]};
      *reinterpret_cast<bf16x4_t*>(vp + 8) = bf16x4_t{v0[4], v0[5], v0[6], v0[7]};
      *reinterpret_cast<bf16x4_t*>(vp + 16) = bf16x4_t{v1[0], v1[1], v1[2], v1[3]};
      *reinterpret_cast<bf16x4_t*>(vp + 24) = bf16x4_t{v1[4], v1[5], v1[6], v1[7]};
    }
    if (lane == 0) groups_on[step & 1][wave] = id_now >= 0;
    bool has_nan = false;
    if (block_whole)
      __syncthreads();
    else
      has_nan = __builtin_amdgcn_readfirstlane(__syncthreads_or(odd));
    if (step + 1 < s_end) {
      request(step + 1);
      if (step + 2 < s_end) id_next = page_of(step + 2);
    }
    if (step * kTile >= span.hi) continue;  // nothing here for this wave's rows

    f32x4 z[MT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int m = 0; m < MT; ++m) z[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const bf16x8_t k = *reinterpret_cast<const bf16x8_t*>(&tile.k[16 * t + r][32 * s + 8 * g]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int p = 0; p < QP; ++p)
            z[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[m][p][s], z[m][t], 0, 0, 0);
      }
    }
    // Scalar, so that whole steps branch past the masks.
    int on[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) on[t] = __builtin_amdgcn_readfirstlane(groups_on[step & 1][t]);
    const bool whole = (step + 1) * kTile <= span.lo && (on[0] & on[1] & on[2] & on[3]);
    if (!whole) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(on[t] && step * kTile + 16 * t + 4 * g + e < lim[m])) z[m][t][e] = -INFINITY;
    }
    float now[MT];
    bool far = false;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, z[m][t][e]);
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      now[m] = fmaxf(mx[m], top);
      far |= (now[m] - mx[m]) * c > kSlack;
    }
    // mx is the running maximum or up to 2^kSlack (of p) below it: moving it
    // rescales everything, and with 32 rows a wave some row's maximum moves in
    // most steps.
    if (__any(far)) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float back = __builtin_amdgcn_exp2f(
            __builtin_fmaf(mx[m], c, now[m] == -INFINITY ? 0.0f : -now[m] * c));
        sum[m] *= back;
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[m][d] *= back;
        mx[m] = now[m];
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float ref = mx[m] == -INFINITY ? 0.0f : mx[m] * c;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(z[m][t][e], c, -ref));
          sum[m] += x;
          z[m][t][e] = x;
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      bf16x8_t p[MT][PP];
#pragma unroll
      for (int m = 0; m < MT; ++m) split8<PP>(z[m][2 * u], z[m][2 * u + 1], p[m]);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const bf16x8_t v =
            *reinterpret_cast<const bf16x8_t*>(&tile.v[16 * d + r][32 * u + 8 * g]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int k = 0; k < PP; ++k)
            acc[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[m][k], acc[m][d], 0, 0, 0);
      }
    }
    if (has_nan) {
      // A row that sees a key with NaN in a channel gets NaN there.  (The empty
      // statement keeps this a branch: as selects it would run in every step.)
      asm volatile("" ::: "memory");
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int seen = min(max(lim[m] - step * kTile, 0), kTile);
        unsigned long long vis = seen == kTile ? ~0ull : (1ull << seen) - 1;
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (!on[t]) vis &= ~(0xffffull << (16 * t));
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (nan_s[step & 1][16 * d + 4 * g + e] & vis) acc[m][d][e] = NAN;
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    sum[m] += __shfl_xor(sum[m], 16, 64);
    sum[m] += __shfl_xor(sum[m], 32, 64);
    if (row0 + 16 * m + r > last) continue;
    if (splits > 1) {
      const Partial o = partial_of(a, splits, orow[m]);
#pragma unroll
      for (int d = 0; d < DT; ++d)
        store4<float>(o.acc + part * D + 16 * d + 4 * g, acc[m][d][0], acc[m][d][1], acc[m][d][2],
                      acc[m][d][3]);
      if (g == 0) {
        o.ml[2 * part] = mx[m] * c;
        o.ml[2 * part + 1] = sum[m];
      }
      continue;
    }
    const float inv = sum[m] == 0.0f ? 0.0f : 1.0f / sum[m];
#pragma unroll
    for (int d = 0; d < DT; ++d)
      store4<T>(static_cast<T*>(a.o) + orow[m] * D + 16 * d + 4 * g, acc[m][d][0] * inv,
                acc[m][d][1] * inv, acc[m][d][2] * inv, acc[m][d][3] * inv);
  }
}

// Joins the splits of a query row, LANES lanes a row.  The loads of a row hang
// on each other (length, splits, maxima, sums).  Where the rows alone fill the
// GPU, 16 lanes put four rows of a wave under way together: 32768 rows of two
// splits 8.7 us, at one row a wave 18.4; few rows of many splits (32 of 64)
// want a whole wave each, 4 us less.
template <typename T, int D, int LANES>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(KvArgs a, int block_rows,
                                                             int splits) {
  constexpr int COLS = D / LANES;
  constexpr int kMost = kMaxSplits / LANES;  // splits whose maximum a lane holds
  const int l = threadIdx.x % LANES;
  const size_t at = static_cast<size_t>(blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES;
  if (at >= static_cast<size_t>(a.B) * a.T * a.H_q) return;
  const int hq = at % a.H_q;
  const int t = at / a.H_q % a.T, b = at / a.H_q / a.T;
  const int n = tokens_of(a, b);
  if (t >= n) return;
  const int group = a.H_q / a.H_kv;
  // The keys of the block of rows that this row was computed in.
  const int row = t * group + hq % group;
  const int last = min((row / block_rows + 1) * block_rows, n * group) - 1;
  const int steps = (key_limit(a, b, last / group) + kTile - 1) / kTile;
  const int per = split_steps(steps, splits);
  const int used = max(1, (steps + per - 1) / per);

  const Partial p = partial_of(a, splits, at);
  float f[kMost], tot = 0.0f, top = -INFINITY;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int s = LANES * k + l;
    f[k] = s < used ? p.ml[2 * s] : -INFINITY;
    top = fmaxf(top, f[k]);
  }
#pragma unroll
  for (int o = 1; o < LANES; o *= 2) top = fmaxf(top, __shfl_xor(top, o, 64));
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int s = LANES * k + l;
    f[k] = s < used ? __builtin_amdgcn_exp2f(f[k] - (top == -INFINITY ? 0.0f : top)) : 0.0f;
    if (s < used) tot += f[k] * p.ml[2 * s + 1];
  }
  tot = LANES == 16 ? row16_sum(tot) : wave_sum(tot);

  float out[COLS] = {};
  constexpr int kAhead = 8;  // splits requested together
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    for (int s0 = LANES * k; s0 < min(used, LANES * (k + 1)); s0 += kAhead) {
      float x[kAhead][COLS];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        load_row<float, COLS>(p.acc + min(s0 + i, used - 1) * D + l * COLS, x[i]);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float w = __shfl(f[k], (s0 + i) % LANES, LANES);  // 0 past the last split
        if (s0 + i < used)
#pragma unroll
          for (int c = 0; c < COLS; ++c) out[c] += w * x[i][c];
      }
    }
  }
  const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
#pragma unroll
  for (int c = 0; c < COLS; ++c)
    static_cast<T*>(a.o)[at * D + l * COLS + c] = from_f32<T>(out[c] * inv);
}

// How a call is cut.
struct Plan {
  bool few;        // the waves of a workgroup share one tile of 16 rows
  int waves;       // of a workgroup
  int block_rows;  // query rows of a workgroup
  int row_blocks;  // workgroups over the rows of a (batch row, kv head)
  int splits;      // workgroups over the keys
};

Plan plan_of(const KvArgs& a, int io_bf16) {
  const long long rows = static_cast<long long>(a.T) * (a.H_q / a.H_kv);
  const long long steps = (static_cast<long long>(a.max_pages) * a.page + kTile - 1) / kTile;
  Plan p;
  // Up to 64 rows go 16 to a workgroup, each reading all keys again; more share
  // them.  Groups of 4 heads of 128, 64 rows against sharing: 16 requests of 2000 to
  // 4000 keys 58 against 67 us, 64 of 1500 to 3000 163 against 153; 96 rows 85
  // against 69 and 231 against 155 (one request 15.5 against 20.7).
  p.few = rows <= 64;
  p.waves = 4;
  p.block_rows = p.few ? 16 : io_bf16 ? kRowsBlock<2> : kRowsBlock<1>;
  p.row_blocks = static_cast<int>((rows + p.block_rows - 1) / p.block_rows);
  const long long base = static_cast<long long>(a.B) * a.H_kv * p.row_blocks;
  // Short tables over few rows: eight waves and no splits, so that one launch
  // does it all.
  if (p.few && steps <= 16 && base <= 256) {
    p.waves = 8;
    p.splits = 1;
    return p;
  }
  // As many workgroups as the GPU holds at a time (two on each of 256 CUs), as
  // far as the table's keys allow: with twice as many, 64 rows of 4096 to 8192
  // keys take 171 us instead of 162, 16 rows of 2000 to 4000 35 instead of 29.
  const long long want = 512 / base;
  const long long most = steps / kMinSteps;
  p.splits = static_cast<int>(min(want, most));
  if (p.splits > kMaxSplits) p.splits = kMaxSplits;
  if (p.splits < 1) p.splits = 1;
  return p;
}

template <typename T, int D>
hipError_t launch_d(const KvArgs& a, hipStream_t stream) {
  const Plan p = plan_of(a, sizeof(T) == 2);
  const dim3 grid(static_cast<unsigned>(a.B) * a.H_kv * p.row_blocks * p.splits);
  constexpr int MT = sizeof(T) == 2 ? 2 : 1;
  if (!p.few)
    hipLaunchKernelGGL((attn_rows_kernel<T, D, MT>), grid, dim3(kThreads), 0, stream, a,
                       p.row_blocks, p.splits);
  else if (p.waves == 8)
    hipLaunchKernelGGL((attn_few_kernel<T, D, 8>), grid, dim3(512), 0, stream, a, p.row_blocks,
                       p.splits);
  else
    hipLaunchKernelGGL((attn_few_kernel<T, D, 4>), grid, dim3(256), 0, stream, a, p.row_blocks,
                       p.splits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const size_t rows = static_cast<size_t>(a.B) * a.T * a.H_q;
  if (rows > 8192)  // 8 waves on every SIMD at one row each
    hipLaunchKernelGGL((attn_join_kernel<T, D, 16>), dim3(static_cast<unsigned>((rows + 15) / 16)),
                       dim3(kThreads), 0, stream, a, p.block_rows, p.splits);
  else
    hipLaunchKernelGGL((attn_join_kernel<T, D, 64>), dim3(static_cast<unsigned>((rows + 3) / 4)),
                       dim3(kThreads), 0, stream, a, p.block_rows, p.splits);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const KvArgs& a, hipStream_t stream) {
  return a.D == 64 ? launch_d<T, 64>(a, stream) : launch_d<T, 128>(a, stream);
}

}  // namespace

size_t attn_workspace_bytes(const KvArgs& a, int io_bf16) {
  const Plan p = plan_of(a, io_bf16);
  if (p.splits == 1) return 0;
  return static_cast<size_t>(a.B) * a.T * a.H_q * p.splits * (a.D + 2) * sizeof(float);
}

hipError_t launch_attn(const KvArgs& a, int io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_t<bf16>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace gdr
