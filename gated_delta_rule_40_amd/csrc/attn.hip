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
// pieces: two for bf16 io (2^-17 of it is lost, far below the output's own
// rounding), three, like q, for fp32 io (2^-25).
//
// Bound by HBM for few query rows (one byte a cached element), by the matrix
// and conversion pipes for prompts.  With few rows the waves of a workgroup
// share the keys and join in LDS (kShare); with many each takes its own rows.
// Where that gives too few workgroups, the keys are also cut into splits over
// workgroups, whose partial sums attn_join_kernel joins.
#include <type_traits>

#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"
#include "kv_device.hpp"

namespace gdr {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kTile = 64;  // keys per step
constexpr float kLog2e = 1.44269504088896340736f;

// Eight e4m3 codes as bf16 (exact).
__device__ __forceinline__ bf16x8_t codes_to_bf16(unsigned w0, unsigned w1) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
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

template <typename T, int D, int MT, bool kShare>
__global__ __launch_bounds__(kThreads) void attn_kernel(KvArgs a, int row_blocks, int splits) {
  constexpr int QP = sizeof(T) == 4 ? 3 : 1;  // pieces of q
  constexpr int PP = sizeof(T) == 4 ? 3 : 2;  // pieces of p
  constexpr int KS = D / 32;                  // contraction steps of S^T
  constexpr int KW = D / 64;                  // 16-byte loads of a lane's key slice
  constexpr int DT = D / 16;                  // row tiles of O^T
  constexpr int kWaves = kThreads / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;

  // Workgroups of one (row, kv head) are B * H_kv apart.
  const int bh = blockIdx.x % (a.B * a.H_kv);
  const int rest = blockIdx.x / (a.B * a.H_kv);
  const int b = bh / a.H_kv, head = bh % a.H_kv;
  const int part = rest % splits;
  const int block = row_blocks - 1 - rest / splits;  // longest first
  const int group = a.H_q / a.H_kv;
  const int n = tokens_of(a, b);
  const int row0 = (kShare ? block : block * kWaves + wave) * 16 * MT;
  if (row0 >= n * group) return;
  const int last = min(row0 + 16 * MT, n * group) - 1;
  const Span span{key_limit(a, b, row0 / group), key_limit(a, b, last / group)};

  const int steps = (span.hi + kTile - 1) / kTile;
  const int per = split_steps(steps, splits);
  const int s_end = min((part + 1) * per, steps);
  constexpr int kStride = kShare ? kWaves : 1;
  int step = part * per + (kShare ? wave : 0);
  if (splits > 1 && part * per >= steps && part > 0) return;  // not read by the join

  // This lane's query rows: one per tile, column r.
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
    const T* src = static_cast<const T*>(a.q) + orow[m] * D + g * (D / 4);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float x[8];
      load_row<T, 8>(src + 8 * s, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bf16 p[QP];
        split<QP>(x[i], p);
#pragma unroll
        for (int c = 0; c < QP; ++c) q[m][c][s][i] = p[c];
      }
    }
  }

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

  f32x4 acc[MT][DT];
  float mx[MT], sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mx[m] = -INFINITY;
    sum[m] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  int idk = -1, idv = -1;
  if (step < s_end) {
    idk = page_of(step, ka);
    idv = page_of(step, g);
    load_k(step, idk);
  }
  for (; step < s_end; step += kStride) {
    load_v(step, idv);
    const size_t ph = static_cast<size_t>(max(idv, 0)) * a.H_kv + head;
    const float ks = a.k_scale[ph] * (a.scale * kLog2e);
    float vs = a.v_scale[ph];
    const int next = step + kStride;
    int idk2 = -1, idv2 = -1;
    if (next < s_end) {
      idk2 = page_of(next, ka);
      idv2 = page_of(next, g);
    }

    f32x4 z[MT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int m = 0; m < MT; ++m) z[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const bf16x8_t k =
            codes_to_bf16(word(kr[t][s / 2], 2 * (s & 1)), word(kr[t][s / 2], 2 * (s & 1) + 1));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int c = 0; c < QP; ++c)
            z[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[m][c][s], z[m][t], 0, 0, 0);
      }
    }
    if (next < s_end) load_k(next, idk2);

    // Every key of the step is there and in sight of every row?
    const int key0 = step * kTile + 16 * g;
    const bool whole = (step + 1) * kTile <= span.lo && __all(idv >= 0);
    const bool group_on = idv >= 0 && key0 < span.hi;
    if (!whole && !group_on) vs = 0.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = z[m][t][e] * ks;
          if (!whole && !(group_on && key0 + 4 * t + e < lim[m])) x = -INFINITY;
          z[m][t][e] = x;
          top = fmaxf(top, x);
        }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float now = fmaxf(mx[m], top);
      if (__any(now > mx[m])) {
        const float back = __builtin_amdgcn_exp2f(mx[m] - (now == -INFINITY ? 0.0f : now));
        sum[m] *= back;
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[m][d] *= back;
        mx[m] = now;
      }
      const float ref = now == -INFINITY ? 0.0f : now;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = __builtin_amdgcn_exp2f(z[m][t][e] - ref);
          sum[m] += p;
          z[m][t][e] = p * vs;
        }
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
      bf16x8_t p[MT][PP];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          bf16 c[PP];
          split<PP>(z[m][2 * u + i / 4][i & 3], c);
#pragma unroll
          for (int k = 0; k < PP; ++k) p[m][k][i] = c[k];
        }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        unsigned w0 = word(vr[d], 2 * u), w1 = word(vr[d], 2 * u + 1);
        if (has_nan) {
          const bf16x8_t bad = nan_codes(w0, w1);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const f32x4 hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                bad, p[m][0], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (hit[e] > 0.0f) acc[m][d][e] = NAN;
          }
          w0 = without_nan(w0);
          w1 = without_nan(w1);
        }
        const bf16x8_t v = codes_to_bf16(w0, w1);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int k = 0; k < PP; ++k)
            acc[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[m][k], acc[m][d], 0, 0, 0);
      }
    }
    idk = idk2;
    idv = idv2;
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    sum[m] += __shfl_xor(sum[m], 16, 64);
    sum[m] += __shfl_xor(sum[m], 32, 64);
  }

  if constexpr (kShare) {
    // Join the waves' sums: every wave leaves its own in LDS, then 16 threads
    // share a row.
    static_assert(MT == 1, "one tile of rows");
    constexpr int LD = D + 4;
    __shared__ float acc_s[kWaves][16][LD], ml_s[kWaves][16][2];
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *reinterpret_cast<f32x4*>(&acc_s[wave][r][16 * d + 4 * g]) = acc[0][d];
    if (g == 0) {
      ml_s[wave][r][0] = mx[0];
      ml_s[wave][r][1] = sum[0];
    }
    __syncthreads();
    const int row = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * (D / 16);
    if (row0 + row > last) return;
    float top = -INFINITY, tot = 0.0f, out[D / 16] = {};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ml_s[w][row][0]);
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
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
  } else {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (row0 + 16 * m + r > last) continue;
      if (splits > 1) {
        const Partial p = partial_of(a, splits, orow[m]);
#pragma unroll
        for (int d = 0; d < DT; ++d)
          store4<float>(p.acc + part * D + 16 * d + 4 * g, acc[m][d][0], acc[m][d][1],
                        acc[m][d][2], acc[m][d][3]);
        if (g == 0) {
          p.ml[2 * part] = mx[m];
          p.ml[2 * part + 1] = sum[m];
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
}

// Joins the splits of a query row: a wave per row, D/64 columns a lane.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(KvArgs a, int wave_rows, int splits) {
  const int lane = threadIdx.x & 63;
  const size_t at = static_cast<size_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
  if (at >= static_cast<size_t>(a.B) * a.T * a.H_q) return;
  const int hq = at % a.H_q;
  const int t = at / a.H_q % a.T, b = at / a.H_q / a.T;
  const int n = tokens_of(a, b);
  if (t >= n) return;
  const int group = a.H_q / a.H_kv;
  // The keys of the tile of rows that this row was computed in.
  const int row = t * group + hq % group;
  const int last = min((row / wave_rows + 1) * wave_rows, n * group) - 1;
  const int steps = (key_limit(a, b, last / group) + kTile - 1) / kTile;
  const int per = split_steps(steps, splits);
  const int used = max(1, (steps + per - 1) / per);

  const Partial p = partial_of(a, splits, at);
  float top = -INFINITY;
  for (int s = 0; s < used; ++s) top = fmaxf(top, p.ml[2 * s]);
  const float ref = top == -INFINITY ? 0.0f : top;
  float tot = 0.0f, out[D / 64] = {};
  for (int s = 0; s < used; ++s) {
    const float f = __builtin_amdgcn_exp2f(p.ml[2 * s] - ref);
    tot += f * p.ml[2 * s + 1];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) out[i] += f * p.acc[s * D + lane * (D / 64) + i];
  }
  const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    static_cast<T*>(a.o)[at * D + lane * (D / 64) + i] = from_f32<T>(out[i] * inv);
}

// How a call is cut.
struct Plan {
  bool share;      // the waves of a workgroup share one tile of rows
  int wave_rows;   // query rows of a wave
  int row_blocks;  // workgroups over the rows of a (batch row, kv head)
  int splits;      // workgroups over the keys
};

Plan plan_of(const KvArgs& a, int io_bf16) {
  const long long rows = static_cast<long long>(a.T) * (a.H_q / a.H_kv);
  Plan p;
  p.share = rows <= 64;
  p.wave_rows = p.share || !io_bf16 ? 16 : 32;
  const int block_rows = p.share ? 16 : p.wave_rows * (kThreads / 64);
  p.row_blocks = static_cast<int>((rows + block_rows - 1) / block_rows);
  // Enough workgroups for every CU to hold several, as far as the table's
  // keys allow.
  const long long base = static_cast<long long>(a.B) * a.H_kv * p.row_blocks;
  const long long steps = (static_cast<long long>(a.max_pages) * a.page + kTile - 1) / kTile;
  const long long want = (1024 + base - 1) / base;
  const long long most = steps / kMinSteps;
  p.splits = static_cast<int>(min(want, most));
  if (p.splits > 64) p.splits = 64;
  if (p.splits < 1) p.splits = 1;
  return p;
}

template <typename T, int D>
hipError_t launch_d(const KvArgs& a, hipStream_t stream) {
  const Plan p = plan_of(a, sizeof(T) == 2);
  const dim3 grid(static_cast<unsigned>(a.B) * a.H_kv * p.row_blocks * p.splits);
  if (p.share) {
    hipLaunchKernelGGL((attn_kernel<T, D, 1, true>), grid, dim3(kThreads), 0, stream, a,
                       p.row_blocks, p.splits);
  } else {
    constexpr int MT = sizeof(T) == 2 ? 2 : 1;
    hipLaunchKernelGGL((attn_kernel<T, D, MT, false>), grid, dim3(kThreads), 0, stream, a,
                       p.row_blocks, p.splits);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const size_t rows = static_cast<size_t>(a.B) * a.T * a.H_q;
  hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3(static_cast<unsigned>((rows + 3) / 4)),
                     dim3(kThreads), 0, stream, a, p.wave_rows, p.splits);
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
