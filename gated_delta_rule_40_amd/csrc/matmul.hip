// matmul.hip -- products of 8-bit rows with an 8-bit weight for gfx950:
//
//   y[m,n] = bias[n] + sum_b sx[m,b] sw[n/128,b] sum_{k in b} x[m,k] w[n,k]
//
// A block of 128 channels is a whole contraction of the matrix pipe, so that its sum
// leaves it at once and takes its two scales in one multiply-add on the way into the
// fp32 accumulator.  The weight is the instruction's first operand: a lane then holds
// four neighbouring outputs of one row, and one row's scale.
//
// Numbers.  The 8-bit matrix instructions add groups of 8 products aligned to the
// largest of them, 13 bits below its exponent (measured: beside 2^16, 2^3 counts and
// 2^2 is lost), and the groups in fp32: a result is off by 1.4e-5 of its norm for
// normal codes, 5e-5 for codes of every magnitude, against the 1.7e-3 that rounding to
// bf16 costs.  So a bf16 output takes them.  An fp32 output takes bf16 instructions
// (e4m3 is exact in bf16, products and sums are fp32: 5e-8) at half their rate.
//
// stream_kernel: few rows.  The weight is read once, straight into registers; the
// blocks of a row are shared by the waves of a workgroup and their sums joined in LDS.
// Bound by HBM.
#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"

namespace gdr {
namespace {

constexpr int kBlock = 128;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Channels of 16 rows of one block as an operand: lane l holds row l % 16, channels
// 32 (l / 16) ... + 31 (any order of the channels does, as long as it is the same for
// both operands).  EXACT: widened to bf16.
template <bool EXACT>
struct Operand;
template <>
struct Operand<false> {
  i32x8 v;
  __device__ __forceinline__ void set(i32x8 codes) { v = codes; }
};
template <>
struct Operand<true> {
  bf16x8 v[4];
  __device__ __forceinline__ void set(i32x8 codes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[2 * i + j], 1.0f, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[2 * i + j], 1.0f, true);
        v[i][4 * j] = lo[0];
        v[i][4 * j + 1] = lo[1];
        v[i][4 * j + 2] = hi[0];
        v[i][4 * j + 3] = hi[1];
      }
    }
  }
};

// Sums over one block.  Result: columns (the second operand's rows) l % 16, rows
// 4 (l / 16) ... + 3.
__device__ __forceinline__ f32x4 block_product(const Operand<false>& w, const Operand<false>& x) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, zero, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_product(const Operand<true>& w, const Operand<true>& x) {
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], s, 0, 0, 0);
  return s;
}

__device__ __forceinline__ i32x8 join(i32x4 lo, i32x4 hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 32 channels from k of a row of K, zeros behind its end (K a multiple of 16).
__device__ __forceinline__ i32x8 load_channels(const uint8_t* row, int k, int K) {
  const i32x4 zero = {0, 0, 0, 0};
  const i32x4 lo = k < K ? *reinterpret_cast<const i32x4*>(row + k) : zero;
  const i32x4 hi = k + 16 < K ? *reinterpret_cast<const i32x4*>(row + k + 16) : zero;
  return join(lo, hi);
}

// Four neighbouring outputs of row m from column n.
template <typename T>
__device__ __forceinline__ void store_out(const MatmulArgs& a, int m, int n, f32x4 v) {
  if (m >= a.M || n >= a.N) return;
  T* y = static_cast<T*>(a.y) + static_cast<size_t>(m) * a.N + n;
  if (a.bias) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (n + u < a.N) v[u] += a.bias[n + u];
  }
  if (a.N % 4 == 0) {
    store4<T>(y, v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (n + u < a.N) y[u] = from_f32<T>(v[u]);
  }
}

// 16 NT outputs of 16 MT rows a workgroup; wave v takes the blocks v, v + WAVES, ...
template <typename T, bool EXACT, int MT, int NT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void stream_kernel(MatmulArgs a, int row_tiles) {
  __shared__ f32x4 part[WAVES][NT * MT][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int m0 = blockIdx.x % row_tiles * (16 * MT), n0 = blockIdx.x / row_tiles * (16 * NT);
  const int K = a.K, blocks = (K + kBlock - 1) / kBlock;
  const int in = lane % 16, k0 = lane / 16 * 32;

  // Rows past the last are read as the last; their results are not stored.
  const uint8_t* w[NT];
  const uint8_t* x[MT];
  const float* sx[MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
    w[i] = a.w + static_cast<size_t>(min(n0 + 16 * i + in, a.N - 1)) * K;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const size_t m = min(m0 + 16 * j + in, a.M - 1);
    x[j] = a.x + m * K;
    sx[j] = a.x_scales + m * blocks;
  }
  const float* sw = a.w_scales + static_cast<size_t>(n0 / kBlock) * blocks;

  f32x4 acc[NT][MT] = {};
  for (int b = wave; b < blocks; b += WAVES) {
    const int k = b * kBlock + k0;
    i32x8 wc[NT], xc[MT];
    float s[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) wc[i] = load_channels(w[i], k, K);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      xc[j] = load_channels(x[j], k, K);
      s[j] = sx[j][b] * sw[b];
    }
    Operand<EXACT> wf[NT], xf[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) wf[i].set(wc[i]);
#pragma unroll
    for (int j = 0; j < MT; ++j) xf[j].set(xc[j]);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] += block_product(wf[i], xf[j]) * s[j];
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[wave][i * MT + j][lane] = acc[i][j];
  __syncthreads();
  for (int t = threadIdx.x; t < NT * MT * 64; t += WAVES * 64) {
    const int tile = t / 64, l = t % 64;
    f32x4 v = part[0][tile][l];
#pragma unroll
    for (int q = 1; q < WAVES; ++q) v += part[q][tile][l];
    store_out<T>(a, m0 + tile % MT * 16 + l % 16, n0 + tile / MT * 16 + l / 16 * 4, v);
  }
}

template <typename T, int MT, int NT, int WAVES>
hipError_t launch_stream(const MatmulArgs& a, hipStream_t stream) {
  const int row_tiles = (a.M + 16 * MT - 1) / (16 * MT);
  const int col_tiles = (a.N + 16 * NT - 1) / (16 * NT);
  constexpr bool kExact = sizeof(T) == 4;
  hipLaunchKernelGGL((stream_kernel<T, kExact, MT, NT, WAVES>),
                     dim3(static_cast<unsigned>(row_tiles) * col_tiles), dim3(WAVES * 64), 0,
                     stream, a, row_tiles);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// tile_kernel: many rows.  A workgroup owns BN outputs of BM rows; a block of both
// operands lies in LDS, the next is on its way there (straight from memory, no
// registers) while its products run.
// ---------------------------------------------------------------------------

// 16 bytes a lane from `base` (the same in every lane) + offset to LDS: lane l's go
// to lds + 16 l.  Nothing waits for it here.
__device__ __forceinline__ void load_to_lds(const uint8_t* base, unsigned offset, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(offset), "s"(base)
               : "memory");
}
__device__ __forceinline__ void load_to_lds(const uint8_t* p, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds), "v"(p)
               : "memory");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// What lanes behind the last channel load.
__device__ const uint4 kZeros = {0, 0, 0, 0};

// Workgroup `id` of `total` in the order in which workgroups that run together on one
// XCD (every eighth) are neighbours.
__device__ __forceinline__ int xcd_order(int id, int total) {
  const int xcd = id % 8, each = total / 8, more = total % 8;
  return xcd * each + min(xcd, more) + id / 8;
}

constexpr int kRowGroup = 8;  // row tiles that are walked before the next column tile

template <typename T, bool EXACT, int WN, int WM, int NT, int MT>
__global__ __launch_bounds__(WN * WM * 64) void tile_kernel(MatmulArgs a, int row_tiles,
                                                            int col_tiles) {
  constexpr int BN = WN * NT * 16, BM = WM * MT * 16, WAVES = WN * WM;
  constexpr int kPieces = (BN + BM) / 8;          // of 8 rows, 1 KiB, one load of a wave
  constexpr int kEach = kPieces / WAVES;
  static_assert(kPieces % WAVES == 0 && BN % 8 == 0, "pieces are shared evenly");
  static_assert(kBlock % (NT * 16) == 0, "a wave's outputs share their scale");
  __shared__ __attribute__((aligned(1024))) uint8_t tile[2][(BN + BM) * kBlock];

  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int t = xcd_order(blockIdx.x, row_tiles * col_tiles);
  const int group = t / (kRowGroup * col_tiles), within = t % (kRowGroup * col_tiles);
  const int tall = min(kRowGroup, row_tiles - group * kRowGroup);
  const int m0 = (group * kRowGroup + within % tall) * BM, n0 = within / tall * BN;
  const int K = a.K, blocks = (K + kBlock - 1) / kBlock;

  // Rows of 128 bytes; 16-byte piece c of row r lies at c ^ (r % 8), so that lanes
  // that read one piece of many rows meet different banks.  A load of a wave fills 8
  // rows: lane l brings piece (l % 8) ^ (l / 8) of row l / 8.  Rows past the last are
  // read as the last; their results are not stored.
  const int from = ((lane % 8) ^ (lane / 8)) * 16;
  unsigned offset[kEach];
  const uint8_t* base[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int row = (wave * kEach + i) * 8;       // of the two tiles, the weight's first
    const bool w = row < BN;
    const int r0 = w ? n0 : m0, last = (w ? a.N : a.M) - 1 - r0;
    base[i] = (w ? a.w : a.x) + static_cast<size_t>(r0) * K;
    offset[i] = static_cast<unsigned>(min((w ? row : row - BN) + lane / 8, last)) *
                    static_cast<unsigned>(K) + from;
  }
  const unsigned lds0 = static_cast<unsigned>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)&tile[0][0]));
  auto fetch = [&](int b) {
    const unsigned lds = lds0 + (b & 1) * ((BN + BM) * kBlock) + wave * kEach * 1024;
    const int k = b * kBlock;
    if (k + kBlock <= K) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) load_to_lds(base[i] + k, offset[i], lds + i * 1024);
    } else {
      const bool on = k + from < K;
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        load_to_lds(on ? base[i] + k + offset[i] : reinterpret_cast<const uint8_t*>(&kZeros),
                    lds + i * 1024);
    }
  };

  const int wn = wave % WN * (NT * 16), wm = wave / WN * (MT * 16);  // within the tile
  const int in = lane % 16, g = lane / 16;
  const float* sx[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
    sx[j] = a.x_scales + static_cast<size_t>(min(m0 + wm + 16 * j + in, a.M - 1)) * blocks;
  // A tile's columns past N may have no scale of their own.
  const float* sw =
      a.w_scales + static_cast<size_t>(min(n0 + wn, a.N - 1) / kBlock) * blocks;
  const int p0 = ((2 * g) ^ (in % 8)) * 16, p1 = ((2 * g + 1) ^ (in % 8)) * 16;

  // A vector load for the weight's scale, too: scalar ones would be waited for with the
  // reads from LDS.
  int zero = 0;
  asm volatile("" : "+v"(zero));
  float rs[MT], ws = 0.0f;
#pragma unroll
  for (int j = 0; j < MT; ++j) rs[j] = 0.0f;
  if (blocks > 0) {
#pragma unroll
    for (int j = 0; j < MT; ++j) rs[j] = sx[j][0];
    ws = sw[zero];
    fetch(0);
  }
  f32x4 acc[NT][MT] = {};
  for (int b = 0; b < blocks; ++b) {
    wait_loads();
    __syncthreads();  // this block is in LDS, and no wave reads the one before
    float s[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      s[j] = rs[j] * ws;
      asm volatile("" : "+v"(s[j]));  // here: a later use would wait for the loads below
    }
    if (b + 1 < blocks) {
      fetch(b + 1);
#pragma unroll
      for (int j = 0; j < MT; ++j) rs[j] = sx[j][b + 1];
      ws = sw[b + 1 + zero];
    }

    const uint8_t* lw = tile[b & 1] + (wn + in) * kBlock;
    const uint8_t* lx = tile[b & 1] + (BN + wm + in) * kBlock;
    auto operand = [&](const uint8_t* row) {
      Operand<EXACT> f;
      f.set(join(*reinterpret_cast<const i32x4*>(row + p0),
                 *reinterpret_cast<const i32x4*>(row + p1)));
      return f;
    };
    // A block's sum is scaled and added kLag products after its own, when it has left
    // the matrix pipe; the weight's operands are read one ahead.
    constexpr int kLag = 3;
    f32x4 sum[kLag + 1];
    Operand<EXACT> wf[2], xf[MT];
    wf[0] = operand(lw);
#pragma unroll
    for (int j = 0; j < MT; ++j) xf[j] = operand(lx + j * 16 * kBlock);
#pragma unroll
    for (int q = 0; q < NT * MT + kLag; ++q) {
      if (q < NT * MT) {
        const int i = q / MT, j = q % MT;
        if (j == 0 && i + 1 < NT) wf[(i + 1) % 2] = operand(lw + (i + 1) * 16 * kBlock);
        sum[q % (kLag + 1)] = block_product(wf[i % 2], xf[j]);
      }
      if (q >= kLag) acc[(q - kLag) / MT][(q - kLag) % MT] += sum[(q - kLag) % (kLag + 1)] * s[(q - kLag) % MT];
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  const int m = m0 + wm + in, n = n0 + wn + 4 * g;
  if (m0 + BM <= a.M && n0 + BN <= a.N && a.N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      f32x4 bias = {0.0f, 0.0f, 0.0f, 0.0f};
      if (a.bias) {
#pragma unroll
        for (int u = 0; u < 4; ++u) bias[u] = a.bias[n + 16 * i + u];
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const f32x4 v = acc[i][j] + bias;
        store4<T>(static_cast<T*>(a.y) + static_cast<size_t>(m + 16 * j) * a.N + n + 16 * i, v[0],
                  v[1], v[2], v[3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) store_out<T>(a, m + 16 * j, n + 16 * i, acc[i][j]);
  }
}

template <typename T, int WN, int WM, int NT, int MT>
hipError_t launch_tile(const MatmulArgs& a, hipStream_t stream) {
  constexpr bool kExact = sizeof(T) == 4;
  const int row_tiles = (a.M + WM * MT * 16 - 1) / (WM * MT * 16);
  const int col_tiles = (a.N + WN * NT * 16 - 1) / (WN * NT * 16);
  hipLaunchKernelGGL((tile_kernel<T, kExact, WN, WM, NT, MT>),
                     dim3(static_cast<unsigned>(row_tiles) * col_tiles), dim3(WN * WM * 64), 0,
                     stream, a, row_tiles, col_tiles);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_io(const MatmulArgs& a, hipStream_t stream) {
  if (a.M <= 16) return launch_stream<T, 1, 1, 8>(a, stream);
  if (a.M <= 32) return launch_stream<T, 2, 1, 8>(a, stream);
  if (a.M <= 256) return launch_stream<T, 4, 2, 8>(a, stream);
  const long long big = ((a.M + 255ll) / 256) * ((a.N + 255ll) / 256);
  // fp32: bf16 operands take twice the registers.
  constexpr int kTall = sizeof(T) == 4 ? 4 : 8;
  if (big >= 128) return launch_tile<T, 2, 4, kTall, 4>(a, stream);
  return launch_tile<T, 2, 2, 4, 4>(a, stream);
}

}  // namespace

long long matmul_max_grid(int M, int N) {
  const long long rows = (static_cast<long long>(M) + 15) / 16;
  return rows * ((static_cast<long long>(N) + 15) / 16);
}

hipError_t launch_matmul(const MatmulArgs& a, int io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_io<bf16>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace gdr
