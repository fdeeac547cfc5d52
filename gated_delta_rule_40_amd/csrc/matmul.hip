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
// (e4m3 is exact in bf16, products and sums are fp32: 7e-8 of the norm for K = 4096 and few
// rows, 1.1e-7 in the tiles of many) at half their rate.
//
// stream_kernel: few rows.  The weight is read once; the blocks of a row are shared by
// the waves of a workgroup and their sums joined in LDS.  Bound by HBM (one row through
// 8192 x 4096 7.9 us, 34 MB), and with the rows by the L2 caches that every workgroup
// reads x from (64 rows 11.2 us; 64 x 1000 x 4096 6.1, K = 14336 12.4, in smaller tiles).
// tile_kernel: many rows.  4000 rows through 8192 x 4096 130 us, 2.1 PFLOP/s; 8192^3 2.3.
// Between the two, 65 to 1000 rows, the one block under way is what bounds it: a step of a
// workgroup waits for loads that began one step before (250 rows through 8192 x 4096 23 us,
// 44 MB; 400 x 1000 12.2 us, 6 MB, with most CUs idle in large tiles and 80 MB loaded in
// small ones, as workgroups share no sum over K).
// The matrix pipes alone reach 3.5 on such codes, held by power (4.9 on zeros).  A step
// of 2048 matrix cycles a SIMD takes about 3600: the loads into LDS cost some 400 of
// the rest, reading operands 100, the barrier and what surrounds it most of it.
// Tried without gain: two groups of waves half a block apart, a second barrier half way
// with loads a block and a half ahead, the barrier before the last row of products (4%
// faster here, 2 to 10% slower for K = 14336, 4080 and 500 rows),
// the weight's operands two ahead, wave priorities.
#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"
#include "store_through.hpp"

namespace gdr {
namespace {

constexpr int kBlock = 128;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Channels of 16 rows of one block as an operand: lane l holds row l % 16, channels
// 16 (l / 16) ... + 15 and 64 behind those (any order of the channels does, as long as
// it is the same for both operands; in this one four lanes read 64 bytes in a row).  EXACT: widened to bf16.
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

// 16 bytes a lane from `base` (the same in every lane) + offset to LDS: lane l's go
// to lds + 16 l.  Nothing waits for it here.  The compiler writes m0, which
// takes the address in LDS, and knows what it holds.  (The wait states: one behind that
// write, five behind a vector instruction's of a scalar base.)
__device__ __forceinline__ void load_to_lds(const uint8_t* base, unsigned offset, unsigned lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "{m0}"(lds), "v"(offset), "s"(base)
               : "memory");
}
__device__ __forceinline__ void load_to_lds(const uint8_t* p, unsigned lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "{m0}"(lds), "v"(p)
               : "memory");
}
// 4 bytes a lane, lane l's to lds + 4 l.
__device__ __forceinline__ void load_word_to_lds(const float* p, unsigned lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dword %1, off"
               :
               : "{m0}"(lds), "v"(p)
               : "memory");
}
__device__ __forceinline__ unsigned lds_address(const void* p) {
  return static_cast<unsigned>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// What lanes behind the last channel load.
__device__ const uint4 kZeros = {0, 0, 0, 0};

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

// Eight neighbouring outputs of row m from column n; `whole`: the columns are there, and
// 16-byte aligned (where N is not of whole 16 bytes no output is: 4000 x 8191 x 4096 186 us,
// 4000 x 8188 185, 4000 x 8192 132).  bf16 goes through the L2 caches at every size: 1000 x
// 4096 x 1024 9.1 us against 10.2 with plain stores, 192 x 8192 x 4096 22.0 against 22.2, 1500
// x 8192 x 4096 55.3 against 57.0.
template <typename T>
__device__ __forceinline__ void store_out8(const MatmulArgs& a, int m, int n, f32x4 lo, f32x4 hi,
                                           bool whole) {
  if (m >= a.M) return;
  T* y = static_cast<T*>(a.y) + static_cast<size_t>(m) * a.N + n;
  if (whole) {
    if (a.bias) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        lo[u] += a.bias[n + u];
        hi[u] += a.bias[n + 4 + u];
      }
    }
    T e[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      e[u] = from_f32<T>(lo[u]);
      e[4 + u] = from_f32<T>(hi[u]);
    }
#pragma unroll
    for (int c = 0; c < static_cast<int>(sizeof(T)) / 2; ++c) {
      if constexpr (sizeof(T) == 2)
        store_through(y, reinterpret_cast<const through_u32x4*>(e)[c]);
      else  // two stores, each of half the bytes of a line: through 310 against 284 us
        reinterpret_cast<through_u32x4*>(y)[c] = reinterpret_cast<const through_u32x4*>(e)[c];
    }
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (n + u < a.N) {
        const float v = u < 4 ? lo[u % 4] : hi[u % 4];
        y[u] = from_f32<T>(v + (a.bias ? a.bias[n + u] : 0.0f));
      }
  }
}

// 16 NT outputs of 16 MT rows a workgroup; wave v takes the blocks v, v + WAVES, ...
// It loads one straight into LDS, in a place of its own, while the products of the one
// before run; nothing but the join at the end waits for other waves.  8 lanes bring a
// row's 128 bytes: lanes that loaded their own operands touched 16 rows at once, four
// times as many lines (64 rows 18.2 against 12.3 us, 16 rows with K = 14336 18.6 against
// 11.5).  Two to four blocks ahead are no faster: the waves of a workgroup are enough.
template <typename T, bool EXACT, int MT, int NT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void stream_kernel(MatmulArgs a, int row_tiles) {
  constexpr int kRows = 16 * (NT + MT), kPieces = kRows / 8;
  constexpr int kPlace = kRows * kBlock + 256;  // the rows, then the scales of x
  __shared__ __attribute__((aligned(1024))) uint8_t places[WAVES][kPlace];
  static_assert(kPlace >= NT * MT * 1024, "the join takes the same place");
  static_assert(MT <= 4, "one lane loads a row's scale");
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int m0 = blockIdx.x % row_tiles * (16 * MT), n0 = blockIdx.x / row_tiles * (16 * NT);
  const int K = a.K, blocks = (K + kBlock - 1) / kBlock;
  const int in = lane % 16, g = lane / 16;

  // The weight's rows, then those of x; piece c of row r lies at c ^ (r % 8).  Rows past
  // the last are read as the last; their results are not stored.
  const uint8_t* wbase = a.w + static_cast<size_t>(n0) * K;
  const uint8_t* xbase = a.x + static_cast<size_t>(m0) * K;
  const int from = (lane % 8 ^ lane / 8) * 16;
  unsigned offset[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int row = i * 8 + lane / 8;
    const int r = i < 2 * NT ? min(row, a.N - 1 - n0) : min(row - 16 * NT, a.M - 1 - m0);
    offset[i] = static_cast<unsigned>(r) * static_cast<unsigned>(K) + from;
  }
  const float* sx = a.x_scales + static_cast<size_t>(min(m0 + lane % (16 * MT), a.M - 1)) * blocks;
  const float* sw = a.w_scales + static_cast<size_t>(n0 / kBlock) * blocks;
  const uint8_t* place = places[wave];
  const unsigned lds = lds_address(place);
  auto fetch = [&](int b) {
    const int k = b * kBlock;
    if (k + kBlock <= K) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        load_to_lds((i < 2 * NT ? wbase : xbase) + k, offset[i], lds + i * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        load_to_lds(k + from < K ? (i < 2 * NT ? wbase : xbase) + k + offset[i]
                                 : reinterpret_cast<const uint8_t*>(&kZeros),
                    lds + i * 1024);
    }
    load_word_to_lds(sx + b, lds + kRows * kBlock);
  };
  // Rows a multiple of 4 KiB apart lie on the same memory channels: workgroups (32 at a time,
  // four of each XCD, which may share a weight's or x's rows) then begin at different blocks.
  // 64 x 4096 x 4096 10.2 -> 8.5 us, 64 x 8192 12.1 -> 11.1, 1 x 8192 8.6 -> 7.8.  Rows an odd
  // multiple of 2 KiB apart gain nothing (64 x 4096, K = 14336 19.3 and 19.8; 64 x 8192, K =
  // 14336 39.5 and 39.9, K = 6144 13.9 and 13.8, K = 10240 21.1 and 26.3; 16 x 4096, K = 14336
  // 11.1 and 11.2).
  const unsigned turn = K % 4096 == 0 ? blockIdx.x / 32 * WAVES : 0;
  const int first = blocks > 0 ? static_cast<int>(turn % blocks) : 0;
  auto block_of = [&](int t) { return t + first < blocks ? t + first : t + first - blocks; };
  if (wave < blocks) fetch(block_of(wave));

  f32x4 acc[NT][MT] = {};
  const int p0 = (g ^ (in % 8)) * 16, p1 = p0 ^ 64;
  for (int t = wave; t < blocks; t += WAVES) {
    const int b = block_of(t);
    wait_loads();
    auto operand = [&](int row) {
      const uint8_t* p = place + (row + in) * kBlock;
      Operand<EXACT> f;
      f.set(join(*reinterpret_cast<const i32x4*>(p + p0), *reinterpret_cast<const i32x4*>(p + p1)));
      return f;
    };
    Operand<EXACT> wf[NT], xf[MT];
    float s[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) wf[i] = operand(16 * i);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      xf[j] = operand(16 * (NT + j));
      s[j] = *reinterpret_cast<const float*>(place + kRows * kBlock + (16 * j + in) * 4) * sw[b];
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // all read: the place is free
    if (t + WAVES < blocks) fetch(block_of(t + WAVES));
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] += block_product(wf[i], xf[j]) * s[j];
  }
  __syncthreads();
  f32x4(*part)[NT * MT][64] = reinterpret_cast<f32x4(*)[NT * MT][64]>(&places[0][0]);
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

// Workgroup `id` of `total` in the order in which workgroups that run together on one
// XCD (every eighth) are neighbours.
__device__ __forceinline__ int xcd_order(int id, int total) {
  const int xcd = id % 8, each = total / 8, more = total % 8;
  return xcd * each + min(xcd, more) + id / 8;
}

// Row tiles that are walked before the next column tile (8192 x 8192 x 8192: 470 us; 475
// with 2, 476 with 8, 494 with 16, 526 with 32).
constexpr int kRowGroup = 4;

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

  // Rows of 128 bytes, of which a load of a wave fills 8, lane l the 16 bytes at l % 8 of
  // row l / 8.  Piece c of row r lies at c ^ key(r): the lanes that the LDS serves
  // together (0-3, 12-15 and 20-27; 4-11, 16-19 and 28-31; the same from 32) then meet
  // different banks, reading pieces g and g + 4 (lane 16 g + in) of the rows that
  // `in` stands for.  Those are 16 neighbouring ones of x (key r % 8); of the weight
  // 4 of every 8 out of 32, so that a lane holds 8 neighbouring outputs in a pair of
  // products (key r % 4 + 4 (r / 8 % 2)).  Rows past the last are read as the last;
  // their results are not stored.
  auto piece = [&](int i) {  // of this lane's in load i, its first byte in the row
    const int p = wave * kEach + i;  // rows 8 p ... 8 p + 7
    const int key = p < BN / 8 ? lane / 8 % 4 + p % 2 * 4 : lane / 8;
    return (lane % 8 ^ key) * 16;
  };
  unsigned offset[kEach];
  const uint8_t* base[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int row = (wave * kEach + i) * 8;       // of the two tiles, the weight's first
    const bool w = row < BN;
    const int r0 = w ? n0 : m0, last = (w ? a.N : a.M) - 1 - r0;
    base[i] = (w ? a.w : a.x) + static_cast<size_t>(r0) * K;
    offset[i] = static_cast<unsigned>(min((w ? row : row - BN) + lane / 8, last)) *
                    static_cast<unsigned>(K) + piece(i);
  }
  const unsigned lds0 = lds_address(&tile[0][0]);
  auto lds_of = [&](int b, int i) {
    return lds0 + (b & 1) * ((BN + BM) * kBlock) + (wave * kEach + i) * 1024;
  };
  auto fetch = [&](int b, int i) {  // load i of this wave for block b, a whole one
    load_to_lds(base[i] + b * kBlock, offset[i], lds_of(b, i));
  };
  auto fetch_all = [&](int b) {  // any block
    const int k = b * kBlock;
    if (k + kBlock <= K) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) fetch(b, i);
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        load_to_lds(k + piece(i) < K ? base[i] + k + offset[i]
                                     : reinterpret_cast<const uint8_t*>(&kZeros),
                    lds_of(b, i));
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
  const int p0 = (g ^ (in % 8)) * 16, p1 = p0 ^ 64;

  // Scales are loaded for many blocks at once and handed out between lanes: of a row's,
  // the four lanes that hold it take one of four blocks each, of the weight's each lane
  // one of 64.  (One load a row and block touched a line for 4 bytes: 157 us without
  // these loads against 192 with them.)
  float rs[MT], ws = 0.0f;
  auto load_scales = [&](int b, bool start) {  // b a multiple of 4; the first one?
#pragma unroll
    for (int j = 0; j < MT; ++j) rs[j] = sx[j][min(b + g, blocks - 1)];
    if (start || b % 64 == 0) ws = sw[min(b / 64 * 64 + lane, blocks - 1)];
  };
  // Every XCD (whose workgroups share what they load) begins at a block of its own, in whole
  // groups of four blocks, so that the XCDs do not ask for the same channels of memory:
  // 4000 x 8192 x 4096 134 -> 129 us, K = 8192 261 -> 250, K = 5120 158 -> 155, 1000 x 8192,
  // K = 14336 163 -> 155; 4000 x 4096, K = 14336 205 -> 207.
  const int first = K % 512 == 0 ? static_cast<int>(blockIdx.x % 8) * (blocks / 32 * 4) : 0;
  auto block_of = [&](int t) { return t + first < blocks ? t + first : t + first - blocks; };
  if (blocks > 0) {
    load_scales(block_of(0), true);
    fetch_all(block_of(0));
  }
  f32x4 acc[NT][MT] = {};
  // One block, the t-th; AHEAD: the next is there, and whole.
  auto step = [&](int t, auto ahead) {
    constexpr bool AHEAD = decltype(ahead)::value;
    const int b = block_of(t), next = block_of(t + 1);
    wait_loads();
    __syncthreads();  // this block is in LDS, and no wave reads the one before
    const float wb = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ws), b % 64));
    float s[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      s[j] = wb * __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(
                                                (in + 16 * (b % 4)) * 4,
                                                __builtin_bit_cast(int, rs[j])));
      asm volatile("" : "+v"(s[j]));  // here: a later use would wait for the loads below
    }
    if (AHEAD || t + 1 < blocks) {
      if (b % 4 == 3) load_scales(next, false);
      if (!AHEAD) fetch_all(next);
    }

    const uint8_t* lw = tile[b & 1] + (wn + in / 4 * 8 + in % 4) * kBlock;
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
    static_assert(kEach <= NT * MT, "every load has its place");
    f32x4 sum[kLag + 1];
    Operand<EXACT> wf[2], xf[MT];
    wf[0] = operand(lw);
#pragma unroll
    for (int j = 0; j < MT; ++j) xf[j] = operand(lx + j * 16 * kBlock);
#pragma unroll
    for (int q = 0; q < NT * MT + kLag; ++q) {
      if (q < NT * MT) {
        const int i = q / MT, j = q % MT;
        if (j == 0 && i + 1 < NT)
          wf[(i + 1) % 2] = operand(lw + ((i + 1) / 2 * 32 + (i + 1) % 2 * 4) * kBlock);
        sum[q % (kLag + 1)] = block_product(wf[i % 2], xf[j]);
        // The next block's loads, one behind each product: all at once they would hold
        // the wave up until the memory pipe has taken them (161 against 154 us), later
        // ones arrive late (156 to 163).
        if (AHEAD && q < kEach) fetch(next, q);
      }
      if (q >= kLag) {
        const int p = q - kLag;
        acc[p / MT][p % MT] += sum[p % (kLag + 1)] * s[p % MT];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const int whole = K / kBlock;
  int t0 = 0;
  for (; t0 + 1 < whole; ++t0) step(t0, std::true_type{});
  for (; t0 < blocks; ++t0) step(t0, std::false_type{});
  // A lane holds 8 neighbouring outputs in a pair of products.
  const int m = m0 + wm + in, n = n0 + wn + 8 * g;
  const bool whole_row = n0 + BN <= a.N && a.N % (16 / static_cast<int>(sizeof(T))) == 0;
#pragma unroll
  for (int i = 0; i < NT; i += 2)
#pragma unroll
    for (int j = 0; j < MT; ++j)
      store_out8<T>(a, m + 16 * j, n + 16 * i, acc[i][j], acc[i + 1][j], whole_row);
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

// ---------------------------------------------------------------------------
// Which kernel.  Up to 16 rows a tile of as many; past that the one with the lowest
// estimate, in microseconds, of a fixed cost and, for each round of 256 workgroups, one of
// its own and one for 4096 channels of the rows that a workgroup loads (704 sizes from 20 x
// 512 to 1000 x 12288, K of 1024 to 14336, both output types: it takes 0.7% longer than the
// fastest of them all on the average, more than 10% at 15 of them, and 38% at the worst, 400
// x 4096, K = 8192: 58.5 us in 64 x 64, where the stream_kernel's time grows faster than K,
// and 42.3 in the tile of 64 x 128; behind it come 17, 16 and 15%).  The tile_kernel is
// left out up to 64 rows, where the weight is read once and HBM is what counts (17 x 65536
// 57 us with 32 x 32, 70 with a tile of 64 x 128).  With few outputs smaller tiles reach
// more CUs, each of which takes in some 68 bytes a ns:
//   64 x 1000 stream 16 x 16 6.1 us, 32 x 16 6.4, 64 x 32 9.2; K = 14336 12.4, 13.3, 24.0
//   128 x 1000 stream 16 x 16 8.5, 32 x 16 6.8, 32 x 32 7.6, 64 x 32 9.6
//   64 x 4096 stream 32 x 32 8.7, 64 x 16 8.7, 64 x 32 10.1; K = 14336 20.5, 22.3, 25.9
//   32 x 8192 stream 32 x 16 9.9, 32 x 32 8.7; 80 x 4096 64 x 16 14.4, 64 x 32 11.1
//   64 x 8192 stream 64 x 32 11.4, stream 64 x 64 13.8; 64 x 12288 18.7, 15.3
//   160 x 8192 stream 64 x 32 26.9, tile 64 x 128 23.0
//   400 x 8192 tile 64 x 128 29.3, tile 128 x 128 28.9
//   1000 x 8192 tile 128 x 128 43.8, tile 256 x 128 41.1
//   1000 x 12288 tile 128 x 128 66.7, tile 256 x 256 58.1
// An fp32 output's operands take twice the registers: the two that would not fit are left
// out, and the tiles' products take longer (1000 x 8192: 69.7 and 66.6).
// ---------------------------------------------------------------------------
enum class Plan {
  kStream16x16,
  kStream32x16,
  kStream32x32,
  kStream64x16,
  kStream64x32,
  kStream64x64,
  kTile64,
  kTile128,
  kTile256,
  kTile256x256
};

struct Option {
  Plan plan;
  int rows, cols;       // of a tile
  struct Cost {
    float fixed, round, channels;
  } bf16, fp32;  // by the type of the outputs
};
constexpr float kNever = 1e30f;
constexpr Option kOptions[] = {
    {Plan::kStream16x16, 16, 16, {0.0f, 1.5f, 2.4f}, {0.0f, 1.5f, 2.4f}},
    {Plan::kStream32x16, 32, 16, {0.4f, 2.2f, 3.0f}, {0.4f, 2.2f, 3.0f}},
    {Plan::kStream32x32, 32, 32, {2.2f, 1.3f, 4.1f}, {2.2f, 1.3f, 4.1f}},
    {Plan::kStream64x16, 64, 16, {1.2f, 2.1f, 5.3f}, {1.2f, 2.1f, 5.3f}},
    {Plan::kStream64x32, 64, 32, {1.6f, 3.0f, 6.2f}, {1.6f, 3.0f, 6.2f}},
    {Plan::kStream64x64, 64, 64, {0.0f, 6.3f, 7.2f}, {kNever, 0.0f, 0.0f}},
    {Plan::kTile64, 64, 128, {3.5f, 1.1f, 19.1f}, {4.5f, 0.0f, 28.8f}},
    {Plan::kTile128, 128, 128, {10.7f, 1.6f, 20.9f}, {11.7f, 1.0f, 35.1f}},
    {Plan::kTile256, 256, 128, {6.5f, 8.2f, 33.3f}, {0.0f, 14.1f, 56.5f}},
    {Plan::kTile256x256, 256, 256, {5.9f, 9.4f, 50.4f}, {kNever, 0.0f, 0.0f}},
};

struct Choice {
  Plan plan;
  long long tiles;
};
long long tiles_of(int M, int N, int rows, int cols) {
  return ((M + rows - 1ll) / rows) * ((N + cols - 1ll) / cols);
}
Choice choose(int M, int N, int K, bool fp32) {
  if (M <= 16) return Choice{Plan::kStream16x16, tiles_of(M, N, 16, 16)};
  Choice best = {};
  float least = 0.0f;
  for (const Option& o : kOptions) {
    const long long tiles = tiles_of(M, N, o.rows, o.cols), rounds = (tiles + 255) / 256;
    const Option::Cost& c = fp32 ? o.fp32 : o.bf16;
    const float loaded = static_cast<float>(std::min(M, o.rows) + o.cols) / (o.rows + o.cols);
    const float cost = c.fixed + (c.round + c.channels * loaded * (K / 4096.0f)) * rounds;
    if (M <= 64 && o.plan >= Plan::kTile64) break;
    if (best.tiles == 0 || cost < least) {
      best = Choice{o.plan, tiles};
      least = cost;
    }
  }
  return best;
}

// Whether 16 x 16 tiles take 16 waves, not 8.  With a workgroup a CU and up to 8 rows a CU
// waits for the weight's loads, of which more waves have more under way (1 x 2560, K =
// 14336 8.6 against 10.9 us).  16 rows gain nothing (16 x 4096, K = 14336 13.0 and 12.3), nor
// do waves without a block of their own (1 x 4096, K = 1024 3.8 and 3.6) or more workgroups
// (1 x 8192, K = 4096 8.1 and 7.9; 1 x 5120, K = 14336 16.3 and 13.5).
bool wide(const MatmulArgs& a, long long tiles) {
  return a.M <= 8 && a.K >= 16 * kBlock && tiles <= 256;
}

template <typename T>
hipError_t launch_io(const MatmulArgs& a, hipStream_t stream) {
  const Choice choice = choose(a.M, a.N, a.K, sizeof(T) == 4);
  switch (choice.plan) {
    case Plan::kStream16x16:
      return wide(a, choice.tiles) ? launch_stream<T, 1, 1, 16>(a, stream)
                                   : launch_stream<T, 1, 1, 8>(a, stream);
    case Plan::kStream32x16: return launch_stream<T, 2, 1, 8>(a, stream);
    case Plan::kStream32x32: return launch_stream<T, 2, 2, 8>(a, stream);
    case Plan::kStream64x16: return launch_stream<T, 4, 1, 8>(a, stream);
    case Plan::kStream64x32: return launch_stream<T, 4, 2, 8>(a, stream);
    case Plan::kTile64: return launch_tile<T, 2, 2, 4, 2>(a, stream);
    case Plan::kTile128: return launch_tile<T, 2, 2, 4, 4>(a, stream);
    case Plan::kTile256: return launch_tile<T, 2, 4, 4, 4>(a, stream);
    case Plan::kStream64x64:
      if constexpr (sizeof(T) == 2) return launch_stream<T, 4, 4, 8>(a, stream);
      break;
    case Plan::kTile256x256:
      if constexpr (sizeof(T) == 2) return launch_tile<T, 2, 4, 8, 4>(a, stream);
      break;
  }
  return hipErrorInvalidValue;  // an fp32 output is never given the last two
}

}  // namespace

long long matmul_grid(int M, int N, int K, int io_bf16) {
  return choose(M, N, K, !io_bf16).tiles;
}

hipError_t launch_matmul(const MatmulArgs& a, int io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_io<bf16>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace gdr
