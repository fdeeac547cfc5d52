// conv.hip -- short causal convolution per channel for gfx950: single tokens
// and prompts, with the last W - 1 inputs carried as a state.
//
//   y_t[c] = act(bias[c] + sum_w weight[c][w] u_{t-W+1+w}[c])
//
// where u_t = x_t for t >= 0 and the state's rows before that.
//
// A thread owns VEC neighbouring channels (16 bytes of a row) over TILE
// consecutive tokens and slides the W-token window down them in registers, so
// every input is read once but for the W - 1 rows before a tile; weights and
// bias stay in registers over the tile.  Bound by HBM: a value costs one read
// and one write, and about 17 issue slots, which is why the sigmoid goes
// through the hardware exp2 and reciprocal.  8192 channels in bf16: 4000 tokens
// 34.5 us (131 MB, 3.8 TB/s), 500 tokens 8.7 us, 64 single tokens 5.8 us.
// Stores past the caches would take 26.8 us for the 4000 tokens, but the scan
// that reads the outputs next then takes 11 us more: the two together are
// faster with plain stores at every length (4000 tokens 104 against 108 us).
//
// The thread of a row's first tile also writes the new state: it alone reads
// the old one, so the state may be updated in place.
#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;
// Threads that a prompt's tiles should give.  With 8192 channels, tiles of 32
// against 16 tokens: 500 tokens (16 or 32 thousand threads) 12.4 against 8.8 us,
// 1500 tokens (48 or 96 thousand) 14.6 against 15.4 us.
constexpr long long kFill = 40000;

template <typename T, int VEC>
struct Pack {
  T e[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p) {
  Pack<T, VEC> r;
  if constexpr (VEC * sizeof(T) == 16) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    __builtin_memcpy(&r, &w, 16);
  } else {
    static_assert(VEC == 1, "16 bytes or one element");
    r.e[0] = *p;
  }
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, VEC>& r) {
  if constexpr (VEC * sizeof(T) == 16) {
    uint4 w;
    __builtin_memcpy(&w, &r, 16);
    *reinterpret_cast<uint4*>(p) = w;
  } else {
    *p = r.e[0];
  }
}

// TILE: tokens per thread (1 for single tokens).
template <typename T, int VEC, int W, bool SILU, int TILE>
__global__ __launch_bounds__(kThreads) void conv_kernel(ConvArgs a, int tiles, int groups) {
  const unsigned idx = blockIdx.x * kThreads + threadIdx.x;
  const unsigned cg = idx % groups;
  const unsigned bt = idx / groups;
  const int tile = bt % tiles;
  const int b = bt / tiles;
  if (b >= a.B) return;
  const int n = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
  const int t0 = tile * TILE;
  if (t0 >= n && tile > 0) return;
  const int c = cg * VEC;

  using P = Pack<T, VEC>;
  const T* x = static_cast<const T*>(a.x) + static_cast<size_t>(b) * a.T * a.x_stride + c;
  const size_t state_row = static_cast<size_t>(a.C);
  const size_t state_at = static_cast<size_t>(b) * (W - 1) * state_row + c;

  // The W - 1 inputs before the tile.
  P win[W - 1];
  if (tile > 0) {
#pragma unroll
    for (int w = 0; w < W - 1; ++w)
      win[w] = load_pack<T, VEC>(x + static_cast<size_t>(t0 - (W - 1) + w) * a.x_stride);
  } else if (a.state_in) {
    const T* s = static_cast<const T*>(a.state_in) + state_at;
#pragma unroll
    for (int w = 0; w < W - 1; ++w) win[w] = load_pack<T, VEC>(s + w * state_row);
  } else {
#pragma unroll
    for (int w = 0; w < W - 1; ++w)
#pragma unroll
      for (int e = 0; e < VEC; ++e) win[w].e[e] = from_f32<T>(0.0f);
  }

  if (tile == 0) {
    // New state: rows n ... n + W - 2 of (old state, x).
    T* s = static_cast<T*>(a.state_out) + state_at;
    P row[W - 1];
#pragma unroll
    for (int w = 0; w < W - 1; ++w) {
      const int r = n + w;  // below W - 1: a row of the old state
      if (r >= W - 1) {
        row[w] = load_pack<T, VEC>(x + static_cast<size_t>(r - (W - 1)) * a.x_stride);
      } else {
        row[w] = win[0];
#pragma unroll
        for (int q = 1; q < W - 1; ++q)
          if (r == q) row[w] = win[q];
      }
    }
#pragma unroll
    for (int w = 0; w < W - 1; ++w) store_pack<T, VEC>(s + w * state_row, row[w]);
    if (n == 0) return;
  }

  float wt[VEC][W], bias[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if constexpr (W == 4) {
      const float4 q = *reinterpret_cast<const float4*>(a.weight + static_cast<size_t>(c + e) * 4);
      wt[e][0] = q.x;
      wt[e][1] = q.y;
      wt[e][2] = q.z;
      wt[e][3] = q.w;
    } else {
#pragma unroll
      for (int w = 0; w < W; ++w) wt[e][w] = a.weight[static_cast<size_t>(c + e) * W + w];
    }
    bias[e] = a.bias ? a.bias[c + e] : 0.0f;
  }

  // The output this channel group belongs to.
  const int which = c < a.c[0] ? 0 : (c < a.c[0] + a.c[1] ? 1 : 2);
  const int width = which == 0 ? a.c[0] : which == 1 ? a.c[1] : a.c[2];
  const int cy = c - (which > 0 ? a.c[0] : 0) - (which > 1 ? a.c[1] : 0);
  T* y = static_cast<T*>(which == 0 ? a.y[0] : which == 1 ? a.y[1] : a.y[2]) +
         static_cast<size_t>(b) * a.T * width + cy;

  float u[W][VEC];  // the window, oldest first; slot W - 1 takes the new input
#pragma unroll
  for (int w = 0; w < W - 1; ++w)
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[w][e] = to_f32(win[w].e[e]);

  constexpr int kAhead = TILE < 8 ? TILE : 8;  // rows requested together
  for (int tb = t0; tb < min(t0 + TILE, n); tb += kAhead) {
    P in[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      in[j] = load_pack<T, VEC>(x + static_cast<size_t>(min(tb + j, n - 1)) * a.x_stride);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      P out;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        u[W - 1][e] = to_f32(in[j].e[e]);
        float s = bias[e];
#pragma unroll
        for (int w = 0; w < W; ++w) s += wt[e][w] * u[w][e];
        out.e[e] = from_f32<T>(SILU ? silu_hw(s) : s);
#pragma unroll
        for (int w = 0; w < W - 1; ++w) u[w][e] = u[w + 1][e];
      }
      if (tb + j < n) store_pack<T, VEC>(y + static_cast<size_t>(tb + j) * width, out);
    }
  }
}

template <typename T, int VEC, int W, int TILE>
hipError_t launch_tile(const ConvArgs& a, hipStream_t stream) {
  const int groups = a.C / VEC;
  const int tiles = a.T > TILE ? (a.T + TILE - 1) / TILE : 1;
  const long long threads = static_cast<long long>(groups) * tiles * a.B;
  const dim3 grid(static_cast<unsigned>((threads + kThreads - 1) / kThreads));
  if (a.silu)
    hipLaunchKernelGGL((conv_kernel<T, VEC, W, true, TILE>), grid, dim3(kThreads), 0, stream, a,
                       tiles, groups);
  else
    hipLaunchKernelGGL((conv_kernel<T, VEC, W, false, TILE>), grid, dim3(kThreads), 0, stream, a,
                       tiles, groups);
  return hipGetLastError();
}

template <typename T, int VEC, int W>
hipError_t launch_w(const ConvArgs& a, hipStream_t stream) {
  if (a.T <= 1) return launch_tile<T, VEC, W, 1>(a, stream);
  // The longest tile (fewest rows read twice) that still gives kFill threads.
  const long long columns = static_cast<long long>(a.C / VEC) * a.B;
  auto fills = [&](int tile) { return columns * ((a.T + tile - 1) / tile) >= kFill; };
  if (fills(32)) return launch_tile<T, VEC, W, 32>(a, stream);
  if (fills(16)) return launch_tile<T, VEC, W, 16>(a, stream);
  if (fills(8)) return launch_tile<T, VEC, W, 8>(a, stream);
  return launch_tile<T, VEC, W, 4>(a, stream);
}

template <typename T, int VEC>
hipError_t launch_vec(const ConvArgs& a, hipStream_t stream) {
  switch (a.W) {
    case 2: return launch_w<T, VEC, 2>(a, stream);
    case 3: return launch_w<T, VEC, 3>(a, stream);
    default: return launch_w<T, VEC, 4>(a, stream);
  }
}

template <typename T>
hipError_t launch_io(const ConvArgs& a, hipStream_t stream) {
  // 16 bytes per thread where every row starts 16-byte aligned, else one
  // channel per thread.
  constexpr int VEC = 16 / static_cast<int>(sizeof(T));
  const bool wide = a.c[0] % VEC == 0 && a.c[1] % VEC == 0 && a.c[2] % VEC == 0 &&
                    a.x_stride % VEC == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
  return wide ? launch_vec<T, VEC>(a, stream) : launch_vec<T, 1>(a, stream);
}

}  // namespace

long long conv_max_grid(int B, int T, int C) {
  const long long tiles = T > 4 ? (static_cast<long long>(T) + 3) / 4 : 1;
  // Each factor is below 2^31; the product of the first two is checked before
  // the third can overflow 64 bits.
  const long long rows = tiles * B;
  if (rows > kMaxGrid * kThreads) return rows;
  return (rows * C + kThreads - 1) / kThreads;
}

hipError_t launch_conv(const ConvArgs& a, int io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_io<bf16>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace gdr
