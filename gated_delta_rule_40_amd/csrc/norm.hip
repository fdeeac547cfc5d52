// norm.hip -- root-mean-square norms of rows and their 8-bit form for gfx950.
//
//   h = x | x + residual | x silu(gate);  y = h / sqrt(mean h^2 + eps) w [silu(gate)]
//   s = max(amax / 448, 2^-100) per 128 channels, code = rne(y / s)
//
// A value is read once, kept in registers over the sum, and written once: bound by
// HBM, and by a launch and one chain of load, sum and store for few rows.  A thread
// owns vectors of 8 neighbouring channels (16 lanes are a block of 128 channels), so
// that a block's amax is a sum-like exchange inside 16 lanes.
//
// Heads of 16 to 512 channels (powers of two) lie within a wave: head_kernel, lanes
// of many heads side by side, no barrier.  Others take a workgroup a head:
// row_kernel, one barrier for the sum.  Inputs that are not 16-byte aligned are loaded
// by elements (WIDE false); rows that are not of whole vectors take row_kernel with
// one channel at a time, a wave's 64 lanes twice over a block.
//
// Squares are summed in 64 bits: they cannot overflow, and rsqrt(mean + eps) = m 2^e
// is applied as h 2^e m, so rows of any finite magnitude keep their digits.
#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"
#include "kv_device.hpp"

namespace gdr {
namespace {

constexpr int kBlock = 128;           // channels that share a scale
constexpr float kMinScale = 0x1p-100f;

// Sum and maximum over the lanes that share lane / N (N a power of two up to 64).
template <int N>
__device__ __forceinline__ double group_sum(double x) {
#pragma unroll
  for (int o = 1; o < N; o *= 2) x += __shfl_xor(x, o, 64);
  return x;
}
template <int N>
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
  for (int o = 1; o < N; o *= 2) x = fmaxf(x, __shfl_xor(x, o, 64));
  return x;
}

// 1 / sqrt(ss / n + eps) = m * p, p a power of two (exact also where fp32 holds it
// only as a subnormal).
struct Root {
  float m, p;
};
__device__ __forceinline__ Root inverse_root(double ss, int n, float eps) {
  const double r = 1.0 / sqrt(ss / n + static_cast<double>(eps));
  int e = 0;
  const double m = frexp(r, &e);
  return Root{static_cast<float>(m), ldexpf(1.0f, e)};
}

// The scale of a block and its inverse.
__device__ __forceinline__ float block_scale(float amax) {
  return fmaxf(amax * (1.0f / kE4m3Max), kMinScale);
}

template <typename T, int VEC, bool WIDE = true>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 1 || !WIDE) {
#pragma unroll
    for (int u = 0; u < VEC; ++u) v[u] = to_f32(p[u]);
  } else {
    load_row<T, VEC>(p, v);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    *p = from_f32<T>(v[0]);
  } else {
    T e[VEC];
#pragma unroll
    for (int u = 0; u < VEC; ++u) e[u] = from_f32<T>(v[u]);
#pragma unroll
    for (int c = 0; c < VEC * static_cast<int>(sizeof(T)) / 16; ++c)
      reinterpret_cast<uint4*>(p)[c] = reinterpret_cast<const uint4*>(e)[c];
  }
}

__device__ __forceinline__ void store_codes8(uint8_t* p, const float (&v)[8], float inv) {
  uint2 w;
  w.x = e4m3_pair(v[0] * inv, v[1] * inv) | e4m3_pair(v[2] * inv, v[3] * inv) << 16;
  w.y = e4m3_pair(v[4] * inv, v[5] * inv) | e4m3_pair(v[6] * inv, v[7] * inv) << 16;
  *reinterpret_cast<uint2*>(p) = w;
}

// h of VEC channels from `at` of a row (x, gate) or of the dense tensors
// (residual, which takes h).  g: silu of the gate where it comes after the norm.
template <typename T, int VEC, bool WIDE>
__device__ __forceinline__ void form_h(const NormArgs& a, size_t row, size_t col, float (&h)[VEC],
                                       float (&g)[VEC]) {
  load_vec<T, VEC, WIDE>(static_cast<const T*>(a.x) + row * a.x_stride + col, h);
  if (a.residual) {
    const size_t at = row * (static_cast<size_t>(a.H) * a.D) + col;
    float r[VEC];
    if (a.res_bf16) {
      bf16* p = static_cast<bf16*>(a.residual) + at;
      load_vec<bf16, VEC>(p, r);
#pragma unroll
      for (int u = 0; u < VEC; ++u) h[u] += r[u];
      store_vec<bf16, VEC>(p, h);
    } else {
      float* p = static_cast<float*>(a.residual) + at;
      load_vec<float, VEC>(p, r);
#pragma unroll
      for (int u = 0; u < VEC; ++u) h[u] += r[u];
      store_vec<float, VEC>(p, h);
    }
  }
  if (a.gate) {
    load_vec<T, VEC, WIDE>(static_cast<const T*>(a.gate) + row * a.gate_stride + col, g);
#pragma unroll
    for (int u = 0; u < VEC; ++u) g[u] = silu_hw(g[u]);
    if (a.gate_first) {
#pragma unroll
      for (int u = 0; u < VEC; ++u) h[u] *= g[u];
    }
  }
}

// y of VEC channels; w points at their weights.
template <int VEC, bool WIDE>
__device__ __forceinline__ void form_y(const NormArgs& a, Root r, const float* w, float (&h)[VEC],
                                       const float (&g)[VEC]) {
#pragma unroll
  for (int u = 0; u < VEC; ++u) h[u] = h[u] * r.p * r.m;
  if (w) {
    float wt[VEC];
    load_vec<float, VEC, WIDE>(w, wt);
#pragma unroll
    for (int u = 0; u < VEC; ++u) h[u] *= wt[u];
  }
  if (a.gate && !a.gate_first) {
#pragma unroll
    for (int u = 0; u < VEC; ++u) h[u] *= g[u];
  }
}

// LANES lanes a head (of 8 LANES channels).  Every row is padded to whole blocks of
// 128 channels with lanes that have nothing, so that 16 lanes are a block.
template <typename T, int LANES, bool WIDE>
__global__ __launch_bounds__(256) void head_kernel(NormArgs a, unsigned slots) {
  const unsigned idx = blockIdx.x * 256u + threadIdx.x;  // rows times slots are within 2^30
  const size_t row = idx / slots;
  const unsigned slot = idx % slots;
  const int W = a.H * a.D;
  const bool on = row < static_cast<size_t>(a.R) && slot * 8 < static_cast<unsigned>(W);
  float h[8] = {}, g[8] = {};
  if (on) form_h<T, 8, WIDE>(a, row, slot * 8, h, g);
  if (a.norm) {
    double ss = 0.0;
#pragma unroll
    for (int u = 0; u < 8; ++u) ss += static_cast<double>(h[u]) * h[u];
    const Root r = inverse_root(group_sum<LANES>(ss), a.D, a.eps);
    if (on) form_y<8, WIDE>(a, r, a.weight ? a.weight + slot * 8 : nullptr, h, g);
  }
  if (on && a.y) store_vec<T, 8>(static_cast<T*>(a.y) + row * W + slot * 8, h);
  if (a.codes) {
    float top = 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) top = fmaxf(top, finite_abs(h[u]));
    const float s = block_scale(group_max<16>(top));
    if (on) {
      store_codes8(a.codes + row * W + slot * 8, h, 1.0f / s);
      if (slot % 16 == 0) a.scales[row * (slots / 16) + slot / 16] = s;
    }
  }
}

// A workgroup of NT threads for each (row, head), NV vectors of VEC channels a thread.
template <typename T, int VEC, int NT, int NV, bool WIDE>
__global__ __launch_bounds__(NT) void row_kernel(NormArgs a) {
  constexpr int NW = NT / 64;
  static_assert(VEC == 8 || NV % 2 == 0, "a wave's lanes go twice over a block");
  const size_t row = blockIdx.x / a.H;
  const int head = blockIdx.x % a.H, D = a.D;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const size_t W = static_cast<size_t>(a.H) * D, col0 = static_cast<size_t>(head) * D;
  // Channel of a thread's vector j within the head.
  auto channel = [&](int j) {
    if constexpr (VEC == 8) return (j * NT + static_cast<int>(threadIdx.x)) * 8;
    return ((j / 2) * NW + wave) * kBlock + (j % 2) * 64 + lane;
  };
  float h[NV][VEC], g[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = channel(j);
#pragma unroll
    for (int u = 0; u < VEC; ++u) h[j][u] = g[j][u] = 0.0f;
    if (c < D) form_h<T, VEC, WIDE>(a, row, col0 + c, h[j], g[j]);
  }
  if (a.norm) {
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int u = 0; u < VEC; ++u) ss += static_cast<double>(h[j][u]) * h[j][u];
    ss = group_sum<64>(ss);
    if constexpr (NW > 1) {
      __shared__ double part[NW];
      if (lane == 0) part[wave] = ss;
      __syncthreads();
      ss = 0.0;
#pragma unroll
      for (int w = 0; w < NW; ++w) ss += part[w];
    }
    const Root r = inverse_root(ss, D, a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel(j);
      if (c < D) form_y<VEC, WIDE>(a, r, a.weight ? a.weight + col0 + c : nullptr, h[j], g[j]);
    }
  }
  if (a.y) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel(j);
      if (c < D) store_vec<T, VEC>(static_cast<T*>(a.y) + row * W + col0 + c, h[j]);
    }
  }
  if (!a.codes) return;
  float* scales = a.scales + row * ((W + kBlock - 1) / kBlock) + col0 / kBlock;
  uint8_t* codes = a.codes + row * W + col0;
  if constexpr (VEC == 8) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel(j);
      float top = 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) top = fmaxf(top, finite_abs(h[j][u]));
      const float s = block_scale(group_max<16>(top));
      if (c < D) {
        store_codes8(codes + c, h[j], 1.0f / s);
        if (lane % 16 == 0) scales[c / kBlock] = s;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; j += 2) {
      const int c = channel(j);
      const float s = block_scale(
          group_max<64>(fmaxf(finite_abs(h[j][0]), finite_abs(h[j + 1][0]))));
      const unsigned pair = e4m3_pair(h[j][0] * (1.0f / s), h[j + 1][0] * (1.0f / s));
      if (c < D) codes[c] = static_cast<uint8_t>(pair);
      if (c + 64 < D) codes[c + 64] = static_cast<uint8_t>(pair >> 8);
      if (lane == 0 && c < D) scales[c / kBlock] = s;
    }
  }
}

template <typename T, int LANES, bool WIDE>
hipError_t launch_heads(const NormArgs& a, hipStream_t stream) {
  const unsigned slots = (a.H * a.D + kBlock - 1) / kBlock * 16;
  const unsigned threads = static_cast<unsigned>(a.R) * slots;
  hipLaunchKernelGGL((head_kernel<T, LANES, WIDE>), dim3((threads + 255) / 256), dim3(256), 0,
                     stream, a, slots);
  return hipGetLastError();
}

template <typename T, int VEC, int NT, int NV, bool WIDE>
hipError_t launch_rows(const NormArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((row_kernel<T, VEC, NT, NV, WIDE>),
                     dim3(static_cast<unsigned>(a.R) * a.H), dim3(NT), 0, stream, a);
  return hipGetLastError();
}

template <typename T, bool WIDE>
hipError_t launch_vectors(const NormArgs& a, hipStream_t stream) {
  switch (a.D) {
    case 16: return launch_heads<T, 2, WIDE>(a, stream);
    case 32: return launch_heads<T, 4, WIDE>(a, stream);
    case 64: return launch_heads<T, 8, WIDE>(a, stream);
    case 128: return launch_heads<T, 16, WIDE>(a, stream);
    case 256: return launch_heads<T, 32, WIDE>(a, stream);
    case 512: return launch_heads<T, 64, WIDE>(a, stream);
    default: break;
  }
  if (a.D <= 512) return launch_rows<T, 8, 64, 1, WIDE>(a, stream);
  if (a.D <= 2048) return launch_rows<T, 8, 256, 1, WIDE>(a, stream);
  if (a.D <= 4096) return launch_rows<T, 8, 256, 2, WIDE>(a, stream);
  if (a.D <= 8192) return launch_rows<T, 8, 256, 4, WIDE>(a, stream);
  return launch_rows<T, 8, 1024, 4, WIDE>(a, stream);
}

template <typename T>
hipError_t launch_io(const NormArgs& a, hipStream_t stream) {
  if (a.D % 8 != 0) {  // H = 1
    if (a.D <= 512) return launch_rows<T, 1, 64, 8, false>(a, stream);
    if (a.D <= 4096) return launch_rows<T, 1, 256, 16, false>(a, stream);
    return launch_rows<T, 1, 1024, 32, false>(a, stream);
  }
  constexpr int kPer = 16 / static_cast<int>(sizeof(T));
  auto rows_aligned = [&](const void* p, long long stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (stride % kPer == 0 || a.R == 1);
  };
  const bool wide = rows_aligned(a.x, a.x_stride) &&
                    (!a.gate || rows_aligned(a.gate, a.gate_stride)) &&
                    reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
  return wide ? launch_vectors<T, true>(a, stream) : launch_vectors<T, false>(a, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_io<bf16>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace gdr
