// norm.hip -- root-mean-square norms of rows and their 8-bit form for gfx950.
//
//   h = x | x + residual | x silu(gate);  y = h / sqrt(mean h^2 + eps) w [silu(gate)]
//   s = max(amax / 448, 2^-100) per 128 channels, code = rne(y / s)
//
// A value is read once, kept in registers over the sum, and written once: bound by
// HBM, and by a launch and one chain of load, sum and store for few rows.  A thread
// owns vectors of 8 neighbouring channels (16 lanes are a block of 128 channels), so
// that a block's amax is an exchange inside 16 lanes; all loads of a thread are under
// way before the first is used.
//
// Heads of 16 to 512 channels (powers of two) lie within a wave: head_kernel, lanes
// of many heads side by side, no barrier.  Others take a workgroup a head:
// row_kernel, one barrier for the sum.  Rows that are not 16-byte aligned (ALIGNED
// false) are loaded and stored by the same vectors at any address, the last few
// channels of a row that is not of whole vectors one by one.
//
// Squares are summed in 64 bits: they cannot overflow, and rsqrt(mean + eps) = m 2^e
// is applied as h 2^e m, so rows of any finite magnitude keep their digits.
//
// 4000 x 4096 bf16 with a residual to 8 bits 20.7 us (115 MB, 5.6 TB/s), one row 3.2 us,
// 4000 x 8 heads x 512 gated 19.3 us, 4000 x 32 x 128 gated to 8 bits 20.0 us, plain rows
// 4000 x 4096 to 8 bits 11.7 us, 777 x 2501 fp32 9.0 us.
#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"
#include "kv_device.hpp"
#include "store_through.hpp"

namespace gdr {
namespace {

constexpr int kBlock = 128;           // channels that share a scale
constexpr float kMinScale = 0x1p-100f;

// x + y and max(x, y), y from the lane OFF further round a row of 16.
template <int OFF>
__device__ __forceinline__ unsigned rotated(unsigned x) {
  return __builtin_amdgcn_update_dpp(0u, x, 0x120 + OFF, 0xf, 0xf, false);  // row_ror:OFF
}
template <int OFF>
__device__ __forceinline__ double rotated(double x) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
  const unsigned lo = rotated<OFF>(static_cast<unsigned>(u));
  const unsigned hi = rotated<OFF>(static_cast<unsigned>(u >> 32));
  return __builtin_bit_cast(double, static_cast<unsigned long long>(hi) << 32 | lo);
}

// Sum over groups of N neighbouring lanes (N a power of two from 2 to 64).  Rotations
// by 8, 4, 2, 1 leave every lane of a row of 16 with the row's sum; for less than 16
// lanes, and across rows, lanes are exchanged through the LDS crossbar.
template <int N>
__device__ __forceinline__ double group_sum(double x) {
  if constexpr (N < 16) {
#pragma unroll
    for (int o = 1; o < N; o *= 2) x += __shfl_xor(x, o, 64);
  } else {
    x += rotated<8>(x);
    x += rotated<4>(x);
    x += rotated<2>(x);
    x += rotated<1>(x);
#pragma unroll
    for (int o = 16; o < N; o *= 2) x += __shfl_xor(x, o, 64);
  }
  return x;
}
// Largest of a row of 16 lanes.
__device__ __forceinline__ float row16_max(float x) {
  auto with = [](float v, unsigned r) { return fmaxf(v, __builtin_bit_cast(float, r)); };
  x = with(x, rotated<8>(__builtin_bit_cast(unsigned, x)));
  x = with(x, rotated<4>(__builtin_bit_cast(unsigned, x)));
  x = with(x, rotated<2>(__builtin_bit_cast(unsigned, x)));
  return with(x, rotated<1>(__builtin_bit_cast(unsigned, x)));
}

// 1 / sqrt(ss / n + eps) = m * p, p a power of two (exact also where fp32 holds it
// only as a subnormal).  The hardware's root is good to 2^-23; one step of Newton's
// method doubles the digits.  A sum that is infinite (as no finite h's is) has the root 0,
// which the step would turn into NaN.
struct Root {
  float m, p;
};
__device__ __forceinline__ Root inverse_root(double ss, double inverse_n, float eps) {
  const double v = ss * inverse_n + static_cast<double>(eps);
  double r = __builtin_amdgcn_rsq(v);
  r = r == 0.0 ? 0.0 : __builtin_fma(0.5 * r, __builtin_fma(-v * r, r, 1.0), r);
  return Root{static_cast<float>(__builtin_amdgcn_frexp_mant(r)),
              ldexpf(1.0f, __builtin_amdgcn_frexp_exp(r))};
}

// Eight neighbouring values in memory.
template <typename T>
struct Vec {
  T e[8];
};
template <typename T>
struct __attribute__((packed, aligned(1))) AnyVec {
  T e[8];
};

// `n` of them are there (8 where rows are ALIGNED).
template <typename T, bool ALIGNED>
__device__ __forceinline__ Vec<T> load_vec(const T* p, int n) {
  Vec<T> v;
  if constexpr (ALIGNED) {
#pragma unroll
    for (int c = 0; c < static_cast<int>(sizeof(T)) / 2; ++c) {
      const uint4 w = reinterpret_cast<const uint4*>(p)[c];
      __builtin_memcpy(&v.e[c * (16 / sizeof(T))], &w, 16);
    }
  } else if (n >= 8) {
    const AnyVec<T> a = *reinterpret_cast<const AnyVec<T>*>(p);
    __builtin_memcpy(&v, &a, sizeof(v));
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) v.e[u] = u < n ? p[u] : from_f32<T>(0.0f);
  }
  return v;
}
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[8], int n, int through) {
  Vec<T> v;
#pragma unroll
  for (int u = 0; u < 8; ++u) v.e[u] = from_f32<T>(x[u]);
  if constexpr (ALIGNED) {
#pragma unroll
    for (int c = 0; c < static_cast<int>(sizeof(T)) / 2; ++c) {
      through_u32x4 w;
      __builtin_memcpy(&w, &v.e[c * (16 / sizeof(T))], 16);
      if (sizeof(T) == 2 && through)  // fp32 takes two stores, each of half the bytes of a line
        store_through(p + c * (16 / sizeof(T)), w);
      else
        reinterpret_cast<through_u32x4*>(p)[c] = w;
    }
  } else if (n >= 8) {
    AnyVec<T> a;
    __builtin_memcpy(&a, &v, sizeof(v));
    *reinterpret_cast<AnyVec<T>*>(p) = a;
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (u < n) p[u] = v.e[u];
  }
}
template <bool ALIGNED>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[8], float inv, int n,
                                            int through) {
  through_u32x2 w;
  w.x = e4m3_pair(v[0] * inv, v[1] * inv) | e4m3_pair(v[2] * inv, v[3] * inv) << 16;
  w.y = e4m3_pair(v[4] * inv, v[5] * inv) | e4m3_pair(v[6] * inv, v[7] * inv) << 16;
  if constexpr (ALIGNED) {
    if (through)
      store_through(p, w);
    else
      *reinterpret_cast<through_u32x2*>(p) = w;
  } else if (n >= 8) {
    AnyVec<uint8_t> a;
    __builtin_memcpy(&a, &w, 8);
    *reinterpret_cast<AnyVec<uint8_t>*>(p) = a;
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (u < n) p[u] = static_cast<uint8_t>((u < 4 ? w.x : w.y) >> u % 4 * 8);
  }
}

// A thread's vectors: where they lie, and their values on the way from x to y.
template <typename T, bool ALIGNED, int NV>
struct Vectors {
  size_t row[NV];
  int col[NV];   // in the row
  int n[NV];     // channels that are there; 0: nothing
  float h[NV][8];
  Vec<T> z[NV];  // the gate, where it comes after the norm

  // h, and the residual's new values.
  __device__ __forceinline__ void load(const NormArgs& a, int W) {
    Vec<T> x[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (n[j] > 0)
        x[j] = load_vec<T, ALIGNED>(static_cast<const T*>(a.x) + row[j] * a.x_stride + col[j], n[j]);
    if (a.gate) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (n[j] > 0)
          z[j] = load_vec<T, ALIGNED>(
              static_cast<const T*>(a.gate) + row[j] * a.gate_stride + col[j], n[j]);
    }
    if (a.residual) {
      if (a.res_bf16)
        add<bf16>(a, W, x);
      else
        add<float>(a, W, x);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          h[j][u] = n[j] > 0 ? to_f32(x[j].e[u]) : 0.0f;
          if (a.gate && a.gate_first && n[j] > 0) h[j][u] *= silu_hw(to_f32(z[j].e[u]));
        }
    }
  }
  template <typename R>
  __device__ __forceinline__ void add(const NormArgs& a, int W, const Vec<T> (&x)[NV]) {
    R* residual = static_cast<R*>(a.residual);
    Vec<R> r[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (n[j] > 0) r[j] = load_vec<R, ALIGNED>(residual + row[j] * W + col[j], n[j]);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int u = 0; u < 8; ++u) h[j][u] = n[j] > 0 ? to_f32(x[j].e[u]) + to_f32(r[j].e[u]) : 0.0f;
      if (n[j] > 0) store_vec<R, ALIGNED>(residual + row[j] * W + col[j], h[j], n[j], a.through);
    }
  }
  __device__ __forceinline__ double squares(int j) const {
    double ss = 0.0;
#pragma unroll
    for (int u = 0; u < 8; ++u) ss = __builtin_fma(static_cast<double>(h[j][u]), h[j][u], ss);
    return ss;
  }
  // y in h's place; w: the weights of vector j, or nullptr.
  __device__ __forceinline__ void scale(const NormArgs& a, int j, Root r, const Vec<float>* w) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      h[j][u] = h[j][u] * r.p * r.m;
      if (w) h[j][u] *= w->e[u];
      if (a.gate && !a.gate_first) h[j][u] *= silu_hw(to_f32(z[j].e[u]));
    }
  }
  __device__ __forceinline__ void store(const NormArgs& a, int W) const {
    if (a.y) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (n[j] > 0)
          store_vec<T, ALIGNED>(static_cast<T*>(a.y) + row[j] * W + col[j], h[j], n[j], a.through);
    }
    if (!a.codes) return;
    const size_t blocks = (static_cast<size_t>(W) + kBlock - 1) / kBlock;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float top = 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) top = fmaxf(top, finite_abs(h[j][u]));
      const float s = fmaxf(row16_max(top) * (1.0f / kE4m3Max), kMinScale);
      if (n[j] > 0) {
        store_codes<ALIGNED>(a.codes + row[j] * W + col[j], h[j], 1.0f / s, n[j], a.through);
        if (threadIdx.x % 16 == 0) a.scales[row[j] * blocks + col[j] / kBlock] = s;
      }
    }
  }
};

// LANES lanes a head (of 8 LANES channels).  Every row is padded to whole blocks of
// 128 channels with lanes that have nothing, so that 16 lanes are a block.
template <typename T, bool ALIGNED, int LANES>
__global__ __launch_bounds__(256) void head_kernel(NormArgs a, unsigned slots, double inverse_n) {
  const int W = a.H * a.D;
  const unsigned idx = blockIdx.x * 256u + threadIdx.x;
  Vectors<T, ALIGNED, 1> v;
  v.row[0] = idx / slots;
  v.col[0] = idx % slots * 8;
  v.n[0] = v.row[0] < static_cast<size_t>(a.R) && v.col[0] < W ? 8 : 0;
  Vec<float> w;
  if (a.weight && v.n[0] > 0) w = load_vec<float, ALIGNED>(a.weight + v.col[0], 8);
  v.load(a, W);
  if (a.norm) {
    const Root r = inverse_root(group_sum<LANES>(v.squares(0)), inverse_n, a.eps);
    v.scale(a, 0, r, a.weight ? &w : nullptr);
  }
  v.store(a, W);
}

// A workgroup of NT threads for each (row, head), NV vectors a thread.
template <typename T, bool ALIGNED, int NT, int NV>
__global__ __launch_bounds__(NT) void row_kernel(NormArgs a, double inverse_n) {
  constexpr int NW = NT / 64;
  const size_t row = blockIdx.x / a.H;
  const int first = blockIdx.x % a.H * a.D, D = a.D, W = a.H * D;
  Vectors<T, ALIGNED, NV> v;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * NT + static_cast<int>(threadIdx.x)) * 8;
    v.row[j] = row;
    v.col[j] = first + c;
    v.n[j] = D - c;
  }
  constexpr bool kEarly = NV <= 2;  // weights with the rest; four vectors' would spill
  Vec<float> w[NV];
  auto weights = [&](int j) {
    if (v.n[j] > 0) w[j] = load_vec<float, ALIGNED>(a.weight + v.col[j], v.n[j]);
  };
  if (kEarly && a.weight) {
#pragma unroll
    for (int j = 0; j < NV; ++j) weights(j);
  }
  v.load(a, W);
  if (a.norm) {
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < NV; ++j) ss += v.squares(j);
    ss = group_sum<64>(ss);
    if constexpr (NW > 1) {
      __shared__ double part[NW];
      if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = ss;
      __syncthreads();
      ss = 0.0;
#pragma unroll
      for (int i = 0; i < NW; ++i) ss += part[i];
    }
    const Root r = inverse_root(ss, inverse_n, a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!kEarly && a.weight) weights(j);
      v.scale(a, j, r, a.weight ? &w[j] : nullptr);
    }
  }
  v.store(a, W);
}

template <typename T, bool ALIGNED, int LANES>
hipError_t launch_heads(const NormArgs& a, hipStream_t stream) {
  const unsigned slots = (a.H * a.D + kBlock - 1) / kBlock * 16;
  const unsigned vectors = static_cast<unsigned>(a.R) * slots;
  hipLaunchKernelGGL((head_kernel<T, ALIGNED, LANES>), dim3((vectors + 255) / 256), dim3(256), 0,
                     stream, a, slots, 1.0 / a.D);
  return hipGetLastError();
}

template <typename T, bool ALIGNED, int NT, int NV>
hipError_t launch_rows(const NormArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((row_kernel<T, ALIGNED, NT, NV>), dim3(static_cast<unsigned>(a.R) * a.H),
                     dim3(NT), 0, stream, a, 1.0 / a.D);
  return hipGetLastError();
}

template <typename T, bool ALIGNED>
hipError_t launch_sizes(const NormArgs& a, hipStream_t stream) {
  switch (a.D) {
    case 16: return launch_heads<T, ALIGNED, 2>(a, stream);
    case 32: return launch_heads<T, ALIGNED, 4>(a, stream);
    case 64: return launch_heads<T, ALIGNED, 8>(a, stream);
    case 128: return launch_heads<T, ALIGNED, 16>(a, stream);
    case 256: return launch_heads<T, ALIGNED, 32>(a, stream);
    case 512: return launch_heads<T, ALIGNED, 64>(a, stream);
    default: break;
  }
  // One vector a thread for few rows, two to four where rows fill the GPU (300 x 8192 7.6
  // against 7.9 us, 1000 x 8192 15.5 against 13.9).
  const bool few = static_cast<long long>(a.R) * a.H < 512;
  if (a.D <= 512) return launch_rows<T, ALIGNED, 64, 1>(a, stream);
  if (a.D <= 2048) return launch_rows<T, ALIGNED, 256, 1>(a, stream);
  if (a.D <= 4096)
    return few ? launch_rows<T, ALIGNED, 512, 1>(a, stream)
               : launch_rows<T, ALIGNED, 256, 2>(a, stream);
  if (a.D <= 8192)
    return few ? launch_rows<T, ALIGNED, 1024, 1>(a, stream)
               : launch_rows<T, ALIGNED, 256, 4>(a, stream);
  return launch_rows<T, ALIGNED, 1024, 4>(a, stream);
}

template <typename T>
hipError_t launch_io(const NormArgs& a, hipStream_t stream) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(T));
  auto rows_aligned = [&](const void* p, long long stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (stride % kPer == 0 || a.R == 1);
  };
  const bool aligned = a.D % 8 == 0 && rows_aligned(a.x, a.x_stride) &&
                       (!a.gate || rows_aligned(a.gate, a.gate_stride)) &&
                       reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
  return aligned ? launch_sizes<T, true>(a, stream) : launch_sizes<T, false>(a, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs& args, int io_bf16, hipStream_t stream) {
  NormArgs a = args;
  // Outputs that would fill the L2 caches go through them: 4000 x 4096 with a residual
  // 24.2 against 21.4 us, 4000 x 2048 14.8 against 13.0, 500 x 4096 5.9 against 5.6, one
  // row 3.7 against 3.9.
  // fp32 rows do not (2000 x 8192 with an fp32 residual 42.3 against 53.4).
  const long long width = (a.residual && a.res_bf16 ? 2 : 0) + (a.y && io_bf16 ? 2 : 0) +
                          (a.codes ? 1 : 0);
  a.through = width * a.R * a.H * a.D >= (4 << 20);
  return io_bf16 ? launch_io<bf16>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace gdr
