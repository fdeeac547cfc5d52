// rope.hip -- rotary positions for gfx950: packed q|k|v rows split into dense
// tensors, the first R channels of each head of q and k turned.
//
//   (a, b) -> magnitude (a cos pf - b sin pf, a sin pf + b cos pf)
//
// A workgroup takes one or a few tokens.  It forms their R/2 sines and cosines once,
// in LDS, for all heads: the angle as 64-bit turns p f / 2 pi, of which only the part
// behind the point counts, so that far positions keep their digits.  Then every
// thread moves 16 bytes (a pair of 16-byte pieces where the halves of a head are
// turned).  Bound by HBM, and by a launch and two chained loads for single tokens.
#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 256;   // R / 2
constexpr int kMaxTokens = 16;   // tokens of a workgroup

template <typename T, int VEC>
struct Piece {
  T e[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> load_piece(const T* p) {
  Piece<T, VEC> r;
  if constexpr (VEC * sizeof(T) == 16) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    __builtin_memcpy(&r, &w, 16);
  } else {
#pragma unroll
    for (int u = 0; u < VEC; ++u) r.e[u] = p[u];
  }
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, VEC>& r) {
  if constexpr (VEC * sizeof(T) == 16) {
    uint4 w;
    __builtin_memcpy(&w, &r, 16);
    *reinterpret_cast<uint4*>(p) = w;
  } else {
#pragma unroll
    for (int u = 0; u < VEC; ++u) p[u] = r.e[u];
  }
}

// A pair (p, q) turned by w = (cos, sin); which product is rounded is fixed, so that
// every form of the kernel gives the same digits.
__device__ __forceinline__ float turn_first(float p, float q, float2 w) {
  return __builtin_fmaf(p, w.x, -(q * w.y));
}
__device__ __forceinline__ float turn_second(float p, float q, float2 w) {
  return __builtin_fmaf(p, w.y, q * w.x);
}

// VEC channels a piece: 16 bytes, or, where rows or pairs do not allow it, one
// (halves) or two (interleaved).  Items of a token: R / 2 VEC pairs of pieces
// (halves) or R / VEC pieces (interleaved) of a head of q and k, and the pieces that
// are copied.
template <typename T, int VEC, bool INTER>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, int tokens, int total) {
  __shared__ float2 turn[kMaxPairs * kMaxTokens];
  const int half = a.R / 2, D = a.D;
  const int row0 = blockIdx.x * tokens, rows = min(tokens, total - row0);
  for (int i = threadIdx.x; i < rows * half; i += kThreads) {
    const int r = row0 + i / half, f = i % half;
    const long long p = static_cast<long long>(a.pos[r / a.T]) + r % a.T;
    const double t = static_cast<double>(p) * (a.freq[f] * 0.15915494309189533576888);
    float s, c;
    sincospif(2.0f * static_cast<float>(t - rint(t)), &s, &c);
    turn[i] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  __syncthreads();

  const int turned = INTER ? a.R / VEC : half / VEC;   // items of a head that turn
  const int moved = (D - a.R) / VEC;                   // items of a head that do not
  const int per = turned + moved, plain = D / VEC;
  const int heads = a.H_q + a.H_kv;
  const int items = heads * per + (a.v ? a.H_kv * plain : 0);
  for (int i = threadIdx.x; i < rows * items; i += kThreads) {
    const int tok = i / items, r = row0 + tok, b = r / a.T;
    if (a.lens && r % a.T >= a.lens[b]) continue;
    const T* x = static_cast<const T*>(a.x) + static_cast<size_t>(r) * a.x_stride;
    int at = i % items;
    if (at >= heads * per) {  // v
      at -= heads * per;
      const T* from = x + static_cast<size_t>(heads) * D + at * VEC;
      T* to = static_cast<T*>(a.v) + static_cast<size_t>(r) * a.H_kv * D + at * VEC;
      store_piece<T, VEC>(to, load_piece<T, VEC>(from));
      continue;
    }
    const int head = at / per;
    at %= per;
    const T* from = x + static_cast<size_t>(head) * D;
    T* to = head < a.H_q
                ? static_cast<T*>(a.q) + (static_cast<size_t>(r) * a.H_q + head) * D
                : static_cast<T*>(a.k) + (static_cast<size_t>(r) * a.H_kv + head - a.H_q) * D;
    if (at >= turned) {
      const int c = a.R + (at - turned) * VEC;
      store_piece<T, VEC>(to + c, load_piece<T, VEC>(from + c));
      continue;
    }
    const float2* cs = turn + tok * half;
    if constexpr (INTER) {
      Piece<T, VEC> v = load_piece<T, VEC>(from + at * VEC);
#pragma unroll
      for (int u = 0; u < VEC; u += 2) {
        const float2 w = cs[(at * VEC + u) / 2];
        const float p = to_f32(v.e[u]), q = to_f32(v.e[u + 1]);
        v.e[u] = from_f32<T>(turn_first(p, q, w));
        v.e[u + 1] = from_f32<T>(turn_second(p, q, w));
      }
      store_piece<T, VEC>(to + at * VEC, v);
    } else {
      Piece<T, VEC> v = load_piece<T, VEC>(from + at * VEC);
      Piece<T, VEC> z = load_piece<T, VEC>(from + half + at * VEC);
#pragma unroll
      for (int u = 0; u < VEC; ++u) {
        const float2 w = cs[at * VEC + u];
        const float p = to_f32(v.e[u]), q = to_f32(z.e[u]);
        v.e[u] = from_f32<T>(turn_first(p, q, w));
        z.e[u] = from_f32<T>(turn_second(p, q, w));
      }
      store_piece<T, VEC>(to + at * VEC, v);
      store_piece<T, VEC>(to + half + at * VEC, z);
    }
  }
}

template <typename T, int VEC, bool INTER>
hipError_t launch_vec(const RopeArgs& a, hipStream_t stream) {
  const int total = a.B * a.T, tokens = 1;
  hipLaunchKernelGGL((rope_kernel<T, VEC, INTER>), dim3((total + tokens - 1) / tokens),
                     dim3(kThreads), 0, stream, a, tokens, total);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_io(const RopeArgs& a, hipStream_t stream) {
  constexpr int VEC = 16 / static_cast<int>(sizeof(T));
  const bool rows = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                    (a.x_stride % VEC == 0 || a.B * a.T == 1);
  if (a.interleaved)
    return rows && a.R % VEC == 0 ? launch_vec<T, VEC, true>(a, stream)
                                  : launch_vec<T, 2, true>(a, stream);
  return rows && a.R % (2 * VEC) == 0 ? launch_vec<T, VEC, false>(a, stream)
                                      : launch_vec<T, 1, false>(a, stream);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_io<bf16>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace gdr
