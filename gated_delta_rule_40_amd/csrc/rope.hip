// rope.hip -- rotary positions for gfx950: packed q|k|v rows split into dense
// tensors, the first R channels of each head of q and k turned.
//
//   (a, b) -> magnitude (a cos pf - b sin pf, a sin pf + b cos pf)
//
// A workgroup takes one or a few tokens.  It forms their R/2 sines and cosines once,
// in LDS, for all heads: the angle as 64-bit turns p f / 2 pi, of which only the part
// behind the point counts, so that far positions keep their digits.  Then every
// thread moves 16 bytes at a time (a pair of 16-byte pieces where the halves of a head
// are turned), the first ones loaded before the angles are formed.  (Two or four under
// way together are slower: 20.0 and 20.8 against 18.5 us for 4000 tokens of 48 heads of
// 128 in bf16.)  Bound by HBM, and by a launch and two chained loads for single tokens.
//
// 4000 tokens of 48 heads of 128 in bf16 18.3 us (98 MB, 5.4 TB/s), four ragged prompts
// of up to 2047 tokens with half of each head turned 13.3 us, 64 single tokens 3.4 us.
#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"
#include "store_through.hpp"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 1024;   // pairs of a workgroup's tokens, at most
constexpr long long kItems = 512;  // of a workgroup with more than one token, at most

// n / d by a multiplication with the rounded-up quotient of 2^32 and d (Granlund and
// Montgomery's method, exact for all 32-bit n).
struct Divisor {
  unsigned d, mul, one, more;
};
Divisor divisor(unsigned d) {
  unsigned bits = 0;
  while (bits < 32 && (1ull << bits) < d) ++bits;
  const unsigned long long mul = ((1ull << 32) * ((1ull << bits) - d)) / d + 1;
  return Divisor{d, static_cast<unsigned>(mul), bits < 1 ? bits : 1, bits > 1 ? bits - 1 : 0};
}
__device__ __forceinline__ unsigned divide(unsigned n, const Divisor& v) {
  const unsigned t = __umulhi(n, v.mul);
  return (t + ((n - t) >> v.one)) >> v.more;
}

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
__device__ __forceinline__ void store_piece(T* p, const Piece<T, VEC>& r, int through) {
  if constexpr (VEC * sizeof(T) == 16) {
    through_u32x4 w;
    __builtin_memcpy(&w, &r, 16);
    if (through)
      store_through(p, w);
    else
      *reinterpret_cast<through_u32x4*>(p) = w;
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

// What the kernel divides by: items of a token, items of a head, tokens of a row, pairs.
struct Divisors {
  Divisor items, per, T, half;
};

// VEC channels a piece: 16 bytes, or, where rows or pairs do not allow it, one
// (halves) or two (interleaved).  Items of a token: for each head of q and k its R / 2
// VEC pairs of pieces (halves) or R / VEC pieces (interleaved), then the pieces that
// are copied; then the pieces of v.
template <typename T, int VEC, bool INTER>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, int tokens, int total,
                                                        Divisors by) {
  __shared__ float2 turn[kTable];
  const int half = a.R / 2, D = a.D;
  const int row0 = blockIdx.x * tokens, rows = min(tokens, total - row0);
  const int turned = INTER ? a.R / VEC : half / VEC;   // items of a head that turn
  const int heads = a.H_q + a.H_kv;
  const int first_v = heads * static_cast<int>(by.per.d);
  const unsigned items = rows * by.items.d;
  Piece<T, VEC> v, z;
  T* to;              // nullptr: nothing to do
  const float2* cs;   // nullptr: copied

  auto load = [&](unsigned i) {
    to = nullptr;
    cs = nullptr;
    if (i >= items) return;
    const unsigned tok = divide(i, by.items), r = row0 + tok;
    int at = i - tok * by.items.d;
    if (a.lens) {
      const unsigned b = divide(r, by.T);
      if (static_cast<int>(r - b * by.T.d) >= a.lens[b]) return;
    }
    const T* x = static_cast<const T*>(a.x) + static_cast<size_t>(r) * a.x_stride;
    if (at >= first_v) {
      at = (at - first_v) * VEC;
      v = load_piece<T, VEC>(x + static_cast<size_t>(heads) * D + at);
      to = static_cast<T*>(a.v) + static_cast<size_t>(r) * a.H_kv * D + at;
      return;
    }
    const int head = divide(at, by.per);
    at -= head * static_cast<int>(by.per.d);
    const int c = at < turned ? at * VEC : a.R + (at - turned) * VEC;
    const T* from = x + static_cast<size_t>(head) * D + c;
    to = c + (head < a.H_q
                     ? static_cast<T*>(a.q) + (static_cast<size_t>(r) * a.H_q + head) * D
                     : static_cast<T*>(a.k) +
                           (static_cast<size_t>(r) * a.H_kv + head - a.H_q) * D);
    v = load_piece<T, VEC>(from);
    if (at < turned) {
      cs = turn + tok * half + (INTER ? c / 2 : c);
      if (!INTER) z = load_piece<T, VEC>(from + half);
    }
  };

  load(threadIdx.x);
  for (unsigned i = threadIdx.x; i < static_cast<unsigned>(rows * half); i += kThreads) {
    const unsigned tok = divide(i, by.half), r = row0 + tok, b = divide(r, by.T);
    const long long p = static_cast<long long>(a.pos[b]) + (r - b * by.T.d);
    const double t = static_cast<double>(p) * (a.freq[i - tok * half] * 0.15915494309189533576888);
    float s, c;
    sincospif(2.0f * static_cast<float>(t - rint(t)), &s, &c);
    turn[i] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  __syncthreads();

  for (unsigned i = threadIdx.x; i < items; load(i += kThreads)) {
    if (!to) continue;
    if (cs) {
      if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 w = cs[e / 2];
          const float p = to_f32(v.e[e]), q = to_f32(v.e[e + 1]);
          v.e[e] = from_f32<T>(turn_first(p, q, w));
          v.e[e + 1] = from_f32<T>(turn_second(p, q, w));
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float2 w = cs[e];
          const float p = to_f32(v.e[e]), q = to_f32(z.e[e]);
          v.e[e] = from_f32<T>(turn_first(p, q, w));
          z.e[e] = from_f32<T>(turn_second(p, q, w));
        }
        store_piece<T, VEC>(to + half, z, a.through);
      }
    }
    store_piece<T, VEC>(to, v, a.through);
  }
}

template <typename T, int VEC, bool INTER>
hipError_t launch_vec(const RopeArgs& a, hipStream_t stream) {
  const int total = a.B * a.T, half = a.R / 2;
  const unsigned per = (INTER ? a.R / VEC : half / VEC) + (a.D - a.R) / VEC;
  const unsigned items =
      (a.H_q + a.H_kv) * per + (a.v ? static_cast<unsigned>(a.H_kv) * (a.D / VEC) : 0);
  // Tokens of a workgroup: as many as its threads take in two items each and the table
  // holds the pairs of, as long as that gives two workgroups a CU.
  int tokens = 1;
  while (tokens < 16 && items * (tokens * 2ll) <= kItems && half * (tokens * 2) <= kTable &&
         total / (tokens * 2) >= 512)
    tokens *= 2;
  const Divisors by = {divisor(items), divisor(per), divisor(a.T), divisor(half ? half : 1)};
  hipLaunchKernelGGL((rope_kernel<T, VEC, INTER>), dim3((total + tokens - 1) / tokens),
                     dim3(kThreads), 0, stream, a, tokens, total, by);
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

hipError_t launch_rope(const RopeArgs& args, int io_bf16, hipStream_t stream) {
  RopeArgs a = args;
  // Outputs that would fill the L2 caches go through them: 4000 tokens of 48 heads of 128
  // 19.5 against 18.3 us, 500 5.1 against 5.2, 64 3.9 against 4.5.
  const long long out = static_cast<long long>(a.B) * a.T * (a.H_q + (a.v ? 2 : 1) * a.H_kv) *
                        a.D * (io_bf16 ? 2 : 4);
  a.through = out >= (16 << 20);
  return io_bf16 ? launch_io<bf16>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace gdr
