// kv_append.hip -- keys and values of new tokens into pages of e4m3 codes, one
// power-of-two scale per (page, head).
//
// With a power of two, scaling a value and shifting a code to a larger scale
// are exact but for the rounding to e4m3's subnormals, so a page that takes
// tokens one by one holds (nearly) what it would hold if they had come at
// once: a growing scale costs no precision each time.
//
// One workgroup per (row, page it may touch, head, keys or values).  A thread
// takes 4 neighbouring slots x 8 channels: it loads the new tokens among them
// once, keeps them in registers while the workgroup finds the largest
// magnitude, and then writes 8 bytes a slot (keys) or 4 bytes a channel
// (transposed values), rewriting older codes only if the scale grew.  Keys:
// neighbouring threads along the channels, 16 D/8 bytes of a token together;
// values: along the slots, so that a channel's row of the page goes out whole.
// Bound by latency, one round of loads and one of stores around the reduction: 4
// prompts of 1024 to 2047 tokens, 8 heads of 128 in bf16, 38 MB, take 13 us (2.9
// TB/s) where a copy of that size takes 7.
#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"
#include "kv_device.hpp"
#include "kv_slots.hpp"

namespace gdr {
namespace {

constexpr int kMaxThreads = 256;

// The codes in a word, shifted to a scale 1 / ratio times theirs.
__device__ __forceinline__ unsigned rescale(unsigned w, float ratio) {
  const unsigned lo = e4m3_pair(e4m3_value(w & 0xff) * ratio, e4m3_value((w >> 8) & 0xff) * ratio);
  const unsigned hi =
      e4m3_pair(e4m3_value((w >> 16) & 0xff) * ratio, e4m3_value(w >> 24) * ratio);
  return lo | hi << 16;
}

// What workgroup `wg` writes: the slots of one page, of one head's keys or values.
struct Target : KvSlots {
  int b, head, is_v;
  int id;  // the page's number, unchecked
};
__device__ __forceinline__ Target target_of(const KvArgs& a, unsigned wg, int touched) {
  Target t = {};
  t.is_v = wg & 1;
  wg >>= 1;
  t.head = wg % a.H_kv;
  wg /= a.H_kv;
  const int j = wg % touched;
  t.b = wg / touched;
  const int n = a.lens ? min(max(a.lens[t.b], 0), a.T) : a.T;
  const int pos = a.pos[t.b];
  const long long page_no = static_cast<long long>(max(pos, 0) / a.page) + j;
  if (page_no >= a.max_pages) return t;
  static_cast<KvSlots&>(t) = kv_slots(pos, n, page_no, a.page);
  t.id = a.block_table[static_cast<size_t>(t.b) * a.max_pages + page_no];
  return t;
}

// Calls of at most this many tokens a row go one wave per (page, head, keys or
// values), a lane per D/64 channels: a short chain of loads and little code.
// One token for 64 requests, 8 heads, pages of 64: 10.1 us as in a prompt, 4.7 us
// like this.
constexpr int kFewTokens = 8;

template <typename T, int D>
__global__ __launch_bounds__(64) void kv_append_few_kernel(KvArgs a, int touched) {
  constexpr int CH = D / 64;  // neighbouring channels of a lane
  const int lane = threadIdx.x;
  const Target t = target_of(a, blockIdx.x, touched);
  if (t.u >= t.w) return;
  const size_t tok = static_cast<size_t>(a.H_kv) * D;
  const T* src = static_cast<const T*>(t.is_v ? a.v : a.k) +
                 (static_cast<size_t>(t.b) * a.T + t.first) * tok +
                 static_cast<size_t>(t.head) * D + lane * CH;
  const int n = t.w - t.u;
  float x[kFewTokens][CH];
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < kFewTokens; ++k) {
    if (k >= n) break;
    load_row<T, CH>(src + k * tok, x[k]);
#pragma unroll
    for (int c = 0; c < CH; ++c) amax = fmaxf(amax, finite_abs(x[k][c]));
  }
  if (t.id < 0 || t.id >= a.n_pages) return;
  const size_t ph = static_cast<size_t>(t.id) * a.H_kv + t.head;
  uint8_t* cache = (t.is_v ? a.v_cache : a.k_cache) + ph * a.page * D;
  float* scale = (t.is_v ? a.v_scale : a.k_scale) + ph;
  const float was = t.had > 0 ? *scale : 0.0f;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
  float now = e4m3_scale(amax);
  if (t.had > 0) now = fmaxf(now, was);
  const float inv = pow2_inverse(now);
  if (t.had > 0 && now > was) {
    // Older codes, a word of 4 at a time: keys lie one after another, a
    // channel's values in the first `had` bytes of its row.
    const float ratio = was * inv;
    const int words = t.is_v ? (t.had + 3) / 4 : t.had * (D / 4);
    const int rows = t.is_v ? D : 1;
    for (int i = lane; i < rows * words; i += 64) {
      const int k = i % words;
      unsigned* p = reinterpret_cast<unsigned*>(cache + (i / words) * a.page) + k;
      const int left = t.is_v ? t.had - 4 * k : 4;
      const unsigned old = left >= 4 ? ~0u : (1u << (8 * left)) - 1;
      const unsigned h = *p;
      *p = (rescale(h, ratio) & old) | (h & ~old);
    }
    // A lane's new bytes may lie in a word that another lane has rewritten.
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
  }
#pragma unroll
  for (int k = 0; k < kFewTokens; ++k) {
    if (k >= n) break;
    const unsigned c = e4m3_pair(x[k][0] * inv, x[k][CH - 1] * inv);
    if (t.is_v) {
#pragma unroll
      for (int e = 0; e < CH; ++e)
        cache[(lane * CH + e) * a.page + t.u + k] = static_cast<uint8_t>(c >> (8 * e));
    } else if constexpr (CH == 2) {
      *reinterpret_cast<uint16_t*>(cache + (t.u + k) * D + 2 * lane) = static_cast<uint16_t>(c);
    } else {
      cache[(t.u + k) * D + lane] = static_cast<uint8_t>(c);
    }
  }
  if (lane == 0) *scale = now;
}

// UNITS: units of 4 slots x 8 channels per thread.
template <typename T, int D, int UNITS>
__global__ __launch_bounds__(kMaxThreads) void kv_append_kernel(KvArgs a, int touched) {
  constexpr int DG = D / 8;
  __shared__ float red[kMaxThreads / 64];
  const int tid = threadIdx.x, nt = blockDim.x;
  const Target t = target_of(a, blockIdx.x, touched);
  if (t.u >= t.w) return;
  const int u = t.u, w = t.w, had = t.had, id = t.id, head = t.head;
  const bool is_v = t.is_v;

  const int page = a.page, quads = page / 4;
  const size_t tok = static_cast<size_t>(a.H_kv) * D;
  // The new token of slot s is at src + (s - u) tok.
  const T* src = static_cast<const T*>(is_v ? a.v : a.k) +
                 (static_cast<size_t>(t.b) * a.T + t.first) * tok + static_cast<size_t>(head) * D;

  float x[UNITS][4][8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int unit = tid + i * nt;
    const int quad = is_v ? unit % quads : unit / DG, dg = is_v ? unit / quads : unit % DG;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = 4 * quad + k;
      if (unit < quads * DG && s >= u && s < w) {
        load_row<T, 8>(src + (s - u) * tok + 8 * dg, x[i][k]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][k][e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite_abs(x[i][k][e]));
    }
  }
  // The page is looked at only now: its number and the new values were under
  // way together.
  if (id < 0 || id >= a.n_pages) return;
  const size_t ph = static_cast<size_t>(id) * a.H_kv + head;
  uint8_t* cache = (is_v ? a.v_cache : a.k_cache) + ph * page * D;
  float* scale = (is_v ? a.v_scale : a.k_scale) + ph;
  const float was = had > 0 ? *scale : 0.0f;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
  if ((tid & 63) == 0) red[tid >> 6] = amax;
  __syncthreads();
  for (int k = 0; k < nt / 64; ++k) amax = fmaxf(amax, red[k]);
  float now = e4m3_scale(amax);
  if (had > 0) now = fmaxf(now, was);
  const float inv = pow2_inverse(now);
  const bool grown = had > 0 && now > was;
  const float ratio = was * inv;

#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int unit = tid + i * nt;
    if (unit >= quads * DG) break;
    const int quad = is_v ? unit % quads : unit / DG, dg = is_v ? unit / quads : unit % DG;
    const int s0 = 4 * quad;
    if (s0 >= w || (s0 + 4 <= u && !grown)) continue;
    unsigned code[4][4];  // [slot][pair of channels]
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        code[k][e] = e4m3_pair(x[i][k][2 * e] * inv, x[i][k][2 * e + 1] * inv);
    if (!is_v) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint2* p = reinterpret_cast<uint2*>(cache + (s0 + k) * D + 8 * dg);
        if (s0 + k >= u && s0 + k < w) {
          *p = make_uint2(code[k][0] | code[k][1] << 16, code[k][2] | code[k][3] << 16);
        } else if (grown && s0 + k < had) {
          const uint2 c = *p;
          *p = make_uint2(rescale(c.x, ratio), rescale(c.y, ratio));
        }
      }
    } else {
      // Bytes of the word: 0xff for a new slot; for an old one where the scale grew.
      unsigned fresh = 0, old = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (s0 + k >= u && s0 + k < w) fresh |= 0xffu << (8 * k);
        if (grown && s0 + k < had) old |= 0xffu << (8 * k);
      }
      uint8_t* row = cache + 8 * dg * page + s0;
      unsigned word[8], here[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        word[e] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) word[e] |= (code[k][e / 2] >> (8 * (e & 1)) & 0xffu) << (8 * k);
      }
      if (old) {  // requested together, ahead of the stores
#pragma unroll
        for (int e = 0; e < 8; ++e) here[e] = *reinterpret_cast<const unsigned*>(row + e * page);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          word[e] = (word[e] & fresh) | (rescale(here[e], ratio) & old) | (here[e] & ~(fresh | old));
      }
      if (old || fresh == 0xffffffffu) {
#pragma unroll
        for (int e = 0; e < 8; ++e) *reinterpret_cast<unsigned*>(row + e * page) = word[e];
      } else {  // single bytes: nothing has to be read first
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (s0 + k >= u && s0 + k < w)
#pragma unroll
            for (int e = 0; e < 8; ++e) row[e * page + k] = static_cast<uint8_t>(word[e] >> (8 * k));
      }
    }
  }
  if (tid == 0) *scale = now;
}

template <typename T, int D>
hipError_t launch_d(const KvArgs& a, hipStream_t stream) {
  const int touched = static_cast<int>(kv_touched_pages(a.T, a.page));
  const dim3 grid(2u * a.H_kv * touched * a.B);
  if (a.T <= kFewTokens) {
    hipLaunchKernelGGL((kv_append_few_kernel<T, D>), grid, dim3(64), 0, stream, a, touched);
    return hipGetLastError();
  }
  const int units = a.page / 4 * (D / 8);
  const int threads = units < 64 ? 64 : units > kMaxThreads ? kMaxThreads : units;
  if (units <= kMaxThreads)
    hipLaunchKernelGGL((kv_append_kernel<T, D, 1>), grid, dim3(threads), 0, stream, a, touched);
  else
    hipLaunchKernelGGL((kv_append_kernel<T, D, 2>), grid, dim3(threads), 0, stream, a, touched);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvArgs& a, int io_bf16, hipStream_t stream) {
  if (io_bf16) return a.D == 64 ? launch_d<bf16, 64>(a, stream) : launch_d<bf16, 128>(a, stream);
  return a.D == 64 ? launch_d<float, 64>(a, stream) : launch_d<float, 128>(a, stream);
}

}  // namespace gdr
