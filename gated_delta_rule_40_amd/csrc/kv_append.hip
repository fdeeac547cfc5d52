// kv_append.hip -- keys and values of new tokens into pages of e4m3 codes, one
// power-of-two scale per (page, head).
//
// With a power of two, scaling a value and shifting a code to a larger scale
// are exact but for the rounding to e4m3's subnormals, so a page that takes
// tokens one by one holds (nearly) what it would hold if they had come at
// once: a growing scale costs no precision each time.
//
// One workgroup per (row, page it may touch, head, keys or values): the
// largest magnitude of the new tokens, the scale, the older codes if the
// scale grew, then the new codes.
#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"
#include "kv_device.hpp"

namespace gdr {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvArgs a, int touched) {
  __shared__ float red[kThreads / 64];
  const int tid = threadIdx.x;
  unsigned wg = blockIdx.x;
  const bool is_v = wg & 1;
  wg >>= 1;
  const int head = wg % a.H_kv;
  wg /= a.H_kv;
  const int j = wg % touched;
  const int b = wg / touched;

  const int n = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
  const long long pos = a.pos[b];
  const long long start = pos > 0 ? pos : 0;
  const long long page_no = start / a.page + j;
  if (page_no >= a.max_pages) return;
  const long long base = page_no * a.page;
  const int u = static_cast<int>(max(start, base) - base);                 // slots [u, w) are new
  const int w = static_cast<int>(min(pos + n, base + a.page) - base);
  if (u >= w) return;
  const int had = pos > base ? static_cast<int>(pos - base) : 0;           // slots [0, had) are old
  const int id = a.block_table[static_cast<size_t>(b) * a.max_pages + page_no];
  if (id < 0 || id >= a.n_pages) return;

  const int D = a.D, page = a.page;
  const size_t ph = static_cast<size_t>(id) * a.H_kv + head;
  uint8_t* cache = (is_v ? a.v_cache : a.k_cache) + ph * page * D;
  float* scale = (is_v ? a.v_scale : a.k_scale) + ph;
  // Token of slot s: t = base + s - pos.
  const T* src = static_cast<const T*>(is_v ? a.v : a.k) +
                 ((static_cast<size_t>(b) * a.T + static_cast<size_t>(base + u - pos)) * a.H_kv +
                  head) * D;
  const size_t tok = static_cast<size_t>(a.H_kv) * D;
  const int count = (w - u) * D;

  float amax = 0.0f;
  for (int i = tid; i < count; i += kThreads)
    amax = fmaxf(amax, finite_abs(to_f32(src[(i / D) * tok + i % D])));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
  if ((tid & 63) == 0) red[tid >> 6] = amax;
  const float was = had > 0 ? *scale : 0.0f;
  __syncthreads();
  amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float now = e4m3_scale(amax);
  if (had > 0) now = fmaxf(now, was);
  const float inv = pow2_inverse(now);

  if (had > 0 && now > was) {
    const float ratio = was * inv;
    for (int i = tid; i < had * D; i += kThreads) {
      uint8_t* p = cache + (is_v ? (i / had) * page + i % had : i);
      *p = static_cast<uint8_t>(e4m3_pair(e4m3_value(*p) * ratio, 0.0f));
    }
  }
  for (int i = tid; i < count; i += kThreads) {
    const float x = to_f32(src[(i / D) * tok + i % D]) * inv;
    const int s = u + i / D, d = i % D;
    cache[is_v ? d * page + s : s * D + d] = static_cast<uint8_t>(e4m3_pair(x, 0.0f));
  }
  if (tid == 0) *scale = now;
}

}  // namespace

hipError_t launch_kv_append(const KvArgs& a, int io_bf16, hipStream_t stream) {
  const int touched = static_cast<int>(kv_touched_pages(a.T, a.page));
  const dim3 grid(2u * a.H_kv * touched * a.B);
  if (io_bf16)
    hipLaunchKernelGGL((kv_append_kernel<bf16>), grid, dim3(kThreads), 0, stream, a, touched);
  else
    hipLaunchKernelGGL((kv_append_kernel<float>), grid, dim3(kThreads), 0, stream, a, touched);
  return hipGetLastError();
}

}  // namespace gdr
