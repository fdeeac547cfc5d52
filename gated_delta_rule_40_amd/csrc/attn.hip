// attn.hip -- softmax attention of new tokens over the 8-bit cache for gfx950.
//
// One workgroup per (row, token, query head) walks the keys in tiles of 256:
// scores, running maximum and sum, then the values, all in fp32.
#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"
#include "kv_device.hpp"

namespace gdr {
namespace {

constexpr int kThreads = 256;

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_kernel(KvArgs a) {
  __shared__ float qs[D], ps[kThreads], red[kThreads / 64], acc_s[kThreads];
  const int tid = threadIdx.x;
  const int hq = blockIdx.x % a.H_q;
  const int t = blockIdx.x / a.H_q % a.T, b = blockIdx.x / a.H_q / a.T;
  const int n = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
  if (t >= n) return;
  const int head = hq / (a.H_q / a.H_kv);
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  const long long keys = min(static_cast<long long>(a.pos[b]) + t + 1, cap);
  const size_t qo = ((static_cast<size_t>(b) * a.T + t) * a.H_q + hq) * D;
  for (int d = tid; d < D; d += kThreads) qs[d] = to_f32(static_cast<const T*>(a.q)[qo + d]);

  constexpr int PARTS = kThreads / D;  // threads that share an output column
  const int d = tid % D, part = tid / D;
  float m = -INFINITY, l = 0.0f, acc = 0.0f;
  for (long long k0 = 0; k0 < keys; k0 += kThreads) {
    __syncthreads();
    const long long key = k0 + tid;
    float z = -INFINITY;
    if (key < keys) {
      const int id = a.block_table[static_cast<size_t>(b) * a.max_pages + key / a.page];
      if (id >= 0 && id < a.n_pages) {
        const size_t ph = static_cast<size_t>(id) * a.H_kv + head;
        const uint8_t* kp = a.k_cache + (ph * a.page + key % a.page) * D;
        float s = 0.0f;
        for (int i = 0; i < D; ++i) s += qs[i] * e4m3_value(kp[i]);
        z = s * a.k_scale[ph] * a.scale;
      }
    }
    float top = z;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if ((tid & 63) == 0) red[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float p = z == -INFINITY ? 0.0f : expf(z - top);
    ps[tid] = p;
    const float back = m == -INFINITY ? 0.0f : expf(m - top);
    float sum = wave_sum(p);
    __syncthreads();
    if ((tid & 63) == 0) red[tid >> 6] = sum;
    __syncthreads();
    l = l * back + red[0] + red[1] + red[2] + red[3];
    acc *= back;
    m = top;
    for (int i = part; i < kThreads && k0 + i < keys; i += PARTS) {
      if (ps[i] == 0.0f) continue;
      const long long kk = k0 + i;
      const int id = a.block_table[static_cast<size_t>(b) * a.max_pages + kk / a.page];
      const size_t ph = static_cast<size_t>(id) * a.H_kv + head;
      acc += ps[i] * a.v_scale[ph] * e4m3_value(a.v_cache[(ph * D + d) * a.page + kk % a.page]);
    }
  }
  acc_s[tid] = acc;
  __syncthreads();
  if (part == 0) {
    for (int i = 1; i < PARTS; ++i) acc += acc_s[i * D + d];
    static_cast<T*>(a.o)[qo + d] = from_f32<T>(l > 0.0f ? acc / l : l == 0.0f ? 0.0f : NAN);
  }
}

template <typename T>
hipError_t launch_t(const KvArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.T * a.H_q);
  if (a.D == 64)
    hipLaunchKernelGGL((attn_kernel<T, 64>), grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((attn_kernel<T, 128>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t attn_workspace_bytes(const KvArgs&, int) { return 0; }

hipError_t launch_attn(const KvArgs& a, int io_bf16, hipStream_t stream) {
  return io_bf16 ? launch_t<bf16>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace gdr
