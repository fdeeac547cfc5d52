// ssm.hip -- selective state space scan for gfx950: single tokens and prompts.
//
// Per batch row and head h of group g = h / (H / G), with x (P), B and C (N):
//   d = softplus(dt + dt_bias[h]),  S <- exp(-exp(A_log[h]) d) S + d B x^T,
//   y = S^T C + D[h] x.
#include "device_common.hpp"
#include "gdr.h"
#include "gdr_internal.h"

namespace gdr {
namespace {

// ---------------------------------------------------------------------------
// One token.  A workgroup owns a head's whole N x P state tile: C4 = P/4 lanes
// cover a row as float4s, RG row groups of RPT consecutive rows each, so the
// state crosses HBM once in each direction and the small inputs are read
// while it arrives.  The column sums of y go over the row groups of a wave by
// lane exchanges, over the waves through LDS.  Bound by HBM.
// ---------------------------------------------------------------------------
template <int N, int P>
struct StepShape {
  static constexpr int C4 = P / 4;
  static constexpr int RG = (N < 256 / C4) ? N : 256 / C4;
  static constexpr int NT = C4 * RG;
  static constexpr int RPT = N / RG;
  static constexpr int NW = NT / 64;
  static_assert(NT % 64 == 0 && N % RG == 0, "whole waves, even rows");
};

// kNt: the state passes the caches by.  A model steps many layers' states in
// turn, so one of 64 MiB or more is gone from the 256 MiB MALL before its next
// step, and keeping it there only evicts what the step needs: six states in
// turn take 27.7 -> 24.3 us at 64 MiB each and 40.6 -> 39.7 at 96, three take
// 51.2 -> 48.2 at 128; states that stay (three of 32 MiB) lose 12.4 -> 14.2 us.
constexpr size_t kNtStateBytes = size_t{64} << 20;

template <typename T, int N, int P, bool kNt>
__global__ __launch_bounds__((StepShape<N, P>::NT)) void ssm_step_kernel(SsmArgs a) {
  using Sh = StepShape<N, P>;
  constexpr int C4 = Sh::C4, RPT = Sh::RPT, NW = Sh::NW;
  __shared__ float4 red[NW][C4];
  const int tid = threadIdx.x;
  const int c4 = tid % C4, row0 = tid / C4 * RPT;
  const int h = blockIdx.x % a.H, b = blockIdx.x / a.H;
  const int g = h / (a.H / a.G);
  const size_t bh = static_cast<size_t>(b) * a.H + h;

  const T* row = static_cast<const T*>(a.x) +
                 static_cast<size_t>(b) * (static_cast<size_t>(a.H) * P + 2 * a.G * N);
  const T* bg = row + static_cast<size_t>(a.H) * P + g * N;
  const T* cg = bg + a.G * N;
  float xv[4], bv[RPT], cv[RPT];
  load_row<T, 4>(row + h * P + 4 * c4, xv);
  load_row<T, RPT>(bg + row0, bv);
  load_row<T, RPT>(cg + row0, cv);
  const float dt = a.dt[bh], al = a.A_log[h];
  const float db = a.dt_bias ? a.dt_bias[h] : 0.0f;
  const float dskip = a.D ? a.D[h] : 0.0f;

  nt_f32x4* S = reinterpret_cast<nt_f32x4*>(a.state_out + bh * N * P) + row0 * C4 + c4;
  nt_f32x4 s[RPT];
#pragma unroll
  for (int m = 0; m < RPT; ++m) s[m] = kNt ? __builtin_nontemporal_load(&S[m * C4]) : S[m * C4];

  const float d = softplusf(dt + db);
  const float decay = expf(decay_rate(al) * d);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int m = 0; m < RPT; ++m) {
    const float w = d * bv[m];
    s[m].x = decay * s[m].x + w * xv[0];
    s[m].y = decay * s[m].y + w * xv[1];
    s[m].z = decay * s[m].z + w * xv[2];
    s[m].w = decay * s[m].w + w * xv[3];
    if constexpr (kNt)
      __builtin_nontemporal_store(s[m], &S[m * C4]);
    else
      S[m * C4] = s[m];
    y.x += cv[m] * s[m].x;
    y.y += cv[m] * s[m].y;
    y.z += cv[m] * s[m].z;
    y.w += cv[m] * s[m].w;
  }
  y.x = lane_class_sum<C4>(y.x);
  y.y = lane_class_sum<C4>(y.y);
  y.z = lane_class_sum<C4>(y.z);
  y.w = lane_class_sum<C4>(y.w);
  if constexpr (NW > 1) {
    if ((tid & 63) < C4) red[tid >> 6][c4] = y;
    __syncthreads();
  }
  if (tid < C4) {
    if constexpr (NW > 1) {
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        const float4 t = red[w][c4];
        y.x += t.x;
        y.y += t.y;
        y.z += t.z;
        y.w += t.w;
      }
    }
    store4<T>(static_cast<T*>(a.y) + bh * P + 4 * c4, y.x + dskip * xv[0], y.y + dskip * xv[1],
              y.z + dskip * xv[2], y.w + dskip * xv[3]);
  }
}

// ---------------------------------------------------------------------------
// Token by token: a wave owns 16 columns of a head's state (4 lanes a row as
// float4s, 16 row groups of N/16 rows) and walks the tokens with the state in
// registers; the column sums stay inside the wave.
// ---------------------------------------------------------------------------
template <typename T, int N>
__global__ __launch_bounds__(64) void ssm_walk_kernel(SsmArgs a) {
  constexpr int RPT = N / 16;
  const int lane = threadIdx.x, c4 = lane & 3, row0 = (lane >> 2) * RPT;
  const int slices = a.P / 16;
  const int slice = blockIdx.x % slices;
  const int h = blockIdx.x / slices % a.H, b = blockIdx.x / slices / a.H;
  const int g = h / (a.H / a.G);
  const int n = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
  const int col = 16 * slice + 4 * c4;

  const size_t at = ((static_cast<size_t>(b) * a.H + h) * N + row0) * a.P + col;
  float4 s[RPT];
#pragma unroll
  for (int m = 0; m < RPT; ++m)
    s[m] = a.state_in ? *reinterpret_cast<const float4*>(a.state_in + at + m * a.P)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
  const float rate = n > 0 ? decay_rate(a.A_log[h]) : 0.0f;  // T = 0 comes without parameters
  const float db = n > 0 && a.dt_bias ? a.dt_bias[h] : 0.0f;
  const float dskip = n > 0 && a.D ? a.D[h] : 0.0f;

  for (int t = 0; t < n; ++t) {
    const size_t bt = static_cast<size_t>(b) * a.T + t;
    float xv[4], bv[RPT], cv[RPT];
    const size_t xo = (bt * a.H + h) * a.P + col;
    load_row<T, 4>(static_cast<const T*>(a.x) + xo, xv);
    load_row<T, RPT>(static_cast<const T*>(a.b) + (bt * a.G + g) * N + row0, bv);
    load_row<T, RPT>(static_cast<const T*>(a.c) + (bt * a.G + g) * N + row0, cv);
    const float d = softplusf(a.dt[bt * a.H + h] + db);
    const float decay = expf(rate * d);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
      const float w = d * bv[m];
      s[m].x = decay * s[m].x + w * xv[0];
      s[m].y = decay * s[m].y + w * xv[1];
      s[m].z = decay * s[m].z + w * xv[2];
      s[m].w = decay * s[m].w + w * xv[3];
      y.x += cv[m] * s[m].x;
      y.y += cv[m] * s[m].y;
      y.z += cv[m] * s[m].z;
      y.w += cv[m] * s[m].w;
    }
    y.x = lane_class_sum<4>(y.x);
    y.y = lane_class_sum<4>(y.y);
    y.z = lane_class_sum<4>(y.z);
    y.w = lane_class_sum<4>(y.w);
    if (lane < 4)
      store4<T>(static_cast<T*>(a.y) + xo, y.x + dskip * xv[0], y.y + dskip * xv[1],
                y.z + dskip * xv[2], y.w + dskip * xv[3]);
  }
#pragma unroll
  for (int m = 0; m < RPT; ++m) *reinterpret_cast<float4*>(a.state_out + at + m * a.P) = s[m];
}

// Walked while that beats a chunk that is mostly padding: 64 heads (N = 128,
// P = 64), one row, 8 tokens 9.0 against 11.2 us, 16 tokens 15.0 against 11.3;
// 32 rows of 8 tokens 49.8 against 46.7.
constexpr int kWalkMaxT = 8;

template <typename T, int N>
hipError_t step_n(const SsmArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H);
  const bool nt = static_cast<size_t>(a.B) * a.H * N * a.P * sizeof(float) >= kNtStateBytes;
#define GDR_STEP(P_)                                                                       \
  case P_:                                                                                 \
    if (nt)                                                                                \
      hipLaunchKernelGGL((ssm_step_kernel<T, N, P_, true>), grid,                          \
                         dim3(StepShape<N, P_>::NT), 0, stream, a);                        \
    else                                                                                   \
      hipLaunchKernelGGL((ssm_step_kernel<T, N, P_, false>), grid,                         \
                         dim3(StepShape<N, P_>::NT), 0, stream, a);                        \
    break
  switch (a.P) {
    GDR_STEP(16);
    GDR_STEP(32);
    GDR_STEP(64);
    GDR_STEP(128);
    default: return hipErrorInvalidValue;
  }
#undef GDR_STEP
  return hipGetLastError();
}

template <typename T, int N>
hipError_t walk_n(const SsmArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H * (a.P / 16));
  hipLaunchKernelGGL((ssm_walk_kernel<T, N>), grid, dim3(64), 0, stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t step_t(const SsmArgs& a, hipStream_t stream) {
  switch (a.N) {
    case 16: return step_n<T, 16>(a, stream);
    case 32: return step_n<T, 32>(a, stream);
    case 64: return step_n<T, 64>(a, stream);
    case 128: return step_n<T, 128>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

template <typename T>
hipError_t walk_t(const SsmArgs& a, hipStream_t stream) {
  switch (a.N) {
    case 16: return walk_n<T, 16>(a, stream);
    case 32: return walk_n<T, 32>(a, stream);
    case 64: return walk_n<T, 64>(a, stream);
    case 128: return walk_n<T, 128>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_ssm_step(const SsmArgs& a, int io_bf16, hipStream_t stream) {
  return io_bf16 ? step_t<bf16>(a, stream) : step_t<float>(a, stream);
}

int ssm_walk_max_t() { return kWalkMaxT; }

hipError_t launch_ssm_prefill(const SsmArgs& a, int io_bf16, hipStream_t stream) {
  if (a.T > kWalkMaxT) return launch_ssm_chunked(a, io_bf16, stream);
  return io_bf16 ? walk_t<bf16>(a, stream) : walk_t<float>(a, stream);
}

}  // namespace gdr
