// gdr_internal.h -- argument blocks and launchers shared by the C-ABI layer
// (api.cpp) and the kernel sources.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace gdr {

// Argument block of the fused decode kernel.  Pointers are device pointers.
struct DecodeArgs {
  const void* qkv;          // [B, 2*H_qk*dk + H_v*dv] io dtype
  const float* gate_in;     // channel [B,H_v,dk] | scalar/fused [B,H_v]
  const float* A_log;       // [H_v] (fused gate only)
  const float* dt_bias;     // [H_v] (fused gate only)
  const float* beta_logit;  // [B,H_v]
  float* state;             // [B,H_v,dk,dv] in place
  void* o;                  // [B,H_v,dv] io dtype
  int B, H_qk, H_v, dk, dv;
  int gate;                 // gdr_gate value
  int l2norm;
  float scale;
};

// Launch the decode kernel; dv_slice columns of the state per workgroup.
hipError_t launch_decode(const DecodeArgs& a, int io_bf16, int dv_slice, hipStream_t stream);

// Columns of the state one decode workgroup owns, for these sizes.
int decode_dv_slice(int B, int H_v, int dv);

// Argument block of the chunked prefill kernels.
struct PrefillArgs {
  const void* q;            // [B,T,H_qk,dk]
  const void* k;            // [B,T,H_qk,dk]
  const void* v;            // [B,T,H_v,dv]
  const float* gate_in;     // channel [B,T,H_v,dk] | scalar/fused [B,T,H_v]
  const float* A_log;       // [H_v]
  const float* dt_bias;     // [H_v]
  const float* beta_logit;  // [B,T,H_v]
  const float* state_in;    // [B,H_v,dk,dv] or nullptr
  float* state_out;         // [B,H_v,dk,dv]
  void* o;                  // [B,T,H_v,dv]
  void* ws;                 // workspace
  void* ws_qk;              // scalar gates: the normalised k and q rows per (b, qk head, chunk),
                            // inside the workspace (set by the chunked launch)
  int B, T, H_qk, H_v, dk, dv, chunk;
  int gate;
  int l2norm;
  float scale;
};

// Workspace bytes of a chunked prefill; scalar gates (any gate but
// GDR_GATE_CHANNEL) take smaller chunk blocks plus the normalised k and q rows
// once per qk head.
size_t prefill_workspace_bytes(int B, int T, int H_qk, int H_v, int dk, int dv, int chunk,
                               int io_bf16, int gate);
hipError_t launch_prefill(const PrefillArgs& a, int io_bf16, hipStream_t stream);

// The allocation-free prefill takes its workspace from a device array of this
// many bytes (one per device, held until the process ends).
constexpr size_t kNoallocScratchBytes = static_cast<size_t>(128) << 20;
// Device address of the current device's array (resolved on the first call
// on that device).
hipError_t noalloc_scratch(void** ptr);

// Short sequences token by token (the state tile held in registers over all
// T tokens; the workspace is not used).  The prefill takes this path for
// T <= recurrent_max_t(B, H_v) when the per-token vectors fit
// kRecurrentMaxLds bytes of LDS per workgroup.
constexpr size_t kRecurrentMaxLds = 64 * 1024;
int recurrent_max_t(int B, int H_v);
int recurrent_dv_slice(int B, int H_v, int dv);
size_t recurrent_lds_bytes(int T, int dk, int dv_slice);
hipError_t launch_recurrent(const PrefillArgs& a, int io_bf16, hipStream_t stream);

// Argument block of the short convolution (step: T = 1, y0 takes all channels).
struct ConvArgs {
  const void* x;        // rows of C channels, x_stride elements apart
  const float* weight;  // [C,W]
  const float* bias;    // [C] or nullptr
  const int* lens;      // [B] or nullptr
  const void* state_in;   // [B,W-1,C] or nullptr
  void* state_out;      // [B,W-1,C]
  void* y[3];
  long long x_stride;
  int B, T, W, C;
  int c[3];             // widths of the outputs
  int silu;
};
hipError_t launch_conv(const ConvArgs& a, int io_bf16, hipStream_t stream);
// Workgroups launch_conv starts for these sizes on the narrow (one channel a
// thread) path, the larger of its two.
long long conv_max_grid(int B, int T, int C);

// Argument block of the selective state space scan.
struct SsmArgs {
  const void* x;          // step: packed x|B|C rows; prefill [B,T,H,P]
  const void* b;          // [B,T,G,N] (prefill)
  const void* c;          // [B,T,G,N] (prefill)
  const float* dt;        // [B,T,H]
  const float* A_log;     // [H]
  const float* dt_bias;   // [H] or nullptr
  const float* D;         // [H] or nullptr
  const int* lens;        // [B] or nullptr
  const float* state_in;  // [B,H,N,P] or nullptr
  float* state_out;       // [B,H,N,P]
  void* y;                // [B,T,H,P]
  void* ws;
  int B, T, G, H, N, P;
};
hipError_t launch_ssm_step(const SsmArgs& a, int io_bf16, hipStream_t stream);
size_t ssm_workspace_bytes(int B, int T, int G, int H, int N, int P, int io_bf16);
// Longest prompt that is walked token by token; longer ones go in chunks.
int ssm_walk_max_t();
hipError_t launch_ssm_chunked(const SsmArgs& a, int io_bf16, hipStream_t stream);
hipError_t launch_ssm_prefill(const SsmArgs& a, int io_bf16, hipStream_t stream);

// Argument blocks of the 8-bit cache.
struct KvArgs {
  const void* k;  // [B,T,H_kv,D] new keys and values (append)
  const void* v;
  const void* q;  // [B,T,H_q,D] (attention)
  void* o;
  const int* block_table;  // [B,max_pages]
  const int* pos;          // [B]
  const int* lens;         // [B] or nullptr
  uint8_t* k_cache;        // [n_pages,H_kv,page,D] e4m3 codes
  uint8_t* v_cache;        // [n_pages,H_kv,D,page]
  float* k_scale;          // [n_pages,H_kv]
  float* v_scale;
  void* ws;
  int B, T, H_q, H_kv, D, page, n_pages, max_pages;
  float scale;
};
hipError_t launch_kv_append(const KvArgs& a, int io_bf16, hipStream_t stream);
// Pages that T consecutive positions can touch at most.
inline long long kv_touched_pages(int T, int page) {
  return (static_cast<long long>(T) + page - 2) / page + 1;
}
size_t attn_workspace_bytes(const KvArgs& a, int io_bf16);
hipError_t launch_attn(const KvArgs& a, int io_bf16, hipStream_t stream);

// Argument block of the norm and of the plain 8-bit rows.
struct NormArgs {
  const void* x;        // rows of H*D channels, x_stride elements apart
  const void* gate;     // rows gate_stride apart, or nullptr
  const float* weight;  // [H,D] or nullptr
  void* residual;       // [R,H*D] or nullptr
  void* y;              // [R,H*D] or nullptr
  uint8_t* codes;       // [R,H*D] or nullptr
  float* scales;        // [R,ceil(H*D/128)]
  long long x_stride, gate_stride;
  int R, H, D;
  int res_bf16;         // dtype of the residual
  int gate_first;       // the gate goes before the norm
  int norm;             // 0: rows as they are
  int through;          // how outputs are stored (set by the launch)
  float eps;
};
constexpr int kNormMaxD = 32768;
// Heads that lie within a wave.
inline bool norm_short_head(int D) {
  return D == 16 || D == 32 || D == 64 || D == 128 || D == 256 || D == 512;
}
hipError_t launch_norm(const NormArgs& a, int io_bf16, hipStream_t stream);

// Argument block of the 8-bit product.
struct MatmulArgs {
  const uint8_t* x;       // [M,K]
  const float* x_scales;  // [M,ceil(K/128)]
  const uint8_t* w;       // [N,K]
  const float* w_scales;  // [ceil(N/128),ceil(K/128)]
  const float* bias;      // [N] or nullptr
  void* y;                // [M,N]
  int M, N, K;
};
constexpr int kMatmulMaxK = 1 << 20;
// Workgroups launch_matmul starts for these sizes.
long long matmul_grid(int M, int N, int K, int io_bf16);
hipError_t launch_matmul(const MatmulArgs& a, int io_bf16, hipStream_t stream);

// Argument block of the rotary positions.
struct RopeArgs {
  const void* x;       // rows of (H_q + 2 H_kv) D channels, x_stride elements apart
  const double* freq;  // [R/2]
  const int* pos;      // [B]
  const int* lens;     // [B] or nullptr
  void* q;
  void* k;
  void* v;             // or nullptr
  long long x_stride;
  int B, T, H_q, H_kv, D, R;
  int interleaved;
  int through;         // how outputs are stored (set by the launch)
  float magnitude;
};
hipError_t launch_rope(const RopeArgs& a, int io_bf16, hipStream_t stream);

// Workgroups a launch may have: 256 threads each within 32 bits of threads.
constexpr long long kMaxGrid = (1ll << 24) - 1;

}  // namespace gdr
