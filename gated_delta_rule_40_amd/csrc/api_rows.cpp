// api_rows.cpp -- the C ABI of the norms, the 8-bit product and the rotary
// positions (include/gdr.h): validation on the host, then the launchers.
// Nothing here allocates, frees or synchronises; errors are returned before
// anything is enqueued.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "api_check.hpp"
#include "gdr.h"
#include "gdr_internal.h"

namespace {

using namespace gdr::check;

// ---- norms -------------------------------------------------------------------

int check_norm_sizes(const gdr_norm_dims* d, gdr_dtype io, int64_t x_stride) {
  if (!d) return GDR_E_NULL;
  if (!known_io(io)) return GDR_E_DTYPE;
  if (d->R < 0 || d->H <= 0 || d->D <= 0) return GDR_E_SHAPE;
  // A row's channels, and those a workgroup's threads reach past its end, are 32-bit.
  if (!within(INT32_MAX - 2 * gdr::kNormMaxD, {d->H, d->D})) return GDR_E_SHAPE;
  if (x_stride < static_cast<int64_t>(d->H) * d->D) return GDR_E_SHAPE;
  if (d->D > gdr::kNormMaxD) return GDR_E_UNSUPPORTED;
  if (d->H > 1 && d->D % 128 != 0 && d->D != 16 && d->D != 32 && d->D != 64)
    return GDR_E_UNSUPPORTED;
  // Short heads: 32-bit numbers of vectors of 8 channels, rows padded to whole blocks;
  // others: a workgroup a head, of 1024 threads past 8192 channels, else (where there are
  // many) of up to 256.
  const long long slots = (static_cast<long long>(d->H) * d->D + 127) / 128 * 16;
  if (gdr::norm_short_head(d->D) ? !within(UINT32_MAX - 512ll, {d->R, slots})
                                 : !within(d->D > 8192 ? gdr::kMaxGrid / 4 : gdr::kMaxGrid,
                                           {d->R, d->H}))
    return GDR_E_SHAPE;
  if (!within(INT64_MAX / 16, {d->R, x_stride})) return GDR_E_SHAPE;
  return GDR_OK;
}

size_t blocks_of(size_t channels) { return (channels + 127) / 128; }

int run_norm(gdr::NormArgs& a, const gdr_norm_dims& d, gdr_dtype io, gdr_dtype res,
             hipStream_t stream) {
  const size_t es = size_of(io), R = d.R, W = static_cast<size_t>(d.H) * d.D;
  if (!aligned(a.x, es) || !aligned(a.gate, es) || !aligned(a.weight, 4) ||
      !aligned(a.residual, 16) || !aligned(a.y, 16) || !aligned(a.codes, 16) ||
      !aligned(a.scales, 4))
    return GDR_E_ALIGN;
  const Range writes[4] = {range_or_none(a.residual, R * W * size_of(res)),
                           range_or_none(a.y, R * W * es), range_or_none(a.codes, R * W),
                           range_or_none(a.scales, R * blocks_of(W) * sizeof(float))};
  const Range reads[3] = {range_of(a.x, rows_extent(R, a.x_stride, W, es)),
                          range_or_none(a.gate, rows_extent(R, a.gate_stride, W, es)),
                          range_or_none(a.weight, W * sizeof(float))};
  if (clash(writes, reads)) return GDR_E_ALIAS;
  a.R = d.R;
  a.H = d.H;
  a.D = d.D;
  return result(gdr::launch_norm(a, io == GDR_BF16, stream));
}

// ---- 8-bit product -------------------------------------------------------------

int check_matmul_sizes(const gdr_matmul_dims* d, gdr_dtype io) {
  if (!d) return GDR_E_NULL;
  if (!known_io(io)) return GDR_E_DTYPE;
  if (d->M < 0 || d->N < 0 || d->K < 0) return GDR_E_SHAPE;
  if (d->K % 16 != 0 || d->K > gdr::kMatmulMaxK) return GDR_E_UNSUPPORTED;
  // The ends of the last tiles are 32-bit.
  if (d->M > INT32_MAX - 256 || d->N > INT32_MAX - 256) return GDR_E_SHAPE;
  // Workgroups of up to 512 threads (of 1024 only where there are few).
  if (gdr::matmul_grid(d->M, d->N, d->K, io == GDR_BF16) > gdr::kMaxGrid / 2) return GDR_E_SHAPE;
  return GDR_OK;
}

// ---- rotary positions ------------------------------------------------------------

int check_rope_sizes(const gdr_rope_dims* d, gdr_dtype io, gdr_rope_pairs pairs, int64_t x_stride,
                     bool with_v) {
  if (!d) return GDR_E_NULL;
  if (!known_io(io) || (pairs != GDR_ROPE_HALF && pairs != GDR_ROPE_INTERLEAVED))
    return GDR_E_DTYPE;
  if (d->B < 0 || d->T < 0 || d->H_q <= 0 || d->H_kv <= 0 || d->D <= 0 || d->R < 0 ||
      d->R > d->D || d->R % 2 != 0)
    return GDR_E_SHAPE;
  if (d->D % 8 != 0 || d->D > 512) return GDR_E_UNSUPPORTED;
  const long long heads = static_cast<long long>(d->H_q) + (with_v ? 2ll : 1ll) * d->H_kv;
  if (!within(INT32_MAX, {heads, d->D}) || x_stride < heads * d->D) return GDR_E_SHAPE;
  if (!within(gdr::kMaxGrid, {d->B, d->T})) return GDR_E_SHAPE;
  if (!within(INT64_MAX / 16, {d->B, d->T, x_stride})) return GDR_E_SHAPE;
  return GDR_OK;
}

}  // namespace

extern "C" {

int gdr_rms_norm(const gdr_norm_dims* dims, gdr_dtype io, const void* x, int64_t x_stride,
                 gdr_dtype res, void* residual, gdr_norm_gate order, const void* gate,
                 int64_t gate_stride, const float* weight, float eps, void* y, void* codes,
                 float* scales, hipStream_t stream) {
  const int rc = check_norm_sizes(dims, io, x_stride);
  if (rc != GDR_OK) return rc;
  const gdr_norm_dims& d = *dims;
  if (residual && !known_io(res)) return GDR_E_DTYPE;
  if (order != GDR_NORM_GATE_NONE && order != GDR_NORM_GATE_AFTER &&
      order != GDR_NORM_GATE_BEFORE)
    return GDR_E_DTYPE;
  const bool gated = order != GDR_NORM_GATE_NONE;
  if (gated && (gate_stride < static_cast<int64_t>(d.H) * d.D ||
                !within(INT64_MAX / 16, {d.R, gate_stride})))
    return GDR_E_SHAPE;
  if (!(eps > 0.0f) || !isfinite(eps) || (gated && residual)) return GDR_E_UNSUPPORTED;
  if (d.R == 0) return GDR_OK;
  if (!x || (gated && !gate) || (!codes != !scales) || (!y && !codes)) return GDR_E_NULL;
  gdr::NormArgs a = {};
  a.x = x;
  a.x_stride = x_stride;
  a.residual = residual;
  a.res_bf16 = res == GDR_BF16;
  if (gated) {
    a.gate = gate;
    a.gate_stride = gate_stride;
    a.gate_first = order == GDR_NORM_GATE_BEFORE;
  }
  a.weight = weight;
  a.y = y;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.norm = 1;
  a.eps = eps;
  return run_norm(a, d, io, res, stream);
}

int gdr_quant_rows(const gdr_norm_dims* dims, gdr_dtype io, const void* x, int64_t x_stride,
                   void* codes, float* scales, hipStream_t stream) {
  const int rc = check_norm_sizes(dims, io, x_stride);
  if (rc != GDR_OK) return rc;
  if (dims->R == 0) return GDR_OK;
  if (!x || !codes || !scales) return GDR_E_NULL;
  gdr::NormArgs a = {};
  a.x = x;
  a.x_stride = x_stride;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  return run_norm(a, *dims, io, io, stream);
}

int gdr_matmul_fp8(const gdr_matmul_dims* dims, gdr_dtype io, const void* x,
                   const float* x_scales, const void* w, const float* w_scales,
                   const float* bias, void* y, hipStream_t stream) {
  const int rc = check_matmul_sizes(dims, io);
  if (rc != GDR_OK) return rc;
  const gdr_matmul_dims& d = *dims;
  if (d.M == 0 || d.N == 0) return GDR_OK;
  if (!y || (d.K > 0 && (!x || !x_scales || !w || !w_scales))) return GDR_E_NULL;
  if (!aligned(y, 16) || !aligned(bias, 4) ||
      (d.K > 0 && (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) ||
                   !aligned(w_scales, 4))))
    return GDR_E_ALIGN;
  const size_t M = d.M, N = d.N, K = d.K, kb = blocks_of(K);
  const Range writes[1] = {range_of(y, M * N * size_of(io))};
  const Range reads[5] = {range_of(x, M * K), range_of(x_scales, M * kb * sizeof(float)),
                          range_of(w, N * K),
                          range_of(w_scales, blocks_of(N) * kb * sizeof(float)),
                          range_or_none(bias, N * sizeof(float))};
  if (clash(writes, reads)) return GDR_E_ALIAS;
  gdr::MatmulArgs a = {};
  a.x = static_cast<const uint8_t*>(x);
  a.x_scales = x_scales;
  a.w = static_cast<const uint8_t*>(w);
  a.w_scales = w_scales;
  a.bias = bias;
  a.y = y;
  a.M = d.M;
  a.N = d.N;
  a.K = d.K;
  return result(gdr::launch_matmul(a, io == GDR_BF16, stream));
}

int gdr_rope(const gdr_rope_dims* dims, gdr_dtype io, gdr_rope_pairs pairs, const void* x,
             int64_t x_stride, const double* freq, float magnitude, const int32_t* pos,
             const int32_t* lens, void* q, void* k, void* v, hipStream_t stream) {
  const int rc = check_rope_sizes(dims, io, pairs, x_stride, v != nullptr);
  if (rc != GDR_OK) return rc;
  const gdr_rope_dims& d = *dims;
  if (d.B == 0 || d.T == 0) return GDR_OK;
  if (!x || !pos || !q || !k || (d.R > 0 && !freq)) return GDR_E_NULL;
  const size_t es = size_of(io);
  if (!aligned(x, es) || !aligned(freq, 8) || !aligned(pos, 4) || !aligned(lens, 4) ||
      !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16))
    return GDR_E_ALIGN;
  const size_t rows = static_cast<size_t>(d.B) * d.T, D = d.D, kv = rows * d.H_kv * D * es;
  const size_t width = (static_cast<size_t>(d.H_q) + (v ? 2 : 1) * static_cast<size_t>(d.H_kv)) * D;
  const Range writes[3] = {range_of(q, rows * d.H_q * D * es), range_of(k, kv),
                           range_or_none(v, kv)};
  const Range reads[4] = {range_of(x, rows_extent(rows, x_stride, width, es)),
                          range_or_none(d.R ? freq : nullptr, d.R / 2 * sizeof(double)),
                          range_of(pos, d.B * sizeof(int32_t)),
                          range_or_none(lens, d.B * sizeof(int32_t))};
  if (clash(writes, reads)) return GDR_E_ALIAS;
  gdr::RopeArgs a = {};
  a.x = x;
  a.freq = freq;
  a.pos = pos;
  a.lens = lens;
  a.q = q;
  a.k = k;
  a.v = v;
  a.x_stride = x_stride;
  a.B = d.B;
  a.T = d.T;
  a.H_q = d.H_q;
  a.H_kv = d.H_kv;
  a.D = d.D;
  a.R = d.R;
  a.interleaved = pairs == GDR_ROPE_INTERLEAVED;
  a.magnitude = magnitude;
  return result(gdr::launch_rope(a, io == GDR_BF16, stream));
}

int gdr_rope_freqs(int32_t R, double base, const gdr_rope_scaling* scaling, double* freq,
                   float* magnitude) {
  if (R < 2 || R > 512 || R % 2 != 0) return GDR_E_SHAPE;
  if (!isfinite(base) || !(base > 1.0)) return GDR_E_UNSUPPORTED;
  gdr_rope_scaling s = {GDR_ROPE_NONE, 1.0, 0.0, 0.0, 0.0};
  if (scaling) s = *scaling;
  const bool ramp = s.kind == GDR_ROPE_TURNS || s.kind == GDR_ROPE_INDEX;
  if (s.kind != GDR_ROPE_NONE) {
    if (s.kind != GDR_ROPE_LINEAR && s.kind != GDR_ROPE_BASE && !ramp) return GDR_E_DTYPE;
    if (!isfinite(s.factor) || !(s.factor >= 1.0)) return GDR_E_UNSUPPORTED;
    if (s.kind == GDR_ROPE_BASE) {
      if (R == 2) return GDR_E_UNSUPPORTED;
      base *= pow(s.factor, static_cast<double>(R) / (R - 2));
      if (!isfinite(base)) return GDR_E_UNSUPPORTED;
    }
    if (ramp && (!isfinite(s.context) || !(s.context > 0.0) || !isfinite(s.high) ||
                 !(s.low > 0.0) || !(s.low < s.high)))
      return GDR_E_UNSUPPORTED;
  }
  if (!freq) return GDR_E_NULL;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  // The index (as a real number) whose frequency makes `turns` turns over the context.
  auto index_of = [&](double turns) {
    return R * log(s.context / (turns * kTwoPi)) / (2.0 * log(base));
  };
  double first = 0.0, last = 0.0;
  if (s.kind == GDR_ROPE_INDEX) {
    first = fmax(floor(index_of(s.high)), 0.0);
    last = fmin(ceil(index_of(s.low)), R - 1.0);
    if (last <= first) last = first + 0.001;  // a step
  }
  for (int i = 0; i < R / 2; ++i) {
    const double f = pow(base, -2.0 * i / R);
    double u = 1.0;  // share of f that is not stretched
    if (s.kind == GDR_ROPE_LINEAR) u = 0.0;
    if (s.kind == GDR_ROPE_TURNS) u = (s.context * f / kTwoPi - s.low) / (s.high - s.low);
    if (s.kind == GDR_ROPE_INDEX) u = 1.0 - (i - first) / (last - first);
    u = fmin(fmax(u, 0.0), 1.0);
    freq[i] = s.kind == GDR_ROPE_NONE || s.kind == GDR_ROPE_BASE
                  ? f
                  : f * (u + (1.0 - u) / s.factor);
  }
  if (magnitude)
    *magnitude =
        s.kind == GDR_ROPE_INDEX ? static_cast<float>(0.1 * log(s.factor) + 1.0) : 1.0f;
  return GDR_OK;
}

}  // extern "C"
