// api_layers.cpp -- the C ABI of the short convolution, the selective state
// space scan and attention over the 8-bit cache (include/gdr.h): validation on
// the host, then the launchers.  Nothing here allocates, frees or
// synchronises; errors are returned before anything is enqueued.
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "api_check.hpp"
#include "gdr.h"
#include "gdr_internal.h"

namespace {

using namespace gdr::check;

// ---- short convolution ----------------------------------------------------

int check_conv_sizes(const gdr_conv_dims* d, gdr_dtype io, gdr_act act, int T, int64_t x_stride) {
  if (!d) return GDR_E_NULL;
  if (!known_io(io) || (act != GDR_ACT_NONE && act != GDR_ACT_SILU)) return GDR_E_DTYPE;
  if (d->B < 0 || T < 0 || d->c0 <= 0 || d->c1 < 0 || d->c2 < 0) return GDR_E_SHAPE;
  const long long C = static_cast<long long>(d->c0) + d->c1 + d->c2;
  if (C > INT32_MAX || x_stride < C || (d->c2 > 0 && d->c1 == 0)) return GDR_E_SHAPE;
  if (T > INT32_MAX - 64) return GDR_E_SHAPE;  // the end of the last tile is 32-bit
  if (d->W < 2 || d->W > 4) return GDR_E_UNSUPPORTED;
  if (gdr::conv_max_grid(d->B, T, static_cast<int>(C)) > gdr::kMaxGrid) return GDR_E_SHAPE;
  // Byte extents stay within 62 bits.
  if (!within(INT64_MAX / 16, {d->B, T > 0 ? T : 1, x_stride})) return GDR_E_SHAPE;
  return GDR_OK;
}

gdr::ConvArgs conv_args(const gdr_conv_dims& d, int T, gdr_act act, const void* x,
                        int64_t x_stride, const float* weight, const float* bias) {
  gdr::ConvArgs a = {};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.x_stride = x_stride;
  a.B = d.B;
  a.T = T;
  a.W = d.W;
  a.C = d.c0 + d.c1 + d.c2;
  a.silu = act == GDR_ACT_SILU;
  return a;
}

// ---- selective state space scan --------------------------------------------

bool supported_width(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

int check_ssm_sizes(const gdr_ssm_dims* d, gdr_dtype io, int T) {
  if (!d) return GDR_E_NULL;
  if (!known_io(io)) return GDR_E_DTYPE;
  if (d->B < 0 || T < 0 || d->G <= 0 || d->H <= 0 || d->N <= 0 || d->P <= 0) return GDR_E_SHAPE;
  if (d->H % d->G != 0) return GDR_E_SHAPE;
  if (!supported_width(d->N) || !supported_width(d->P)) return GDR_E_UNSUPPORTED;
  // The rows of a chunk of 64 tokens are reached through 32-bit byte offsets.
  if (!within(UINT32_MAX, {64, 4, d->H, d->P}) || !within(UINT32_MAX, {64, 4, d->G, d->N}))
    return GDR_E_SHAPE;
  // Workgroups: one per (row, head, 16 columns, chunk of 64 tokens) at most.
  const long long chunks = (static_cast<long long>(T) + 63) / 64;
  if (!within(gdr::kMaxGrid, {d->B, d->H, d->P / 16, chunks > 0 ? chunks : 1}))
    return GDR_E_SHAPE;
  return GDR_OK;
}

int check_ssm_params(const float* dt, const float* A_log, const float* dt_bias, const float* D) {
  if (!dt || !A_log) return GDR_E_NULL;
  if (!aligned(dt, 4) || !aligned(A_log, 4) || !aligned(dt_bias, 4) || !aligned(D, 4))
    return GDR_E_ALIGN;
  return GDR_OK;
}

// ---- 8-bit cache -----------------------------------------------------------

int check_kv_sizes(const gdr_kv_dims* d, gdr_dtype io, bool attn) {
  if (!d) return GDR_E_NULL;
  if (!known_io(io)) return GDR_E_DTYPE;
  if (d->B < 0 || d->T < 0 || d->H_kv <= 0 || d->D <= 0 || d->page <= 0 || d->n_pages < 0 ||
      d->max_pages < 0)
    return GDR_E_SHAPE;
  if (attn && (d->H_q <= 0 || d->H_q % d->H_kv != 0)) return GDR_E_SHAPE;
  if ((d->D != 64 && d->D != 128) ||
      (d->page != 16 && d->page != 32 && d->page != 64 && d->page != 128))
    return GDR_E_UNSUPPORTED;
  if (attn ? !within(gdr::kMaxGrid, {d->B, d->T, d->H_q})
           : !within(gdr::kMaxGrid, {2, d->B, gdr::kv_touched_pages(d->T, d->page), d->H_kv}))
    return GDR_E_SHAPE;
  // Positions, and the end of the step they fall into, are 32-bit.
  if (!within(INT32_MAX - 128, {d->max_pages, d->page})) return GDR_E_SHAPE;
  if (!within(INT64_MAX / 16, {d->n_pages, d->H_kv, d->page, d->D})) return GDR_E_SHAPE;
  return GDR_OK;
}

gdr::KvArgs kv_args(const gdr_kv_dims& d) {
  gdr::KvArgs a = {};
  a.B = d.B;
  a.T = d.T;
  a.H_q = d.H_q;
  a.H_kv = d.H_kv;
  a.D = d.D;
  a.page = d.page;
  a.n_pages = d.n_pages;
  a.max_pages = d.max_pages;
  return a;
}

struct KvRanges {
  Range k_cache, v_cache, k_scale, v_scale, table, pos, lens;
};

// The pointers both entry points take, and where they lie.
int check_kv_ptrs(const gdr_kv_dims& d, const void* k_cache, const void* v_cache,
                  const float* k_scale, const float* v_scale, const int32_t* table,
                  const int32_t* pos, const int32_t* lens, KvRanges* r) {
  // An empty pool or table may come as NULL: neither is followed.
  if (d.n_pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale)) return GDR_E_NULL;
  if ((d.max_pages > 0 && !table) || !pos) return GDR_E_NULL;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(table, 4) || !aligned(pos, 4) || !aligned(lens, 4))
    return GDR_E_ALIGN;
  const size_t heads = static_cast<size_t>(d.n_pages) * d.H_kv;
  const size_t codes = heads * d.page * d.D;
  r->k_cache = range_of(k_cache, codes);
  r->v_cache = range_of(v_cache, codes);
  r->k_scale = range_of(k_scale, heads * sizeof(float));
  r->v_scale = range_of(v_scale, heads * sizeof(float));
  r->table = range_of(table, static_cast<size_t>(d.B) * d.max_pages * sizeof(int32_t));
  r->pos = range_of(pos, static_cast<size_t>(d.B) * sizeof(int32_t));
  r->lens = range_or_none(lens, static_cast<size_t>(d.B) * sizeof(int32_t));
  return GDR_OK;
}

}  // namespace

extern "C" {

int gdr_conv_step(const gdr_conv_dims* dims, gdr_dtype io, gdr_act act, const void* x,
                  int64_t x_stride, const float* weight, const float* bias, void* state, void* y,
                  hipStream_t stream) {
  const int rc = check_conv_sizes(dims, io, act, 1, x_stride);
  if (rc != GDR_OK) return rc;
  const gdr_conv_dims& d = *dims;
  if (d.B == 0) return GDR_OK;
  if (!x || !weight || !state || !y) return GDR_E_NULL;
  const size_t es = size_of(io);
  if (!aligned(x, es) || !aligned(weight, 16) || !aligned(bias, 4) || !aligned(state, 16) ||
      !aligned(y, 16))
    return GDR_E_ALIGN;
  gdr::ConvArgs a = conv_args(d, 1, act, x, x_stride, weight, bias);
  const size_t B = d.B, C = a.C;
  const Range writes[2] = {range_of(state, B * (d.W - 1) * C * es), range_of(y, B * C * es)};
  const Range reads[3] = {range_of(x, rows_extent(B, x_stride, C, es)),
                          range_of(weight, C * d.W * sizeof(float)),
                          range_or_none(bias, C * sizeof(float))};
  if (clash(writes, reads)) return GDR_E_ALIAS;
  a.state_in = state;
  a.state_out = state;
  a.y[0] = y;
  a.c[0] = a.C;
  return result(gdr::launch_conv(a, io == GDR_BF16, stream));
}

int gdr_conv_prefill(const gdr_conv_dims* dims, gdr_dtype io, gdr_act act, const void* x,
                     int64_t x_stride, const float* weight, const float* bias,
                     const int32_t* lens, const void* state_in, void* state_out, void* y0,
                     void* y1, void* y2, hipStream_t stream) {
  const int rc = check_conv_sizes(dims, io, act, dims ? dims->T : 0, x_stride);
  if (rc != GDR_OK) return rc;
  const gdr_conv_dims& d = *dims;
  if (d.B == 0) return GDR_OK;
  const bool any = d.T > 0;
  if (!state_out || (any && (!x || !weight || !y0 || (d.c1 && !y1) || (d.c2 && !y2))))
    return GDR_E_NULL;
  if (!any && state_in == state_out) return GDR_OK;
  const size_t es = size_of(io);
  if (!aligned(state_in, 16) || !aligned(state_out, 16) || !aligned(lens, 4)) return GDR_E_ALIGN;
  if (any && (!aligned(x, es) || !aligned(weight, 16) || !aligned(bias, 4) || !aligned(y0, 16) ||
              (d.c1 && !aligned(y1, 16)) || (d.c2 && !aligned(y2, 16))))
    return GDR_E_ALIGN;
  gdr::ConvArgs a = conv_args(d, d.T, act, x, x_stride, weight, bias);
  const size_t B = d.B, T = d.T, C = a.C, st = B * (d.W - 1) * C * es;
  const bool in_place = state_in == state_out;
  const Range writes[4] = {range_of(state_out, st), range_of(y0, B * T * d.c0 * es),
                           d.c1 ? range_of(y1, B * T * d.c1 * es) : Range{0, 0},
                           d.c2 ? range_of(y2, B * T * d.c2 * es) : Range{0, 0}};
  const Range reads[5] = {range_of(x, rows_extent(B * T, x_stride, C, es)),
                          range_or_none(any ? weight : nullptr, C * d.W * sizeof(float)),
                          range_or_none(any ? bias : nullptr, C * sizeof(float)),
                          range_or_none(lens, B * sizeof(int32_t)),
                          in_place ? Range{0, 0} : range_or_none(state_in, st)};
  if (clash(writes, reads)) return GDR_E_ALIAS;
  a.lens = lens;
  a.state_in = state_in;
  a.state_out = state_out;
  a.y[0] = y0;
  a.y[1] = y1;
  a.y[2] = y2;
  a.c[0] = d.c0;
  a.c[1] = d.c1;
  a.c[2] = d.c2;
  return result(gdr::launch_conv(a, io == GDR_BF16, stream));
}

int gdr_ssm_step(const gdr_ssm_dims* dims, gdr_dtype io, const void* xbc, const float* dt,
                 const float* A_log, const float* dt_bias, const float* D, float* state, void* y,
                 hipStream_t stream) {
  int rc = check_ssm_sizes(dims, io, 1);
  if (rc != GDR_OK) return rc;
  const gdr_ssm_dims& d = *dims;
  if (d.B == 0) return GDR_OK;
  if (!xbc || !state || !y) return GDR_E_NULL;
  rc = check_ssm_params(dt, A_log, dt_bias, D);
  if (rc != GDR_OK) return rc;
  if (!aligned(xbc, 16) || !aligned(state, 16) || !aligned(y, 16)) return GDR_E_ALIGN;
  const size_t es = size_of(io), B = d.B, H = d.H;
  const Range writes[2] = {range_of(state, B * H * d.N * d.P * sizeof(float)),
                           range_of(y, B * H * d.P * es)};
  const Range reads[5] = {
      range_of(xbc, B * (H * d.P + 2 * static_cast<size_t>(d.G) * d.N) * es),
      range_of(dt, B * H * sizeof(float)), range_of(A_log, H * sizeof(float)),
      range_or_none(dt_bias, H * sizeof(float)), range_or_none(D, H * sizeof(float))};
  if (clash(writes, reads)) return GDR_E_ALIAS;
  gdr::SsmArgs a = {};
  a.x = xbc;
  a.dt = dt;
  a.A_log = A_log;
  a.dt_bias = dt_bias;
  a.D = D;
  a.state_in = state;
  a.state_out = state;
  a.y = y;
  a.B = d.B;
  a.T = 1;
  a.G = d.G;
  a.H = d.H;
  a.N = d.N;
  a.P = d.P;
  return result(gdr::launch_ssm_step(a, io == GDR_BF16, stream));
}

size_t gdr_ssm_workspace_size(const gdr_ssm_dims* dims, gdr_dtype io) {
  if (!dims || check_ssm_sizes(dims, io, dims->T) != GDR_OK || dims->B == 0 || dims->T == 0)
    return 0;
  return gdr::ssm_workspace_bytes(dims->B, dims->T, dims->G, dims->H, dims->N, dims->P,
                                  io == GDR_BF16);
}

int gdr_ssm_prefill(const gdr_ssm_dims* dims, gdr_dtype io, const void* x, const void* b,
                    const void* c, const float* dt, const float* A_log, const float* dt_bias,
                    const float* D, const int32_t* lens, const float* state_in, float* state_out,
                    void* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int rc = check_ssm_sizes(dims, io, dims ? dims->T : 0);
  if (rc != GDR_OK) return rc;
  const gdr_ssm_dims& d = *dims;
  if (d.B == 0) return GDR_OK;
  const bool any = d.T > 0;
  if (!state_out || (any && (!x || !b || !c || !y))) return GDR_E_NULL;
  if (!any && state_in == state_out) return GDR_OK;
  if (!aligned(state_in, 16) || !aligned(state_out, 16) || !aligned(lens, 4)) return GDR_E_ALIGN;
  const size_t need = gdr_ssm_workspace_size(dims, io);
  if (any) {
    rc = check_ssm_params(dt, A_log, dt_bias, D);
    if (rc != GDR_OK) return rc;
    if (!aligned(x, 16) || !aligned(b, 16) || !aligned(c, 16) || !aligned(y, 16))
      return GDR_E_ALIGN;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDR_E_WORKSPACE;
    if (need > 0 && !aligned(workspace, 16)) return GDR_E_ALIGN;
  }
  const size_t es = size_of(io), B = d.B, T = d.T, H = d.H;
  const size_t st = B * H * d.N * d.P * sizeof(float), bc = B * T * d.G * d.N * es;
  const Range writes[3] = {range_of(state_out, st), range_of(y, B * T * H * d.P * es),
                           need ? range_of(workspace, need) : Range{0, 0}};
  const Range reads[8] = {range_of(x, B * T * H * d.P * es), range_of(b, bc), range_of(c, bc),
                          range_of(dt, B * T * H * sizeof(float)),
                          range_or_none(any ? A_log : nullptr, H * sizeof(float)),
                          range_or_none(any ? dt_bias : nullptr, H * sizeof(float)),
                          range_or_none(any ? D : nullptr, H * sizeof(float)),
                          range_or_none(any ? lens : nullptr, B * sizeof(int32_t))};
  const Range from = range_or_none(state_in, st);
  if (clash(writes, reads) || overlap(writes[1], from) || overlap(writes[2], from) ||
      (state_in != state_out && overlap(writes[0], from)))
    return GDR_E_ALIAS;
  gdr::SsmArgs a = {};
  a.x = x;
  a.b = b;
  a.c = c;
  a.dt = dt;
  a.A_log = A_log;
  a.dt_bias = dt_bias;
  a.D = D;
  a.lens = lens;
  a.state_in = state_in;
  a.state_out = state_out;
  a.y = y;
  a.ws = workspace;
  a.B = d.B;
  a.T = d.T;
  a.G = d.G;
  a.H = d.H;
  a.N = d.N;
  a.P = d.P;
  return result(gdr::launch_ssm_prefill(a, io == GDR_BF16, stream));
}

int gdr_kv_append(const gdr_kv_dims* dims, gdr_dtype io, const void* k, const void* v,
                  const int32_t* block_table, const int32_t* pos, const int32_t* lens,
                  void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                  hipStream_t stream) {
  int rc = check_kv_sizes(dims, io, false);
  if (rc != GDR_OK) return rc;
  const gdr_kv_dims& d = *dims;
  if (d.B == 0 || d.T == 0 || d.n_pages == 0 || d.max_pages == 0) return GDR_OK;
  if (!k || !v) return GDR_E_NULL;
  KvRanges r;
  rc = check_kv_ptrs(d, k_cache, v_cache, k_scale, v_scale, block_table, pos, lens, &r);
  if (rc != GDR_OK) return rc;
  if (!aligned(k, 16) || !aligned(v, 16)) return GDR_E_ALIGN;
  const size_t in = static_cast<size_t>(d.B) * d.T * d.H_kv * d.D * size_of(io);
  const Range writes[4] = {r.k_cache, r.v_cache, r.k_scale, r.v_scale};
  const Range reads[5] = {range_of(k, in), range_of(v, in), r.table, r.pos, r.lens};
  if (clash(writes, reads)) return GDR_E_ALIAS;
  gdr::KvArgs a = kv_args(d);
  a.k = k;
  a.v = v;
  a.block_table = block_table;
  a.pos = pos;
  a.lens = lens;
  a.k_cache = static_cast<uint8_t*>(k_cache);
  a.v_cache = static_cast<uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return result(gdr::launch_kv_append(a, io == GDR_BF16, stream));
}

size_t gdr_attn_workspace_size(const gdr_kv_dims* dims, gdr_dtype io) {
  if (check_kv_sizes(dims, io, true) != GDR_OK || dims->B == 0 || dims->T == 0) return 0;
  return gdr::attn_workspace_bytes(kv_args(*dims), io == GDR_BF16);
}

int gdr_attn_cached(const gdr_kv_dims* dims, gdr_dtype io, const void* q, const void* k_cache,
                    const void* v_cache, const float* k_scale, const float* v_scale,
                    const int32_t* block_table, const int32_t* pos, const int32_t* lens, void* o,
                    float scale, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int rc = check_kv_sizes(dims, io, true);
  if (rc != GDR_OK) return rc;
  const gdr_kv_dims& d = *dims;
  if (d.B == 0 || d.T == 0) return GDR_OK;
  if (!q || !o) return GDR_E_NULL;
  KvRanges r;
  rc = check_kv_ptrs(d, k_cache, v_cache, k_scale, v_scale, block_table, pos, lens, &r);
  if (rc != GDR_OK) return rc;
  if (!aligned(q, 16) || !aligned(o, 16)) return GDR_E_ALIGN;
  const size_t need = gdr_attn_workspace_size(dims, io);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GDR_E_WORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return GDR_E_ALIGN;
  const size_t bytes = static_cast<size_t>(d.B) * d.T * d.H_q * d.D * size_of(io);
  const Range writes[2] = {range_of(o, bytes), need ? range_of(workspace, need) : Range{0, 0}};
  const Range reads[8] = {range_of(q, bytes), r.k_cache, r.v_cache, r.k_scale,
                          r.v_scale,          r.table,   r.pos,     r.lens};
  if (clash(writes, reads)) return GDR_E_ALIAS;
  gdr::KvArgs a = kv_args(d);
  a.q = q;
  a.o = o;
  a.block_table = block_table;
  a.pos = pos;
  a.lens = lens;
  a.k_cache = static_cast<uint8_t*>(const_cast<void*>(k_cache));
  a.v_cache = static_cast<uint8_t*>(const_cast<void*>(v_cache));
  a.k_scale = const_cast<float*>(k_scale);
  a.v_scale = const_cast<float*>(v_scale);
  a.ws = workspace;
  a.scale = scale;
  return result(gdr::launch_attn(a, io == GDR_BF16, stream));
}

}  // extern "C"
