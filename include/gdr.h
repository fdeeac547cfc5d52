/*
 * gdr.h -- C ABI of the gated delta rule library for AMD Instinct MI355X (gfx950).
 * The layers beside it (short convolution, state space scan, attention over an
 * 8-bit cache; norms, 8-bit products, rotary positions) follow in the second half.
 *
 * The gated delta rule is the GatedDeltaNet linear-attention recurrence.  Per
 * batch row b and value head h it keeps a state S (dk x dv, fp32) and, for each
 * token with query q, key k (dk), value v (dv), write strength beta in (0,1) and
 * log-decay g <= 0 (one per key channel, or one per token for the scalar gate):
 *
 *     S   <- diag(exp(g)) S                       decay
 *     S   <- S + beta * k * (v - S^T k)^T         delta-rule write
 *     o    = scale * S^T q                        read the updated state
 *
 * Sources: the fused decode step (Q/K/V split, L2 normalisation, head repeat,
 * gating, recurrent update) is the one described on the page "Add fused
 * GatedDeltaNet decode Triton kernel" (executorch PR #18865, summary); the
 * two-pass state update on "Two-pass optimization for channelwise gated delta
 * rule kernel" (executorch PR #21020, Summary); routing by sequence length and
 * the chunkwise WY/UT prefill with a ragged final chunk on "Add parallel
 * chunked prefill for channelwise gated delta rule" (executorch PR #21061,
 * Summary).  The pages print no formulas; the conventions below are the
 * library's reading of them and are fixed:
 *
 *   - L2 normalisation (when l2norm_qk != 0): x / sqrt(sum x^2 + 1e-6);
 *   - head repeat: value head h uses query/key head h / (H_v / H_qk);
 *   - beta = sigmoid(beta_logit), computed in the kernel;
 *   - gates (gdr_gate): channel g per key channel; scalar g per token/head;
 *     fused g = -exp(A_log[h]) * softplus(x + dt_bias[h]);
 *   - output from the post-update state, times `scale`.
 *
 * Conventions shared by every entry point
 *   - All tensors are dense, row-major (last index fastest), in device memory,
 *     16-byte aligned, owned by the caller.  The library never allocates,
 *     frees or synchronises; it only enqueues kernels on `stream` (a
 *     hipStream_t; NULL means the default stream) and returns.
 *   - fp32 tensors are `float`; bf16 tensors are IEEE bfloat16 bit patterns.
 *     The state is always fp32.  q/k/v (or qkv) and o use the io dtype.
 *   - Return value: GDR_OK or a negative gdr_status.  Arguments are validated
 *     on the host before any launch; on error nothing is enqueued and no
 *     buffer is touched.  GDR_E_HIP reports a failed launch.
 *   - Supported sizes: dk, dv in {16, 32, 64, 128}; H_v a multiple of H_qk;
 *     chunk in {16, 32, 64}.  B = 0 (and T = 0 for prefill) is a valid no-op.
 *     GDR_E_SHAPE also reports sizes past the 32-bit limits of the launch:
 *     B * H_v * dv and, for prefill, B * H_v * ceil(T / chunk) at most
 *     2^31 - 1, and chunk * H_v * dv at most 2^32 - 1.  The layers in the
 *     second half state theirs in the same way: workgroups within 2^24 and
 *     their threads within 2^32, positions and lengths within 2^31 - 129,
 *     256 H P and 256 G N bytes (a chunk of the scan) within 2^32.
 */
#ifndef GDR_H_
#define GDR_H_

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* dtype of q/k/v (or the packed qkv row) and of o. */
typedef enum gdr_dtype { GDR_F32 = 0, GDR_BF16 = 1 } gdr_dtype;

/* How the log-decay g is given.  Shapes are listed as [decode] / [prefill].
 *   GDR_GATE_CHANNEL      gate_in = g  [B,H_v,dk] / [B,T,H_v,dk]
 *   GDR_GATE_SCALAR       gate_in = g  [B,H_v]    / [B,T,H_v]
 *   GDR_GATE_SCALAR_FUSED gate_in = x  [B,H_v]    / [B,T,H_v], with A_log and
 *                         dt_bias [H_v]: g = -exp(A_log[h]) * softplus(x + dt_bias[h])
 * All gate tensors are fp32.  A_log and dt_bias must be NULL for the other kinds
 * or are ignored.  Channel and scalar g must be <= 0 (a decay, not a growth);
 * any strength of decay is supported: the chunked prefill evaluates only
 * exponentials of non-positive arguments (it forms the chunk's causal terms
 * exactly once a chunk decays by more than e^-64 on some channel). */
typedef enum gdr_gate {
  GDR_GATE_CHANNEL = 0,
  GDR_GATE_SCALAR = 1,
  GDR_GATE_SCALAR_FUSED = 2
} gdr_gate;

/* Problem sizes.  Decode ignores T and chunk. */
typedef struct gdr_dims {
  int32_t B, T, H_qk, H_v, dk, dv, chunk;
} gdr_dims;

typedef enum gdr_status {
  GDR_OK = 0,
  GDR_E_NULL = -1,        /* a required pointer is NULL                         */
  GDR_E_SHAPE = -2,       /* negative size, H_v % H_qk != 0, H % G != 0, ...    */
  GDR_E_DTYPE = -3,       /* unknown io dtype, gate kind or activation          */
  GDR_E_UNSUPPORTED = -4, /* dk/dv/chunk/W/N/P/D/page outside the compiled set, */
                          /* or a value outside what an entry point takes       */
  GDR_E_WORKSPACE = -5,   /* workspace NULL or smaller than the size query      */
  GDR_E_HIP = -6,         /* the HIP runtime reported an error at launch        */
  GDR_E_ALIAS = -7,       /* o, the state or the workspace overlaps a buffer    */
                          /* it must not (see each entry point)                 */
  GDR_E_ALIGN = -8,       /* a tensor is not 16-byte aligned (fp32 vectors and  */
                          /* int32 tensors of the layers: to their element)     */
  GDR_E_SCRATCH = -9      /* the call needs more workspace than the             */
                          /* allocation-free entry point holds                  */
} gdr_status;

/*
 * gdr_decode_step -- one token (T = 1) for every (batch row, value head), one kernel.
 *
 * Fuses, per the page "Add fused GatedDeltaNet decode Triton kernel" (PR #18865,
 * summary): the Q/K/V split of the packed row, L2 normalisation of q and k, the
 * head repeat H_qk -> H_v, the gates (beta and the decay) and the state update.
 * The update reads and writes the state once each, in the two-pass order of
 * "Two-pass optimization for channelwise gated delta rule kernel" (PR #21020,
 * Summary): pass 1 forms vhat = (diag(a) S)^T k with the decay a = exp(g)
 * folded in; pass 2 writes S = diag(a) S + beta k (v - vhat)^T and accumulates
 * o = scale S^T q.
 *
 *   dims        B, H_qk, H_v, dk, dv (T and chunk ignored)
 *   io          dtype of qkv and o
 *   gate        see gdr_gate; gate_in shape [B,H_v,dk] or [B,H_v]
 *   qkv         [B, 2*H_qk*dk + H_v*dv]: q heads, then k heads, then v heads,
 *               each head's channels contiguous
 *   A_log, dt_bias  [H_v] fp32 for GDR_GATE_SCALAR_FUSED, else ignored
 *   beta_logit  [B,H_v] fp32
 *   state       [B,H_v,dk,dv] fp32, read and updated IN PLACE; must not
 *               overlap qkv, gate_in, A_log, dt_bias or beta_logit
 *   o           [B,H_v,dv] io dtype, written; must not overlap the state or
 *               any input
 *   scale       output multiplier
 *   l2norm_qk   nonzero: normalise q and k rows; zero: use them as given
 */
int gdr_decode_step(const gdr_dims* dims, gdr_dtype io, gdr_gate gate, const void* qkv,
                    const float* gate_in, const float* A_log, const float* dt_bias,
                    const float* beta_logit, float* state, void* o, float scale,
                    int l2norm_qk, hipStream_t stream);

/*
 * gdr_prefill_workspace_size -- bytes of device workspace gdr_prefill_chunked
 * needs for these sizes and this gate kind (0 when B or T is 0).  Returns 0 as
 * well for unsupported arguments; gdr_prefill_chunked then reports the reason.
 * Scalar gates need less per value head: with one decay per token the decayed
 * keys and queries are row scalings of the normalised k and q rows, which are
 * kept once per qk head.
 */
size_t gdr_prefill_workspace_size(const gdr_dims* dims, gdr_dtype io, gdr_gate gate);

/*
 * gdr_prefill_chunked -- T tokens per (batch row, value head), chunkwise WY/UT form.
 *
 * Follows "Add parallel chunked prefill for channelwise gated delta rule"
 * (PR #21061, Summary): per chunk of `chunk` tokens (the last chunk may be
 * shorter and runs through the same code), per-channel log-decay prefix sums,
 * the causal query/key and key/key terms, the beta-folded unit-lower-triangular
 * transform, WY pseudo-keys / pseudo-values, and the carry of the state from
 * chunk to chunk.  Independent (batch, head) units run in parallel, each with a
 * disjoint slice of the caller's workspace.  The result equals T applications
 * of the token update (up to rounding).
 *
 * Short sequences (T <= 16 at up to 64 (batch, head) units, T <= 24 above)
 * are run token by token instead, each token the two-pass update above, with
 * the state held on chip across the tokens: the fixed cost of the chunked form
 * does not pay off there.  The workspace is then not touched, but the same
 * size is still required.
 *
 * Long sequences over few units (at most 128 sixteen-column state slices,
 * B * H_v * dv / 16, and segments of at least 8 chunks) carry the state by a
 * parallel scan instead of one walk: the carry over a range of chunks is an
 * affine map of the state, S_out = M S_in + N, so the sequence is cut into
 * segments whose maps are formed side by side, composed in fp32, and each
 * segment is then run from its start state.  The workspace then also holds
 * fp32 segment states and maps, which the size query includes.  The result
 * matches the single walk to rounding.
 *
 *   dims        B, T, H_qk, H_v, dk, dv, chunk
 *   io          dtype of q, k, v and o
 *   gate        see gdr_gate; gate_in shape [B,T,H_v,dk] or [B,T,H_v]
 *   q, k        [B,T,H_qk,dk]
 *   v           [B,T,H_v,dv]
 *   A_log, dt_bias  [H_v] fp32 for GDR_GATE_SCALAR_FUSED, else ignored
 *   beta_logit  [B,T,H_v] fp32
 *   state_in    [B,H_v,dk,dv] fp32 initial state, or NULL for zeros
 *   state_out   [B,H_v,dk,dv] fp32 final state; either equal to state_in
 *               (in place) or not overlapping it, and not overlapping any
 *               other input
 *   o           [B,T,H_v,dv] io dtype; must not overlap any input or the state
 *   workspace   device memory of at least gdr_prefill_workspace_size() bytes,
 *               16-byte aligned, contents need not be initialised; it must not
 *               overlap any input, o or the state, and may be reused once the
 *               enqueued work has finished
 *   T == 0      copies state_in to state_out (zeros when state_in is NULL)
 */
int gdr_prefill_chunked(const gdr_dims* dims, gdr_dtype io, gdr_gate gate, const void* q,
                        const void* k, const void* v, const float* gate_in, const float* A_log,
                        const float* dt_bias, const float* beta_logit, const float* state_in,
                        float* state_out, void* o, float scale, int l2norm_qk, void* workspace,
                        size_t workspace_bytes, hipStream_t stream);

/*
 * gdr_prefill_chunked_noalloc -- gdr_prefill_chunked without a workspace
 * argument, for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation.
 *
 * Same arguments, results, validation and status codes as
 * gdr_prefill_chunked, minus workspace / workspace_bytes.  The workspace is a
 * device array inside the library, GDR_NOALLOC_SCRATCH_BYTES bytes on each
 * device it runs on, held until the process ends; the library allocates and
 * frees nothing on any call.  The first call on a device (the current device)
 * looks up that device's array address.
 *
 *   - A call whose gdr_prefill_workspace_size() exceeds
 *     GDR_NOALLOC_SCRATCH_BYTES returns GDR_E_SCRATCH and enqueues nothing
 *     (B = 1, H_v = 32, dk = dv = 128, chunk 64, bf16 fits up to T = 4032).
 *   - Every call on a device shares that device's array and leaves its
 *     contents behind; no content needs to be cleared between calls.  Calls
 *     that may run at the same time on one device (other streams, other
 *     threads) RACE on the array: order them on one stream, or use
 *     gdr_prefill_chunked with a workspace per concurrent call.
 */
#define GDR_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)
int gdr_prefill_chunked_noalloc(const gdr_dims* dims, gdr_dtype io, gdr_gate gate,
                                const void* q, const void* k, const void* v,
                                const float* gate_in, const float* A_log, const float* dt_bias,
                                const float* beta_logit, const float* state_in, float* state_out,
                                void* o, float scale, int l2norm_qk, hipStream_t stream);

/* ------------------------------------------------------------------------
 * The layers beside the gated delta rule: the short causal convolution that a
 * recurrent layer's input row passes first, the selective state space scan,
 * and attention over a cache of 8-bit keys and values.  The conventions at
 * the top of this file hold; what differs is stated at each function.
 *
 * Padded batches: where a function takes `lens` ([B] int32 in device memory,
 * NULL for T tokens in every row), row b holds lens[b] tokens (taken as 0 if
 * negative, as T if larger).  Tokens behind them are not read, and their
 * output rows are left as they were.
 *
 * Alignment: tensors 16 bytes, but for fp32 vectors (bias, dt, A_log, dt_bias, D,
 * scales) and int32 tensors (lens, pos, block_table), which need that of their
 * element, and x of the convolution.
 *
 * Numbers: states, sums and softmax statistics are fp32 or wider.  An output in
 * bf16 is rounded once, from a sum whose terms are within 2^-15 of themselves or
 * better (gdr_matmul_fp8 states its own).  What depends on an input that is not finite may be infinite or NaN
 * (which of the two can differ between a function's forms); nothing else is.
 * ------------------------------------------------------------------------ */

/* Sizes of the short convolution: W taps over c0 + c1 + c2 channels, written
 * as one to three dense outputs (c1 = c2 = 0 for one, c2 = 0 for two). */
typedef struct gdr_conv_dims {
  int32_t B, T, W, c0, c1, c2;
} gdr_conv_dims;

typedef enum gdr_act { GDR_ACT_NONE = 0, GDR_ACT_SILU = 1 } gdr_act;

/*
 * gdr_conv_step -- one token of a short causal convolution per channel:
 *
 *     y[c] = act(bias[c] + sum_w weight[c][w] * u[w][c])
 *
 * where u is the row's last W inputs, oldest first: the state, then x.  The
 * state then drops its oldest row and takes x.  With C = 2*H_qk*dk + H_v*dv
 * the output is the packed row of gdr_decode_step, with C = H*P + 2*G*N that
 * of gdr_ssm_step.
 *
 *   dims      B, W (2, 3 or 4), C = c0 + c1 + c2 channels (T ignored; the
 *             output is one row of C channels however they are given)
 *   x         [B] rows of C channels, io dtype, x_stride elements apart
 *             (x_stride >= C); aligned to its element.  Rows and outputs that
 *             are 16-byte aligned throughout take the wide path.
 *   weight    [C,W] fp32, 16-byte aligned; weight[c][W-1] multiplies x
 *   bias      [C] fp32 or NULL
 *   state     [B,W-1,C] io dtype, oldest input first, updated IN PLACE; must
 *             not overlap x, weight or bias
 *   y         [B,C] io dtype, must not overlap the state or an input
 */
int gdr_conv_step(const gdr_conv_dims* dims, gdr_dtype io, gdr_act act, const void* x,
                  int64_t x_stride, const float* weight, const float* bias, void* state, void* y,
                  hipStream_t stream);

/*
 * gdr_conv_prefill -- gdr_conv_step for T tokens per row, with the channels
 * split over up to three outputs: c0 | c1 | c2 become the dense q | k | v of
 * gdr_prefill_chunked or the x | b | c of gdr_ssm_prefill.
 *
 *   x          [B,T] rows of C channels, x_stride elements apart
 *   lens       [B] int32 or NULL
 *   state_in   [B,W-1,C] io dtype, the inputs before the first token, oldest
 *              first, or NULL for zeros
 *   state_out  [B,W-1,C] io dtype, the last W-1 inputs (those of state_in
 *              count); may be state_in itself, else must not overlap it, nor
 *              x, weight or bias
 *   y0, y1, y2 [B,T,c0], [B,T,c1], [B,T,c2] io dtype (ignored where the width
 *              is 0), no two overlapping, nor any input or state
 *   T == 0     copies state_in to state_out (zeros when it is NULL)
 */
int gdr_conv_prefill(const gdr_conv_dims* dims, gdr_dtype io, gdr_act act, const void* x,
                     int64_t x_stride, const float* weight, const float* bias,
                     const int32_t* lens, const void* state_in, void* state_out, void* y0,
                     void* y1, void* y2, hipStream_t stream);

/* Sizes of the selective state space scan: H heads of width P with a state of
 * N rows each, in G groups of H / G neighbouring heads that share B and C.
 * N and P in {16, 32, 64, 128}.  A step ignores T. */
typedef struct gdr_ssm_dims {
  int32_t B, T, G, H, N, P;
} gdr_ssm_dims;

/*
 * gdr_ssm_step -- one token of the selective state space scan.  Per batch row
 * and head h of group g = h / (H / G), with input x (P), B and C (N):
 *
 *     d = softplus(dt + dt_bias[h])
 *     S <- exp(-exp(A_log[h]) d) S + d B x^T
 *     y  = S^T C + D[h] x
 *
 * (exp(A_log) past fp32's largest value counts as that value.)
 *
 *   xbc      [B, H*P + 2*G*N] io dtype: x heads, then B groups, then C groups
 *   dt       [B,H] fp32
 *   A_log    [H] fp32
 *   dt_bias  [H] fp32 or NULL (zeros)
 *   D        [H] fp32 or NULL (zeros)
 *   state    [B,H,N,P] fp32, updated IN PLACE; must not overlap an input
 *   y        [B,H,P] io dtype; must not overlap the state or an input
 */
int gdr_ssm_step(const gdr_ssm_dims* dims, gdr_dtype io, const void* xbc, const float* dt,
                 const float* A_log, const float* dt_bias, const float* D, float* state, void* y,
                 hipStream_t stream);

/* gdr_ssm_workspace_size -- bytes of device workspace gdr_ssm_prefill needs
 * (may be 0); 0 as well for unsupported arguments. */
size_t gdr_ssm_workspace_size(const gdr_ssm_dims* dims, gdr_dtype io);

/*
 * gdr_ssm_prefill -- T tokens of the scan; equals T steps up to rounding.
 *
 *   x          [B,T,H,P] io dtype
 *   b, c       [B,T,G,N] io dtype
 *   dt         [B,T,H] fp32
 *   A_log, dt_bias, D   as in gdr_ssm_step
 *   lens       [B] int32 or NULL
 *   state_in   [B,H,N,P] fp32 or NULL for zeros
 *   state_out  [B,H,N,P] fp32, the state behind the last token of each row;
 *              may be state_in itself, else must not overlap it, nor any
 *              other input
 *   y          [B,T,H,P] io dtype; must not overlap any input or the state
 *   workspace  gdr_ssm_workspace_size() bytes (NULL if that is 0), 16-byte
 *              aligned, uninitialised, overlapping nothing else; one for each
 *              call that may run at the same time
 *   T == 0     copies state_in to state_out (zeros when it is NULL)
 */
int gdr_ssm_prefill(const gdr_ssm_dims* dims, gdr_dtype io, const void* x, const void* b,
                    const void* c, const float* dt, const float* A_log, const float* dt_bias,
                    const float* D, const int32_t* lens, const float* state_in, float* state_out,
                    void* y, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The key/value cache is a pool of n_pages pages of `page` tokens.  A page
 * holds e4m3 codes (OCP, 448 at most, no infinity) and one fp32 scale per
 * head for its keys and one for its values; a code c stands for c * scale:
 *
 *     k_cache [n_pages,H_kv,page,D]    k_scale [n_pages,H_kv]
 *     v_cache [n_pages,H_kv,D,page]    v_scale [n_pages,H_kv]
 *
 * Values are stored transposed: attention contracts over the tokens, and so
 * reads them in the order in which the matrix instructions take them.  Scales
 * are powers of two from 2^-100 up.
 *
 * block_table [B,max_pages] int32 names row b's pages in order: its position
 * p lies in page block_table[b][p / page], slot p % page.  pos [B] int32 is
 * the position of the row's first new token (what is cached before the call
 * is [0, pos)).  Entries outside [0, n_pages) and positions outside the table
 * (negative ones, or past max_pages * page) are not followed: such tokens are
 * not written, and attention takes them as absent.  A pool or table without
 * pages may be NULL.
 *
 * H_q a multiple of H_kv; D in {64, 128}; page in {16, 32, 64, 128}.
 * gdr_kv_append ignores H_q.
 */
typedef struct gdr_kv_dims {
  int32_t B, T, H_q, H_kv, D, page, n_pages, max_pages;
} gdr_kv_dims;

/*
 * gdr_kv_append -- writes the keys and values of up to T new tokens per row
 * into their pages.  A page's scale is the smallest power of two s >= 2^-100
 * with max|x| <= 448 s over the finite values written; where the page already
 * holds tokens of the row (positions before pos) it is at least the scale it
 * had, and if it grows, their codes are rounded to the new scale (exact but
 * for values that become subnormal).  Codes round to nearest even; infinities
 * become +-448, NaN stays NaN.  Slots behind the last new token keep their
 * codes.
 *
 *   k, v         [B,T,H_kv,D] io dtype
 *   pos          [B] int32
 *   lens         [B] int32 or NULL
 *   caches, scales   updated in place; must not overlap an input.  Pages that
 *                the call writes must be named once in the table (two writers
 *                of one page race, and its contents are then undefined)
 */
int gdr_kv_append(const gdr_kv_dims* dims, gdr_dtype io, const void* k, const void* v,
                  const int32_t* block_table, const int32_t* pos, const int32_t* lens,
                  void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                  hipStream_t stream);

/* gdr_attn_workspace_size -- bytes of device workspace gdr_attn_cached needs
 * (may be 0); 0 as well for unsupported arguments.  n_pages is not used. */
size_t gdr_attn_workspace_size(const gdr_kv_dims* dims, gdr_dtype io);

/*
 * gdr_attn_cached -- softmax attention of T new tokens per row over the cache:
 * token t of row b, at position pos[b] + t, attends to the cached positions
 * 0 ... pos[b] + t (append the new tokens first); query head h reads kv head
 * h / (H_q / H_kv).
 *
 *     o = sum_j softmax_j(scale q . k_j) v_j
 *
 * A query with nothing to attend to gives zeros.  What lies in the pages
 * behind a row's last position does not matter, NaN included.
 *
 *   q          [B,T,H_q,D] io dtype
 *   o          [B,T,H_q,D] io dtype; must not overlap any input
 *   workspace  gdr_attn_workspace_size() bytes (NULL if that is 0), 16-byte
 *              aligned, uninitialised, overlapping nothing else; one for each
 *              call that may run at the same time
 */
int gdr_attn_cached(const gdr_kv_dims* dims, gdr_dtype io, const void* q, const void* k_cache,
                    const void* v_cache, const float* k_scale, const float* v_scale,
                    const int32_t* block_table, const int32_t* pos, const int32_t* lens, void* o,
                    float scale, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * What stands between the residual stream and the mixers above: the norm that a
 * layer begins with, the 8-bit product that makes the packed row, rotary
 * positions, and the norm or plain 8 bits on the way to the output's product.
 *
 * 8-bit rows: a row of K channels is K e4m3 codes (OCP, 448 at most, no
 * infinity) and one fp32 scale for each block of 128 channels (the last block
 * may be short); a code c stands for c * scale.
 *
 *     codes [R,K]    scales [R,ceil(K/128)]
 *
 * The library writes s = max(amax / 448, 2^-100), amax the largest finite
 * magnitude of the block, and c = value / s rounded to nearest even (each quotient
 * a product with the fp32 reciprocal, first); infinities become +-448, NaN stays
 * NaN.  The product takes any scales whose products
 * x_scales w_scales, which it forms first, are 0 or normal fp32 numbers: smaller
 * ones lose digits, and what a larger one reaches is infinite or NaN.
 * ------------------------------------------------------------------------ */

/* R rows of H heads of D channels. */
typedef struct gdr_norm_dims {
  int32_t R, H, D;
} gdr_norm_dims;

/* Where the gate of gdr_rms_norm goes: behind the norm (the gated delta rule's
 * output) or before it (the scan's). */
typedef enum gdr_norm_gate {
  GDR_NORM_GATE_NONE = 0,
  GDR_NORM_GATE_AFTER = 1,
  GDR_NORM_GATE_BEFORE = 2
} gdr_norm_gate;

/*
 * gdr_rms_norm -- root-mean-square norm of rows, head by head:
 *
 *     h = x | x + residual | x silu(gate)     (nothing, a residual, a gate BEFORE)
 *     y = h / sqrt(mean_D h^2 + eps) * weight [* silu(gate)]        (a gate AFTER)
 *
 * With a residual, h is stored back to it (rounded to its type; the norm takes
 * h as summed in fp32).  H = 1 for whole rows.
 *
 *   dims      R, H, D.  D up to 32768; where H > 1, D is a multiple of 128 or
 *             one of 16, 32, 64
 *   io        dtype of x, gate and y
 *   x         R rows of H*D channels, x_stride elements apart; aligned to its
 *             element, and so is gate.  16-byte aligned rows and D a multiple of
 *             8 take the wide path.
 *   residual  [R,H*D] of dtype res, updated IN PLACE, or NULL (res is then
 *             ignored); not together with a gate (GDR_E_UNSUPPORTED)
 *   order     where the gate goes; gate and gate_stride are ignored for NONE
 *   gate      R rows of H*D channels, gate_stride elements apart
 *   weight    [H,D] fp32 or NULL (ones)
 *   eps       finite and above 0, else GDR_E_UNSUPPORTED
 *   y         [R,H*D] io dtype or NULL
 *   codes, scales   8-bit rows of K = H*D channels, from y before it is rounded
 *             to the io dtype; both or neither NULL, and not NULL together with y
 *
 * residual, y, codes and scales must not overlap each other or an input.  Sums
 * of squares are 64-bit: rows of any finite fp32 magnitude have a finite norm.
 * An h past fp32's range is infinite; a head that holds an infinity is 0 at its
 * finite channels and NaN at the infinite ones.
 */
int gdr_rms_norm(const gdr_norm_dims* dims, gdr_dtype io, const void* x, int64_t x_stride,
                 gdr_dtype res, void* residual, gdr_norm_gate order, const void* gate,
                 int64_t gate_stride, const float* weight, float eps, void* y, void* codes,
                 float* scales, hipStream_t stream);

/*
 * gdr_quant_rows -- rows of H*D channels to 8-bit rows as they are (an
 * attention's output has no norm before its product).  Arguments and conditions
 * as in gdr_rms_norm.
 */
int gdr_quant_rows(const gdr_norm_dims* dims, gdr_dtype io, const void* x, int64_t x_stride,
                   void* codes, float* scales, hipStream_t stream);

typedef struct gdr_matmul_dims {
  int32_t M, N, K;
} gdr_matmul_dims;

/*
 * gdr_matmul_fp8 -- product of 8-bit rows with an 8-bit weight:
 *
 *     y[m,n] = bias[n] + sum_b x_scales[m,b] w_scales[n/128,b]
 *                                sum_{k in block b} x[m,k] w[n,k]
 *
 * over blocks b of 128 channels.  The sum over blocks is fp32 and y is rounded
 * once.  Within a block the output's type chooses the arithmetic:
 *
 *     fp32   products are exact and their sum is fp32
 *     bf16   products are added 8 at a time, what lies 13 bits below the largest
 *            of the 8 is dropped, and the groups' sums are added in fp32.  Next
 *            to y's own rounding that is a hundredth for ordinary rows, but it can
 *            reach 2^-10 of the sum of the terms' magnitudes, so that of a y that
 *            its terms nearly cancel to no digit may be left.  Take fp32 for those
 *
 * The order in which blocks are added depends on the sizes and on the place of
 * the row and column: the same call gives the same digits every time, equal rows
 * at different places, or in calls of different sizes, may differ in their last.
 *
 *   dims      M rows, N outputs (within 2^31 - 257), K channels: a multiple of 16, up
 *             to 2^20
 *   io        dtype of y
 *   x         [M,K] e4m3 codes, 16-byte aligned
 *   x_scales  [M,ceil(K/128)] fp32
 *   w         [N,K] e4m3 codes, 16-byte aligned
 *   w_scales  [ceil(N/128),ceil(K/128)] fp32
 *   bias      [N] fp32 or NULL
 *   y         [M,N] io dtype; must not overlap an input
 *   K == 0    y is the bias (zeros without one)
 */
int gdr_matmul_fp8(const gdr_matmul_dims* dims, gdr_dtype io, const void* x,
                   const float* x_scales, const void* w, const float* w_scales,
                   const float* bias, void* y, hipStream_t stream);

/* Rows of B sequences of T tokens; H_q query heads and H_kv key and value heads
 * of D channels, the first R of which are turned. */
typedef struct gdr_rope_dims {
  int32_t B, T, H_q, H_kv, D, R;
} gdr_rope_dims;

/* Which channels of a head's first R make a pair: (i, i + R/2) or (2i, 2i + 1). */
typedef enum gdr_rope_pairs { GDR_ROPE_HALF = 0, GDR_ROPE_INTERLEAVED = 1 } gdr_rope_pairs;

/*
 * gdr_rope -- splits packed rows of q heads | k heads | v heads and turns q and k
 * by their positions: pair i = (a, b) of token t of row b, at position
 * p = pos[b] + t, becomes
 *
 *     magnitude * (a cos(p freq[i]) - b sin(p freq[i]),
 *                  a sin(p freq[i]) + b cos(p freq[i]))
 *
 * The other channels are copied.  Outputs are as gdr_kv_append and
 * gdr_attn_cached take them.  Angles are 64-bit: exact to 2^-24 of a turn at
 * positions up to 2^24 and frequencies up to 1, and to 2^-20 at any position.
 *
 *   dims      B, T, H_q, H_kv, D (a multiple of 8 up to 512), R (even, 0 to D)
 *   io        dtype of x, q, k and v
 *   x         [B,T] rows of (H_q + 2 H_kv) D channels, x_stride elements apart;
 *             aligned to its element.  16-byte aligned rows and pairs that fill
 *             16 bytes (R a multiple of 8 or, in halves, of 16) take the wide path.
 *   freq      [R/2] fp64 radians a position, finite (NULL if R is 0)
 *   pos       [B] int32, the position of each row's first token
 *   lens      [B] int32 or NULL
 *   q, k, v   [B,T,H_q,D], [B,T,H_kv,D] twice, io dtype; v may be NULL (not
 *             copied; x then has no v heads to show).  Not overlapping each
 *             other or an input
 */
int gdr_rope(const gdr_rope_dims* dims, gdr_dtype io, gdr_rope_pairs pairs, const void* x,
             int64_t x_stride, const double* freq, float magnitude, const int32_t* pos,
             const int32_t* lens, void* q, void* k, void* v, hipStream_t stream);

/* How frequencies base^(-2i/R) are stretched to contexts `factor` times as long
 * as the `context` tokens that a model was trained on:
 *
 *   NONE    not at all
 *   LINEAR  all by 1 / factor
 *   BASE    by a larger base, base * factor^(R / (R - 2)): the first frequency
 *           stays, the last is divided by factor
 *   TURNS   by 1 / factor below `low` turns over the context, not at all above
 *           `high`, and between by 1 / factor + u (1 - 1 / factor),
 *           u = (turns - low) / (high - low)
 *   INDEX   as TURNS, but u falls linearly in the index i, from 1 at the index
 *           (rounded down, at least 0) that makes `high` turns to 0 at the one
 *           (rounded up, at most R - 1) that makes `low`; the magnitude is
 *           0.1 ln(factor) + 1 */
typedef enum gdr_rope_kind {
  GDR_ROPE_NONE = 0,
  GDR_ROPE_LINEAR = 1,
  GDR_ROPE_BASE = 2,
  GDR_ROPE_TURNS = 3,
  GDR_ROPE_INDEX = 4
} gdr_rope_kind;

typedef struct gdr_rope_scaling {
  int32_t kind;  /* gdr_rope_kind */
  double factor, context, low, high;
} gdr_rope_scaling;

/*
 * gdr_rope_freqs -- the frequencies of gdr_rope, computed on the HOST into
 * host memory (copy them to the device once).
 *
 *   R          even, 2 to 512
 *   base       finite and above 1
 *   scaling    NULL for none; factor >= 1; TURNS and INDEX: context > 0,
 *              0 < low < high; BASE: R > 2, its larger base finite.  Else
 *              GDR_E_UNSUPPORTED
 *   freq       [R/2] written; magnitude (may be NULL) written
 */
int gdr_rope_freqs(int32_t R, double base, const gdr_rope_scaling* scaling, double* freq,
                   float* magnitude);

/* Static, human-readable text for a gdr_status value. */
const char* gdr_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H_ */
