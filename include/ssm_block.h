/*
 * libssm_block: what stands around the state-space mixers of libssm in a
 * model of hybrid blocks, on AMD MI355X (gfx950): a gated linear recurrence,
 * the residual addition with RMS norm, and sliding-window attention with
 * sinks, each with its backward or its single-token form.  Plain C ABI:
 * device pointers, sizes, a HIP stream; no torch types.
 *
 * The conventions are those of ssm.h (whose status and dtype codes these
 * calls share):
 *   - Tensor pointers are DEVICE pointers owned by the caller.  The library
 *     never allocates, frees or synchronises; scratch memory ("workspace") is
 *     passed in by the caller and need not be initialised.
 *   - Every tensor is dense, row-major, with the last listed index
 *     contiguous, except where a stride is given.
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL = null stream)
 *     and may be captured into a HIP graph.
 *   - All argument checks run on the host before any HIP call.  A call that
 *     fails a check returns a negative ssm_status_t, launches nothing and
 *     writes nothing; ssm_block_last_error() then holds a one-line reason
 *     (per host thread).  SSM_ERR_HIP is returned when a launch itself fails.
 *   - Pointers must be aligned to their element size, and more where an entry
 *     point says so; otherwise SSM_ERR_ALIGN.
 *   - Outputs must not overlap inputs or each other, except where an entry
 *     point says so, and the workspace none of them; otherwise SSM_ERR_SHAPE.
 *   - Unsupported sizes return SSM_ERR_UNSUPPORTED; there is no fallback path.
 *   - Indices and offsets are 64-bit throughout.
 *   - The same inputs give the same bits on every call: no result depends on
 *     the order in which workgroups finish.
 */
#ifndef SSM_BLOCK_H
#define SSM_BLOCK_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The reason of this thread's last failed call ("" after a call that passed). */
SSM_API const char *ssm_block_last_error(void);

/* ------------------------------------------------------------------------ */
/* Gated linear recurrence                                                   */
/* ------------------------------------------------------------------------ */

/*
 * Sizes of one call.  in_dtype: x, rec, inp (and dy, dx, drec, dinp);
 * out_dtype: y.  reserved must be 0.  Supported: any batch, seqlen, dim >= 0
 * with dim <= 2^22 and batch * ceil(dim / 32) * ceil(seqlen / 128) < 2^31.
 */
typedef struct {
  int64_t batch, seqlen, dim;
  int32_t in_dtype, out_dtype;
  int32_t reserved;
  int32_t reserved2;
  void *workspace;
  size_t workspace_bytes;
} ssm_glr_dims_t;

/* Steps between two saved states (see `states` below). */
enum { SSM_GLR_STATE_STEP = 16 };

/*
 * Per batch row and channel, with s(v) = 1 / (1 + exp(-v)):
 *   r_t = s(rec_t), i_t = s(inp_t), a_t = exp(A r_t), b_t = sqrt(1 - a_t^2)
 *   h_t = a_t h_{t-1} + b_t i_t x_t,   y_t = h_t
 * h_{-1} = h0; where reset_t is not 0, h_{t-1} counts as zero in step t.
 *   x, rec, inp : (batch, seqlen, dim) in_dtype
 *   A           : (dim) float32, A <= 0 (a positive A gives NaN)
 *   h0          : (batch, dim) float32, nullable (zero)
 *   reset       : (batch, seqlen) bytes, nullable (no resets)
 *   y           : (batch, seqlen, dim) out_dtype
 *   h_last      : (batch, dim) float32, nullable; may be exactly h0
 *   states      : (batch, ceil(seqlen / 16), dim) float32, nullable: the
 *                 state before step 16 k, which ssm_glr_bwd starts from
 * seqlen = 0 writes h_last = h0.  1 - a^2 is computed without cancellation
 * where a is near 1.  A sequence's tiles wait for their predecessors' states in
 * the workspace; a wait of several seconds, which only a fault could cause,
 * ends in NaN.
 */
SSM_API int ssm_glr_workspace_size(const ssm_glr_dims_t *dims, size_t *bytes);
SSM_API int ssm_glr_fwd(const void *x, const void *rec, const void *inp, const float *A, const float *h0,
                        const uint8_t *reset, void *y, float *h_last, float *states,
                        const ssm_glr_dims_t *dims, void *stream);

/*
 * Backward: with g_t = dy_t + a_{t+1} g_{t+1} (the second term absent where
 * reset_{t+1}, and a_L g_L = dh_last), hp_t = h_{t-1} (zero where reset_t):
 *   w_t = g_t (a_t hp_t - a_t^2 / b_t i_t x_t)           (d / d log a_t)
 *   dx_t = g_t b_t i_t        dinp_t = g_t b_t x_t i_t (1 - i_t)
 *   drec_t = w_t A r_t (1 - r_t)     dA = sum over batch and t of w_t r_t
 *   dh0 = a_0 g_0 (zero where reset_0)
 * Where 1 - a_t^2 is below 2^-126 (the gate is shut) b_t and its term of w_t
 * count as 0.
 *   states : what ssm_glr_fwd saved for these inputs
 *   dy     : (batch, seqlen, dim) in_dtype (out_dtype is not used)
 *   dh_last: (batch, dim) float32, nullable (zero)
 *   dx, drec, dinp: (batch, seqlen, dim) in_dtype; dA: (dim) float32;
 *   dh0    : (batch, dim) float32, nullable
 */
SSM_API int ssm_glr_bwd_workspace_size(const ssm_glr_dims_t *dims, size_t *bytes);
SSM_API int ssm_glr_bwd(const void *x, const void *rec, const void *inp, const float *A, const uint8_t *reset,
                        const float *states, const void *dy, const float *dh_last, void *dx, void *drec,
                        void *dinp, float *dA, float *dh0, const ssm_glr_dims_t *dims, void *stream);

/*
 * One step (dims.seqlen must be 1; no workspace): x, rec, inp, y are
 * (batch, dim), h the state before the step and h_out (which may be exactly
 * h) the state after it, (batch, dim) float32.
 */
SSM_API int ssm_glr_step(const void *x, const void *rec, const void *inp, const float *A, const float *h,
                         void *y, float *h_out, const ssm_glr_dims_t *dims, void *stream);

/* ------------------------------------------------------------------------ */
/* Residual addition with RMS norm                                           */
/* ------------------------------------------------------------------------ */

/*
 * Sizes of one call.  in_dtype: x, residual, residual_out (and dy, s, dres,
 * dx); out_dtype: y.  group: values that share a scale in the 8-bit form: 0
 * (the whole row) or a multiple of 32.  Supported: rows >= 0, dim >= 1.
 */
typedef struct {
  int64_t rows, dim, group;
  int32_t in_dtype, out_dtype;
  float eps;
  int32_t reserved;
  void *workspace;
  size_t workspace_bytes;
} ssm_rms_dims_t;

/*
 * Per row: s = x + residual, rstd = 1 / sqrt(mean(s^2) + eps),
 * y = s rstd w.  s is summed and normalised in float32; residual_out holds it
 * rounded to in_dtype.
 *   x, residual, residual_out: (rows, dim) in_dtype; residual is nullable
 *     (s = x), residual_out is nullable and may be exactly x or residual
 *   w: (dim) float32;  y: (rows, dim) out_dtype, may be exactly x
 */
SSM_API int ssm_rms_add_fwd(const void *x, const void *residual, const float *w, void *y, void *residual_out,
                            const ssm_rms_dims_t *dims, void *stream);

/*
 * The same with y in 8 bits: y stands for q * scale, where scale is
 * max |y| / 448 over the group (the row with group = 0; a row's last group
 * may be short) and q = y / scale rounded to the nearest e4m3 value (OCP:
 * 4 exponent and 3 mantissa bits, largest 448).  A group of zeros has scale
 * 0 and q 0; a NaN in a group makes its scale NaN.
 *   q: (rows, dim) bytes; scale: (rows, ceil(dim / group)) float32
 * out_dtype is not used.
 */
SSM_API int ssm_rms_add_q8_fwd(const void *x, const void *residual, const float *w, void *q, float *scale,
                               void *residual_out, const ssm_rms_dims_t *dims, void *stream);

/*
 * Backward of y with respect to the sum s (what residual_out holds) and w:
 * with n = s rstd and dn = dy w,
 *   dx = rstd (dn - n mean(dn n)) + dres,   dw = sum over rows of dy n
 * dx is the gradient of x and of residual alike; dres (nullable) is what
 * arrives through residual_out.
 *   dy, s, dres, dx: (rows, dim) in_dtype (dx may be exactly dy or dres);
 *   w, dw: (dim) float32, dw nullable
 */
SSM_API int ssm_rms_add_bwd_workspace_size(const ssm_rms_dims_t *dims, size_t *bytes);
SSM_API int ssm_rms_add_bwd(const void *dy, const void *s, const float *w, const void *dres, void *dx, float *dw,
                            const ssm_rms_dims_t *dims, void *stream);

/* ------------------------------------------------------------------------ */
/* Sliding-window attention with sinks                                       */
/* ------------------------------------------------------------------------ */

/*
 * Sizes of one call.  nheads query heads, nkv key heads (nkv divides nheads;
 * query head h reads key head h / (nheads / nkv)), headdim 64 or 128.  All
 * storage is bfloat16, lse is float32.  window >= 1, sinks >= 0.
 * q_batch, q_token, ...: elements between two batch rows and two tokens of q,
 * k and v (heads of a token are adjacent: head stride headdim); the batch and
 * token strides must be multiples of 8 and q, k, v 16-byte aligned, and so
 * must y, dy, dq, dk and dv, which are dense; token strides are at most 2^24.
 * scale multiplies q.k.  seqlen <= 2^30, nheads and batch * nheads <= 65535,
 * batch * nheads * seqlen < 2^31 (seqlen counted in whole blocks of 128), and
 * in the backward batch * nkv * sinks < 2^27.
 */
typedef struct {
  int64_t batch, seqlen, nheads, nkv, headdim;
  int64_t window, sinks;
  int64_t q_batch, q_token, k_batch, k_token, v_batch, v_token;
  float scale;
  int32_t reserved;
  void *workspace;
  size_t workspace_bytes;
} ssm_swa_dims_t;

/*
 * Query t of a batch row sees key j when j <= t, j < length, t < length and
 * (t - j < window or j < sinks):
 *   y_t = sum_j p_tj v_j,  p_tj = exp(scale q_t.k_j) / sum over the seen keys
 * A query at or past the row's length sees nothing: y = 0, lse = -inf.
 *   q, y   : (batch, seqlen, nheads, headdim);  k, v: (batch, seqlen, nkv, headdim)
 *   lengths: (batch) int32, nullable (seqlen); values outside 0 .. seqlen are
 *            taken as the nearer end.  Rows of q, k and v at or past the length
 *            are not used: they may hold anything.
 *   lse    : (batch, nheads, seqlen) float32, nullable: log of the sum of
 *            exp(scale q.k) over the seen keys
 * An infinity or NaN in a key or value reaches the queries that see it only.
 */
SSM_API int ssm_swa_fwd(const void *q, const void *k, const void *v, const int32_t *lengths, void *y, float *lse,
                        const ssm_swa_dims_t *dims, void *stream);

/*
 * Backward: with p from q, k and lse, and dp_tj = dy_t.v_j,
 *   ds_tj = p_tj (dp_tj - dy_t.y_t)
 *   dq_t = scale sum_j ds_tj k_j, dk_j = scale sum ds_tj q_t, dv_j = sum p_tj dy_t
 * the last two over the queries and query heads that see j.
 *   dy, y, dq: (batch, seqlen, nheads, headdim); dk, dv: (batch, seqlen, nkv, headdim)
 * Rows at or past the length are not used and get zero gradients.  An infinity
 * or NaN in a key or value reaches the queries that see it, and through their
 * gradients the keys and values that those see; one in a query or its dy, the
 * keys and values that it sees.
 */
SSM_API int ssm_swa_bwd_workspace_size(const ssm_swa_dims_t *dims, size_t *bytes);
SSM_API int ssm_swa_bwd(const void *q, const void *k, const void *v, const int32_t *lengths, const void *y,
                        const float *lse, const void *dy, void *dq, void *dk, void *dv, const ssm_swa_dims_t *dims,
                        void *stream);

/*
 * One token per batch row against a cache of sinks + window slots, in which
 * position p lives in slot p when p < sinks, else in slot
 * sinks + (p - sinks) mod window: the first `sinks` positions stay, the last
 * `window` others are kept.  The call stores k and v of position pos in its
 * slot and attends over every position the cache then holds.
 *   q, y            : (batch, nheads, headdim);  k, v: (batch, nkv, headdim);
 *                     q_token, k_token and v_token are not used
 *   k_cache, v_cache: (batch, nkv, sinks + window, headdim), 16-byte aligned;
 *                     slots of positions not yet stored may hold anything
 *   pos             : (batch) int32; a negative value marks a row without a
 *                     token: y = 0 and its cache stays as it is
 * dims.seqlen must be 1.  sinks + window <= 2^30.
 */
SSM_API int ssm_swa_step_workspace_size(const ssm_swa_dims_t *dims, size_t *bytes);
SSM_API int ssm_swa_step(const void *q, const void *k, const void *v, void *k_cache, void *v_cache,
                         const int32_t *pos, void *y, const ssm_swa_dims_t *dims, void *stream);

/*
 * Store the keys and values of a prompt into such a cache: of every batch
 * row the positions below its length that a next token would still see.
 *   k, v: (batch, seqlen, nkv, headdim); lengths as ssm_swa_fwd
 * Slots that no such position owns keep what they hold.
 */
SSM_API int ssm_swa_fill(const void *k, const void *v, const int32_t *lengths, void *k_cache, void *v_cache,
                         const ssm_swa_dims_t *dims, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_BLOCK_H */
