/*
 * libssm_delta: blocks of delta-rule layers and of attention with normalised
 * keys, beside the operators of libssm_block, on AMD MI355X (gfx950): the
 * gated delta rule, norms of queries and keys with the rotation by position,
 * and sliding-window attention steps over a cache held in 8 bits.  Plain C
 * ABI: device pointers, sizes, a HIP stream; no torch types.
 *
 * The conventions are those of ssm_block.h (status and dtype codes of ssm.h):
 *   - Tensor pointers are DEVICE pointers owned by the caller, all on the
 *     device of `stream`.  The library never allocates, frees or synchronises;
 *     scratch memory ("workspace") is passed in by the caller, aligned to 256
 *     bytes, and need not be initialised.  Calls that may run at the same time
 *     (on two streams, or in two captured graphs that are replayed at once)
 *     need a workspace each.
 *   - Every tensor is dense, row-major, with the last listed index
 *     contiguous, except where a stride is given.
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL = null stream)
 *     and may be captured into a HIP graph.
 *   - All argument checks run on the host before any HIP call.  A call that
 *     fails a check returns a negative ssm_status_t, launches nothing and
 *     writes nothing; ssm_delta_last_error() then holds a one-line reason
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
#ifndef SSM_DELTA_H
#define SSM_DELTA_H

#include "ssm_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The reason of this thread's last failed call ("" after a call that passed). */
SSM_API const char *ssm_delta_last_error(void);

/* ------------------------------------------------------------------------ */
/* Gated delta rule                                                          */
/* ------------------------------------------------------------------------ */

/*
 * Sizes of one call.  nheads value heads share nqk query and key heads (nqk
 * divides nheads; value head h has query and key head h / (nheads / nqk)).
 * kdim and vdim: 64 or 128 each.  q, k, v, y and their gradients are bfloat16;
 * gate_dtype: g, beta (and dg, dbeta).
 * q_batch, q_token, ...: elements between two batch rows and two tokens of q,
 * k and v (heads of a token are adjacent: head stride kdim or vdim); batch and
 * token strides must be multiples of 8, token strides at most 2^24, and q, k,
 * v, y, dy, dq, dk, dv and the states 16-byte aligned; all but q, k and v are
 * dense.  scale multiplies y.  seqlen <= 2^30, nqk * kdim and nheads * vdim
 * <= 2^24, and batch * nheads * max(4, ceil(seqlen / 64)) < 2^24.
 */
typedef struct {
  int64_t batch, seqlen, nqk, nheads, kdim, vdim;
  int64_t q_batch, q_token, k_batch, k_token, v_batch, v_token;
  float scale;
  int32_t gate_dtype;
  void *workspace;
  size_t workspace_bytes;
} ssm_gdr_dims_t;

/* Tokens that are taken at a time. */
enum { SSM_GDR_STATE_STEP = 64 };

/*
 * Per batch row and value head, with the state S (vdim x kdim), a_t = exp(g_t):
 *   u_t = beta_t (v_t - a_t S_{t-1} k_t)
 *   S_t = a_t S_{t-1} + u_t k_t^T,   y_t = scale S_t q_t
 * over the tokens below the row's length; y is 0 from there on.
 *   q, k   : (batch, seqlen, nqk, kdim);  v, y: (batch, seqlen, nheads, vdim)
 *   g, beta: (batch, seqlen, nheads) gate_dtype; g is the logarithm of the
 *            decay (at or below 0 for a state that fades; -inf forgets, and
 *            so does anything below -200; above 0 the sum over a block of 64
 *            tokens must stay below 88, where exp leaves float32)
 *   h0     : (batch, nheads, vdim, kdim) float32, nullable (zero)
 *   lengths: (batch) int32, nullable (seqlen); values outside 0 .. seqlen are
 *            taken as the nearer end.  Rows at or past the length are not used.
 *   h_last : as h0, nullable: the state after the row's last token (h0 where
 *            there is none); may be exactly h0.  Where it is asked for, the
 *            state is held to float32 on its way (it ends less than 1e-6 of its
 *            norm off, as float32 token by token would), else to 2^-18: y's last
 *            bits may differ with and without it
 *   states : ssm_gdr_states_size() bytes, 16-byte aligned, nullable: what
 *            ssm_gdr_bwd starts from (the state before every 64th token, the
 *            u_t / beta_t, and what of v, g and beta it needs), in an order of its own;
 *            what is of tokens past a row's last block of 64 is not written
 * The rule is stable for beta |k|^2 from 0 to 2: keys are meant to have unit
 * length.
 * Tokens are taken 64 at a time: a value that is not finite reaches y from the
 * start of its block of 64 tokens (of its channel, if it is one of v; of the
 * value heads that share it, if it is one of q or k; of its own, if it is one of
 * beta, or of g and not -inf) and what comes after.
 */
/* (Of a call without states: one with them takes as many bytes, and uses fewer.) */
SSM_API int ssm_gdr_workspace_size(const ssm_gdr_dims_t *dims, size_t *bytes);
SSM_API int ssm_gdr_states_size(const ssm_gdr_dims_t *dims, size_t *bytes);
SSM_API int ssm_gdr_fwd(const void *q, const void *k, const void *v, const void *g, const void *beta, const float *h0,
                        const int32_t *lengths, void *y, float *h_last, void *states, const ssm_gdr_dims_t *dims,
                        void *stream);

/*
 * Backward: with dS_t the gradient of S_t (dS_t = a_{t+1} (dS_{t+1} -
 * dv_{t+1} k_{t+1}^T) + scale dy_t q_t^T, from dh_last after the last token),
 *   e_t = dS_t k_t,  dv_t = beta_t e_t,  dbeta_t = e_t.(v_t - a_t S_{t-1} k_t)
 *   dq_t = scale S_t^T dy_t,  dk_t = dS_t^T u_t - a_t S_{t-1}^T dv_t
 *   dg_t = a_t (<dS_t, S_{t-1}> - dv_t.S_{t-1} k_t)
 * dq and dk are summed over the value heads that share a head.  Rows at or
 * past the length get zero gradients.  dg, dbeta and dh0 are right to about
 * 1e-5 of their norms, also where they are float32, the others to their own
 * rounding.
 *   q, k, lengths: as in the forward;  states: what it saved for them
 *   dh_last, dh0: (batch, nheads, vdim, kdim) float32, both nullable
 *   dq, dk : (batch, seqlen, nqk, kdim);  dv, dy: (batch, seqlen, nheads, vdim)
 *   dg, dbeta: (batch, seqlen, nheads) gate_dtype
 */
SSM_API int ssm_gdr_bwd_workspace_size(const ssm_gdr_dims_t *dims, size_t *bytes);
SSM_API int ssm_gdr_bwd(const void *q, const void *k, const int32_t *lengths, const void *states, const void *dy,
                        const float *dh_last, void *dq, void *dk, void *dv, void *dg, void *dbeta, float *dh0,
                        const ssm_gdr_dims_t *dims, void *stream);

/*
 * One token per batch row (dims.seqlen must be 1; no workspace): q, k are
 * (batch, nqk, kdim), v, y (batch, nheads, vdim), g, beta (batch, nheads), h
 * the state before the token and h_out (which may be exactly h) the state
 * after it.  The token strides are not used.
 */
SSM_API int ssm_gdr_step(const void *q, const void *k, const void *v, const void *g, const void *beta, const float *h,
                         void *y, float *h_out, const ssm_gdr_dims_t *dims, void *stream);

/* ------------------------------------------------------------------------ */
/* Norms of queries and keys with the rotation by position                   */
/* ------------------------------------------------------------------------ */

/*
 * Sizes of one call.  dtype: q, k and what becomes of them (and gradients).
 * headdim: a multiple of 16 up to 256; rot: how many of a head's elements are
 * rotated, a multiple of 16 from 0 to headdim.  neighbours: 0 pairs element i
 * with i + rot / 2, 1 pairs 2 i with 2 i + 1.
 * q_batch, q_token, k_..: elements between batch rows and tokens of q and k;
 * oq_.., ok_..: of q_out and k_out (dq and dk).  Heads of a token are
 * adjacent.  Strides are multiples of 16 bytes, and q, k, wq, wk and the
 * outputs aligned to 16 bytes.  nheads, nkv >= 1, at most 2^20.
 */
typedef struct {
  int64_t batch, seqlen, nheads, nkv, headdim, rot;
  int64_t q_batch, q_token, k_batch, k_token, oq_batch, oq_token, ok_batch, ok_token;
  int32_t dtype, neighbours;
  float eps;
  int32_t reserved;
  void *workspace;
  size_t workspace_bytes;
} ssm_qk_norm_dims_t;

/*
 * Per token and head of q, with w = wq, and of k, with w = wk:
 *   n = x / sqrt(mean(x^2) + eps) w
 *   (n_a, n_b) of pair i < rot / 2 becomes (n_a cos - n_b sin, n_b cos + n_a sin)
 *   of the angle pos inv_freq_i, which is taken in float64; the others stay.
 *   q, q_out: (batch, seqlen, nheads, headdim);  k, k_out: (batch, seqlen, nkv, headdim)
 *   wq, wk  : (headdim) float32, nullable (ones): shared by all heads
 *   inv_freq: (rot / 2) float32;  pos: (batch, seqlen) int32, nullable (0, 1, ..
 *             in each batch row); neither is used with rot = 0
 * q_out may be exactly q, and k_out exactly k (with the same strides); tensors
 * that lie side by side in one (the same strides, as parts of one projection)
 * do not count as overlapping.  w = headdim^-0.5 makes heads of unit length.
 */
SSM_API int ssm_qk_norm_fwd(const void *q, const void *k, const float *wq, const float *wk, const float *inv_freq,
                            const int32_t *pos, void *q_out, void *k_out, const ssm_qk_norm_dims_t *dims, void *stream);

/*
 * Backward: with d the gradient of an output, rotated back, and m = x rstd,
 *   dw = sum over tokens and heads of d m,   dx = rstd (d w - m mean(d w m))
 *   q, k        : as in the forward, with its other arguments
 *   dq_out, dk_out: the gradients of q_out and k_out, dense
 *   dq, dk      : shaped like q and k, with the output strides
 *   dwq, dwk    : (headdim) float32, both nullable; the workspace is used for
 *                 them only
 */
SSM_API int ssm_qk_norm_bwd_workspace_size(const ssm_qk_norm_dims_t *dims, size_t *bytes);
SSM_API int ssm_qk_norm_bwd(const void *q, const void *k, const float *wq, const float *wk, const float *inv_freq,
                            const int32_t *pos, const void *dq_out, const void *dk_out, void *dq, void *dk, float *dwq,
                            float *dwk, const ssm_qk_norm_dims_t *dims, void *stream);

/* ------------------------------------------------------------------------ */
/* Sliding-window attention over a cache in 8 bits                           */
/* ------------------------------------------------------------------------ */

/*
 * One token per batch row, as ssm_swa_step (whose sizes, ssm_swa_dims_t, and
 * rules these calls share), against a cache that holds most of the window in
 * e4m3 floats (OCP: 4 exponent and 3 mantissa bits, largest 448).  window must
 * be a multiple of 64.  The positions behind the sinks, sinks + 64 n .., form
 * blocks of 64; per batch row and key head the cache has
 *   near : (batch, nkv, sinks + 64, headdim) bfloat16: the sinks, then the
 *          positions of the last block, as they came
 *   ring : (batch, nkv, window, headdim) bytes: block n, once it is whole, at
 *          64 (n mod (window / 64)), each value v as v / scale, rounded to the
 *          nearest even
 *   scale: (batch, nkv, window / 64) float32: max |v| / 448 over a block's 64
 *          positions and headdim elements (0 for a block of zeros; a value
 *          that is not finite makes its block NaN)
 * each of them for keys and for values, 16-byte aligned (scales: 4).  The call
 * stores k and v of position pos near, attends to what ssm_swa_step would
 * (pos's block in bfloat16, the rest of the window as the ring holds it, and
 * the sinks), and, if pos is its block's last, stores that in the ring.
 * Places of positions not yet stored may hold anything.  A position is
 * rounded once, when its block is whole; storing the same position again
 * gives the same cache.
 *   q, y: (batch, nheads, headdim);  k, v: (batch, nkv, headdim) bfloat16
 *   pos : (batch) int32, negative for a row without a token: y = 0 and its
 *         cache stays as it is
 */
SSM_API int ssm_swa_q8_step_workspace_size(const ssm_swa_dims_t *dims, size_t *bytes);
SSM_API int ssm_swa_q8_step(const void *q, const void *k, const void *v, void *k_near, void *v_near, void *k_ring,
                            void *v_ring, float *k_scale, float *v_scale, const int32_t *pos, void *y,
                            const ssm_swa_dims_t *dims, void *stream);

/*
 * Store the keys and values of a prompt into such a cache: of every batch row
 * the positions below its length that a next token would still see.
 *   k, v: (batch, seqlen, nkv, headdim); lengths as ssm_swa_fwd
 * Places that no such position owns keep what they hold.
 */
SSM_API int ssm_swa_q8_fill(const void *k, const void *v, const int32_t *lengths, void *k_near, void *v_near,
                            void *k_ring, void *v_ring, float *k_scale, float *v_scale, const ssm_swa_dims_t *dims,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_DELTA_H */
