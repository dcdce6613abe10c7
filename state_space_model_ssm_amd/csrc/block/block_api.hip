// C ABI of libssm_block (declared in include/ssm_block.h): argument checks,
// workspace sizing and dispatch to the HIP launchers.
//
// Every check runs on the host before any HIP call, so a rejected request
// launches nothing and writes nothing.  Nothing here throws: the last error
// is a fixed buffer per thread.
#include "ssm_block.h"

#include <math.h>

#include "block_check.h"
#include "block_internal.h"
#include "swa_check.h"

using namespace ssmb;

namespace {

// ---------------------------------------------------------------------------
// Gated linear recurrence
// ---------------------------------------------------------------------------

int check_glr(const ssm_glr_dims_t *d) {
  if (!d) return fail(SSM_ERR_NULL, "dims is NULL");
  if (d->batch < 0 || d->seqlen < 0 || d->dim < 0)
    return fail(SSM_ERR_SHAPE, "negative size (batch=%lld seqlen=%lld dim=%lld)", (long long)d->batch,
                (long long)d->seqlen, (long long)d->dim);
  if (!valid_dtype(d->in_dtype) || !valid_dtype(d->out_dtype))
    return fail(SSM_ERR_DTYPE, "in_dtype %d or out_dtype %d is not an ssm_dtype_t", d->in_dtype, d->out_dtype);
  if (d->reserved != 0 || d->reserved2 != 0) return fail(SSM_ERR_SHAPE, "reserved fields must be 0");
  const int64_t tiles = mul(d->batch, ceil_div(d->dim, 32)), n = mul(mul(d->batch, d->dim), d->seqlen);
  const int64_t all = mul(tiles, ceil_div(d->seqlen, 128));
  if (tiles < 0 || n < 0 || mul(n, 4) < 0 || all < 0 || all > kMaxGrid || tiles > kMaxGrid)
    return fail(SSM_ERR_UNSUPPORTED, "batch * ceil(dim / 32) * ceil(seqlen / 128) must be below 2^31");
  if (d->dim > (int64_t{1} << 22)) return fail(SSM_ERR_UNSUPPORTED, "dim must be at most 2^22");
  return SSM_OK;
}

size_t glr_workspace(const ssm_glr_dims_t &d) {
  const size_t chain = ssmb::glr_chain_bytes(d.batch, d.seqlen, d.dim);
  return chain > 0 ? up256(ssmb::kGlrSets * ssmb::kGlrCounterBytes + chain) : 0;
}
size_t glr_bwd_workspace(const ssm_glr_dims_t &d) {  // and the terms of dA
  return glr_workspace(d) + up256(static_cast<size_t>(ssmb::glr_bwd_parts(d.batch, d.seqlen)) * d.dim * 4);
}

// ---------------------------------------------------------------------------
// Residual addition with RMS norm
// ---------------------------------------------------------------------------

int check_rms(const ssm_rms_dims_t *d, bool q8) {
  if (!d) return fail(SSM_ERR_NULL, "dims is NULL");
  if (d->rows < 0 || d->dim < 1)
    return fail(SSM_ERR_SHAPE, "rows must be >= 0 and dim >= 1 (rows=%lld dim=%lld)", (long long)d->rows,
                (long long)d->dim);
  if (!valid_dtype(d->in_dtype) || !valid_dtype(d->out_dtype))
    return fail(SSM_ERR_DTYPE, "in_dtype %d or out_dtype %d is not an ssm_dtype_t", d->in_dtype, d->out_dtype);
  if (d->reserved != 0) return fail(SSM_ERR_SHAPE, "reserved must be 0");
  if (!(d->eps >= 0.0f) || isinf(d->eps)) return fail(SSM_ERR_SHAPE, "eps must be finite and >= 0");
  if (q8 ? (d->group < 0 || d->group % 32 != 0) : d->group != 0)
    return fail(SSM_ERR_SHAPE, q8 ? "group must be 0 or a multiple of 32 (got %lld)" : "group must be 0 here (got %lld)",
                (long long)d->group);
  if (d->rows > kMaxGrid || mul(mul(d->rows, d->dim), 4) < 0)
    return fail(SSM_ERR_UNSUPPORTED, "rows must be below 2^31");
  return SSM_OK;
}

size_t rms_bwd_workspace(const ssm_rms_dims_t &d) {
  return up256(static_cast<size_t>(ssmb::rms_bwd_parts(d.rows, d.dim)) * d.dim * 4);
}

int rms_fwd_run(const void *x, const void *residual, const float *w, void *y, float *scale, void *residual_out,
                bool q8, const ssm_rms_dims_t *dims, void *stream) {
  int rc = check_rms(dims, q8);
  if (rc != SSM_OK) return rc;
  const ssm_rms_dims_t &d = *dims;
  const size_t n = static_cast<size_t>(d.rows) * d.dim, ei = dtype_size(d.in_dtype);
  const size_t eo = q8 ? 1 : dtype_size(d.out_dtype);
  const int64_t group = d.group > 0 && d.group < d.dim ? d.group : d.dim;
  const Arg ins[] = {{"x", x, n * ei, ei, true},
                     {"residual", residual, n * ei, ei, false},
                     {"w", w, static_cast<size_t>(d.rows > 0 ? d.dim : 0) * 4, 4, true}};
  const Arg outs[] = {{q8 ? "q" : "y", y, n * eo, eo, true},
                      {"scale", scale, q8 ? static_cast<size_t>(d.rows) * ceil_div(d.dim, group) * 4 : 0, 4, q8},
                      {"residual_out", residual_out, n * ei, ei, false}};
  const void *const same[3][2] = {{!q8 && ei == eo ? x : nullptr, nullptr}, {nullptr, nullptr}, {x, residual}};
  rc = check_args(ins, outs, same);
  if (rc != SSM_OK) return rc;
  if (d.rows == 0) return ok();
  ssmb::RmsParams p{};
  p.x = x;
  p.residual = residual;
  p.w = w;
  p.y = y;
  p.scale = q8 ? scale : nullptr;
  p.residual_out = residual_out;
  p.eps = d.eps;
  p.rows = d.rows;
  p.dim = d.dim;
  p.group = group;
  return launched(ssmb::launch_rms(p, d.in_dtype == SSM_BF16, d.out_dtype == SSM_BF16, static_cast<hipStream_t>(stream)),
                  "rms_add");
}

// ---------------------------------------------------------------------------
// Sliding-window attention
// ---------------------------------------------------------------------------

ssmb::SwaParams swa_params(const ssm_swa_dims_t &d, const void *q, const void *k, const void *v,
                           const int32_t *lengths) {
  ssmb::SwaParams p{};
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.lengths = lengths;
  p.batch = d.batch;
  p.seqlen = d.seqlen;
  p.nheads = d.nheads;
  p.nkv = d.nkv;
  // A window or sinks past the sequence's end see what its length does.
  p.window = d.window < d.seqlen ? d.window : (d.seqlen > 0 ? d.seqlen : 1);
  p.sinks = d.sinks < d.seqlen ? d.sinks : d.seqlen;
  p.q_batch = d.q_batch;
  p.q_token = d.q_token;
  p.k_batch = d.k_batch;
  p.k_token = d.k_token;
  p.v_batch = d.v_batch;
  p.v_token = d.v_token;
  p.scale = d.scale;
  p.headdim = static_cast<int32_t>(d.headdim);
  return p;
}

ssmb::SwaBwdPlan swa_plan(const ssm_swa_dims_t &d) {
  return ssmb::swa_bwd_plan(d.batch, d.seqlen, d.nheads, d.nkv, d.headdim, d.window, d.sinks);
}

int check_swa_bwd(const ssm_swa_dims_t *d) {
  const int rc = check_swa(d, false);
  if (rc != SSM_OK) return rc;
  const ssmb::SwaBwdPlan plan = swa_plan(*d);
  const int64_t heads = d->batch * d->nkv, sums = int64_t{plan.sum_blocks} * 4 * (d->headdim / 32);
  if (plan.items * heads > ssmb::kMaxGroups || sums * heads > ssmb::kMaxGroups)
    return fail(SSM_ERR_UNSUPPORTED, "batch * nkv * sinks is too large for the backward");
  return SSM_OK;
}

// log2(e) lse and dy.y of every query, then the terms of dk and dv.
size_t swa_bwd_stats(const ssm_swa_dims_t &d) { return up256(static_cast<size_t>(d.batch) * d.nheads * d.seqlen * 4); }
size_t swa_bwd_terms(const ssm_swa_dims_t &d) {
  const ssmb::SwaBwdPlan plan = swa_plan(d);
  return up256(static_cast<size_t>(d.batch) * d.nkv * plan.sum_blocks * plan.slices * 2 * 128 * d.headdim * 4);
}
size_t swa_bwd_workspace(const ssm_swa_dims_t &d) {
  const ssmb::SwaBwdPlan plan = swa_plan(d);
  const size_t far = static_cast<size_t>(d.batch) * d.nkv * plan.far_blocks * plan.far_chunks * 2 * 32 * d.headdim * 4;
  return 2 * swa_bwd_stats(d) + swa_bwd_terms(d) + up256(far);
}

int swa_splits(const ssm_swa_dims_t &d) { return ssmb::swa_step_splits(d.batch, d.nheads, d.nkv, d.sinks + d.window); }

// Per (row, head, split): the sum of values, then the maximum and sum of weights.
size_t swa_step_sums(const ssm_swa_dims_t &d) {
  return up256(static_cast<size_t>(d.batch) * d.nheads * swa_splits(d) * d.headdim * 4);
}
size_t swa_step_workspace(const ssm_swa_dims_t &d) {
  const size_t rows = static_cast<size_t>(d.batch) * d.nheads * swa_splits(d);
  return swa_splits(d) > 1 ? swa_step_sums(d) + up256(rows * 8) : 0;
}

}  // namespace

extern "C" {

const char *ssm_block_last_error(void) { return ssmb::g_last_error; }

int ssm_glr_workspace_size(const ssm_glr_dims_t *dims, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_NULL, "bytes is NULL");
  const int rc = check_glr(dims);
  if (rc != SSM_OK) return rc;
  *bytes = glr_workspace(*dims);
  return ok();
}

int ssm_glr_fwd(const void *x, const void *rec, const void *inp, const float *A, const float *h0,
                const uint8_t *reset, void *y, float *h_last, float *states, const ssm_glr_dims_t *dims,
                void *stream) {
  int rc = check_glr(dims);
  if (rc != SSM_OK) return rc;
  const ssm_glr_dims_t &d = *dims;
  const size_t bd = static_cast<size_t>(d.batch) * d.dim, n = bd * d.seqlen;
  const size_t ei = dtype_size(d.in_dtype), eo = dtype_size(d.out_dtype);
  const Arg ins[] = {{"x", x, n * ei, ei, true},
                     {"rec", rec, n * ei, ei, true},
                     {"inp", inp, n * ei, ei, true},
                     {"A", A, bd > 0 ? d.dim * size_t{4} : 0, 4, true},
                     {"h0", h0, bd * 4, 4, false},
                     {"reset", reset, bd > 0 ? static_cast<size_t>(d.batch) * d.seqlen : 0, 1, false},
                     {"workspace", d.workspace, d.workspace ? d.workspace_bytes : 0, 1, false}};
  const Arg outs[] = {{"y", y, n * eo, eo, true},
                      {"h_last", h_last, bd * 4, 4, false},
                      {"states", states, bd * ceil_div(d.seqlen, SSM_GLR_STATE_STEP) * 4, 4, false}};
  const void *const same[3][2] = {{nullptr, nullptr}, {h0, nullptr}, {nullptr, nullptr}};
  rc = check_args(ins, outs, same);
  if (rc == SSM_OK) rc = check_workspace(ins, glr_workspace(d));
  if (rc != SSM_OK) return rc;
  if (bd == 0 || (d.seqlen == 0 && h_last == nullptr)) return ok();
  ssmb::GlrParams p{};
  p.x = x;
  p.rec = rec;
  p.inp = inp;
  p.A = A;
  p.h0 = h0;
  p.reset = reset;
  p.y = y;
  p.h_last = h_last;
  p.states = states;
  p.batch = d.batch;
  p.seqlen = d.seqlen;
  p.dim = d.dim;
  p.chain = ssmb::glr_chain(d.workspace, d.batch, d.seqlen, d.dim);
  return launched(ssmb::launch_glr(p, d.in_dtype == SSM_BF16, d.out_dtype == SSM_BF16, static_cast<hipStream_t>(stream)),
                  "glr_fwd");
}

int ssm_glr_step(const void *x, const void *rec, const void *inp, const float *A, const float *h, void *y,
                 float *h_out, const ssm_glr_dims_t *dims, void *stream) {
  int rc = check_glr(dims);
  if (rc != SSM_OK) return rc;
  const ssm_glr_dims_t &d = *dims;
  if (d.seqlen != 1) return fail(SSM_ERR_SHAPE, "seqlen must be 1 in a step (got %lld)", (long long)d.seqlen);
  const size_t n = static_cast<size_t>(d.batch) * d.dim;
  const size_t ei = dtype_size(d.in_dtype), eo = dtype_size(d.out_dtype);
  const Arg ins[] = {{"x", x, n * ei, ei, true},
                     {"rec", rec, n * ei, ei, true},
                     {"inp", inp, n * ei, ei, true},
                     {"A", A, n > 0 ? d.dim * size_t{4} : 0, 4, true},
                     {"h", h, n * 4, 4, true}};
  const Arg outs[] = {{"y", y, n * eo, eo, true}, {"h_out", h_out, n * 4, 4, true}};
  const void *const same[2][2] = {{nullptr, nullptr}, {h, nullptr}};
  rc = check_args(ins, outs, same);
  if (rc != SSM_OK) return rc;
  if (n == 0) return ok();
  ssmb::GlrParams p{};
  p.x = x;
  p.rec = rec;
  p.inp = inp;
  p.A = A;
  p.h0 = h;
  p.y = y;
  p.h_last = h_out;
  p.batch = d.batch;
  p.seqlen = 1;
  p.dim = d.dim;
  return launched(
      ssmb::launch_glr_step(p, d.in_dtype == SSM_BF16, d.out_dtype == SSM_BF16, static_cast<hipStream_t>(stream)),
      "glr_step");
}

int ssm_glr_bwd_workspace_size(const ssm_glr_dims_t *dims, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_NULL, "bytes is NULL");
  const int rc = check_glr(dims);
  if (rc != SSM_OK) return rc;
  *bytes = glr_bwd_workspace(*dims);
  return ok();
}

int ssm_glr_bwd(const void *x, const void *rec, const void *inp, const float *A, const uint8_t *reset,
                const float *states, const void *dy, const float *dh_last, void *dx, void *drec, void *dinp,
                float *dA, float *dh0, const ssm_glr_dims_t *dims, void *stream) {
  int rc = check_glr(dims);
  if (rc != SSM_OK) return rc;
  const ssm_glr_dims_t &d = *dims;
  const size_t bd = static_cast<size_t>(d.batch) * d.dim, n = bd * d.seqlen, ei = dtype_size(d.in_dtype);
  const size_t need = glr_bwd_workspace(d);
  const Arg ins[] = {{"x", x, n * ei, ei, true},
                     {"rec", rec, n * ei, ei, true},
                     {"inp", inp, n * ei, ei, true},
                     {"dy", dy, n * ei, ei, true},
                     {"A", A, bd > 0 ? d.dim * size_t{4} : 0, 4, true},
                     {"reset", reset, bd > 0 ? static_cast<size_t>(d.batch) * d.seqlen : 0, 1, false},
                     {"states", states, bd * ceil_div(d.seqlen, SSM_GLR_STATE_STEP) * 4, 4, true},
                     {"dh_last", dh_last, bd * 4, 4, false},
                     {"workspace", d.workspace, d.workspace ? d.workspace_bytes : 0, 1, false}};
  const Arg outs[] = {{"dx", dx, n * ei, ei, true},
                      {"drec", drec, n * ei, ei, true},
                      {"dinp", dinp, n * ei, ei, true},
                      {"dA", dA, d.dim * size_t{4}, 4, true},
                      {"dh0", dh0, bd * 4, 4, false}};
  const void *const same[5][2] = {};
  rc = check_args(ins, outs, same);
  if (rc == SSM_OK) rc = check_workspace(ins, need);
  if (rc != SSM_OK) return rc;
  if (d.dim == 0) return ok();
  ssmb::GlrBwdParams p{};
  p.x = x;
  p.rec = rec;
  p.inp = inp;
  p.dy = dy;
  p.A = A;
  p.states = states;
  p.dh_last = dh_last;
  p.reset = reset;
  p.dx = dx;
  p.drec = drec;
  p.dinp = dinp;
  p.dA = dA;
  p.dh0 = dh0;
  p.chain = ssmb::glr_chain(d.workspace, d.batch, d.seqlen, d.dim);
  p.ws_dA = reinterpret_cast<float *>(static_cast<char *>(d.workspace) + glr_workspace(d));
  p.batch = d.batch;
  p.seqlen = d.seqlen;
  p.dim = d.dim;
  return launched(ssmb::launch_glr_bwd(p, d.in_dtype == SSM_BF16, static_cast<hipStream_t>(stream)), "glr_bwd");
}

int ssm_rms_add_fwd(const void *x, const void *residual, const float *w, void *y, void *residual_out,
                    const ssm_rms_dims_t *dims, void *stream) {
  return rms_fwd_run(x, residual, w, y, nullptr, residual_out, false, dims, stream);
}

int ssm_rms_add_q8_fwd(const void *x, const void *residual, const float *w, void *q, float *scale,
                       void *residual_out, const ssm_rms_dims_t *dims, void *stream) {
  return rms_fwd_run(x, residual, w, q, scale, residual_out, true, dims, stream);
}

int ssm_rms_add_bwd_workspace_size(const ssm_rms_dims_t *dims, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_NULL, "bytes is NULL");
  const int rc = check_rms(dims, false);
  if (rc != SSM_OK) return rc;
  *bytes = rms_bwd_workspace(*dims);
  return ok();
}

int ssm_rms_add_bwd(const void *dy, const void *s, const float *w, const void *dres, void *dx, float *dw,
                    const ssm_rms_dims_t *dims, void *stream) {
  int rc = check_rms(dims, false);
  if (rc != SSM_OK) return rc;
  const ssm_rms_dims_t &d = *dims;
  const size_t n = static_cast<size_t>(d.rows) * d.dim, ei = dtype_size(d.in_dtype);
  const Arg ins[] = {{"dy", dy, n * ei, ei, true},
                     {"s", s, n * ei, ei, true},
                     {"w", w, static_cast<size_t>(d.rows > 0 ? d.dim : 0) * 4, 4, true},
                     {"dres", dres, n * ei, ei, false},
                     {"workspace", d.workspace, d.workspace ? d.workspace_bytes : 0, 1, false}};
  const Arg outs[] = {{"dx", dx, n * ei, ei, true}, {"dw", dw, static_cast<size_t>(d.dim) * 4, 4, false}};
  const void *const same[2][2] = {{dy, dres}, {nullptr, nullptr}};
  rc = check_args(ins, outs, same);
  if (rc == SSM_OK && dw != nullptr) rc = check_workspace(ins, rms_bwd_workspace(d));
  if (rc != SSM_OK) return rc;
  if (d.rows == 0 && dw == nullptr) return ok();
  ssmb::RmsBwdParams p{};
  p.dy = dy;
  p.s = s;
  p.dres = dres;
  p.w = w;
  p.dx = dx;
  p.dw = dw;
  p.ws = static_cast<float *>(d.workspace);
  p.eps = d.eps;
  p.rows = d.rows;
  p.dim = d.dim;
  p.parts = ssmb::rms_bwd_parts(d.rows, d.dim);
  return launched(ssmb::launch_rms_bwd(p, d.in_dtype == SSM_BF16, static_cast<hipStream_t>(stream)), "rms_add_bwd");
}

int ssm_swa_fwd(const void *q, const void *k, const void *v, const int32_t *lengths, void *y, float *lse,
                const ssm_swa_dims_t *dims, void *stream) {
  int rc = check_swa(dims, false);
  if (rc != SSM_OK) return rc;
  const ssm_swa_dims_t &d = *dims;
  const size_t rows = static_cast<size_t>(d.batch) * d.seqlen;
  const Arg ins[] = {{"q", q, span(d, d.q_batch, d.q_token, d.nheads), 16, true},
                     {"k", k, span(d, d.k_batch, d.k_token, d.nkv), 16, true},
                     {"v", v, span(d, d.v_batch, d.v_token, d.nkv), 16, true},
                     {"lengths", lengths, static_cast<size_t>(d.batch) * 4, 4, false}};
  const Arg outs[] = {{"y", y, rows * d.nheads * d.headdim * 2, 16, true}, {"lse", lse, rows * d.nheads * 4, 4, false}};
  const void *const same[2][2] = {};
  rc = check_args(ins, outs, same);
  if (rc != SSM_OK) return rc;
  if (rows == 0) return ok();
  ssmb::SwaParams p = swa_params(d, q, k, v, lengths);
  p.y = static_cast<uint16_t *>(y);
  p.lse = lse;
  return launched(ssmb::launch_swa_fwd(p, static_cast<hipStream_t>(stream)), "swa_fwd");
}

int ssm_swa_bwd_workspace_size(const ssm_swa_dims_t *dims, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_NULL, "bytes is NULL");
  const int rc = check_swa_bwd(dims);
  if (rc != SSM_OK) return rc;
  *bytes = swa_bwd_workspace(*dims);
  return ok();
}

int ssm_swa_bwd(const void *q, const void *k, const void *v, const int32_t *lengths, const void *y, const float *lse,
                const void *dy, void *dq, void *dk, void *dv, const ssm_swa_dims_t *dims, void *stream) {
  int rc = check_swa_bwd(dims);
  if (rc != SSM_OK) return rc;
  const ssm_swa_dims_t &d = *dims;
  const size_t rows = static_cast<size_t>(d.batch) * d.seqlen;
  const size_t nq = rows * d.nheads * d.headdim * 2, nk = rows * d.nkv * d.headdim * 2;
  const Arg ins[] = {{"q", q, span(d, d.q_batch, d.q_token, d.nheads), 16, true},
                     {"k", k, span(d, d.k_batch, d.k_token, d.nkv), 16, true},
                     {"v", v, span(d, d.v_batch, d.v_token, d.nkv), 16, true},
                     {"lengths", lengths, static_cast<size_t>(d.batch) * 4, 4, false},
                     {"y", y, nq, 16, true},
                     {"lse", lse, rows * d.nheads * 4, 4, true},
                     {"dy", dy, nq, 16, true},
                     {"workspace", d.workspace, d.workspace ? d.workspace_bytes : 0, 1, false}};
  const Arg outs[] = {{"dq", dq, nq, 16, true}, {"dk", dk, nk, 16, true}, {"dv", dv, nk, 16, true}};
  const void *const same[3][2] = {};
  rc = check_args(ins, outs, same);
  if (rc == SSM_OK) rc = check_workspace(ins, swa_bwd_workspace(d));
  if (rc != SSM_OK) return rc;
  if (rows == 0) return ok();
  ssmb::SwaParams p = swa_params(d, q, k, v, lengths);
  p.y = static_cast<uint16_t *>(const_cast<void *>(y));
  p.lse = const_cast<float *>(lse);
  p.dy = static_cast<const uint16_t *>(dy);
  p.dq = static_cast<uint16_t *>(dq);
  p.dk = static_cast<uint16_t *>(dk);
  p.dv = static_cast<uint16_t *>(dv);
  char *ws = static_cast<char *>(d.workspace);
  p.ws_lse2 = reinterpret_cast<float *>(ws);
  p.ws_delta = reinterpret_cast<float *>(ws + swa_bwd_stats(d));
  p.ws_part = reinterpret_cast<float *>(ws + 2 * swa_bwd_stats(d));
  p.ws_far = reinterpret_cast<float *>(ws + 2 * swa_bwd_stats(d) + swa_bwd_terms(d));
  return launched(ssmb::launch_swa_bwd(p, swa_plan(d), static_cast<hipStream_t>(stream)), "swa_bwd");
}

int ssm_swa_step_workspace_size(const ssm_swa_dims_t *dims, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_NULL, "bytes is NULL");
  const int rc = check_swa(dims, true);
  if (rc != SSM_OK) return rc;
  *bytes = swa_step_workspace(*dims);
  return ok();
}

int ssm_swa_step(const void *q, const void *k, const void *v, void *k_cache, void *v_cache, const int32_t *pos,
                 void *y, const ssm_swa_dims_t *dims, void *stream) {
  int rc = check_swa(dims, true);
  if (rc != SSM_OK) return rc;
  const ssm_swa_dims_t &d = *dims;
  if (d.sinks + d.window > (int64_t{1} << 30))
    return fail(SSM_ERR_UNSUPPORTED, "sinks + window must be at most 2^30");
  const size_t cache = static_cast<size_t>(d.batch) * d.nkv * (d.sinks + d.window) * d.headdim * 2;
  const Arg ins[] = {{"q", q, span(d, d.q_batch, d.q_token, d.nheads), 16, true},
                     {"k", k, span(d, d.k_batch, d.k_token, d.nkv), 16, true},
                     {"v", v, span(d, d.v_batch, d.v_token, d.nkv), 16, true},
                     {"pos", pos, static_cast<size_t>(d.batch) * 4, 4, true},
                     {"workspace", d.workspace, d.workspace ? d.workspace_bytes : 0, 1, false}};
  const Arg outs[] = {{"k_cache", k_cache, cache, 16, true},
                      {"v_cache", v_cache, cache, 16, true},
                      {"y", y, static_cast<size_t>(d.batch) * d.nheads * d.headdim * 2, 16, true}};
  const void *const same[3][2] = {};
  rc = check_args(ins, outs, same);
  if (rc == SSM_OK) rc = check_workspace(ins, swa_step_workspace(d));
  if (rc != SSM_OK) return rc;
  if (d.batch == 0) return ok();
  ssmb::SwaStepParams p{};
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.k_cache = static_cast<uint16_t *>(k_cache);
  p.v_cache = static_cast<uint16_t *>(v_cache);
  p.pos = pos;
  p.y = static_cast<uint16_t *>(y);
  p.batch = d.batch;
  p.nheads = d.nheads;
  p.nkv = d.nkv;
  p.window = d.window;
  p.sinks = d.sinks;
  p.q_batch = d.q_batch;
  p.k_batch = d.k_batch;
  p.v_batch = d.v_batch;
  p.scale = d.scale;
  p.headdim = static_cast<int32_t>(d.headdim);
  p.ws_o = static_cast<float *>(d.workspace);
  if (d.workspace) p.ws_stat = reinterpret_cast<float *>(static_cast<char *>(d.workspace) + swa_step_sums(d));
  return launched(ssmb::launch_swa_step(p, swa_splits(d), static_cast<hipStream_t>(stream)), "swa_step");
}

int ssm_swa_fill(const void *k, const void *v, const int32_t *lengths, void *k_cache, void *v_cache,
                 const ssm_swa_dims_t *dims, void *stream) {
  int rc = check_swa(dims, false);
  if (rc != SSM_OK) return rc;
  const ssm_swa_dims_t &d = *dims;
  if (d.sinks + d.window > (int64_t{1} << 30))
    return fail(SSM_ERR_UNSUPPORTED, "sinks + window must be at most 2^30");
  const size_t cache = static_cast<size_t>(d.batch) * d.nkv * (d.sinks + d.window) * d.headdim * 2;
  const Arg ins[] = {{"k", k, span(d, d.k_batch, d.k_token, d.nkv), 16, true},
                     {"v", v, span(d, d.v_batch, d.v_token, d.nkv), 16, true},
                     {"lengths", lengths, static_cast<size_t>(d.batch) * 4, 4, false}};
  const Arg outs[] = {{"k_cache", k_cache, cache, 16, true}, {"v_cache", v_cache, cache, 16, true}};
  const void *const same[2][2] = {};
  rc = check_args(ins, outs, same);
  if (rc != SSM_OK) return rc;
  if (d.batch == 0 || d.seqlen == 0) return ok();
  ssmb::SwaParams p = swa_params(d, nullptr, k, v, lengths);
  p.window = d.window;
  p.sinks = d.sinks;
  return launched(ssmb::launch_swa_fill(p, static_cast<uint16_t *>(k_cache), static_cast<uint16_t *>(v_cache),
                                        static_cast<hipStream_t>(stream)),
                  "swa_fill");
}

}  // extern "C"
