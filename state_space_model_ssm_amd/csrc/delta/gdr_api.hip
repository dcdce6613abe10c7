// C ABI of the gated delta rule (declared in include/ssm_delta.h): argument
// checks, workspace sizing and dispatch.
#include "ssm_delta.h"

#include <math.h>

#include "block/block_check.h"
#include "gdr_internal.h"

using namespace ssmb;

namespace {

int check_gdr(const ssm_gdr_dims_t *d, bool step) {
  if (!d) return fail(SSM_ERR_NULL, "dims is NULL");
  if (d->batch < 0 || d->seqlen < 0)
    return fail(SSM_ERR_SHAPE, "negative size (batch=%lld seqlen=%lld)", (long long)d->batch, (long long)d->seqlen);
  if (step && d->seqlen != 1) return fail(SSM_ERR_SHAPE, "seqlen must be 1 in a step (got %lld)", (long long)d->seqlen);
  if (d->nheads < 1 || d->nqk < 1 || d->nheads % d->nqk != 0)
    return fail(SSM_ERR_SHAPE, "nqk (%lld) must divide nheads (%lld)", (long long)d->nqk, (long long)d->nheads);
  if ((d->kdim != 64 && d->kdim != 128) || (d->vdim != 64 && d->vdim != 128))
    return fail(SSM_ERR_UNSUPPORTED, "kdim %lld or vdim %lld not supported (64 or 128 each)", (long long)d->kdim,
                (long long)d->vdim);
  if (!valid_dtype(d->gate_dtype)) return fail(SSM_ERR_DTYPE, "gate_dtype %d is not an ssm_dtype_t", d->gate_dtype);
  if (!isfinite(d->scale)) return fail(SSM_ERR_SHAPE, "scale must be finite");
  if (d->seqlen > (int64_t{1} << 30)) return fail(SSM_ERR_UNSUPPORTED, "seqlen must be at most 2^30");
  const int64_t chunks = ceil_div(d->seqlen, SSM_GDR_STATE_STEP), heads = mul(d->batch, d->nheads);
  const int64_t all = mul(heads, chunks > 4 ? chunks : 4);  // a workgroup per chunk, and per 32 values
  if (d->nheads > kMaxGroups || heads < 0 || all < 0 || all > kMaxGroups)
    return fail(SSM_ERR_UNSUPPORTED, "batch * nheads * max(4, ceil(seqlen / 64)) must be below 2^24");
  const int64_t strides[] = {d->q_batch, d->q_token, d->k_batch, d->k_token, d->v_batch, d->v_token};
  for (const int64_t s : strides)
    if (s < 0 || s % 8 != 0 || s > (int64_t{1} << 40))
      return fail(SSM_ERR_SHAPE, "strides must be multiples of 8 elements, not negative (got %lld)", (long long)s);
  if (d->q_token > kMaxToken || d->k_token > kMaxToken || d->v_token > kMaxToken)
    return fail(SSM_ERR_UNSUPPORTED, "token strides must be at most 2^24 elements");
  // (Outputs are dense, and a block's 64 tokens are addressed in 32 bits.)
  const int64_t nk = d->nqk * d->kdim, nv = d->nheads * d->vdim;
  if (nk > kMaxToken || nv > kMaxToken)
    return fail(SSM_ERR_UNSUPPORTED, "nqk * kdim and nheads * vdim must be at most 2^24");
  if (d->seqlen > 1 && (d->q_token < nk || d->k_token < nk || d->v_token < nv))
    return fail(SSM_ERR_SHAPE, "a token stride is smaller than the token");
  if (d->batch > 1 && (d->q_batch < nk || d->k_batch < nk || d->v_batch < nv))
    return fail(SSM_ERR_SHAPE, "a batch stride is smaller than a token");
  return SSM_OK;
}

// Bytes that a strided (batch, seqlen, heads, dim) tensor spans.
size_t span(const ssm_gdr_dims_t &d, int64_t batch_stride, int64_t token_stride, int64_t token) {
  if (d.batch == 0 || d.seqlen == 0) return 0;
  return static_cast<size_t>((d.batch - 1) * batch_stride + (d.seqlen - 1) * token_stride + token) * 2;
}

size_t saved_bytes(const ssm_gdr_dims_t &d) {
  return static_cast<size_t>(d.batch) * d.nheads * ceil_div(d.seqlen, SSM_GDR_STATE_STEP) * gdr_saved_bytes(d.kdim, d.vdim);
}

GdrParams params(const ssm_gdr_dims_t &d, bool bwd = false) {
  GdrParams p{};
  p.ws = static_cast<char *>(d.workspace);
  p.batch = d.batch;
  p.seqlen = d.seqlen;
  p.nqk = d.nqk;
  p.nheads = d.nheads;
  p.chunks = ceil_div(d.seqlen, SSM_GDR_STATE_STEP);
  p.q_batch = d.q_batch;
  p.q_token = d.q_token;
  p.k_batch = d.k_batch;
  p.k_token = d.k_token;
  p.v_batch = d.v_batch;
  p.v_token = d.v_token;
  p.scale = d.scale;
  p.kdim = static_cast<int32_t>(d.kdim);
  p.vdim = static_cast<int32_t>(d.vdim);
  p.gates_bf16 = d.gate_dtype == SSM_BF16;
  p.seg = bwd ? gdr_bwd_segments(d.batch * d.nheads, d.kdim, d.vdim, p.chunks)
              : gdr_segments(d.batch * d.nheads, d.kdim, d.vdim, p.chunks);
  return p;
}

}  // namespace

extern "C" {

const char *ssm_delta_last_error(void) { return g_last_error; }

int ssm_gdr_workspace_size(const ssm_gdr_dims_t *dims, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_NULL, "bytes is NULL");
  const int rc = check_gdr(dims, false);
  if (rc != SSM_OK) return rc;
  const GdrSizes n = gdr_sizes(params(*dims));
  *bytes = n.all();
  return ok();
}

int ssm_gdr_states_size(const ssm_gdr_dims_t *dims, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_NULL, "bytes is NULL");
  const int rc = check_gdr(dims, false);
  if (rc != SSM_OK) return rc;
  *bytes = saved_bytes(*dims);
  return ok();
}

int ssm_gdr_fwd(const void *q, const void *k, const void *v, const void *g, const void *beta, const float *h0,
                const int32_t *lengths, void *y, float *h_last, void *states, const ssm_gdr_dims_t *dims,
                void *stream) {
  int rc = check_gdr(dims, false);
  if (rc != SSM_OK) return rc;
  const ssm_gdr_dims_t &d = *dims;
  GdrParams p = params(d);
  const size_t eg = dtype_size(d.gate_dtype), rows = static_cast<size_t>(d.batch) * d.seqlen;
  const size_t state = static_cast<size_t>(d.batch) * d.nheads * d.vdim * d.kdim * 4;
  const Arg ins[] = {{"q", q, span(d, d.q_batch, d.q_token, d.nqk * d.kdim), 16, true},
                     {"k", k, span(d, d.k_batch, d.k_token, d.nqk * d.kdim), 16, true},
                     {"v", v, span(d, d.v_batch, d.v_token, d.nheads * d.vdim), 16, true},
                     {"g", g, rows * d.nheads * eg, eg, true},
                     {"beta", beta, rows * d.nheads * eg, eg, true},
                     {"h0", h0, state, 16, false},
                     {"lengths", lengths, static_cast<size_t>(d.batch) * 4, 4, false},
                     {"workspace", d.workspace, d.workspace ? d.workspace_bytes : 0, 1, false}};
  const Arg outs[] = {{"y", y, rows * d.nheads * d.vdim * 2, 16, true},
                      {"h_last", h_last, state, 16, false},
                      {"states", states, saved_bytes(d), 16, false}};
  const void *const same[3][2] = {{nullptr, nullptr}, {h0, nullptr}, {nullptr, nullptr}};
  rc = check_args(ins, outs, same);
  const GdrSizes n = gdr_sizes(p);
  if (rc == SSM_OK) rc = check_workspace(ins, n.all());
  if (rc != SSM_OK) return rc;
  if (d.batch == 0 || (d.seqlen == 0 && h_last == nullptr)) return ok();
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.g = g;
  p.beta = beta;
  p.h0 = h0;
  p.lengths = lengths;
  p.y = static_cast<uint16_t *>(y);
  p.h_last = h_last;
  p.saved = static_cast<char *>(states);
  p.ops = states ? p.saved + gdr_both_bytes(d.kdim, d.vdim) : p.ws;
  p.ops_step = static_cast<int64_t>(states ? gdr_saved_bytes(d.kdim, d.vdim) : kGdrChunkBytes);
  p.rest = h_last != nullptr || p.seg.count > 1 ? p.ws + n.chunks : nullptr;
  p.ws_state = reinterpret_cast<float *>(p.ws + n.chunks + n.rest);
  p.ws_carry = reinterpret_cast<uint16_t *>(p.ws + n.chunks + n.rest + n.state);
  return launched(launch_gdr_fwd(p, static_cast<hipStream_t>(stream)), "gdr_fwd");
}

int ssm_gdr_bwd_workspace_size(const ssm_gdr_dims_t *dims, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_NULL, "bytes is NULL");
  const int rc = check_gdr(dims, false);
  if (rc != SSM_OK) return rc;
  const GdrSizes n = gdr_bwd_sizes(params(*dims, true));
  *bytes = n.all();
  return ok();
}

int ssm_gdr_bwd(const void *q, const void *k, const int32_t *lengths, const void *states, const void *dy,
                const float *dh_last, void *dq, void *dk, void *dv, void *dg, void *dbeta, float *dh0,
                const ssm_gdr_dims_t *dims, void *stream) {
  int rc = check_gdr(dims, false);
  if (rc != SSM_OK) return rc;
  const ssm_gdr_dims_t &d = *dims;
  GdrParams p = params(d, true);
  const size_t eg = dtype_size(d.gate_dtype), rows = static_cast<size_t>(d.batch) * d.seqlen;
  const size_t state = static_cast<size_t>(d.batch) * d.nheads * d.vdim * d.kdim * 4;
  const Arg ins[] = {{"q", q, span(d, d.q_batch, d.q_token, d.nqk * d.kdim), 16, true},
                     {"k", k, span(d, d.k_batch, d.k_token, d.nqk * d.kdim), 16, true},
                     {"lengths", lengths, static_cast<size_t>(d.batch) * 4, 4, false},
                     {"states", states, saved_bytes(d), 16, true},
                     {"dy", dy, rows * d.nheads * d.vdim * 2, 16, true},
                     {"dh_last", dh_last, state, 16, false},
                     {"workspace", d.workspace, d.workspace ? d.workspace_bytes : 0, 1, false}};
  const Arg outs[] = {{"dq", dq, rows * d.nqk * d.kdim * 2, 16, true},   {"dk", dk, rows * d.nqk * d.kdim * 2, 16, true},
                      {"dv", dv, rows * d.nheads * d.vdim * 2, 16, true}, {"dg", dg, rows * d.nheads * eg, eg, true},
                      {"dbeta", dbeta, rows * d.nheads * eg, eg, true},  {"dh0", dh0, state, 16, false}};
  const void *const same[6][2] = {};
  rc = check_args(ins, outs, same);
  const GdrSizes n = gdr_bwd_sizes(p);
  if (rc == SSM_OK) rc = check_workspace(ins, n.all());
  if (rc != SSM_OK) return rc;
  if (d.batch == 0 || (d.seqlen == 0 && dh0 == nullptr)) return ok();
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.lengths = lengths;
  p.saved = static_cast<char *>(const_cast<void *>(states));
  p.dy = static_cast<const uint16_t *>(dy);
  p.dh_last = dh_last;
  p.dq = static_cast<uint16_t *>(dq);
  p.dk = static_cast<uint16_t *>(dk);
  p.dv = static_cast<uint16_t *>(dv);
  p.dg = dg;
  p.dbeta = dbeta;
  p.dh0 = dh0;
  p.ws_both = p.ws;
  p.ops = p.saved + gdr_both_bytes(d.kdim, d.vdim);
  p.ops_step = static_cast<int64_t>(gdr_saved_bytes(d.kdim, d.vdim));
  p.ws_state = reinterpret_cast<float *>(p.ws + n.chunks + n.rest);
  p.ws_carry = reinterpret_cast<uint16_t *>(p.ws + n.chunks + n.rest + n.state);
  return launched(launch_gdr_bwd(p, static_cast<hipStream_t>(stream)), "gdr_bwd");
}

int ssm_gdr_step(const void *q, const void *k, const void *v, const void *g, const void *beta, const float *h, void *y,
                 float *h_out, const ssm_gdr_dims_t *dims, void *stream) {
  int rc = check_gdr(dims, true);
  if (rc != SSM_OK) return rc;
  const ssm_gdr_dims_t &d = *dims;
  const size_t eg = dtype_size(d.gate_dtype), heads = static_cast<size_t>(d.batch) * d.nheads;
  const Arg ins[] = {{"q", q, span(d, d.q_batch, d.q_token, d.nqk * d.kdim), 16, true},
                     {"k", k, span(d, d.k_batch, d.k_token, d.nqk * d.kdim), 16, true},
                     {"v", v, span(d, d.v_batch, d.v_token, d.nheads * d.vdim), 16, true},
                     {"g", g, heads * eg, eg, true},
                     {"beta", beta, heads * eg, eg, true},
                     {"h", h, heads * d.vdim * d.kdim * 4, 16, true}};
  const Arg outs[] = {{"y", y, heads * d.vdim * 2, 16, true}, {"h_out", h_out, heads * d.vdim * d.kdim * 4, 16, true}};
  const void *const same[2][2] = {{nullptr, nullptr}, {h, nullptr}};
  rc = check_args(ins, outs, same);
  if (rc != SSM_OK) return rc;
  if (d.batch == 0) return ok();
  GdrParams p = params(d);
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.g = g;
  p.beta = beta;
  p.h0 = h;
  p.y = static_cast<uint16_t *>(y);
  p.h_last = h_out;
  return launched(launch_gdr_step(p, static_cast<hipStream_t>(stream)), "gdr_step");
}

}  // extern "C"
