// C ABI of the norms of queries and keys and of the attention over a cache in 8
// bits (declared in include/ssm_delta.h): argument checks, workspace sizing and
// dispatch.
#include "ssm_delta.h"

#include <math.h>

#include "block/block_check.h"
#include "block/swa_check.h"
#include "delta_internal.h"

using namespace ssmb;

namespace {

// ---------------------------------------------------------------------------
// Norms of queries and keys
// ---------------------------------------------------------------------------

int check_qk(const ssm_qk_norm_dims_t *d) {
  if (!d) return fail(SSM_ERR_NULL, "dims is NULL");
  if (d->batch < 0 || d->seqlen < 0)
    return fail(SSM_ERR_SHAPE, "negative size (batch=%lld seqlen=%lld)", (long long)d->batch, (long long)d->seqlen);
  if (d->nheads < 1 || d->nkv < 1)
    return fail(SSM_ERR_SHAPE, "nheads and nkv must be at least 1 (got %lld, %lld)", (long long)d->nheads, (long long)d->nkv);
  if (d->headdim < 16 || d->headdim > 256 || d->headdim % 16 != 0)
    return fail(SSM_ERR_UNSUPPORTED, "headdim %lld not supported (a multiple of 16, at most 256)", (long long)d->headdim);
  if (d->rot < 0 || d->rot > d->headdim || d->rot % 16 != 0)
    return fail(SSM_ERR_SHAPE, "rot must be a multiple of 16 from 0 to headdim (got %lld)", (long long)d->rot);
  if (!valid_dtype(d->dtype)) return fail(SSM_ERR_DTYPE, "dtype %d is not an ssm_dtype_t", d->dtype);
  if (d->neighbours != 0 && d->neighbours != 1) return fail(SSM_ERR_SHAPE, "neighbours must be 0 or 1 (got %d)", d->neighbours);
  if (!(d->eps >= 0.0f) || isinf(d->eps)) return fail(SSM_ERR_SHAPE, "eps must be finite and >= 0");
  if (d->reserved != 0) return fail(SSM_ERR_SHAPE, "reserved must be 0");
  constexpr int64_t kMaxHeads = int64_t{1} << 20;
  if (d->nheads > kMaxHeads || d->nkv > kMaxHeads || d->seqlen > (int64_t{1} << 31) - 1)
    return fail(SSM_ERR_UNSUPPORTED, "nheads and nkv must be at most 2^20 and seqlen below 2^31");
  const int64_t n = mul(mul(d->batch, d->seqlen), (d->nheads + d->nkv) * d->headdim);
  if (n < 0 || mul(n, 4) < 0) return fail(SSM_ERR_UNSUPPORTED, "the tensors are too large");
  const int64_t each = 16 / static_cast<int64_t>(dtype_size(d->dtype));
  const int64_t strides[] = {d->q_batch,  d->q_token,  d->k_batch,  d->k_token,
                             d->oq_batch, d->oq_token, d->ok_batch, d->ok_token};
  for (int k = 0; k < 8; ++k) {
    const int64_t s = strides[k], token = (k % 4 < 2 ? d->nheads : d->nkv) * d->headdim;
    if (s < 0 || s % each != 0 || s > (int64_t{1} << 40))
      return fail(SSM_ERR_SHAPE, "strides must be multiples of %lld elements, not negative (got %lld)", (long long)each, (long long)s);
    if ((k % 2 == 0 ? d->batch : d->seqlen) > 1 && s < token) return fail(SSM_ERR_SHAPE, "a stride is smaller than a token");
  }
  // Bytes from the first token to the last: below 2^62.
  for (int k = 0; k < 8; k += 2) {
    const int64_t rows = mul(d->batch > 1 ? d->batch - 1 : 0, strides[k]);
    const int64_t far = mul(d->seqlen > 1 ? d->seqlen - 1 : 0, strides[k + 1]);
    if (rows < 0 || far < 0 || mul(rows + far, 8) < 0) return fail(SSM_ERR_UNSUPPORTED, "the tensors are too large");
  }
  // Rows of one output must not meet: a batch row's tokens end before the next one's, or between them.
  for (int k = 4; k < 8; k += 2) {
    const int64_t token = (k == 4 ? d->nheads : d->nkv) * d->headdim, sb = strides[k], st = strides[k + 1];
    if (d->batch > 1 && d->seqlen > 1 && sb < (d->seqlen - 1) * st + token && st < (d->batch - 1) * sb + token)
      return fail(SSM_ERR_SHAPE, "the rows of an output overlap");
  }
  return SSM_OK;
}

size_t dw_workspace(const ssm_qk_norm_dims_t &d) {
  const QkNormGroups n = qk_norm_groups(d.batch * d.seqlen, d.nheads, d.nkv, d.headdim, true);
  return up256(static_cast<size_t>(n.q + n.k) * d.headdim * 4);
}

// A strided (batch, seqlen, heads, headdim) tensor of a call.
struct Rows {
  const char *name;
  const void *p;
  int64_t batch_stride, token_stride, token;  // in bytes
  size_t bytes;
};
Rows rows_of(const ssm_qk_norm_dims_t &d, const char *name, const void *p, int64_t sb, int64_t st, int64_t heads) {
  const int64_t e = static_cast<int64_t>(dtype_size(d.dtype));
  Rows r{name, p, sb * e, st * e, heads * d.headdim * e, 0};
  if (d.batch > 0 && d.seqlen > 0)
    r.bytes = static_cast<size_t>((d.batch - 1) * r.batch_stride + (d.seqlen - 1) * r.token_stride + r.token);
  return r;
}
// Parts of one tensor side by side (same strides, no token of one within the other's) do not meet.
bool side_by_side(const ssm_qk_norm_dims_t &d, const Rows &a, const Rows &b) {
  const bool tokens = d.seqlen > 1, batches = d.batch > 1;
  if ((tokens && a.token_stride != b.token_stride) || (batches && a.batch_stride != b.batch_stride)) return false;
  const int64_t step = tokens ? a.token_stride : a.batch_stride;
  if (!tokens && !batches) return false;  // one token each: the bytes say all
  if (tokens && batches && (a.batch_stride % step != 0 || a.batch_stride < step * d.seqlen)) return false;
  const int64_t gap = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  return gap >= 0 ? gap >= a.token && gap + b.token <= step : -gap >= b.token && -gap + a.token <= step;
}
int meets(const ssm_qk_norm_dims_t &d, const Rows &out, const Rows &other) {
  const Arg a = {out.name, out.p, out.bytes, 16, true}, b = {other.name, other.p, other.bytes, 16, true};
  if (!overlap(a, b) || side_by_side(d, out, other)) return SSM_OK;
  return fail(SSM_ERR_SHAPE, "%s overlaps %s", out.name, other.name);
}

int qk_run(const void *q, const void *k, const float *wq, const float *wk, const float *inv_freq, const int32_t *pos,
           const void *dyq, const void *dyk, void *out_q, void *out_k, float *dwq, float *dwk,
           const ssm_qk_norm_dims_t *dims, void *stream, bool bwd) {
  int rc = check_qk(dims);
  if (rc != SSM_OK) return rc;
  const ssm_qk_norm_dims_t &d = *dims;
  const int64_t tokens = d.batch * d.seqlen;
  const size_t e = dtype_size(d.dtype), n = static_cast<size_t>(tokens), w = static_cast<size_t>(d.headdim) * 4;
  const Rows rq = rows_of(d, "q", q, d.q_batch, d.q_token, d.nheads), rk = rows_of(d, "k", k, d.k_batch, d.k_token, d.nkv);
  const Rows oq = rows_of(d, bwd ? "dq" : "q_out", out_q, d.oq_batch, d.oq_token, d.nheads);
  const Rows ok_ = rows_of(d, bwd ? "dk" : "k_out", out_k, d.ok_batch, d.ok_token, d.nkv);
  // q and k are compared with the outputs below, by their rows.
  const Arg rows[] = {{"q", q, rq.bytes, 16, true}, {"k", k, rk.bytes, 16, true}};
  for (const Arg &a : rows)
    if ((rc = check_in(a)) != SSM_OK) return rc;
  const size_t need = bwd && (dwq != nullptr || dwk != nullptr) ? dw_workspace(d) : 0;
  const Arg ins[] = {{"wq", wq, w, 16, false},
                     {"wk", wk, w, 16, false},
                     {"inv_freq", inv_freq, static_cast<size_t>(d.rot) / 2 * 4, 4, n > 0},
                     {"pos", pos, d.rot > 0 ? n * 4 : 0, 4, false},
                     {"dq_out", dyq, bwd ? n * d.nheads * d.headdim * e : 0, 16, bwd},
                     {"dk_out", dyk, bwd ? n * d.nkv * d.headdim * e : 0, 16, bwd},
                     {"workspace", d.workspace, bwd && d.workspace ? d.workspace_bytes : 0, 1, false}};
  const Arg outs[] = {{oq.name, out_q, oq.bytes, 16, true},
                      {"dwq", dwq, w, 4, false},
                      {"dwk", dwk, w, 4, false}};
  const Arg outs_k[] = {{ok_.name, out_k, ok_.bytes, 16, true}, {"dwq", dwq, w, 4, false}, {"dwk", dwk, w, 4, false}};
  const void *const same[3][2] = {};
  rc = check_args(ins, outs, same);
  if (rc == SSM_OK) rc = check_args(ins, outs_k, same);
  if (rc == SSM_OK) rc = check_workspace(ins, need);
  if (rc != SSM_OK) return rc;
  // An output may take exactly its input's place.
  const bool place_q = out_q == q && oq.batch_stride == rq.batch_stride && oq.token_stride == rq.token_stride;
  const bool place_k = out_k == k && ok_.batch_stride == rk.batch_stride && ok_.token_stride == rk.token_stride;
  if ((!place_q && (rc = meets(d, oq, rq)) != SSM_OK) || (rc = meets(d, oq, rk)) != SSM_OK) return rc;
  if ((!place_k && (rc = meets(d, ok_, rk)) != SSM_OK) || (rc = meets(d, ok_, rq)) != SSM_OK) return rc;
  if ((rc = meets(d, ok_, oq)) != SSM_OK) return rc;
  for (const Arg &o : {outs[1], outs[2]})
    for (const Arg &a : rows)
      if (overlap(o, a)) return fail(SSM_ERR_SHAPE, "%s overlaps %s", o.name, a.name);
  if (need > 0) {
    const Arg ws = {"workspace", d.workspace, need, 1, true};
    for (const Arg &a : rows)
      if (overlap(ws, a)) return fail(SSM_ERR_SHAPE, "workspace overlaps %s", a.name);
  }
  if (tokens == 0 && need == 0 && dwq == nullptr && dwk == nullptr) return ok();
  QkNormParams p{};
  p.q = q;
  p.k = k;
  p.wq = wq;
  p.wk = wk;
  p.inv_freq = inv_freq;
  p.pos = pos;
  p.dyq = dyq;
  p.dyk = dyk;
  p.out_q = out_q;
  p.out_k = out_k;
  p.dwq = dwq;
  p.dwk = dwk;
  p.ws = dwq != nullptr || dwk != nullptr ? static_cast<float *>(d.workspace) : nullptr;
  p.tokens = tokens;
  p.seqlen = d.seqlen;
  p.nheads = d.nheads;
  p.nkv = d.nkv;
  p.q_batch = d.q_batch;
  p.q_token = d.q_token;
  p.k_batch = d.k_batch;
  p.k_token = d.k_token;
  p.oq_batch = d.oq_batch;
  p.oq_token = d.oq_token;
  p.ok_batch = d.ok_batch;
  p.ok_token = d.ok_token;
  p.eps = d.eps;
  p.headdim = static_cast<int32_t>(d.headdim);
  p.rot = static_cast<int32_t>(d.rot);
  p.neighbours = d.neighbours;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return bwd ? launched(launch_qk_norm_bwd(p, d.dtype == SSM_BF16, s), "qk_norm_bwd")
             : launched(launch_qk_norm(p, d.dtype == SSM_BF16, s), "qk_norm_fwd");
}

// ---------------------------------------------------------------------------
// Attention over a cache in 8 bits
// ---------------------------------------------------------------------------

int check_q8(const ssm_swa_dims_t *d, bool step) {
  const int rc = check_swa(d, step);
  if (rc != SSM_OK) return rc;
  if (d->window % kSwaBlock != 0) return fail(SSM_ERR_SHAPE, "window must be a multiple of 64 (got %lld)", (long long)d->window);
  if (d->sinks + d->window > (int64_t{1} << 30)) return fail(SSM_ERR_UNSUPPORTED, "sinks + window must be at most 2^30");
  return SSM_OK;
}

struct CacheBytes {
  size_t near, ring, scale;
};
CacheBytes cache_bytes(const ssm_swa_dims_t &d) {
  const size_t rows = static_cast<size_t>(d.batch) * d.nkv;
  return {rows * (d.sinks + kSwaBlock) * d.headdim * 2, rows * d.window * d.headdim, rows * (d.window / kSwaBlock) * 4};
}

SwaQ8Plan q8_plan(const ssm_swa_dims_t &d) { return swa_q8_plan(d.batch, d.nheads, d.nkv, d.window, d.sinks); }
size_t q8_sums(const ssm_swa_dims_t &d) {
  return up256(static_cast<size_t>(d.batch) * d.nheads * q8_plan(d).splits * d.headdim * 4);
}
size_t q8_workspace(const ssm_swa_dims_t &d) {
  const int splits = q8_plan(d).splits;
  const size_t rows = static_cast<size_t>(d.batch) * d.nheads * splits;
  return splits > 1 ? q8_sums(d) + up256(rows * 8) : 0;
}

SwaQ8Cache cache_of(void *k_near, void *v_near, void *k_ring, void *v_ring, float *k_scale, float *v_scale) {
  return {static_cast<uint16_t *>(k_near), static_cast<uint16_t *>(v_near), static_cast<uint8_t *>(k_ring),
          static_cast<uint8_t *>(v_ring),  k_scale,                         v_scale};
}

}  // namespace

extern "C" {

int ssm_qk_norm_fwd(const void *q, const void *k, const float *wq, const float *wk, const float *inv_freq,
                    const int32_t *pos, void *q_out, void *k_out, const ssm_qk_norm_dims_t *dims, void *stream) {
  return qk_run(q, k, wq, wk, inv_freq, pos, nullptr, nullptr, q_out, k_out, nullptr, nullptr, dims, stream, false);
}

int ssm_qk_norm_bwd_workspace_size(const ssm_qk_norm_dims_t *dims, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_NULL, "bytes is NULL");
  const int rc = check_qk(dims);
  if (rc != SSM_OK) return rc;
  *bytes = dw_workspace(*dims);
  return ok();
}

int ssm_qk_norm_bwd(const void *q, const void *k, const float *wq, const float *wk, const float *inv_freq,
                    const int32_t *pos, const void *dq_out, const void *dk_out, void *dq, void *dk, float *dwq, float *dwk,
                    const ssm_qk_norm_dims_t *dims, void *stream) {
  return qk_run(q, k, wq, wk, inv_freq, pos, dq_out, dk_out, dq, dk, dwq, dwk, dims, stream, true);
}

int ssm_swa_q8_step_workspace_size(const ssm_swa_dims_t *dims, size_t *bytes) {
  if (!bytes) return fail(SSM_ERR_NULL, "bytes is NULL");
  const int rc = check_q8(dims, true);
  if (rc != SSM_OK) return rc;
  *bytes = q8_workspace(*dims);
  return ok();
}

int ssm_swa_q8_step(const void *q, const void *k, const void *v, void *k_near, void *v_near, void *k_ring, void *v_ring,
                    float *k_scale, float *v_scale, const int32_t *pos, void *y, const ssm_swa_dims_t *dims,
                    void *stream) {
  int rc = check_q8(dims, true);
  if (rc != SSM_OK) return rc;
  const ssm_swa_dims_t &d = *dims;
  const CacheBytes n = cache_bytes(d);
  const Arg ins[] = {{"q", q, span(d, d.q_batch, d.q_token, d.nheads), 16, true},
                     {"k", k, span(d, d.k_batch, d.k_token, d.nkv), 16, true},
                     {"v", v, span(d, d.v_batch, d.v_token, d.nkv), 16, true},
                     {"pos", pos, static_cast<size_t>(d.batch) * 4, 4, true},
                     {"workspace", d.workspace, d.workspace ? d.workspace_bytes : 0, 1, false}};
  const Arg outs[] = {{"k_near", k_near, n.near, 16, true},   {"v_near", v_near, n.near, 16, true},
                      {"k_ring", k_ring, n.ring, 16, true},   {"v_ring", v_ring, n.ring, 16, true},
                      {"k_scale", k_scale, n.scale, 4, true}, {"v_scale", v_scale, n.scale, 4, true},
                      {"y", y, static_cast<size_t>(d.batch) * d.nheads * d.headdim * 2, 16, true}};
  const void *const same[7][2] = {};
  rc = check_args(ins, outs, same);
  if (rc == SSM_OK) rc = check_workspace(ins, q8_workspace(d));
  if (rc != SSM_OK) return rc;
  if (d.batch == 0) return ok();
  SwaStepParams p{};
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
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
  if (d.workspace) p.ws_stat = reinterpret_cast<float *>(static_cast<char *>(d.workspace) + q8_sums(d));
  return launched(launch_swa_q8_step(p, cache_of(k_near, v_near, k_ring, v_ring, k_scale, v_scale), q8_plan(d),
                                     static_cast<hipStream_t>(stream)),
                  "swa_q8_step");
}

int ssm_swa_q8_fill(const void *k, const void *v, const int32_t *lengths, void *k_near, void *v_near, void *k_ring,
                    void *v_ring, float *k_scale, float *v_scale, const ssm_swa_dims_t *dims, void *stream) {
  int rc = check_q8(dims, false);
  if (rc != SSM_OK) return rc;
  const ssm_swa_dims_t &d = *dims;
  const CacheBytes n = cache_bytes(d);
  const Arg ins[] = {{"k", k, span(d, d.k_batch, d.k_token, d.nkv), 16, true},
                     {"v", v, span(d, d.v_batch, d.v_token, d.nkv), 16, true},
                     {"lengths", lengths, static_cast<size_t>(d.batch) * 4, 4, false}};
  const Arg outs[] = {{"k_near", k_near, n.near, 16, true},   {"v_near", v_near, n.near, 16, true},
                      {"k_ring", k_ring, n.ring, 16, true},   {"v_ring", v_ring, n.ring, 16, true},
                      {"k_scale", k_scale, n.scale, 4, true}, {"v_scale", v_scale, n.scale, 4, true}};
  const void *const same[6][2] = {};
  rc = check_args(ins, outs, same);
  if (rc != SSM_OK) return rc;
  if (d.batch == 0 || d.seqlen == 0) return ok();
  SwaParams p{};
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.lengths = lengths;
  p.batch = d.batch;
  p.seqlen = d.seqlen;
  p.nkv = d.nkv;
  p.window = d.window;
  p.sinks = d.sinks;
  p.k_batch = d.k_batch;
  p.k_token = d.k_token;
  p.v_batch = d.v_batch;
  p.v_token = d.v_token;
  p.headdim = static_cast<int32_t>(d.headdim);
  return launched(launch_swa_q8_fill(p, cache_of(k_near, v_near, k_ring, v_ring, k_scale, v_scale), static_cast<hipStream_t>(stream)),
                  "swa_q8_fill");
}

}  // extern "C"
