// Checks of the sizes of sliding-window attention, for the entry points of
// libssm_block and libssm_delta.
#pragma once

#include <math.h>

#include "block_check.h"
#include "block_internal.h"
#include "ssm_block.h"

namespace ssmb {

inline int check_swa(const ssm_swa_dims_t *d, bool step) {
  if (!d) return fail(SSM_ERR_NULL, "dims is NULL");
  if (d->batch < 0 || d->seqlen < 0)
    return fail(SSM_ERR_SHAPE, "negative size (batch=%lld seqlen=%lld)", (long long)d->batch, (long long)d->seqlen);
  if (step && d->seqlen != 1) return fail(SSM_ERR_SHAPE, "seqlen must be 1 in a step (got %lld)", (long long)d->seqlen);
  if (d->nheads < 1 || d->nkv < 1 || d->nheads % d->nkv != 0)
    return fail(SSM_ERR_SHAPE, "nkv (%lld) must divide nheads (%lld)", (long long)d->nkv, (long long)d->nheads);
  if (d->window < 1 || d->sinks < 0)
    return fail(SSM_ERR_SHAPE, "window must be >= 1 and sinks >= 0 (window=%lld sinks=%lld)", (long long)d->window,
                (long long)d->sinks);
  if (!isfinite(d->scale)) return fail(SSM_ERR_SHAPE, "scale must be finite");
  if (d->reserved != 0) return fail(SSM_ERR_SHAPE, "reserved must be 0");
  if (d->headdim != 64 && d->headdim != 128)
    return fail(SSM_ERR_UNSUPPORTED, "headdim %lld not supported (64 or 128)", (long long)d->headdim);
  constexpr int64_t kMax = int64_t{1} << 30;
  if (d->seqlen > kMax || d->window > kMax || d->sinks > kMax)
    return fail(SSM_ERR_UNSUPPORTED, "seqlen, window and sinks must be at most 2^30");
  const int64_t rows = mul(d->batch, d->nheads);
  if (rows < 0 || rows > 65535 || d->nheads > 65535)
    return fail(SSM_ERR_UNSUPPORTED, "nheads and batch * nheads must be at most 65535");
  // A workgroup has 128 (query, head) pairs, queries in blocks of 32, 64 or 128.
  if (rows * ceil_div(d->seqlen, 128) > kMaxGroups)
    return fail(SSM_ERR_UNSUPPORTED, "batch * nheads * seqlen must be below 2^31");
  const int64_t strides[] = {d->q_batch, d->q_token, d->k_batch, d->k_token, d->v_batch, d->v_token};
  for (const int64_t s : strides)
    if (s < 0 || s % 8 != 0 || s > (int64_t{1} << 40))
      return fail(SSM_ERR_SHAPE, "strides must be multiples of 8 elements, not negative (got %lld)", (long long)s);
  if (d->q_token > kMaxToken || d->k_token > kMaxToken || d->v_token > kMaxToken)
    return fail(SSM_ERR_UNSUPPORTED, "token strides must be at most 2^24 elements");
  if (d->seqlen > 1 && (d->q_token < d->nheads * d->headdim || d->k_token < d->nkv * d->headdim ||
                        d->v_token < d->nkv * d->headdim))
    return fail(SSM_ERR_SHAPE, "a token stride is smaller than the token");
  if (d->batch > 1 && (d->q_batch < d->nheads * d->headdim || d->k_batch < d->nkv * d->headdim ||
                       d->v_batch < d->nkv * d->headdim))
    return fail(SSM_ERR_SHAPE, "a batch stride is smaller than a token");
  return SSM_OK;
}

// Bytes that a strided (batch, seqlen, heads, headdim) tensor spans.
inline size_t span(const ssm_swa_dims_t &d, int64_t batch_stride, int64_t token_stride, int64_t heads) {
  if (d.batch == 0 || d.seqlen == 0) return 0;
  return static_cast<size_t>((d.batch - 1) * batch_stride + (d.seqlen - 1) * token_stride + heads * d.headdim) * 2;
}

}  // namespace ssmb
