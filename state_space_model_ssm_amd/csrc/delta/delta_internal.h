// Internal declarations of the norms of queries and keys and of the attention
// over a cache in 8 bits: kernel parameters, and the launchers that
// delta_api.hip calls.
#pragma once

#include "block/block_internal.h"

namespace ssmb {

// Norms of queries and keys with rotation (see ssm_qk_norm_fwd and its neighbour).
struct QkNormParams {
  const void *q, *k;              // dtype
  const float *wq, *wk, *inv_freq;  // wq, wk nullable (ones)
  const int32_t *pos;             // nullable (0, 1, ..)
  const void *dyq, *dyk;          // backward: gradients of the outputs, dense
  void *out_q, *out_k;            // outputs, or dq and dk
  float *dwq, *dwk, *ws;          // nullable; (workgroups, headdim) terms, of those of q and then of k
  int64_t tokens, seqlen, nheads, nkv;
  int64_t q_batch, q_token, k_batch, k_token, oq_batch, oq_token, ok_batch, ok_token;
  float eps;
  int32_t headdim, rot, neighbours;
  int32_t tile_q, tile_k;         // tokens that a workgroup of either takes at a time
  int64_t nq;                     // workgroups of q
};
struct QkNormGroups {
  int64_t q, k;
  int tile_q, tile_k;
};
QkNormGroups qk_norm_groups(int64_t tokens, int64_t nheads, int64_t nkv, int64_t headdim, bool bwd);
hipError_t launch_qk_norm(const QkNormParams &p, int bf16, hipStream_t stream);
hipError_t launch_qk_norm_bwd(const QkNormParams &p, int bf16, hipStream_t stream);

// Attention over a ring of e4m3 blocks (see ssm_swa_q8_step).
constexpr int kSwaBlock = 64;
struct SwaQ8Cache {
  uint16_t *k_near, *v_near;      // (batch, nkv, sinks + 64, headdim) bf16
  uint8_t *k_ring, *v_ring;       // (batch, nkv, window, headdim) e4m3
  float *k_scale, *v_scale;       // (batch, nkv, window / 64)
};
struct SwaQ8Plan {
  int splits, waves;  // workgroups that share a row's tiles, and wavefronts of each
};
SwaQ8Plan swa_q8_plan(int64_t batch, int64_t nheads, int64_t nkv, int64_t window, int64_t sinks);
hipError_t launch_swa_q8_step(const SwaStepParams &p, const SwaQ8Cache &cache, const SwaQ8Plan &plan, hipStream_t stream);
hipError_t launch_swa_q8_fill(const SwaParams &p, const SwaQ8Cache &cache, hipStream_t stream);

}  // namespace ssmb
