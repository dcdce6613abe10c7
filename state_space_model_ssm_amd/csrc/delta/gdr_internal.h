// Internal declarations of the gated delta rule: kernel parameters, the
// workspace's layout, and the launchers that gdr_api.hip calls.
#pragma once

#include "block/block_internal.h"

namespace ssmb {

constexpr int kGdrChunk = 64;

// What the forward knows of a chunk of 64 tokens and a value head before it
// has a state: T = (I + L)^-1 and the attention A within the chunk, as
// operands in bfloat16 parts (see gdr_tile.h), and the gates' factors.
constexpr int kGdrFrags = 6;                                   // operands of a lower triangle: 16 rows x 32 columns each
constexpr size_t kGdrTriBytes = size_t{2} * kGdrFrags * 1024;  // both parts
constexpr size_t kGdrGateBytes = 4 * kGdrChunk * 4;
constexpr size_t kGdrChunkBytes = 2 * kGdrTriBytes + kGdrGateBytes;

struct GdrParams {
  const uint16_t *q, *k, *v;   // bf16
  const void *g, *beta;        // gate dtype
  const float *h0;             // nullable
  const int32_t *lengths;      // nullable
  uint16_t *y;
  float *h_last, *states;      // nullable
  char *ws;                    // kGdrChunkBytes per (row, value head, chunk)
  int64_t batch, seqlen, nqk, nheads, chunks;
  int64_t q_batch, q_token, k_batch, k_token, v_batch, v_token;
  float scale;
  int32_t kdim, vdim, gates_bf16;
};
size_t gdr_workspace(const GdrParams &p);
hipError_t launch_gdr_fwd(const GdrParams &p, hipStream_t stream);
hipError_t launch_gdr_step(const GdrParams &p, hipStream_t stream);  // h0 -> h_last

}  // namespace ssmb
