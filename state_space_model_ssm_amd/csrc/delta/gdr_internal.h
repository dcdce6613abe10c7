// Internal declarations of the gated delta rule: kernel parameters, the
// workspace's layout, and the launchers that gdr_api.hip calls.
#pragma once

#include "block/block_internal.h"

namespace ssmb {

// What is known of a chunk of 64 tokens and a value head before its state is:
// T = (I + L)^-1 less I and the attention A within the chunk, as operands in
// bfloat16 parts (see gdr_tile.h), then the gates' factors.
constexpr int kGdrFrags = 6;                                   // operands of a triangle: 16 rows x 32 columns each
constexpr size_t kGdrTriBytes = size_t{2} * kGdrFrags * 1024;  // both parts
// Factors, 64 of each: scale e^G, e^G, beta e^(GC - G), beta (float32), G log2(e) (float64), e^(GC - G).
constexpr size_t kGdrGateBytes = 2048;
constexpr size_t kGdrChunkBytes = 2 * kGdrTriBytes + kGdrGateBytes;
constexpr size_t kGdrRestBytes = kGdrTriBytes / 2;  // T's third part, where the state is held to float32
// Of a chunk and value head, in two bfloat16 parts as operands over 32 values
// (see gdr_tile.h): the state before it or dS behind it, [16 key elements][32
// values][part], then Z or D, [32 values][16 tokens][part], 1 KiB each.
constexpr size_t gdr_state_bytes(int64_t kdim, int64_t vdim) { return static_cast<size_t>(kdim * vdim) * 4; }
constexpr size_t gdr_both_bytes(int64_t kdim, int64_t vdim) { return gdr_state_bytes(kdim, vdim) + static_cast<size_t>(64 * vdim) * 4; }
// What the forward saves: those, and what is known of the chunk.
constexpr size_t gdr_saved_bytes(int64_t kdim, int64_t vdim) { return gdr_both_bytes(kdim, vdim) + kGdrChunkBytes; }

// Long sequences of few heads are cut into segments of `chunks` chunks, and the
// state at the start of each is found before y is made: with S_0 = 0 and with
// S_0 = I a segment gives E and P, and its end is P S_0 + E.
// Backwards alike: from dS = 0 a segment gives an E of its own, and dS before
// it is P^T dS + E.
struct GdrSegments {
  int64_t count, chunks;
};
GdrSegments gdr_segments(int64_t heads, int64_t kdim, int64_t vdim, int64_t chunks);

struct GdrParams {
  const uint16_t *q, *k, *v;   // bf16
  const void *g, *beta;        // gate dtype
  const float *h0;             // nullable
  const int32_t *lengths;      // nullable
  uint16_t *y;
  float *h_last;               // nullable
  char *saved;                 // gdr_saved_bytes() per (row, value head, chunk), nullable in the forward
  char *ws;
  char *ops;                   // kGdrChunkBytes per (row, value head, chunk), ops_step bytes apart: in `saved` or the workspace
  int64_t ops_step;
  char *rest;                  // kGdrRestBytes per (row, value head, chunk), in the workspace; null where T is taken in two parts
  const uint16_t *dy;          // backward
  const float *dh_last;        // nullable
  uint16_t *dq, *dk, *dv;
  void *dg, *dbeta;            // gate dtype
  float *dh0;                  // nullable
  char *ws_both;               // the backward's dS and D: gdr_both_bytes() each
  GdrSegments seg;
  float *ws_state;             // (row, value head, segment): E, and then the state before the segment, or dS behind it
  uint16_t *ws_carry;          // (row, value head, segment): P in three parts (backward: P^T in two), as operands
  int64_t batch, seqlen, nqk, nheads, chunks;
  int64_t q_batch, q_token, k_batch, k_token, v_batch, v_token;
  float scale;
  int32_t kdim, vdim, gates_bf16;
};
// Sizes of the forward's workspace: ws, rest, ws_state and ws_carry in turn.
struct GdrSizes {
  size_t chunks, rest, state, carry;
  size_t all() const { return chunks + rest + state + carry; }
};
GdrSizes gdr_sizes(const GdrParams &p);
GdrSegments gdr_bwd_segments(int64_t heads, int64_t kdim, int64_t vdim, int64_t chunks);
GdrSizes gdr_bwd_sizes(const GdrParams &p);  // of the backward's: ws_both, ws_state and ws_carry
void launch_gdr_bwd_carry(const GdrParams &p, hipStream_t stream);
void launch_gdr_bwd_join(const GdrParams &p, hipStream_t stream);
hipError_t launch_gdr_bwd(const GdrParams &p, hipStream_t stream);
hipError_t launch_gdr_fwd(const GdrParams &p, hipStream_t stream);
hipError_t launch_gdr_step(const GdrParams &p, hipStream_t stream);  // h0 -> h_last

}  // namespace ssmb
