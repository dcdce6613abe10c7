// Internal declarations of libssm_block: kernel parameter blocks and the
// launchers that block_api.hip calls after validating a request.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssmb {

// Workgroups of 256 that a launch may have along an axis: fewer than 2^32 threads.
constexpr int64_t kMaxGroups = (int64_t{1} << 24) - 1;
// Workgroups along x of a launch that takes two axes, where there are more.
constexpr unsigned kGridWidth = 1u << 20;

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ld(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float ld(const uint16_t *p, int64_t i) {
  return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}
__device__ __forceinline__ void st(float *p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void st(uint16_t *p, int64_t i, float v) {
  p[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));  // round to nearest even
}

// What tiles of a recurrence tell each other, in the workspace: counters (one
// per set of channel blocks, 128 bytes apart), a summary (product, end) per (row, tile, channel), and
// the state at the start of each group of tiles.  Nothing for one tile.
struct GlrChain {
  unsigned *counter;
  uint64_t *sums;
  unsigned *starts;
  int64_t bytes;               // of sums and starts
};
constexpr unsigned kGlrSets = 32, kGlrCounterBytes = 128;
// Sets of `rows` channel blocks: the most that share them evenly.
__host__ __device__ inline unsigned glr_sets(unsigned rows) {
  unsigned n = rows < kGlrSets ? rows : kGlrSets;
  while (rows % n != 0) --n;
  return n;
}
size_t glr_chain_bytes(int64_t batch, int64_t seqlen, int64_t dim);
GlrChain glr_chain(void *workspace, int64_t batch, int64_t seqlen, int64_t dim);

// Gated linear recurrence (see ssm_glr_fwd and ssm_glr_bwd in ssm_block.h).
struct GlrParams {
  const void *x, *rec, *inp;   // in dtype
  const float *A, *h0;         // h0 nullable
  const uint8_t *reset;        // nullable
  void *y;                     // out dtype
  float *h_last, *states;      // nullable
  GlrChain chain;
  int64_t batch, seqlen, dim;
};
hipError_t launch_glr(const GlrParams &p, int in_bf16, int out_bf16, hipStream_t stream);
hipError_t launch_glr_step(const GlrParams &p, int in_bf16, int out_bf16, hipStream_t stream);

struct GlrBwdParams {
  const void *x, *rec, *inp, *dy;  // in dtype
  const float *A, *states, *dh_last;
  const uint8_t *reset;
  void *dx, *drec, *dinp;
  float *dA, *dh0;             // dh0 nullable
  float *ws_dA;                // (glr_bwd_parts, dim)
  GlrChain chain;
  int64_t batch, seqlen, dim;
};
int64_t glr_bwd_parts(int64_t batch, int64_t seqlen);
hipError_t launch_glr_bwd(const GlrBwdParams &p, int in_bf16, hipStream_t stream);

// Residual addition with RMS norm (see ssm_rms_add_fwd and its neighbours).
struct RmsParams {
  const void *x, *residual;    // in dtype; residual nullable
  const float *w;
  void *y;                     // out dtype, or e4m3 bytes with scale
  float *scale;                // non-null: the 8-bit form
  void *residual_out;          // in dtype, nullable
  float eps;
  int64_t rows, dim, group;    // group > 0
};
hipError_t launch_rms(const RmsParams &p, int in_bf16, int out_bf16, hipStream_t stream);

struct RmsBwdParams {
  const void *dy, *s, *dres;   // dres nullable
  const float *w;
  void *dx;
  float *dw;                   // nullable
  float *ws;                   // (parts, dim) terms of dw
  float eps;
  int64_t rows, dim, parts;
};
// Workgroups of the backward, and so the terms of dw.
int64_t rms_bwd_parts(int64_t rows, int64_t dim);
hipError_t launch_rms_bwd(const RmsBwdParams &p, int in_bf16, hipStream_t stream);

// Sliding-window attention (see ssm_swa_fwd and its neighbours).
struct SwaParams {
  const uint16_t *q, *k, *v;   // bf16
  const int32_t *lengths;      // nullable
  uint16_t *y;
  float *lse;                  // nullable in the forward
  const uint16_t *dy;          // backward
  uint16_t *dq, *dk, *dv;
  float *ws_lse2, *ws_delta;   // (batch, nheads, seqlen): log2(e) lse and dy.y
  float *ws_part, *ws_far;     // terms of dk and dv (see SwaBwdPlan)
  int64_t batch, seqlen, nheads, nkv, window, sinks;
  int64_t q_batch, q_token, k_batch, k_token, v_batch, v_token;
  float scale;
  int32_t headdim;
};
hipError_t launch_swa_fwd(const SwaParams &p, hipStream_t stream);

// How the work of dk and dv is shared out, per (batch row, key head).  A
// workgroup has a block of 128 keys, over the queries that see them through
// the window; the group's heads are shared by `slices` workgroups.  Sinks are
// also seen by all queries after those: where there are any, each of the first
// far_blocks blocks of 32 keys has far_chunks more workgroups, whose wavefronts
// take queries in turn.  The first sum_blocks blocks of 128 have more than one
// workgroup: each writes its terms, (2, 128, headdim) or (2, 32, headdim)
// floats, and another launch adds them in their order.
struct SwaBwdPlan {
  unsigned blocks, slices, far_blocks, far_chunks, sum_blocks;
  int64_t items;               // workgroups per (batch row, key head)
};
SwaBwdPlan swa_bwd_plan(int64_t batch, int64_t seqlen, int64_t nheads, int64_t nkv, int64_t headdim, int64_t window,
                        int64_t sinks);
hipError_t launch_swa_bwd(const SwaParams &p, const SwaBwdPlan &plan, hipStream_t stream);

struct SwaStepParams {
  const uint16_t *q, *k, *v;
  uint16_t *k_cache, *v_cache;
  const int32_t *pos;
  uint16_t *y;
  float *ws_o, *ws_stat;       // per (row, head, split): [headdim], and maximum and sum
  int64_t batch, nheads, nkv, window, sinks;
  int64_t q_batch, k_batch, v_batch;
  float scale;
  int32_t headdim;
};
// Workgroups that share the slots of a (row, key head).
int swa_step_splits(int64_t batch, int64_t nheads, int64_t nkv, int64_t slots);
hipError_t launch_swa_step(const SwaStepParams &p, int splits, hipStream_t stream);

// Cache fill: k, v (batch, seqlen, nkv, headdim) into the ring.
hipError_t launch_swa_fill(const SwaParams &p, uint16_t *k_cache, uint16_t *v_cache, hipStream_t stream);

}  // namespace ssmb
