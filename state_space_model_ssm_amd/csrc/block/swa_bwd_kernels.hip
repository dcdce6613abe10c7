// Backward of sliding-window attention with sinks for gfx950.
//
// Query t sees key j when j <= t < length and (t - j < window or j < sinks).
// Simplest form: one wavefront per query (dq) or per key (dk, dv), lanes over
// the head's elements.
#include "block_internal.h"

namespace ssmb {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ int64_t row_length(const SwaParams &p, int64_t b) {
  if (p.lengths == nullptr) return p.seqlen;
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : n > p.seqlen ? p.seqlen : n;
}

// dq and delta = dy.y of one query.
template <int D>
__global__ void __launch_bounds__(64) swa_dq_kernel(const SwaParams p) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x, b = blockIdx.y / p.nheads, h = blockIdx.y % p.nheads;
  const int64_t c = h / (p.nheads / p.nkv);
  const int64_t out = ((b * p.seqlen + t) * p.nheads + h) * D;
  float acc[E] = {}, delta = 0.0f;
  if (t < row_length(p, b)) {
    const float lse = p.lse[(b * p.nheads + h) * p.seqlen + t];
    float q[E], dy[E];
    for (int e = 0; e < E; ++e) {
      q[e] = ld(p.q, b * p.q_batch + t * p.q_token + h * D + lane + 64 * e) * p.scale;
      dy[e] = ld(p.dy, out + lane + 64 * e);
      delta = fmaf(dy[e], ld(p.y, out + lane + 64 * e), delta);
    }
    delta = wave_sum(delta);
    const int64_t lo = t - p.window + 1 > 0 ? t - p.window + 1 : 0;
    for (int64_t j = p.sinks > 0 ? 0 : lo; j <= t; ++j) {
      if (j >= p.sinks && j < lo) j = lo;
      float s = 0.0f, dp = 0.0f, k[E];
      for (int e = 0; e < E; ++e) {
        k[e] = ld(p.k, b * p.k_batch + j * p.k_token + c * D + lane + 64 * e);
        s = fmaf(q[e], k[e], s);
        dp = fmaf(dy[e], ld(p.v, b * p.v_batch + j * p.v_token + c * D + lane + 64 * e), dp);
      }
      const float w = __builtin_amdgcn_exp2f((wave_sum(s) - lse) * kLog2e);
      const float ds = w * (wave_sum(dp) - delta) * p.scale;
      for (int e = 0; e < E; ++e) acc[e] = fmaf(ds, k[e], acc[e]);
    }
  }
  for (int e = 0; e < E; ++e) st(p.dq, out + lane + 64 * e, acc[e]);
  if (lane == 0) p.ws_delta[(b * p.nheads + h) * p.seqlen + t] = delta;
}

// dk and dv of one key, over the queries and the group's heads that see it.
template <int D>
__global__ void __launch_bounds__(64) swa_dkv_kernel(const SwaParams p) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x;
  const int64_t j = blockIdx.x, b = blockIdx.y / p.nkv, c = blockIdx.y % p.nkv, group = p.nheads / p.nkv;
  const int64_t n = row_length(p, b);
  float dk[E] = {}, dv[E] = {};
  if (j < n) {
    float k[E], v[E];
    for (int e = 0; e < E; ++e) {
      k[e] = ld(p.k, b * p.k_batch + j * p.k_token + c * D + lane + 64 * e);
      v[e] = ld(p.v, b * p.v_batch + j * p.v_token + c * D + lane + 64 * e);
    }
    const int64_t hi = j < p.sinks || n - j < p.window ? n : j + p.window;
    for (int64_t h = c * group; h < (c + 1) * group; ++h) {
      for (int64_t t = j; t < hi; ++t) {
        const int64_t row = ((b * p.seqlen + t) * p.nheads + h) * D, at = (b * p.nheads + h) * p.seqlen + t;
        float q[E], dy[E], s = 0.0f, dp = 0.0f;
        for (int e = 0; e < E; ++e) {
          q[e] = ld(p.q, b * p.q_batch + t * p.q_token + h * D + lane + 64 * e) * p.scale;
          dy[e] = ld(p.dy, row + lane + 64 * e);
          s = fmaf(q[e], k[e], s);
          dp = fmaf(dy[e], v[e], dp);
        }
        const float w = __builtin_amdgcn_exp2f((wave_sum(s) - p.lse[at]) * kLog2e);
        const float ds = w * (wave_sum(dp) - p.ws_delta[at]);
        for (int e = 0; e < E; ++e) {
          dk[e] = fmaf(ds, q[e], dk[e]);
          dv[e] = fmaf(w, dy[e], dv[e]);
        }
      }
    }
  }
  const int64_t out = ((b * p.seqlen + j) * p.nkv + c) * D;
  for (int e = 0; e < E; ++e) {
    st(p.dk, out + lane + 64 * e, dk[e]);
    st(p.dv, out + lane + 64 * e, dv[e]);
  }
}

}  // namespace

hipError_t launch_swa_bwd(const SwaParams &p, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(p.seqlen), static_cast<uint32_t>(p.batch * p.nheads)), t(64);
  const dim3 gk(static_cast<uint32_t>(p.seqlen), static_cast<uint32_t>(p.batch * p.nkv));
  if (p.headdim == 64) {
    hipLaunchKernelGGL((swa_dq_kernel<64>), g, t, 0, s, p);
    hipLaunchKernelGGL((swa_dkv_kernel<64>), gk, t, 0, s, p);
  } else {
    hipLaunchKernelGGL((swa_dq_kernel<128>), g, t, 0, s, p);
    hipLaunchKernelGGL((swa_dkv_kernel<128>), gk, t, 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace ssmb
