// Gated linear recurrence for gfx950: forward, backward and one step.
//
//   r = s(rec), i = s(inp), a = exp(A r), b = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + b_t i_t x_t
//
// Simplest form: one lane per (batch row, channel) walks the sequence.
#include "block_internal.h"
#include "ssm_block.h"

namespace ssmb {
namespace {

// The smallest normal float: below it the reciprocal square root has no use.
constexpr float kSmallest = 0x1p-126f;

// 1 - exp(u) for u <= 0.  Above -0.5, where the subtraction would cancel, the
// series -u (1 + u/2 (1 + u/3 (...))) to the 9th power (error below 1.1e-8 of
// the result); below, 1 - a^2 with a = exp(u / 2) at hand.
__device__ __forceinline__ float one_minus_exp(float u, float a) {
  float p = fmaf(u, 1.0f / 9.0f, 1.0f);
  p = fmaf(u * (1.0f / 8.0f), p, 1.0f);
  p = fmaf(u * (1.0f / 7.0f), p, 1.0f);
  p = fmaf(u * (1.0f / 6.0f), p, 1.0f);
  p = fmaf(u * (1.0f / 5.0f), p, 1.0f);
  p = fmaf(u * (1.0f / 4.0f), p, 1.0f);
  p = fmaf(u * (1.0f / 3.0f), p, 1.0f);
  p = fmaf(u * (1.0f / 2.0f), p, 1.0f);
  return u > -0.5f ? -u * p : fmaf(-a, a, 1.0f);
}

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// The decay a and the weighted input u = b i x of one step.
__device__ __forceinline__ void gates(float x, float rec, float inp, float A, float &a, float &u) {
  const float la = A * sigmoid(rec);
  a = __builtin_amdgcn_exp2f(la * kLog2e);
  u = __builtin_amdgcn_sqrtf(one_minus_exp(2.0f * la, a)) * sigmoid(inp) * x;
}

template <typename Tin, typename Tout>
__global__ void __launch_bounds__(64) glr_fwd_kernel(const GlrParams p) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (id >= p.batch * p.dim) return;
  const int64_t b = id / p.dim, d = id % p.dim;
  const Tin *x = static_cast<const Tin *>(p.x), *rec = static_cast<const Tin *>(p.rec);
  const Tin *inp = static_cast<const Tin *>(p.inp);
  const int64_t nstate = (p.seqlen + SSM_GLR_STATE_STEP - 1) / SSM_GLR_STATE_STEP;
  const float A = p.A[d];
  float h = p.h0 != nullptr ? p.h0[id] : 0.0f;
  for (int64_t t = 0; t < p.seqlen; ++t) {
    const int64_t at = (b * p.seqlen + t) * p.dim + d;
    if (p.states != nullptr && t % SSM_GLR_STATE_STEP == 0)
      p.states[(b * nstate + t / SSM_GLR_STATE_STEP) * p.dim + d] = h;
    float a, u;
    gates(ld(x, at), ld(rec, at), ld(inp, at), A, a, u);
    if (p.reset != nullptr && p.reset[b * p.seqlen + t]) h = 0.0f;
    h = fmaf(a, h, u);
    st(static_cast<Tout *>(p.y), at, h);
  }
  if (p.h_last != nullptr) p.h_last[id] = h;
}

template <typename Tin>
__global__ void __launch_bounds__(64) glr_bwd_kernel(const GlrBwdParams p) {
  constexpr int T = SSM_GLR_STATE_STEP;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (id >= p.batch * p.dim) return;
  const int64_t b = id / p.dim, d = id % p.dim;
  const Tin *gx = static_cast<const Tin *>(p.x), *grec = static_cast<const Tin *>(p.rec);
  const Tin *ginp = static_cast<const Tin *>(p.inp), *gdy = static_cast<const Tin *>(p.dy);
  const int64_t nstate = (p.seqlen + T - 1) / T;
  const float A = p.A[d];
  float carry = p.dh_last != nullptr ? p.dh_last[id] : 0.0f, dA = 0.0f;  // carry: a_{t+1} g_{t+1}
  for (int64_t k = nstate - 1; k >= 0; --k) {
    float hp[T];  // the state each step starts from, zero where it is reset
    float h = p.states[(b * nstate + k) * p.dim + d];
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const int64_t t = k * T + j;
      hp[j] = 0.0f;
      if (t < p.seqlen) {
        const int64_t at = (b * p.seqlen + t) * p.dim + d;
        float a, u;
        gates(ld(gx, at), ld(grec, at), ld(ginp, at), A, a, u);
        if (p.reset != nullptr && p.reset[b * p.seqlen + t]) h = 0.0f;
        hp[j] = h;
        h = fmaf(a, h, u);
      }
    }
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      const int64_t t = k * T + j;
      if (t < p.seqlen) {
        const int64_t at = (b * p.seqlen + t) * p.dim + d;
        const float x = ld(gx, at);
        // s(v) with 1 - s(v) = e s(v), e = exp(-v): no cancellation at either end.
        float v = ld(grec, at);
        v = v < -87.0f ? -87.0f : v;
        const float er = __builtin_amdgcn_exp2f(-v * kLog2e), r = __builtin_amdgcn_rcpf(1.0f + er);
        v = ld(ginp, at);
        v = v < -87.0f ? -87.0f : v;
        const float ei = __builtin_amdgcn_exp2f(-v * kLog2e), i = __builtin_amdgcn_rcpf(1.0f + ei);
        const float la = A * r, a = __builtin_amdgcn_exp2f(la * kLog2e);
        const float q = one_minus_exp(2.0f * la, a);
        const float rb = q >= kSmallest ? __builtin_amdgcn_rsqf(q) : 0.0f;  // 1 / b
        const float beta = q * rb;
        const float g = ld(gdy, at) + carry;
        const float ix = i * x;
        const float w = g * (a * hp[j] - a * a * rb * ix);
        st(static_cast<Tin *>(p.dx), at, g * beta * i);
        st(static_cast<Tin *>(p.drec), at, w * la * (er * r));
        st(static_cast<Tin *>(p.dinp), at, g * beta * ix * (ei * i));
        dA = fmaf(w, r, dA);
        carry = (p.reset != nullptr && p.reset[b * p.seqlen + t]) ? 0.0f : a * g;
      }
    }
  }
  p.ws_dA[id] = dA;
  if (p.dh0 != nullptr) p.dh0[id] = carry;
}

__global__ void __launch_bounds__(256) glr_sum_kernel(const float *part, float *dA, int64_t parts, int64_t dim) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (d >= dim) return;
  float s = 0.0f;
  for (int64_t k = 0; k < parts; ++k) s += part[k * dim + d];
  dA[d] = s;
}

template <typename Tin, typename Tout>
__global__ void __launch_bounds__(256) glr_step_kernel(const GlrParams p) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= p.batch * p.dim) return;
  float a, u;
  gates(ld(static_cast<const Tin *>(p.x), id), ld(static_cast<const Tin *>(p.rec), id),
        ld(static_cast<const Tin *>(p.inp), id), p.A[id % p.dim], a, u);
  const float h = fmaf(a, p.h0[id], u);
  p.h_last[id] = h;
  st(static_cast<Tout *>(p.y), id, h);
}

dim3 blocks(int64_t n, int64_t per) { return dim3(static_cast<uint32_t>((n + per - 1) / per)); }

}  // namespace

hipError_t launch_glr(const GlrParams &p, int in_bf16, int out_bf16, hipStream_t s) {
  const dim3 g = blocks(p.batch * p.dim, 64), t(64);
  if (in_bf16 && out_bf16) hipLaunchKernelGGL((glr_fwd_kernel<uint16_t, uint16_t>), g, t, 0, s, p);
  else if (in_bf16) hipLaunchKernelGGL((glr_fwd_kernel<uint16_t, float>), g, t, 0, s, p);
  else if (out_bf16) hipLaunchKernelGGL((glr_fwd_kernel<float, uint16_t>), g, t, 0, s, p);
  else hipLaunchKernelGGL((glr_fwd_kernel<float, float>), g, t, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_glr_step(const GlrParams &p, int in_bf16, int out_bf16, hipStream_t s) {
  const dim3 g = blocks(p.batch * p.dim, 256), t(256);
  if (in_bf16 && out_bf16) hipLaunchKernelGGL((glr_step_kernel<uint16_t, uint16_t>), g, t, 0, s, p);
  else if (in_bf16) hipLaunchKernelGGL((glr_step_kernel<uint16_t, float>), g, t, 0, s, p);
  else if (out_bf16) hipLaunchKernelGGL((glr_step_kernel<float, uint16_t>), g, t, 0, s, p);
  else hipLaunchKernelGGL((glr_step_kernel<float, float>), g, t, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_glr_bwd(const GlrBwdParams &p, int in_bf16, hipStream_t s) {
  const dim3 g = blocks(p.batch * p.dim, 64), t(64);
  if (p.batch * p.dim > 0) {
    if (in_bf16) hipLaunchKernelGGL((glr_bwd_kernel<uint16_t>), g, t, 0, s, p);
    else hipLaunchKernelGGL((glr_bwd_kernel<float>), g, t, 0, s, p);
  }
  if (p.dim > 0)
    hipLaunchKernelGGL(glr_sum_kernel, blocks(p.dim, 256), dim3(256), 0, s, p.ws_dA, p.dA, p.batch, p.dim);
  return hipGetLastError();
}

}  // namespace ssmb
