// One token of sliding-window attention against a ring cache, and the ring's
// fill from a prompt, for gfx950.
//
// Simplest form: one wavefront per (batch row, query head) walks the slots;
// the token's own key and value come from the arguments, and the group's
// first head stores them.
#include "block_internal.h"

namespace ssmb {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

template <int D>
__global__ void __launch_bounds__(64) swa_step_kernel(const SwaStepParams p) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x;
  const int64_t b = blockIdx.x / p.nheads, h = blockIdx.x % p.nheads;
  const int64_t group = p.nheads / p.nkv, c = h / group, slots = p.sinks + p.window;
  const int64_t pos = p.pos[b], out = (b * p.nheads + h) * D;
  float acc[E] = {}, top = -INFINITY, sum = 0.0f;
  if (pos >= 0) {
    const int64_t own = pos < p.sinks ? pos : p.sinks + (pos - p.sinks) % p.window;
    const int64_t count = pos + 1 < slots ? pos + 1 : slots, base = (b * p.nkv + c) * slots * D;
    float q[E], kn[E], vn[E];
    for (int e = 0; e < E; ++e) {
      q[e] = ld(p.q, b * p.q_batch + h * D + lane + 64 * e) * p.scale;
      kn[e] = ld(p.k, b * p.k_batch + c * D + lane + 64 * e);
      vn[e] = ld(p.v, b * p.v_batch + c * D + lane + 64 * e);
    }
    for (int64_t j = 0; j < count; ++j) {
      float s = 0.0f, v[E];
      for (int e = 0; e < E; ++e) {
        const int64_t at = base + j * D + lane + 64 * e;
        s = fmaf(q[e], j == own ? kn[e] : ld(p.k_cache, at), s);
        v[e] = j == own ? vn[e] : ld(p.v_cache, at);
      }
      s = wave_sum(s);
      const float m = s > top ? s : top;
      const float keep = __builtin_amdgcn_exp2f((top - m) * kLog2e), w = __builtin_amdgcn_exp2f((s - m) * kLog2e);
      sum = fmaf(sum, keep, w);
      for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], keep, w * v[e]);
      top = m;
    }
    if (h % group == 0) {
      for (int e = 0; e < E; ++e) {
        st(p.k_cache, base + own * D + lane + 64 * e, kn[e]);
        st(p.v_cache, base + own * D + lane + 64 * e, vn[e]);
      }
    }
  }
  for (int e = 0; e < E; ++e) st(p.y, out + lane + 64 * e, sum > 0.0f ? acc[e] / sum : 0.0f);
}

// One thread per 16 bytes of a slot: slot s of a row of length n holds
// position s below the sinks, else the largest position p < n with
// (p - sinks) mod window = s - sinks.
__global__ void __launch_bounds__(256) swa_fill_kernel(const SwaParams p, uint16_t *kc, uint16_t *vc) {
  const int64_t chunks = p.headdim / 8, slots = p.sinks + p.window;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= p.batch * p.nkv * slots * chunks) return;
  const int64_t e = id % chunks, s = id / chunks % slots, c = id / chunks / slots % p.nkv;
  const int64_t b = id / chunks / slots / p.nkv;
  int64_t n = p.lengths != nullptr ? p.lengths[b] : p.seqlen;
  n = n < 0 ? 0 : n > p.seqlen ? p.seqlen : n;
  int64_t pos = s;
  if (s >= n) return;
  if (s >= p.sinks) pos += (n - 1 - s) / p.window * p.window;
  const uint4 k = *reinterpret_cast<const uint4 *>(p.k + b * p.k_batch + pos * p.k_token + c * p.headdim + e * 8);
  const uint4 v = *reinterpret_cast<const uint4 *>(p.v + b * p.v_batch + pos * p.v_token + c * p.headdim + e * 8);
  reinterpret_cast<uint4 *>(kc)[id] = k;
  reinterpret_cast<uint4 *>(vc)[id] = v;
}

}  // namespace

hipError_t launch_swa_step(const SwaStepParams &p, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(p.batch * p.nheads)), t(64);
  if (p.headdim == 64) hipLaunchKernelGGL((swa_step_kernel<64>), g, t, 0, s, p);
  else hipLaunchKernelGGL((swa_step_kernel<128>), g, t, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_swa_fill(const SwaParams &p, uint16_t *kc, uint16_t *vc, hipStream_t s) {
  const int64_t n = p.batch * p.nkv * (p.sinks + p.window) * (p.headdim / 8);
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(swa_fill_kernel, dim3(static_cast<uint32_t>((n + 255) / 256)), dim3(256), 0, s, p, kc, vc);
  return hipGetLastError();
}

}  // namespace ssmb
