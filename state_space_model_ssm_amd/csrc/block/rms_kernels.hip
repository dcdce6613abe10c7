// Residual addition with RMS norm for gfx950: y = s / sqrt(mean(s^2) + eps) w
// with s = x + residual, in storage types or in e4m3 bytes with scales, and
// its backward.
//
// Simplest form: one wavefront per row, which it reads again for each pass.
#include "block_internal.h"

namespace ssmb {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// The larger of a and |b|, NaN if either is one.
__device__ __forceinline__ float amax(float a, float b) {
  const float c = fabsf(b);
  return (a != a || a > c) ? a : c;
}

__device__ __forceinline__ float wave_amax(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = amax(v, __shfl_xor(v, m));
  return v;
}

// v (within +-448 or NaN) as an e4m3 byte, rounded to nearest even.
__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xff);
}

template <typename Tin, typename Tout, bool Q8>
__global__ void __launch_bounds__(64) rms_fwd_kernel(const RmsParams p) {
  const int64_t row = blockIdx.x, base = row * p.dim;
  const int lane = threadIdx.x;
  const Tin *x = static_cast<const Tin *>(p.x), *res = static_cast<const Tin *>(p.residual);
  auto sum_at = [&](int64_t c) { return ld(x, base + c) + (res != nullptr ? ld(res, base + c) : 0.0f); };
  float ss = 0.0f;
  for (int64_t c = lane; c < p.dim; c += 64) {
    const float s = sum_at(c);
    ss = fmaf(s, s, ss);
  }
  const float rstd = 1.0f / sqrtf(wave_sum(ss) / static_cast<float>(p.dim) + p.eps);
  if constexpr (Q8) {
    const int64_t ngroup = (p.dim + p.group - 1) / p.group;
    for (int64_t g = 0; g < ngroup; ++g) {
      const int64_t lo = g * p.group, hi = lo + p.group < p.dim ? lo + p.group : p.dim;
      float top = 0.0f;
      for (int64_t c = lo + lane; c < hi; c += 64) top = amax(top, sum_at(c) * rstd * p.w[c]);
      const float scale = wave_amax(top) / 448.0f;
      if (lane == 0) p.scale[row * ngroup + g] = scale;
      for (int64_t c = lo + lane; c < hi; c += 64) {
        const float v = sum_at(c) * rstd * p.w[c] / (scale > 0.0f ? scale : 1.0f);
        static_cast<uint8_t *>(p.y)[base + c] = to_e4m3(v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v);
      }
    }
  }
  for (int64_t c = lane; c < p.dim; c += 64) {
    const float s = sum_at(c);
    if (p.residual_out != nullptr) st(static_cast<Tin *>(p.residual_out), base + c, s);
    if constexpr (!Q8) st(static_cast<Tout *>(p.y), base + c, s * rstd * p.w[c]);
  }
}

template <typename Tin>
__global__ void __launch_bounds__(64) rms_bwd_kernel(const RmsBwdParams p) {
  const int lane = threadIdx.x;
  const Tin *dy = static_cast<const Tin *>(p.dy), *s = static_cast<const Tin *>(p.s);
  const Tin *dres = static_cast<const Tin *>(p.dres);
  float *part = p.ws + static_cast<int64_t>(blockIdx.x) * p.dim;
  if (p.dw != nullptr)
    for (int64_t c = lane; c < p.dim; c += 64) part[c] = 0.0f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t base = row * p.dim;
    float ss = 0.0f, dot = 0.0f;
    for (int64_t c = lane; c < p.dim; c += 64) {
      const float v = ld(s, base + c);
      ss = fmaf(v, v, ss);
      dot = fmaf(ld(dy, base + c) * p.w[c], v, dot);
    }
    const float inv = 1.0f / static_cast<float>(p.dim);
    const float rstd = 1.0f / sqrtf(wave_sum(ss) * inv + p.eps);
    const float mean = wave_sum(dot) * rstd * inv;
    for (int64_t c = lane; c < p.dim; c += 64) {
      const float n = ld(s, base + c) * rstd, d = ld(dy, base + c);
      const float r = dres != nullptr ? ld(dres, base + c) : 0.0f;
      st(static_cast<Tin *>(p.dx), base + c, fmaf(rstd, d * p.w[c] - n * mean, r));
      if (p.dw != nullptr) part[c] = fmaf(d, n, part[c]);
    }
  }
}

__global__ void __launch_bounds__(256) rms_sum_kernel(const float *part, float *dw, int64_t parts, int64_t dim) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= dim) return;
  float s = 0.0f;
  for (int64_t k = 0; k < parts; ++k) s += part[k * dim + c];
  dw[c] = s;
}

}  // namespace

hipError_t launch_rms(const RmsParams &p, int in_bf16, int out_bf16, hipStream_t st) {
  const dim3 g(static_cast<uint32_t>(p.rows)), t(64);
  if (p.scale != nullptr) {
    if (in_bf16) hipLaunchKernelGGL((rms_fwd_kernel<uint16_t, uint16_t, true>), g, t, 0, st, p);
    else hipLaunchKernelGGL((rms_fwd_kernel<float, float, true>), g, t, 0, st, p);
  } else if (in_bf16 && out_bf16) hipLaunchKernelGGL((rms_fwd_kernel<uint16_t, uint16_t, false>), g, t, 0, st, p);
  else if (in_bf16) hipLaunchKernelGGL((rms_fwd_kernel<uint16_t, float, false>), g, t, 0, st, p);
  else if (out_bf16) hipLaunchKernelGGL((rms_fwd_kernel<float, uint16_t, false>), g, t, 0, st, p);
  else hipLaunchKernelGGL((rms_fwd_kernel<float, float, false>), g, t, 0, st, p);
  return hipGetLastError();
}

int64_t rms_bwd_parts(int64_t rows, int64_t) { return rows < 1024 ? rows : 1024; }

hipError_t launch_rms_bwd(const RmsBwdParams &p, int in_bf16, hipStream_t st) {
  const dim3 g(static_cast<uint32_t>(p.parts)), t(64);
  if (p.rows > 0) {
    if (in_bf16) hipLaunchKernelGGL((rms_bwd_kernel<uint16_t>), g, t, 0, st, p);
    else hipLaunchKernelGGL((rms_bwd_kernel<float>), g, t, 0, st, p);
  }
  if (p.dw != nullptr)
    hipLaunchKernelGGL(rms_sum_kernel, dim3(static_cast<uint32_t>((p.dim + 255) / 256)), dim3(256), 0, st, p.ws, p.dw,
                       p.parts, p.dim);
  return hipGetLastError();
}

}  // namespace ssmb
