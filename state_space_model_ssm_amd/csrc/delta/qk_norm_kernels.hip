// Norms of queries and keys for each head, with the rotation by position in
// the same pass, and their backward, for gfx950.
//
// Bound by memory: an element is read once and written once.  A head is 16
// elements per lane, in two pieces of 8 that hold the two elements of each
// pair that is rotated together; a workgroup takes all heads of a few tokens,
// whose sines and cosines it makes once, in LDS.  The angle pos * inv_freq is
// taken in float64 and reduced to a fraction of a turn there: in float32 a
// position of 10^6 would have lost a sixteenth of a radian.
#include "delta_internal.h"

namespace ssmb {
namespace {

typedef __attribute__((ext_vector_type(4))) unsigned int u4;
typedef __attribute__((ext_vector_type(4))) float f4;
constexpr int kMaxTile = 8;    // tokens
constexpr int kMaxPairs = 128;

__device__ __forceinline__ void load8(float (&x)[8], const uint16_t *p) {
  const u4 v = *reinterpret_cast<const u4 *>(p);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(v[k] << 16);
    x[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(float (&x)[8], const float *p) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const f4 v = reinterpret_cast<const f4 *>(p)[k];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * k + e] = v[e];
  }
}
__device__ __forceinline__ void store8(const float (&x)[8], uint16_t *p) {
  typedef __attribute__((ext_vector_type(8))) __bf16 bf8;
  bf8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = static_cast<__bf16>(x[e]);
  *reinterpret_cast<bf8 *>(p) = v;
}
__device__ __forceinline__ void store8(const float (&x)[8], float *p) {
#pragma unroll
  for (int k = 0; k < 2; ++k) reinterpret_cast<f4 *>(p)[k] = f4{x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]};
}

// The sum over the G lanes (a power of two, at most 16) that share a head.
template <int G>
__device__ __forceinline__ float sum_lanes(float v) {
  if constexpr (G > 1) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, true));
  if constexpr (G > 2) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, true));
  if constexpr (G > 4) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));
  if constexpr (G > 8) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, true));
  return v;
}

// Where lane j's two pieces lie in a head, and the first of its pairs.
struct Place {
  int lo, hi, pair;
  bool live, turns;
};
__device__ __forceinline__ Place place_of(const QkNormParams &p, int j) {
  Place at;
  at.live = 16 * j < p.headdim;
  at.turns = 16 * j < p.rot;
  at.pair = 8 * j;
  if (at.turns && !p.neighbours) {
    at.lo = 8 * j;
    at.hi = p.rot / 2 + 8 * j;
  } else {
    at.lo = 16 * j;
    at.hi = 16 * j + 8;
  }
  if (!at.live) at.lo = at.hi = 0;
  return at;
}

// Rotate the lane's pairs by the token's angles (SIGN -1: back).
template <bool NEIGHBOURS, int SIGN>
__device__ __forceinline__ void rotate(float (&lo)[8], float (&hi)[8], const float2 *turn) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 cs = turn[k];
    const float s = SIGN * cs.y;
    float &a = NEIGHBOURS ? (k < 4 ? lo[2 * (k % 4)] : hi[2 * (k % 4)]) : lo[k];
    float &b = NEIGHBOURS ? (k < 4 ? lo[2 * (k % 4) + 1] : hi[2 * (k % 4) + 1]) : hi[k];
    const float x = a, y = b;
    a = x * cs.x - y * s;
    b = y * cs.x + x * s;
  }
}

struct Shared {
  float2 turn[kMaxTile][kMaxPairs];  // cosine and sine
  int64_t q[kMaxTile], k[kMaxTile], oq[kMaxTile], ok[kMaxTile];  // offsets of the tokens
};

// Angles and offsets of tokens first .. first + count - 1.
__device__ __forceinline__ void begin(const QkNormParams &p, Shared &sh, int64_t first, int count) {
  const int tid = threadIdx.x, half = p.rot / 2;
  if (tid < count) {
    const int64_t b = (first + tid) / p.seqlen, t = (first + tid) % p.seqlen;
    sh.q[tid] = b * p.q_batch + t * p.q_token;
    sh.k[tid] = b * p.k_batch + t * p.k_token;
    sh.oq[tid] = b * p.oq_batch + t * p.oq_token;
    sh.ok[tid] = b * p.ok_batch + t * p.ok_token;
  }
  for (int i = tid; i < count * half; i += 256) {
    const int t = i / half, f = i % half;
    const double pos = p.pos != nullptr ? static_cast<double>(p.pos[first + t]) : static_cast<double>((first + t) % p.seqlen);
    const double turns = pos * (static_cast<double>(p.inv_freq[f]) * 0.15915494309189533577);
    float s, c;
    sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
    sh.turn[t][f] = make_float2(c, s);
  }
}

// G lanes share a head of 16 G elements or fewer.
template <typename T, int G, bool NEIGHBOURS>
__global__ void __launch_bounds__(256) qk_norm_kernel(const QkNormParams p) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, j = tid % G, heads = static_cast<int>(p.nheads + p.nkv);
  const Place at = place_of(p, j);
  float wq[2][8], wk[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) wq[0][e] = wq[1][e] = wk[0][e] = wk[1][e] = 1.0f;
  if (p.wq != nullptr) load8(wq[0], p.wq + at.lo), load8(wq[1], p.wq + at.hi);
  if (p.wk != nullptr) load8(wk[0], p.wk + at.lo), load8(wk[1], p.wk + at.hi);
  const float mean = 1.0f / static_cast<float>(p.headdim);
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * p.tile; first < p.tokens; first += static_cast<int64_t>(gridDim.x) * p.tile) {
    const int count = p.tokens - first < p.tile ? static_cast<int>(p.tokens - first) : p.tile;
    begin(p, sh, first, count);
    __syncthreads();
    const int rows = count * heads;
    for (int row0 = 0; row0 < rows; row0 += 256 / G) {
      const int row = row0 + tid / G;
      if (row >= rows) continue;
      const int t = row / heads, h = row % heads;
      const bool key = h >= p.nheads;
      const int64_t head = static_cast<int64_t>(key ? h - p.nheads : h) * p.headdim;
      const T *x = key ? static_cast<const T *>(p.k) + sh.k[t] + head : static_cast<const T *>(p.q) + sh.q[t] + head;
      float lo[8], hi[8], sum = 0.0f;
      load8(lo, x + at.lo);
      load8(hi, x + at.hi);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], sum));
      sum = sum_lanes<G>(at.live ? sum : 0.0f);
      const float rstd = 1.0f / sqrtf(fmaf(sum, mean, p.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] *= rstd * (key ? wk[0][e] : wq[0][e]);
        hi[e] *= rstd * (key ? wk[1][e] : wq[1][e]);
      }
      if (at.turns) rotate<NEIGHBOURS, 1>(lo, hi, sh.turn[t] + at.pair);
      if (at.live) {
        T *y = key ? static_cast<T *>(p.out_k) + sh.ok[t] + head : static_cast<T *>(p.out_q) + sh.oq[t] + head;
        store8(lo, y + at.lo);
        store8(hi, y + at.hi);
      }
    }
    __syncthreads();
  }
}

// With n = x rstd and the gradient dn of n w after the rotation is taken back:
// dw = sum of dn n, dx = rstd (dn w - n mean(dn w n)).
template <typename T, int G, bool NEIGHBOURS>
__global__ void __launch_bounds__(256) qk_norm_bwd_kernel(const QkNormParams p) {
  __shared__ Shared sh;
  __shared__ float part[256 / G * 16 * G / 2];  // (wavefronts' halves in turn) [group][16 G]
  const int tid = threadIdx.x, j = tid % G, heads = static_cast<int>(p.nheads + p.nkv);
  const Place at = place_of(p, j);
  float w[2][2][8], dw[2][2][8] = {};  // [q or k][piece]
#pragma unroll
  for (int e = 0; e < 8; ++e) w[0][0][e] = w[0][1][e] = w[1][0][e] = w[1][1][e] = 1.0f;
  if (p.wq != nullptr) load8(w[0][0], p.wq + at.lo), load8(w[0][1], p.wq + at.hi);
  if (p.wk != nullptr) load8(w[1][0], p.wk + at.lo), load8(w[1][1], p.wk + at.hi);
  const float mean = 1.0f / static_cast<float>(p.headdim);
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * p.tile; first < p.tokens; first += static_cast<int64_t>(gridDim.x) * p.tile) {
    const int count = p.tokens - first < p.tile ? static_cast<int>(p.tokens - first) : p.tile;
    begin(p, sh, first, count);
    __syncthreads();
    const int rows = count * heads;
    for (int row0 = 0; row0 < rows; row0 += 256 / G) {
      const int row = row0 + tid / G;
      if (row >= rows) continue;
      const int t = row / heads, h = row % heads;
      const bool key = h >= p.nheads;
      const int64_t n = key ? h - p.nheads : h, head = n * p.headdim;
      const T *x = key ? static_cast<const T *>(p.k) + sh.k[t] + head : static_cast<const T *>(p.q) + sh.q[t] + head;
      const T *dy = key ? static_cast<const T *>(p.dyk) + ((first + t) * p.nkv + n) * p.headdim
                        : static_cast<const T *>(p.dyq) + ((first + t) * p.nheads + n) * p.headdim;
      float lo[8], hi[8], dlo[8], dhi[8], sum = 0.0f;
      load8(lo, x + at.lo);
      load8(hi, x + at.hi);
      load8(dlo, dy + at.lo);
      load8(dhi, dy + at.hi);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], sum));
      sum = sum_lanes<G>(at.live ? sum : 0.0f);
      const float rstd = 1.0f / sqrtf(fmaf(sum, mean, p.eps));
      if (at.turns) rotate<NEIGHBOURS, -1>(dlo, dhi, sh.turn[t] + at.pair);
      float dot = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] *= rstd;
        hi[e] *= rstd;
        const float a = dlo[e] * lo[e], b = dhi[e] * hi[e];
        dw[0][0][e] += key ? 0.0f : a;
        dw[0][1][e] += key ? 0.0f : b;
        dw[1][0][e] += key ? a : 0.0f;
        dw[1][1][e] += key ? b : 0.0f;
        dlo[e] *= key ? w[1][0][e] : w[0][0][e];
        dhi[e] *= key ? w[1][1][e] : w[0][1][e];
        dot = fmaf(dlo[e], lo[e], fmaf(dhi[e], hi[e], dot));
      }
      dot = sum_lanes<G>(at.live ? dot : 0.0f) * mean;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] = rstd * fmaf(-lo[e], dot, dlo[e]);
        hi[e] = rstd * fmaf(-hi[e], dot, dhi[e]);
      }
      if (at.live) {
        T *dx = key ? static_cast<T *>(p.out_k) + sh.ok[t] + head : static_cast<T *>(p.out_q) + sh.oq[t] + head;
        store8(lo, dx + at.lo);
        store8(hi, dx + at.hi);
      }
    }
    __syncthreads();
  }
  if (p.ws == nullptr) return;
  // The groups' terms, one piece at a time, in a fixed order.
  constexpr int N = 256 / G;
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int piece = 0; piece < 2; ++piece) {
#pragma unroll
      for (int e = 0; e < 8; ++e) part[tid * 8 + e] = dw[x][piece][e];
      __syncthreads();
      if (tid < 8 * G && 16 * (tid / 8) < p.headdim) {
        float sum = 0.0f;
        for (int k = 0; k < N; ++k) sum += part[k * 8 * G + tid];
        const Place to = place_of(p, tid / 8);
        p.ws[(static_cast<int64_t>(blockIdx.x) * 2 + x) * p.headdim + (piece != 0 ? to.hi : to.lo) + tid % 8] = sum;
      }
      __syncthreads();
    }
}

// dw = the sum over the workgroups' terms: 16 columns by 64 threads of a share each.
__global__ void __launch_bounds__(1024) qk_norm_sum_kernel(const QkNormParams p, int parts) {
  __shared__ float sums[64][17];
  const int c = threadIdx.x % 16, k = threadIdx.x / 16, col = blockIdx.x * 16 + c;
  const int64_t step = 2 * p.headdim;
  float sum = 0.0f;
  for (int i = k; i < parts; i += 64) sum += p.ws[i * step + col];
  sums[k][c] = sum;
  __syncthreads();
  if (k >= 4) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) sum += sums[16 * k + i][c];
  sum += __shfl_down(sum, 32);
  sum += __shfl_down(sum, 16);
  if (k != 0) return;
  float *to = col < p.headdim ? p.dwq : p.dwk;
  if (to != nullptr) to[col % p.headdim] = sum;
}

template <typename T, int G>
void run(const QkNormParams &p, bool bwd, unsigned groups, hipStream_t s) {
  const dim3 g(groups), t(256);
  if (bwd) {
    if (p.neighbours) hipLaunchKernelGGL((qk_norm_bwd_kernel<T, G, true>), g, t, 0, s, p);
    else hipLaunchKernelGGL((qk_norm_bwd_kernel<T, G, false>), g, t, 0, s, p);
  } else {
    if (p.neighbours) hipLaunchKernelGGL((qk_norm_kernel<T, G, true>), g, t, 0, s, p);
    else hipLaunchKernelGGL((qk_norm_kernel<T, G, false>), g, t, 0, s, p);
  }
}

template <typename T>
void run(const QkNormParams &p, bool bwd, unsigned groups, hipStream_t s) {
  if (p.headdim > 128) run<T, 16>(p, bwd, groups, s);
  else if (p.headdim > 64) run<T, 8>(p, bwd, groups, s);
  else if (p.headdim > 32) run<T, 4>(p, bwd, groups, s);
  else run<T, 2>(p, bwd, groups, s);
}

// Tokens that a workgroup takes at a time: one where there are few, so that
// all of the chip has some; more share the work of a workgroup's beginning.
int tile_of(int64_t tokens) { return tokens >= 16384 ? kMaxTile : tokens >= 4096 ? 2 : 1; }

}  // namespace

// Workgroups of the backward, and so the terms of dwq and dwk.
int64_t qk_norm_parts(int64_t tokens) {
  const int64_t n = (tokens + tile_of(tokens) - 1) / tile_of(tokens);
  return n < 1024 ? n : 1024;
}

hipError_t launch_qk_norm(const QkNormParams &p0, int bf16, hipStream_t s) {
  QkNormParams p = p0;
  p.tile = tile_of(p.tokens);
  const int64_t n = (p.tokens + p.tile - 1) / p.tile;
  const unsigned groups = static_cast<unsigned>(n < (1 << 20) ? n : 1 << 20);
  bf16 ? run<uint16_t>(p, false, groups, s) : run<float>(p, false, groups, s);
  return hipGetLastError();
}

hipError_t launch_qk_norm_bwd(const QkNormParams &p0, int bf16, hipStream_t s) {
  QkNormParams p = p0;
  p.tile = tile_of(p.tokens);
  const int parts = static_cast<int>(qk_norm_parts(p.tokens));
  if (parts > 0) bf16 ? run<uint16_t>(p, true, static_cast<unsigned>(parts), s) : run<float>(p, true, static_cast<unsigned>(parts), s);
  if (p.dwq != nullptr || p.dwk != nullptr)  // (without tokens, too: zeros)
    hipLaunchKernelGGL(qk_norm_sum_kernel, dim3(static_cast<uint32_t>(2 * p.headdim / 16)), dim3(1024), 0, s, p, parts);
  return hipGetLastError();
}

}  // namespace ssmb
