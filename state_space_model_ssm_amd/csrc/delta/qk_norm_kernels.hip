// Norms of queries and keys for each head, with the rotation by position in
// the same pass, and their backward, for gfx950.
//
// Bound by memory: an element is read once and written once.  A head is 16
// elements per lane, in two pieces of 8 that hold the two elements of each
// pair that is rotated together; a workgroup takes all of q's heads of a few
// tokens, or all of k's, whose sines and cosines it makes once, in LDS.  (One
// that took both kept two sets of weights and of their gradients in registers:
// 170 in the backward, now 131.)  The angle pos * inv_freq is
// taken in float64 and reduced to a fraction of a turn there: in float32 a
// position of 10^6 would have lost a sixteenth of a radian.
//
// Measured: 32749 tokens of 16 and 4 heads of 128 in 68 us, 4.9 TB/s of what is
// read and written (a large copy: 4.8); training's 8192 tokens of 32 and 8 heads
// of 64 forward in 17.9 us (4.7 TB/s), backward in 27.0 (4.7) and the sum of the
// weights' gradients in 4.0, which is the latency of two reads; one token of 32
// sequences in 4.2 us.
#include "delta_internal.h"

namespace ssmb {
namespace {

typedef __attribute__((ext_vector_type(4))) unsigned int u4;
typedef __attribute__((ext_vector_type(4))) float f4;
constexpr int kMaxTile = 16;   // tokens
constexpr int kMaxPairs = 128;

// Eight elements as they lie in memory, and as numbers.
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  u4 v;
  __device__ __forceinline__ void load(const uint16_t *p) { v = *reinterpret_cast<const u4 *>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(v[k] << 16);
      x[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
    }
  }
};
template <>
struct Eight<float> {
  f4 v[2];
  __device__ __forceinline__ void load(const float *p) {
#pragma unroll
    for (int k = 0; k < 2; ++k) v[k] = reinterpret_cast<const f4 *>(p)[k];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v[e / 4][e % 4];
  }
};
__device__ __forceinline__ void load8(float (&x)[8], const float *p) {
  Eight<float> v;
  v.load(p);
  v.get(x);
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

// What a workgroup works on: the first `nq` take q's heads, the others k's.
struct Side {
  bool key;
  int heads, tile;
  int64_t group, groups;  // its number among the workgroups of its side
  int64_t x_batch, x_token, y_batch, y_token;
};
__device__ __forceinline__ Side side_of(const QkNormParams &p) {
  const bool key = blockIdx.x >= p.nq;
  const unsigned nq = static_cast<unsigned>(p.nq);
  if (key) return {true, static_cast<int>(p.nkv), p.tile_k, blockIdx.x - nq, gridDim.x - nq, p.k_batch, p.k_token, p.ok_batch, p.ok_token};
  return {false, static_cast<int>(p.nheads), p.tile_q, blockIdx.x, nq, p.q_batch, p.q_token, p.oq_batch, p.oq_token};
}

struct Shared {
  float2 turn[kMaxTile][kMaxPairs];    // cosine and sine
  int64_t x[kMaxTile], y[kMaxTile];    // offsets of the tokens, of what is read and written
};

// Angles and offsets of tokens first .. first + count - 1.
__device__ __forceinline__ void begin(const QkNormParams &p, const Side &side, Shared &sh, int64_t first, int count) {
  const int tid = threadIdx.x, half = p.rot / 2;
  if (tid < count) {
    const int64_t b = (first + tid) / p.seqlen, t = (first + tid) % p.seqlen;
    sh.x[tid] = b * side.x_batch + t * side.x_token;
    sh.y[tid] = b * side.y_batch + t * side.y_token;
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
  const int tid = threadIdx.x, j = tid % G;
  const Side side = side_of(p);
  const Place at = place_of(p, j);
  const T *x = static_cast<const T *>(side.key ? p.k : p.q);
  T *y = static_cast<T *>(side.key ? p.out_k : p.out_q);
  const float *weights = side.key ? p.wk : p.wq;
  float w[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[0][e] = w[1][e] = 1.0f;
  if (weights != nullptr) load8(w[0], weights + at.lo), load8(w[1], weights + at.hi);
  const float mean = 1.0f / static_cast<float>(p.headdim);
  for (int64_t first = side.group * side.tile; first < p.tokens; first += side.groups * side.tile) {
    const int count = p.tokens - first < side.tile ? static_cast<int>(p.tokens - first) : side.tile;
    begin(p, side, sh, first, count);
    __syncthreads();
    const int rows = count * side.heads;
    // A row's elements are on their way while the one before is worked on.
    Eight<T> next[2];
    auto fetch = [&](int row) {
      row = row < rows ? row : rows - 1;
      const T *from = x + sh.x[row / side.heads] + static_cast<int64_t>(row % side.heads) * p.headdim;
      next[0].load(from + at.lo);
      next[1].load(from + at.hi);
    };
    fetch(tid / G);
    for (int row = tid / G; row < rows; row += 256 / G) {
      const int t = row / side.heads;
      float lo[8], hi[8], sum = 0.0f;
      next[0].get(lo);
      next[1].get(hi);
      fetch(row + 256 / G);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], sum));
      sum = sum_lanes<G>(at.live ? sum : 0.0f);
      const float rstd = 1.0f / sqrtf(fmaf(sum, mean, p.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] *= rstd * w[0][e];
        hi[e] *= rstd * w[1][e];
      }
      if (at.turns) rotate<NEIGHBOURS, 1>(lo, hi, sh.turn[t] + at.pair);
      if (at.live) {
        T *to = y + sh.y[t] + static_cast<int64_t>(row % side.heads) * p.headdim;
        store8(lo, to + at.lo);
        store8(hi, to + at.hi);
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
  __shared__ float part[256 * 8];  // a piece of every thread
  const int tid = threadIdx.x, j = tid % G;
  const Side side = side_of(p);
  const Place at = place_of(p, j);
  const T *x = static_cast<const T *>(side.key ? p.k : p.q), *dy = static_cast<const T *>(side.key ? p.dyk : p.dyq);
  T *dx = static_cast<T *>(side.key ? p.out_k : p.out_q);
  const float *weights = side.key ? p.wk : p.wq;
  float w[2][8], dw[2][8] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e) w[0][e] = w[1][e] = 1.0f;
  if (weights != nullptr) load8(w[0], weights + at.lo), load8(w[1], weights + at.hi);
  const float mean = 1.0f / static_cast<float>(p.headdim);
  for (int64_t first = side.group * side.tile; first < p.tokens; first += side.groups * side.tile) {
    const int count = p.tokens - first < side.tile ? static_cast<int>(p.tokens - first) : side.tile;
    begin(p, side, sh, first, count);
    __syncthreads();
    const int rows = count * side.heads;
    Eight<T> next[4];  // x and its output's gradient, as in the forward
    auto fetch = [&](int row) {
      row = row < rows ? row : rows - 1;
      const T *from = x + sh.x[row / side.heads] + static_cast<int64_t>(row % side.heads) * p.headdim;
      const T *grad = dy + (first * side.heads + row) * p.headdim;
      next[0].load(from + at.lo);
      next[1].load(from + at.hi);
      next[2].load(grad + at.lo);
      next[3].load(grad + at.hi);
    };
    fetch(tid / G);
    for (int row = tid / G; row < rows; row += 256 / G) {
      const int t = row / side.heads;
      float lo[8], hi[8], dlo[8], dhi[8], sum = 0.0f;
      next[0].get(lo);
      next[1].get(hi);
      next[2].get(dlo);
      next[3].get(dhi);
      fetch(row + 256 / G);
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
        dw[0][e] = fmaf(dlo[e], lo[e], dw[0][e]);
        dw[1][e] = fmaf(dhi[e], hi[e], dw[1][e]);
        dlo[e] *= w[0][e];
        dhi[e] *= w[1][e];
        dot = fmaf(dlo[e], lo[e], fmaf(dhi[e], hi[e], dot));
      }
      dot = sum_lanes<G>(at.live ? dot : 0.0f) * mean;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] = rstd * fmaf(-lo[e], dot, dlo[e]);
        hi[e] = rstd * fmaf(-hi[e], dot, dhi[e]);
      }
      if (at.live) {
        T *to = dx + sh.y[t] + static_cast<int64_t>(row % side.heads) * p.headdim;
        store8(lo, to + at.lo);
        store8(hi, to + at.hi);
      }
    }
    __syncthreads();
  }
  if (p.ws == nullptr) return;
  // The groups' terms, one piece at a time, in a fixed order.
  constexpr int N = 256 / G;
#pragma unroll
  for (int piece = 0; piece < 2; ++piece) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[tid * 8 + e] = dw[piece][e];
    __syncthreads();
    if (tid < 8 * G && 16 * (tid / 8) < p.headdim) {
      float sum = 0.0f;
      for (int k = 0; k < N; ++k) sum += part[k * 8 * G + tid];
      const Place to = place_of(p, tid / 8);
      p.ws[static_cast<int64_t>(blockIdx.x) * p.headdim + (piece != 0 ? to.hi : to.lo) + tid % 8] = sum;
    }
    __syncthreads();
  }
}

// dw = the sum over the workgroups' terms: 16 columns by 64 threads of a share each.
__global__ void __launch_bounds__(1024) qk_norm_sum_kernel(const QkNormParams p, int nk) {
  __shared__ float sums[64][17];
  const int tiles = p.headdim / 16;
  const bool key = static_cast<int>(blockIdx.x) >= tiles;
  const int c = threadIdx.x % 16, k = threadIdx.x / 16, col = (blockIdx.x - (key ? tiles : 0)) * 16 + c;
  float *to = key ? p.dwk : p.dwq;
  if (to == nullptr) return;
  const int64_t parts = key ? nk : p.nq;
  const float *from = p.ws + (key ? p.nq * p.headdim : 0) + col;
  float sum = 0.0f;
  for (int64_t i = k; i < parts; i += 64) sum += from[i * p.headdim];
  sums[k][c] = sum;
  __syncthreads();
  if (k >= 4) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) sum += sums[16 * k + i][c];
  sum += __shfl_down(sum, 32);
  sum += __shfl_down(sum, 16);
  if (k == 0) to[col] = sum;
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

// Lanes of 16 elements that share a head.
int lanes_of(int64_t headdim) { return headdim > 128 ? 16 : headdim > 64 ? 8 : headdim > 32 ? 4 : 2; }

template <typename T>
void run(const QkNormParams &p, bool bwd, unsigned groups, hipStream_t s) {
  switch (lanes_of(p.headdim)) {
    case 16: run<T, 16>(p, bwd, groups, s); break;
    case 8: run<T, 8>(p, bwd, groups, s); break;
    case 4: run<T, 4>(p, bwd, groups, s); break;
    default: run<T, 2>(p, bwd, groups, s);
  }
}

// Tokens that a workgroup takes at a time: as many as its lanes have heads for,
// and up to four times those while 512 workgroups are left, which share the
// work of a workgroup's beginning.  Forward of 16 and 4 heads of 128: 512 tokens
// take 6.1 us, with 8 at a time 10.5; 8192 take 26.8, with 1 at a time 30.6.
int tile_of(int64_t tokens, int64_t heads, int64_t headdim) {
  const int64_t rows = 256 / lanes_of(headdim), most = tokens / 512;
  int tile = 1;
  while (tile < kMaxTile && (2 * tile * heads <= rows || (2 * tile * heads <= 4 * rows && 2 * tile <= most))) tile *= 2;
  return tile;
}

}  // namespace

QkNormGroups qk_norm_groups(int64_t tokens, int64_t nheads, int64_t nkv, int64_t headdim, bool bwd) {
  QkNormGroups n;
  n.tile_q = tile_of(tokens, nheads, headdim);
  n.tile_k = tile_of(tokens, nkv, headdim);
  const int64_t tq = (tokens + n.tile_q - 1) / n.tile_q, tk = (tokens + n.tile_k - 1) / n.tile_k;
  // The backward's workgroups each leave a term of dw.  768 are there at once
  // (2048 tokens of 16 and 4 heads of 128: 13.6 us, with at most 512 17.6); what
  // takes more goes round in 512 (4096 tokens of 64 and 8: 78 us, in 768 80; the
  // sum of their terms 4.7, of 1024 6.8).
  const int64_t most = bwd ? (tq + tk <= 768 ? 768 : 512) : int64_t{1} << 21;
  // Shares by the heads: a workgroup of either side has about the same rows.
  const int64_t share = most * nheads / (nheads + nkv), mq = share < 1 ? 1 : share < most ? share : most - 1;
  n.q = tq + tk <= most || tq < mq ? tq : mq;
  n.k = tq + tk <= most || tk < most - mq ? tk : most - mq;
  return n;
}

namespace {
hipError_t launch(const QkNormParams &p0, int bf16, bool bwd, hipStream_t s) {
  QkNormParams p = p0;
  const QkNormGroups n = qk_norm_groups(p.tokens, p.nheads, p.nkv, p.headdim, bwd);
  p.nq = n.q;
  p.tile_q = n.tile_q;
  p.tile_k = n.tile_k;
  const unsigned groups = static_cast<unsigned>(n.q + n.k);
  if (groups > 0) bf16 ? run<uint16_t>(p, bwd, groups, s) : run<float>(p, bwd, groups, s);
  if (p.dwq != nullptr || p.dwk != nullptr)  // (without tokens, too: zeros)
    hipLaunchKernelGGL(qk_norm_sum_kernel, dim3(static_cast<uint32_t>(2 * p.headdim / 16)), dim3(1024), 0, s, p, static_cast<int>(n.k));
  return hipGetLastError();
}
}  // namespace

hipError_t launch_qk_norm(const QkNormParams &p, int bf16, hipStream_t s) { return launch(p, bf16, false, s); }
hipError_t launch_qk_norm_bwd(const QkNormParams &p, int bf16, hipStream_t s) { return launch(p, bf16, true, s); }

}  // namespace ssmb
