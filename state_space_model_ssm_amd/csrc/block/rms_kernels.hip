// Residual addition with RMS norm for gfx950: y = s / sqrt(mean(s^2) + eps) w
// with s = x + residual, in storage types or in e4m3 bytes with scales, and
// its backward.
//
// All of it is bound by memory: a row is read once into registers (16 bytes
// per lane and load, by 16 or 64 lanes or the whole workgroup, whichever
// leaves a lane the fewest idle loads), summed across its lanes, and written:
// 16384 x 2048 bfloat16, out of the caches, forward 52 us (5.2 TB/s), backward
// 48; in 8 bits 16384 x 5120 131 us (4.5 TB/s).
// Workgroups walk rows with w in registers, and with the backward's sums over
// rows for dw, which they write once each; a second launch adds those in
// order.  Where rows do not start on 16 bytes the same loads start at any value
// (16384 x 2047 bfloat16, a call forward and one backward: 110 us against 108
// for 2048; value by value they were 203).  Rows too short or too long for that,
// and groups that fit no lanes, go value by value, the forward's through LDS, or
// are read again per pass if they are too long for LDS.
#include "block_internal.h"

namespace ssmb {
namespace {

// Sum over the TPR lanes of a row (in one wavefront, or the workgroup's four
// through `lds`, which nobody else uses until the next barrier but one).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *lds) {
#pragma unroll
  for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) v += __shfl_xor(v, m);
  if constexpr (TPR == 256) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  }
  return v;
}

// The larger of a and |b|, NaN if either is one.
__device__ __forceinline__ float amax(float a, float b) {
  const float c = fabsf(b);
  return (a != a || a > c) ? a : c;
}

// amax over `lanes` neighbours, a power of two up to 64.
__device__ __forceinline__ float lanes_amax(float v, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) v = amax(v, __shfl_xor(v, m));
  return v;
}

// Values of a group are divided by its scale as (v * lift) * inverse: lift
// keeps the inverse of a tiny scale finite.  A scale of 0 (whose values are
// all 0) counts as 1.
__device__ __forceinline__ float lift(float scale) { return scale < 0x1p-90f ? 0x1p90f : 1.0f; }
__device__ __forceinline__ float inverse(float scale) { return 1.0f / (scale != 0.0f ? scale * lift(scale) : 1.0f); }

// Two values within +-448 (or NaN) as e4m3 bytes, rounded to nearest even.
// (A value can pass 448 by the rounding of the scale; it is held there.)
__device__ __forceinline__ float hold(float v) { return v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v; }
__device__ __forceinline__ int to_e4m3(float a, float b, int old, bool high) {
  return high ? __builtin_amdgcn_cvt_pk_fp8_f32(hold(a), hold(b), old, true)
              : __builtin_amdgcn_cvt_pk_fp8_f32(hold(a), hold(b), old, false);
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf2;
  const bf2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}

// V values of a row in a lane, as words in loads of up to 16 bytes that start
// at any value if LOOSE.
template <int N, int ALIGN>
struct Words {
  typedef unsigned type __attribute__((ext_vector_type(N), aligned(ALIGN)));
};
template <typename E, int V, bool LOOSE>
struct Piece {
  static constexpr int kWords = V * sizeof(E) / 4, kAtOnce = kWords < 4 ? kWords : 4;
  typedef typename Words<kAtOnce, LOOSE ? sizeof(E) : 4 * kAtOnce>::type type;
  __device__ static __forceinline__ void get(const void *from, int64_t at, float (&f)[V]) {
    const type *p = reinterpret_cast<const type *>(static_cast<const E *>(from) + at);
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const unsigned v = p[k / kAtOnce][k % kAtOnce];
      if constexpr (sizeof(E) == 4) {
        f[k] = __uint_as_float(v);
      } else {
        f[2 * k] = __uint_as_float(v << 16);
        f[2 * k + 1] = __uint_as_float(v & 0xffff0000u);
      }
    }
  }
  __device__ static __forceinline__ void put(void *to, int64_t at, const float (&f)[V]) {
    type *p = reinterpret_cast<type *>(static_cast<E *>(to) + at);
#pragma unroll
    for (int k = 0; k < kWords; k += kAtOnce) {
      type v;
#pragma unroll
      for (int n = 0; n < kAtOnce; ++n) {
        if constexpr (sizeof(E) == 4) v[n] = __float_as_uint(f[k + n]);
        else v[n] = pack(f[2 * (k + n)], f[2 * (k + n) + 1]);
      }
      p[k / kAtOnce] = v;
    }
  }
};

// Where piece k of a row starts.  LOOSE: the last piece ends with the row, and
// takes over values of the piece before it where the row is no multiple of V:
// both lanes then write the same, and sums leave the first seen() out.
template <int V, bool LOOSE>
__device__ __forceinline__ int piece_at(int k, int dim) {
  return LOOSE && k * V > dim - V ? dim - V : k * V;
}
template <int V, bool LOOSE>
__device__ __forceinline__ int seen(int k, int at) {
  int n = k * V - at;
  if constexpr (!LOOSE) return 0;
  asm volatile("" : "+v"(n));  // comparisons with it are not to be kept across rows: they would take 128 scalar registers
  return n;
}

// Rows in registers: piece n of lane l is piece l + TPR n of the row.
// Q8: groups are the row or 2^k neighbouring lanes of a wavefront (group_lanes).
template <typename Tin, typename Tout, int TPR, int NV, bool Q8, bool LOOSE>
__global__ void __launch_bounds__(256) rms_rows_kernel(const RmsParams p, int group_lanes) {
  constexpr int V = 16 / sizeof(Tin), kRows = 256 / TPR;
  __shared__ float lds[2][2][4];
  const int l = threadIdx.x % TPR, dim = static_cast<int>(p.dim), pieces = (dim + V - 1) / V;
  const float inv = 1.0f / static_cast<float>(p.dim);
  float w[NV][V];
#pragma unroll
  for (int n = 0; n < NV; ++n)
    Piece<float, V, LOOSE>::get(p.w, piece_at<V, LOOSE>(l + TPR * n < pieces ? l + TPR * n : 0, dim), w[n]);
  int odd = 0;  // turns of the workgroup-wide sums' scratch
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < p.rows; first += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t row = first + threadIdx.x / TPR;
    const bool live = row < p.rows;
    const int64_t base = (live ? row : first) * p.dim;
    float s[NV][V], ss = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int k = l + TPR * n, at = piece_at<V, LOOSE>(k, dim);
#pragma unroll
      for (int e = 0; e < V; ++e) s[n][e] = 0.0f;
      if (k < pieces) {
        Piece<Tin, V, LOOSE>::get(p.x, base + at, s[n]);
        if (p.residual != nullptr) {
          float r[V];
          Piece<Tin, V, LOOSE>::get(p.residual, base + at, r);
#pragma unroll
          for (int e = 0; e < V; ++e) s[n][e] += r[e];
        }
      }
      const int skip = seen<V, LOOSE>(k, at);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float v = e < skip ? 0.0f : s[n][e];
        ss = fmaf(v, v, ss);
      }
    }
    const float rstd = 1.0f / sqrtf(fmaf(row_sum<TPR>(ss, lds[odd][0]), inv, p.eps));
    if (p.residual_out != nullptr && live) {
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (l + TPR * n < pieces) Piece<Tin, V, LOOSE>::put(p.residual_out, base + piece_at<V, LOOSE>(l + TPR * n, dim), s[n]);
    }
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < V; ++e) s[n][e] = s[n][e] * rstd * w[n][e];
    if constexpr (!Q8) {
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (l + TPR * n < pieces && live) Piece<Tout, V, LOOSE>::put(p.y, base + piece_at<V, LOOSE>(l + TPR * n, dim), s[n]);
    } else {
      float top[NV];
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        top[n] = 0.0f;
        if (l + TPR * n < pieces) {
#pragma unroll
          for (int e = 0; e < V; ++e) top[n] = amax(top[n], s[n][e]);
        }
      }
      if (group_lanes == 0) {  // the row
        float all = top[0];
#pragma unroll
        for (int n = 1; n < NV; ++n) all = amax(all, top[n]);
        all = lanes_amax(all, TPR < 64 ? TPR : 64);
        if constexpr (TPR == 256) {
          float *scratch = lds[odd][1];
          if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = all;
          __syncthreads();
          all = amax(amax(scratch[0], scratch[1]), amax(scratch[2], scratch[3]));
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) top[n] = all;
        if (l == 0 && live) p.scale[row] = all * (1.0f / 448.0f);
      } else {
        const int64_t ngroup = (p.dim + p.group - 1) / p.group;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          top[n] = lanes_amax(top[n], group_lanes);
          const int piece = l + TPR * n;
          if (piece < pieces && live && piece % group_lanes == 0)
            p.scale[row * ngroup + piece / group_lanes] = top[n] * (1.0f / 448.0f);
        }
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const float scale = top[n] * (1.0f / 448.0f), k = inverse(scale);
        if (scale < 0x1p-90f) {
#pragma unroll
          for (int e = 0; e < V; ++e) s[n][e] *= lift(scale);
        }
        if (l + TPR * n < pieces && live) {
          uint8_t *q = static_cast<uint8_t *>(p.y) + base + piece_at<V, LOOSE>(l + TPR * n, dim);
          int b[V / 4];
#pragma unroll
          for (int e = 0; e < V; e += 4) {
            b[e / 4] = to_e4m3(s[n][e] * k, s[n][e + 1] * k, 0, false);
            b[e / 4] = to_e4m3(s[n][e + 2] * k, s[n][e + 3] * k, b[e / 4], true);
          }
          typedef typename Words<V / 4, LOOSE ? 1 : V>::type bytes;
          bytes v;
#pragma unroll
          for (int n4 = 0; n4 < V / 4; ++n4) v[n4] = static_cast<unsigned>(b[n4]);
          *reinterpret_cast<bytes *>(q) = v;
        }
      }
    }
    odd ^= 1;
  }
}

// Rows that are read in a loop are summed in runs of 256 terms per thread, and
// the runs in float64: added up one by one in float32, equal values of a row of
// 2^27 moved the sum by a thousandth.
constexpr int64_t kRun = 256 * 256;
__device__ __forceinline__ int64_t run_end(int64_t run, int64_t dim) { return run + kRun < dim ? run + kRun : dim; }

// Rows of any alignment, a workgroup per row, through LDS (`keep`: the row's
// sums stay there between the passes) or, too long for that, read again.  Rows
// past kGridWidth go along the grid's other axis (workgroups that walk rows took
// 55 us against 49 for 32768 x 100 bfloat16 in 8 bits, groups of 32).
template <typename Tin, typename Tout, bool Q8>
__global__ void __launch_bounds__(256) rms_any_kernel(const RmsParams p, int keep) {
  extern __shared__ float held[];
  __shared__ float lds[4];
  const Tin *x = static_cast<const Tin *>(p.x), *res = static_cast<const Tin *>(p.residual);
  const int64_t row = static_cast<int64_t>(blockIdx.y) * kGridWidth + blockIdx.x, base = row * p.dim;
  if (row >= p.rows) return;
  auto sum_at = [&](int64_t c) { return ld(x, base + c) + (res != nullptr ? ld(res, base + c) : 0.0f); };
  auto squares = [&](int64_t c, int64_t end) {
    float ss = 0.0f;
    for (c += threadIdx.x; c < end; c += 256) {
      const float s = sum_at(c);
      if (keep) held[c] = s;
      ss = fmaf(s, s, ss);
    }
    return ss;
  };
  float ss = squares(0, run_end(0, p.dim));
  if (p.dim > kRun) {
    double total = ss;
    for (int64_t run = kRun; run < p.dim; run += kRun) total += squares(run, run_end(run, p.dim));
    ss = static_cast<float>(total);
  }
  const float rstd = 1.0f / sqrtf(fmaf(row_sum<256>(ss, lds), 1.0f / static_cast<float>(p.dim), p.eps));
  auto value = [&](int64_t c) { return keep ? held[c] : sum_at(c); };  // (row_sum() has a barrier)
  if constexpr (Q8) {
    // A wavefront per group in turn.
    const int lane = threadIdx.x & 63;
    const int64_t ngroup = (p.dim + p.group - 1) / p.group;
    for (int64_t g = threadIdx.x >> 6; g < ngroup; g += 4) {
      const int64_t lo = g * p.group, hi = lo + p.group < p.dim ? lo + p.group : p.dim;
      float top = 0.0f;
      for (int64_t c = lo + lane; c < hi; c += 64) top = amax(top, value(c) * rstd * p.w[c]);
      const float scale = lanes_amax(top, 64) * (1.0f / 448.0f), k = inverse(scale);
      if (lane == 0) p.scale[row * ngroup + g] = scale;
      for (int64_t c = lo + lane; c < hi; c += 64)
        static_cast<uint8_t *>(p.y)[base + c] =
            static_cast<uint8_t>(to_e4m3(value(c) * rstd * p.w[c] * lift(scale) * k, 0.0f, 0, false) & 0xff);
    }
    if (!keep) __syncthreads();  // residual_out may be x: every group has been read
  }
  for (int64_t c = threadIdx.x; c < p.dim; c += 256) {
    const float s = value(c);
    if (p.residual_out != nullptr) st(static_cast<Tin *>(p.residual_out), base + c, s);
    if constexpr (!Q8) st(static_cast<Tout *>(p.y), base + c, s * rstd * p.w[c]);
  }
}

// Backward with rows in registers.
template <typename Tin, int TPR, int NV, bool LOOSE>
__global__ void __launch_bounds__(256) rms_bwd_rows_kernel(const RmsBwdParams p) {
  constexpr int V = 16 / sizeof(Tin), kRows = 256 / TPR;
  __shared__ float lds[2][2][4];
  __shared__ __align__(16) float sums[kRows > 1 ? kRows * TPR * V : 1];
  const int l = threadIdx.x % TPR, dim = static_cast<int>(p.dim), pieces = (dim + V - 1) / V;
  const float inv = 1.0f / static_cast<float>(p.dim);
  float w[NV][V], dw[NV][V];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    Piece<float, V, LOOSE>::get(p.w, piece_at<V, LOOSE>(l + TPR * n < pieces ? l + TPR * n : 0, dim), w[n]);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[n][e] = 0.0f;
  }
  int odd = 0;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < p.rows; first += p.parts * kRows) {
    const int64_t row = first + threadIdx.x / TPR;
    const bool live = row < p.rows;
    const int64_t base = (live ? row : first) * p.dim;
    float s[NV][V], d[NV][V], r[NV][V], ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int k = l + TPR * n, at = piece_at<V, LOOSE>(k, dim);
#pragma unroll
      for (int e = 0; e < V; ++e) s[n][e] = d[n][e] = r[n][e] = 0.0f;
      if (k < pieces) {
        Piece<Tin, V, LOOSE>::get(p.s, base + at, s[n]);
        Piece<Tin, V, LOOSE>::get(p.dy, base + at, d[n]);
        if (p.dres != nullptr) Piece<Tin, V, LOOSE>::get(p.dres, base + at, r[n]);
      }
      const int skip = seen<V, LOOSE>(k, at);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float v = e < skip ? 0.0f : s[n][e], dv = e < skip ? 0.0f : d[n][e] * w[n][e];
        ss = fmaf(v, v, ss);
        dot = fmaf(dv, v, dot);
      }
    }
    const float rstd = 1.0f / sqrtf(fmaf(row_sum<TPR>(ss, lds[odd][0]), inv, p.eps));
    const float mean = row_sum<TPR>(dot, lds[odd][1]) * rstd * inv;
    odd ^= 1;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float norm = s[n][e] * rstd;
        if (live) dw[n][e] = fmaf(d[n][e], norm, dw[n][e]);
        r[n][e] = fmaf(rstd, d[n][e] * w[n][e] - norm * mean, r[n][e]);
      }
      if (l + TPR * n < pieces && live) Piece<Tin, V, LOOSE>::put(p.dx, base + piece_at<V, LOOSE>(l + TPR * n, dim), r[n]);
    }
  }
  if (p.dw == nullptr) return;
  float *part = p.ws + static_cast<int64_t>(blockIdx.x) * p.dim;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    if constexpr (kRows > 1) {  // over the rows in turn of the workgroup
      const int k = l + TPR * n, skip = seen<V, LOOSE>(k, piece_at<V, LOOSE>(k, dim));
      __syncthreads();
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e >= skip && k < pieces) sums[threadIdx.x * V + e - skip] = dw[n][e];
      __syncthreads();
      for (int c = threadIdx.x; c < TPR * V; c += 256) {
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < kRows; ++k) t += sums[k * TPR * V + c];
        const int64_t at = static_cast<int64_t>(TPR) * n * V + c;
        if (at < p.dim) part[at] = t;
      }
    } else if (l + TPR * n < pieces) {
      Piece<float, V, LOOSE>::put(part, piece_at<V, LOOSE>(l + TPR * n, dim), dw[n]);
    }
  }
}

// Backward of rows too long for registers: a workgroup per row in turn, which
// it reads twice.
template <typename Tin>
__global__ void __launch_bounds__(256) rms_bwd_any_kernel(const RmsBwdParams p) {
  __shared__ float lds[2][4];
  const Tin *dy = static_cast<const Tin *>(p.dy), *s = static_cast<const Tin *>(p.s);
  const Tin *dres = static_cast<const Tin *>(p.dres);
  float *part = p.ws + static_cast<int64_t>(blockIdx.x) * p.dim;
  if (p.dw != nullptr)
    for (int64_t c = threadIdx.x; c < p.dim; c += 256) part[c] = 0.0f;
  for (int64_t row = blockIdx.x; row < p.rows; row += p.parts) {
    const int64_t base = row * p.dim;
    double squares = 0.0, products = 0.0;
    for (int64_t run = 0; run < p.dim; run += kRun) {
      float ss = 0.0f, dot = 0.0f;
      for (int64_t c = run + threadIdx.x, end = run_end(run, p.dim); c < end; c += 256) {
        const float v = ld(s, base + c);
        ss = fmaf(v, v, ss);
        dot = fmaf(ld(dy, base + c) * p.w[c], v, dot);
      }
      squares += ss;
      products += dot;
    }
    const float ss = static_cast<float>(squares), dot = static_cast<float>(products);
    const float inv = 1.0f / static_cast<float>(p.dim);
    __syncthreads();  // the last row's sums have been read
    const float rstd = 1.0f / sqrtf(fmaf(row_sum<256>(ss, lds[0]), inv, p.eps));
    const float mean = row_sum<256>(dot, lds[1]) * rstd * inv;
    for (int64_t c = threadIdx.x; c < p.dim; c += 256) {
      const float n = ld(s, base + c) * rstd, d = ld(dy, base + c);
      const float r = dres != nullptr ? ld(dres, base + c) : 0.0f;
      st(static_cast<Tin *>(p.dx), base + c, fmaf(rstd, d * p.w[c] - n * mean, r));
      if (p.dw != nullptr) part[c] = fmaf(d, n, part[c]);
    }
  }
}

// dw: 16 threads share the terms of a column, a workgroup has 64 columns at a time.
__global__ void __launch_bounds__(1024) rms_sum_kernel(const float *part, float *dw, int64_t parts, int64_t dim) {
  __shared__ float lds[16][64];
  const int k0 = threadIdx.x / 64, col = threadIdx.x % 64;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * 64; first < dim; first += static_cast<int64_t>(gridDim.x) * 64) {
    const int64_t c = first + col;
    float s = 0.0f;
    if (c < dim) {
#pragma unroll 8
      for (int64_t k = k0; k < parts; k += 16) s += part[k * dim + c];
    }
    lds[k0][col] = s;
    __syncthreads();
    if (k0 == 0 && c < dim) {
#pragma unroll
      for (int k = 1; k < 16; ++k) s += lds[k][col];
      dw[c] = s;
    }
    __syncthreads();  // the next columns take `lds`
  }
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Lanes per row and pieces per lane for `pieces` of a row, and the kernel's
// instance for them; false where they are too many.
template <typename F>
bool with_shape(int64_t pieces, F f) {
  if (pieces <= 16) f.template operator()<16, 1>();
  else if (pieces <= 32) f.template operator()<16, 2>();
  else if (pieces <= 64) f.template operator()<64, 1>();
  else if (pieces <= 128) f.template operator()<64, 2>();
  else if (pieces <= 256) f.template operator()<64, 4>();
  else if (pieces <= 512) f.template operator()<256, 2>();
  else if (pieces <= 768) f.template operator()<256, 3>();
  else if (pieces <= 1024) f.template operator()<256, 4>();
  else if (pieces <= 2048) f.template operator()<256, 8>();
  else return false;
  return true;
}

// Workgroups of 256 / lanes rows each; more than fit at once walk the rows.
constexpr int64_t kMostGroups = 2048;
// Past this many workgroups the sum of dw walks its columns.
constexpr int64_t kMostSums = 65536;

template <typename Tin, typename Tout, bool Q8, bool LOOSE>
struct RowsLaunch {
  const RmsParams &p;
  int group_lanes;
  hipStream_t st;
  template <int TPR, int NV>
  void operator()() {
    const int64_t n = (p.rows + 256 / TPR - 1) / (256 / TPR);
    hipLaunchKernelGGL((rms_rows_kernel<Tin, Tout, TPR, NV, Q8, LOOSE>), dim3(static_cast<uint32_t>(n < kMostGroups ? n : kMostGroups)),
                       dim3(256), 0, st, p, group_lanes);
  }
};

template <typename Tin, typename Tout, bool Q8>
hipError_t run_fwd(const RmsParams &p, hipStream_t st) {
  constexpr int V = 16 / sizeof(Tin);
  // Stores of y are 4 to 32 bytes wide, by its type; its rows start on as many
  // where they start on 16 bytes of x.
  const bool loose = p.dim % V != 0 || !aligned16(p.x) || !aligned16(p.residual) || !aligned16(p.residual_out) ||
                     !aligned16(p.y) || !aligned16(p.w);
  const int64_t pieces = (p.dim + V - 1) / V;
  bool rows = p.dim >= V;
  int lanes = 0;
  if (Q8 && p.group < p.dim) {
    if (p.dim % V != 0) rows = false;  // the last piece would span two groups
    lanes = p.group % V == 0 && p.group / V <= 64 ? static_cast<int>(p.group / V) : -1;
    if (lanes < 1 || (lanes & (lanes - 1)) != 0 || (lanes > 16 && pieces <= 32)) rows = false;
  }
  if (rows && (loose ? with_shape(pieces, RowsLaunch<Tin, Tout, Q8, true>{p, lanes, st})
                     : with_shape(pieces, RowsLaunch<Tin, Tout, Q8, false>{p, lanes, st})))
    return hipGetLastError();
  const int keep = p.dim <= 8192;  // 32 KiB of LDS: four workgroups per CU and more
  const dim3 grid = p.rows <= kGridWidth ? dim3(static_cast<uint32_t>(p.rows))
                                         : dim3(kGridWidth, static_cast<uint32_t>((p.rows + kGridWidth - 1) / kGridWidth));
  hipLaunchKernelGGL((rms_any_kernel<Tin, Tout, Q8>), grid, dim3(256),
                     keep ? static_cast<size_t>(p.dim) * 4 : 0, st, p, keep);
  return hipGetLastError();
}

template <typename Tin, bool LOOSE>
struct BwdLaunch {
  const RmsBwdParams &p;
  hipStream_t st;
  template <int TPR, int NV>
  void operator()() {
    hipLaunchKernelGGL((rms_bwd_rows_kernel<Tin, TPR, NV, LOOSE>), dim3(static_cast<uint32_t>(p.parts)), dim3(256), 0, st, p);
  }
};

template <typename Tin>
void run_bwd(const RmsBwdParams &p, hipStream_t st) {
  constexpr int V = 16 / sizeof(Tin);
  const bool loose = p.dim % V != 0 || !aligned16(p.dy) || !aligned16(p.s) || !aligned16(p.dres) || !aligned16(p.dx) ||
                     !aligned16(p.w) || !aligned16(p.ws);
  const int64_t pieces = (p.dim + V - 1) / V;
  if (p.dim >= V &&
      (loose ? with_shape(pieces, BwdLaunch<Tin, true>{p, st}) : with_shape(pieces, BwdLaunch<Tin, false>{p, st})))
    return;
  hipLaunchKernelGGL((rms_bwd_any_kernel<Tin>), dim3(static_cast<uint32_t>(p.parts)), dim3(256), 0, st, p);
}

}  // namespace

hipError_t launch_rms(const RmsParams &p, int in_bf16, int out_bf16, hipStream_t st) {
  if (p.scale != nullptr) return in_bf16 ? run_fwd<uint16_t, uint16_t, true>(p, st) : run_fwd<float, float, true>(p, st);
  if (in_bf16) return out_bf16 ? run_fwd<uint16_t, uint16_t, false>(p, st) : run_fwd<uint16_t, float, false>(p, st);
  return out_bf16 ? run_fwd<float, uint16_t, false>(p, st) : run_fwd<float, float, false>(p, st);
}

int64_t rms_bwd_parts(int64_t rows, int64_t) { return rows < 512 ? rows : 512; }

hipError_t launch_rms_bwd(const RmsBwdParams &p, int in_bf16, hipStream_t st) {
  if (p.rows > 0) {
    if (in_bf16) run_bwd<uint16_t>(p, st);
    else run_bwd<float>(p, st);
  }
  const int64_t groups = (p.dim + 63) / 64;
  if (p.dw != nullptr)
    hipLaunchKernelGGL(rms_sum_kernel, dim3(static_cast<uint32_t>(groups < kMostSums ? groups : kMostSums)), dim3(1024), 0, st, p.ws,
                       p.dw, p.parts, p.dim);
  return hipGetLastError();
}

}  // namespace ssmb
