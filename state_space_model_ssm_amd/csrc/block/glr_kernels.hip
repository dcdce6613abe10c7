// Gated linear recurrence for gfx950: forward, backward and one step.
//
//   r = s(rec), i = s(inp), a = exp(A r), b = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + b_t i_t x_t
//
// A lane takes 16 steps of one channel, or of two that share a dword, in
// registers; a workgroup's tile is 128 steps by 32 lanes of channels (rows of
// 128 bytes).  A lane's steps are summed up as (product of a, end state from
// zero), the 8 summaries of a channel meet in LDS, and each lane then runs its
// steps from the state it starts with, so the tile is read once.  A workgroup
// walks its tiles in time with the state in registers; where there are too few
// channels to fill the GPU, the sequence is cut into segments, a first launch
// sums up the segments, and each workgroup starts from its predecessors'
// summaries, taken in order (so the result does not depend on timing).
//
// 1 - a^2 is computed as -expm1(2 A r) (see one_minus_exp), since a is close
// to 1 in slow channels.
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

constexpr int T = SSM_GLR_STATE_STEP;  // steps of a lane
constexpr int kSubs = 8;               // lanes in time
constexpr int kLanes = 32;             // lanes in channels

// C channels of a lane as they lie in memory: one value, or two bfloat16.
template <typename E, int C>
struct Raw;
template <>
struct Raw<float, 1> {
  typedef float type;
  __device__ static __forceinline__ void get(type v, float (&f)[1]) { f[0] = v; }
  __device__ static __forceinline__ type put(const float (&f)[1]) { return f[0]; }
};
template <>
struct Raw<uint16_t, 1> {
  typedef uint16_t type;
  __device__ static __forceinline__ void get(type v, float (&f)[1]) { f[0] = __uint_as_float(static_cast<uint32_t>(v) << 16); }
  __device__ static __forceinline__ type put(const float (&f)[1]) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f[0]));
  }
};
template <>
struct Raw<uint16_t, 2> {
  typedef uint32_t type;
  __device__ static __forceinline__ void get(type v, float (&f)[2]) {
    f[0] = __uint_as_float(v << 16);
    f[1] = __uint_as_float(v & 0xffff0000u);
  }
  __device__ static __forceinline__ type put(const float (&f)[2]) {
    typedef __attribute__((ext_vector_type(2))) __bf16 bf2;
    const bf2 v = {static_cast<__bf16>(f[0]), static_cast<__bf16>(f[1])};
    return __builtin_bit_cast(uint32_t, v);
  }
};
template <>
struct Raw<float, 2> {
  typedef float2 type;
  __device__ static __forceinline__ void get(type v, float (&f)[2]) { f[0] = v.x; f[1] = v.y; }
  __device__ static __forceinline__ type put(const float (&f)[2]) { return make_float2(f[0], f[1]); }
};

// Where a workgroup and its lanes stand.
struct Place {
  int64_t b, dim, seqlen;
  int sub, c, seg;      // place in time within a tile; first channel; segment
  int64_t tile0, tile1; // tiles of the segment
  unsigned off;         // of the first of the lane's steps in a tile, in elements
  bool live;            // c is a channel (a pair never ends past dim: dim is even there)
};
template <int C>
__device__ __forceinline__ Place place(int64_t dim, int64_t seqlen, unsigned segs, int64_t seg_tiles) {
  Place w;
  const unsigned ct = static_cast<unsigned>((dim + kLanes * C - 1) / (kLanes * C));
  const unsigned id = blockIdx.x, seg = id % segs, rest = id / segs;
  w.b = rest / ct;
  w.dim = dim;
  w.seqlen = seqlen;
  w.sub = threadIdx.x / kLanes;
  w.c = static_cast<int>(rest % ct) * kLanes * C + (threadIdx.x % kLanes) * C;
  w.live = w.c < dim;
  if (!w.live) w.c = static_cast<int>(dim) - C;
  w.off = static_cast<unsigned>(w.sub * T) * static_cast<unsigned>(dim) + w.c;
  w.seg = seg;
  const int64_t tiles = (seqlen + T * kSubs - 1) / (T * kSubs);
  w.tile0 = seg * seg_tiles;
  w.tile1 = w.tile0 + seg_tiles < tiles ? w.tile0 + seg_tiles : tiles;
  return w;
}

// Rows of a tensor from row `row` on, at most `most` of them, as a buffer:
// what lies past its last row reads as zero and is not written, so the last
// tile needs no other code.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void *p, int64_t row, int64_t rows, int most, int64_t bytes) {
  const int64_t left = rows < most ? (rows > 0 ? rows : 0) : most;
  char *at = static_cast<char *>(const_cast<void *>(p)) + row * bytes;
  return __builtin_amdgcn_make_buffer_rsrc(at, 0, static_cast<int>(left * bytes), 0x00020000);
}
template <int BYTES>
struct Word;
template <>
struct Word<2> {
  typedef uint16_t type;
  __device__ static __forceinline__ type get(__amdgpu_buffer_rsrc_t r, unsigned at) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
  }
  __device__ static __forceinline__ void put(type v, __amdgpu_buffer_rsrc_t r, unsigned at) {
    __builtin_amdgcn_raw_buffer_store_b16(v, r, at, 0, 0);
  }
};
template <>
struct Word<4> {
  typedef uint32_t type;
  __device__ static __forceinline__ type get(__amdgpu_buffer_rsrc_t r, unsigned at) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
  }
  __device__ static __forceinline__ void put(type v, __amdgpu_buffer_rsrc_t r, unsigned at) {
    __builtin_amdgcn_raw_buffer_store_b32(v, r, at, 0, 0);
  }
};
template <>
struct Word<8> {
  typedef __attribute__((ext_vector_type(2))) unsigned int type;
  __device__ static __forceinline__ type get(__amdgpu_buffer_rsrc_t r, unsigned at) {
    return __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
  }
  __device__ static __forceinline__ void put(type v, __amdgpu_buffer_rsrc_t r, unsigned at) {
    __builtin_amdgcn_raw_buffer_store_b64(v, r, at, 0, 0);
  }
};
template <typename R>
__device__ __forceinline__ R fetch(__amdgpu_buffer_rsrc_t r, unsigned at) {
  return __builtin_bit_cast(R, Word<sizeof(R)>::get(r, at));
}
template <typename R>
__device__ __forceinline__ void write(R v, __amdgpu_buffer_rsrc_t r, unsigned at) {
  Word<sizeof(R)>::put(__builtin_bit_cast(typename Word<sizeof(R)>::type, v), r, at);
}

// Tile k of a tensor, and where in it this lane's step j lies (out of it for
// the stores of a lane without a channel).
template <typename E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_of(const void *p, const Place &w, int64_t k) {
  const int64_t t0 = k * T * kSubs;
  return rows_of(p, w.b * w.seqlen + t0, w.seqlen - t0, T * kSubs, w.dim * sizeof(E));
}
template <typename E>
__device__ __forceinline__ unsigned step_at(const Place &w, int j) {
  return (w.off + static_cast<unsigned>(j) * static_cast<unsigned>(w.dim)) * static_cast<unsigned>(sizeof(E));
}
template <typename E>
__device__ __forceinline__ unsigned store_at(const Place &w, int j) {
  return w.live ? step_at<E>(w, j) : 0xfffffff0u;
}

template <typename E, int C>
__device__ __forceinline__ void load(const void *p, const Place &w, int64_t k, typename Raw<E, C>::type (&v)[T]) {
  const __amdgpu_buffer_rsrc_t r = tile_of<E>(p, w, k);
#pragma unroll
  for (int j = 0; j < T; ++j) v[j] = fetch<typename Raw<E, C>::type>(r, step_at<E>(w, j));
}

// The reset byte of step threadIdx.x % 32 of this lane's 16, and from all 16
// of them a bit per step.
__device__ __forceinline__ unsigned load_reset(const uint8_t *reset, const Place &w, int64_t k) {
  if (reset == nullptr) return 0;
  const int64_t t0 = k * T * kSubs;
  const __amdgpu_buffer_rsrc_t r = rows_of(reset, w.b * w.seqlen + t0, w.seqlen - t0, T * kSubs, 1);
  const unsigned l = threadIdx.x % kLanes;
  return __builtin_amdgcn_raw_buffer_load_b8(r, l < T ? w.sub * T + l : 0xfffffff0u, 0, 0);
}
__device__ __forceinline__ unsigned reset_bits(unsigned byte) {
  const uint64_t all = __ballot(byte != 0);
  return static_cast<unsigned>(all >> (threadIdx.x & 32)) & 0xffffu;
}

template <typename Tin, int C>
struct Tile {
  typename Raw<Tin, C>::type x[T], rec[T], inp[T];
  unsigned reset;
  __device__ __forceinline__ void get(const GlrParams &p, const Place &w, int64_t k) {
    load<Tin, C>(p.rec, w, k, rec);
    load<Tin, C>(p.inp, w, k, inp);
    load<Tin, C>(p.x, w, k, x);
    reset = load_reset(p.reset, w, k);
  }
};

// A product of a that has a reset among its steps is negative: what comes
// before does not pass, be it NaN or infinite.
constexpr float kReset = -1.0f;
__device__ __forceinline__ float after(float prod, float start, float end) {
  return __float_as_int(prod) < 0 ? end : fmaf(prod, start, end);
}
// The product over two stretches of steps.
__device__ __forceinline__ float both(float p, float q) {
  return __uint_as_float((__float_as_uint(p * q) & 0x7fffffffu) | ((__float_as_uint(p) | __float_as_uint(q)) & 0x80000000u));
}

// The state a lane starts tile `it` with, and (next) the tile's end state:
// from `carry` through the lanes' summaries prod, end.  REVERSE: time runs
// from the last lane to the first.
template <int C, bool REVERSE>
__device__ __forceinline__ void join(float (&lds)[2][kSubs][kLanes][2 * C], int it, const Place &w,
                                     const float (&prod)[C], const float (&end)[C], const float (&carry)[C],
                                     float (&start)[C], float (&next)[C]) {
  const int l = threadIdx.x % kLanes;
  float *mine = lds[it & 1][w.sub][l];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    mine[2 * c] = prod[c];
    mine[2 * c + 1] = end[c];
  }
  __syncthreads();  // (the other buffer is written two tiles later, past the next barrier)
  float s[C];
#pragma unroll
  for (int c = 0; c < C; ++c) s[c] = start[c] = carry[c];
#pragma unroll
  for (int k = 0; k < kSubs; ++k) {
    const int sub = REVERSE ? kSubs - 1 - k : k;
    const float *v = lds[it & 1][sub][l];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (sub == w.sub) start[c] = s[c];
      s[c] = after(v[2 * c], s[c], v[2 * c + 1]);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) next[c] = s[c];
}

// SUM: only the segment's summary, (product of a, end state from zero), into ws.
template <typename Tin, typename Tout, int C, bool SUM>
__global__ void __launch_bounds__(256, 3) glr_fwd_kernel(const GlrParams p, unsigned segs, int64_t seg_tiles) {
  __shared__ __align__(16) float lds[2][kSubs][kLanes][2 * C];
  const Place w = place<C>(p.dim, p.seqlen, SUM ? segs - 1 : segs, seg_tiles);
  float A[C], carry[C], whole[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    A[c] = p.A[w.c + c];
    carry[c] = SUM || p.h0 == nullptr ? 0.0f : p.h0[w.b * p.dim + w.c + c];
    whole[c] = 1.0f;
  }
  if constexpr (!SUM) {
    for (int k = 0; k < w.seg; ++k) {
      const float *s = p.ws + ((w.b * (segs - 1) + k) * p.dim + w.c) * 2;
#pragma unroll
      for (int c = 0; c < C; ++c) carry[c] = after(s[2 * c], carry[c], s[2 * c + 1]);
    }
  }
  const int64_t nstate = (p.seqlen + T - 1) / T;
  Tile<Tin, C> now;
  if (w.tile0 < w.tile1) now.get(p, w, w.tile0);
  for (int64_t k = w.tile0; k < w.tile1; ++k) {
    const int64_t t0 = k * T * kSubs + w.sub * T;
    const int steps = p.seqlen - t0 < T ? static_cast<int>(p.seqlen - t0) : T;  // of this lane
    float a[T][C], u[T][C], prod[C], end[C], start[C], next[C];
#pragma unroll
    for (int j = 0; j < T; ++j) {
      float x[C], rec[C], inp[C];
      Raw<Tin, C>::get(now.x[j], x);
      Raw<Tin, C>::get(now.rec[j], rec);
      Raw<Tin, C>::get(now.inp[j], inp);
#pragma unroll
      for (int c = 0; c < C; ++c) gates(x[c], rec[c], inp[c], A[c], a[j][c], u[j][c]);
      if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // bounds the registers of interleaved steps
    }
    const unsigned reset = reset_bits(now.reset);
    if (k + 1 < w.tile1) now.get(p, w, k + 1);  // on its way during the rest of this tile
    if ((k + 1) * T * kSubs > p.seqlen) {       // steps past the end change nothing
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          a[j][c] = j < steps ? a[j][c] : 1.0f;
          u[j][c] = j < steps ? u[j][c] : 0.0f;
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      prod[c] = 1.0f;
      end[c] = 0.0f;
    }
    const bool resets = __any(reset != 0);  // few tiles have one
    if (!resets) {
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          prod[c] *= a[j][c];
          end[c] = fmaf(a[j][c], end[c], u[j][c]);
        }
    } else {
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const bool cut = reset >> j & 1;
          prod[c] = (cut ? kReset : prod[c]) * a[j][c];
          end[c] = fmaf(a[j][c], cut ? 0.0f : end[c], u[j][c]);
        }
    }
    join<C, false>(lds, static_cast<int>(k - w.tile0), w, prod, end, carry, start, next);
    if constexpr (SUM) {
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
        for (int c = 0; c < C; ++c)
          whole[c] = both(whole[c], lds[(k - w.tile0) & 1][sub][threadIdx.x % kLanes][2 * c]);
    } else {
      if (p.states != nullptr) {
        const __amdgpu_buffer_rsrc_t r = rows_of(p.states, w.b * nstate + k * kSubs, nstate - k * kSubs, kSubs, p.dim * 4);
        const unsigned at = (static_cast<unsigned>(w.sub) * static_cast<unsigned>(p.dim) + w.c) * 4;
        write(Raw<float, C>::put(start), r, w.live ? at : 0xfffffff0u);
      }
      const __amdgpu_buffer_rsrc_t r = tile_of<Tout>(p.y, w, k);
#pragma unroll
      for (int j = 0; j < T; ++j) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          start[c] = fmaf(a[j][c], resets && (reset >> j & 1) ? 0.0f : start[c], u[j][c]);
        write(Raw<Tout, C>::put(start), r, store_at<Tout>(w, j));
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) carry[c] = next[c];
  }
  if (!w.live || w.sub != 0) return;
  if constexpr (SUM) {
    float *s = p.ws + ((w.b * (segs - 1) + w.seg) * p.dim + w.c) * 2;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s[2 * c] = whole[c];
      s[2 * c + 1] = carry[c];
    }
  } else if (p.h_last != nullptr && w.seg + 1 == static_cast<int>(segs)) {
#pragma unroll
    for (int c = 0; c < C; ++c) p.h_last[w.b * p.dim + w.c + c] = carry[c];
  }
}

// The backward of a tile needs a state per lane, which the forward saved, and
// the gradient that comes from later steps.  A first pass over the lane's
// steps takes a alone and sums up (product of a, what arrives before the
// lane); once joined, one pass back in time gives g, and one forward the state
// and every output, so each gate is computed once (r twice).
// SUM: only the segment's summary, from rec and dy.
template <typename Tin, int C, bool SUM>
__global__ void __launch_bounds__(256, C == 2 ? 2 : 3) glr_bwd_kernel(const GlrBwdParams p, unsigned segs, int64_t seg_tiles) {
  __shared__ __align__(16) float lds[2][kSubs][kLanes][2 * C];
  typedef typename Raw<Tin, C>::type raw;
  Place w = place<C>(p.dim, p.seqlen, SUM ? segs - 1 : segs, seg_tiles);
  if constexpr (SUM) {  // segments 1 ..: nothing is carried out of the first
    w.seg += 1;
    w.tile0 += seg_tiles;
    const int64_t tiles = (p.seqlen + T * kSubs - 1) / (T * kSubs);
    w.tile1 = w.tile0 + seg_tiles < tiles ? w.tile0 + seg_tiles : tiles;
  }
  float A[C], carry[C], whole[C], dA[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    A[c] = p.A[w.c + c];
    carry[c] = SUM || p.dh_last == nullptr ? 0.0f : p.dh_last[w.b * p.dim + w.c + c];
    whole[c] = 1.0f;
    dA[c] = 0.0f;
  }
  if constexpr (!SUM) {
    for (int k = static_cast<int>(segs) - 1; k > w.seg; --k) {
      const float *s = p.ws_seg + ((w.b * (segs - 1) + k - 1) * p.dim + w.c) * 2;
#pragma unroll
      for (int c = 0; c < C; ++c) carry[c] = after(s[2 * c], carry[c], s[2 * c + 1]);
    }
  }
  const int64_t nstate = (p.seqlen + T - 1) / T;
  for (int64_t k = w.tile1 - 1; k >= w.tile0; --k) {
    raw rec[T], dy[T], x[T], inp[T];
    const int64_t t0 = k * T * kSubs + w.sub * T;
    load<Tin, C>(p.rec, w, k, rec);
    load<Tin, C>(p.dy, w, k, dy);
    float h[C];
    if constexpr (!SUM) {
      load<Tin, C>(p.x, w, k, x);
      load<Tin, C>(p.inp, w, k, inp);
      const __amdgpu_buffer_rsrc_t r = rows_of(p.states, w.b * nstate + k * kSubs, nstate - k * kSubs, kSubs, p.dim * 4);
      const unsigned at = (static_cast<unsigned>(w.sub) * static_cast<unsigned>(p.dim) + w.c) * 4;
      Raw<float, C>::get(fetch<typename Raw<float, C>::type>(r, at), h);
    }
    const unsigned reset = reset_bits(load_reset(p.reset, w, k));
    const int steps = p.seqlen - t0 < T ? static_cast<int>(p.seqlen - t0) : T;  // of this lane
    float a[T][C], g[T][C], prod[C], end[C], start[C], next[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      prod[c] = 1.0f;
      end[c] = 0.0f;
    }
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      float r[C];
      Raw<Tin, C>::get(rec[j], r);
      Raw<Tin, C>::get(dy[j], g[j]);
#pragma unroll
      for (int c = 0; c < C; ++c) a[j][c] = __builtin_amdgcn_exp2f(A[c] * sigmoid(r[c]) * kLog2e);
    }
    if ((k + 1) * T * kSubs > p.seqlen) {  // steps past the end change nothing
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          a[j][c] = j < steps ? a[j][c] : 1.0f;
          g[j][c] = j < steps ? g[j][c] : 0.0f;
        }
    }
#pragma unroll
    for (int j = T - 1; j >= 0; --j)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const bool cut = reset >> j & 1;
        end[c] = cut ? 0.0f : a[j][c] * (end[c] + g[j][c]);
        prod[c] = cut ? kReset : a[j][c] * prod[c];
      }
    join<C, true>(lds, static_cast<int>(w.tile1 - 1 - k), w, prod, end, carry, start, next);
    if constexpr (SUM) {
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
        for (int c = 0; c < C; ++c)
          whole[c] = both(whole[c], lds[(w.tile1 - 1 - k) & 1][sub][threadIdx.x % kLanes][2 * c]);
    } else {
#pragma unroll
      for (int j = T - 1; j >= 0; --j)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          g[j][c] += start[c];
          start[c] = (reset >> j & 1) ? 0.0f : a[j][c] * g[j][c];
        }
      if ((k + 1) * T * kSubs > p.seqlen) {  // dh_last has passed the steps past the end: they add nothing to dA
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
          for (int c = 0; c < C; ++c) g[j][c] = j < steps ? g[j][c] : 0.0f;
      }
      const __amdgpu_buffer_rsrc_t rdx = tile_of<Tin>(p.dx, w, k), rdr = tile_of<Tin>(p.drec, w, k);
      const __amdgpu_buffer_rsrc_t rdi = tile_of<Tin>(p.dinp, w, k);
#pragma unroll
      for (int j = 0; j < T; ++j) {
        float fx[C], fr[C], fi[C], dx[C], dr[C], di[C];
        Raw<Tin, C>::get(x[j], fx);
        Raw<Tin, C>::get(rec[j], fr);
        Raw<Tin, C>::get(inp[j], fi);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          // s(v) with 1 - s(v) = e s(v), e = exp(-v): no cancellation at either end.
          const float vr = fr[c] < -87.0f ? -87.0f : fr[c], vi = fi[c] < -87.0f ? -87.0f : fi[c];
          const float er = __builtin_amdgcn_exp2f(-vr * kLog2e), r = __builtin_amdgcn_rcpf(1.0f + er);
          const float ei = __builtin_amdgcn_exp2f(-vi * kLog2e), i = __builtin_amdgcn_rcpf(1.0f + ei);
          const float la = A[c] * r, q = one_minus_exp(2.0f * la, a[j][c]);
          const float rb = q >= kSmallest ? __builtin_amdgcn_rsqf(q) : 0.0f;  // 1 / b
          const float ix = i * fx[c], gb = g[j][c] * (q * rb), hp = (reset >> j & 1) ? 0.0f : h[c];
          const float wt = g[j][c] * a[j][c] * fmaf(-a[j][c] * rb, ix, hp);
          dx[c] = gb * i;
          dr[c] = wt * la * (er * r);
          di[c] = gb * ix * (ei * i);
          dA[c] = fmaf(wt, r, dA[c]);
          h[c] = fmaf(a[j][c], hp, q * rb * ix);
        }
        const unsigned at = store_at<Tin>(w, j);
        write(Raw<Tin, C>::put(dx), rdx, at);
        write(Raw<Tin, C>::put(dr), rdr, at);
        write(Raw<Tin, C>::put(di), rdi, at);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) carry[c] = next[c];
  }
  if constexpr (SUM) {
    if (!w.live || w.sub != 0) return;
    float *s = p.ws_seg + ((w.b * (segs - 1) + w.seg - 1) * p.dim + w.c) * 2;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s[2 * c] = whole[c];
      s[2 * c + 1] = carry[c];
    }
  } else {
    // dA over the lanes of a channel, in their order.
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) lds[0][w.sub][threadIdx.x % kLanes][c] = dA[c];
    __syncthreads();
    if (!w.live || w.sub != 0) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float s = 0.0f;
      for (int sub = 0; sub < kSubs; ++sub) s += lds[0][sub][threadIdx.x % kLanes][c];
      p.ws_dA[(w.b * segs + w.seg) * p.dim + w.c + c] = s;
      if (p.dh0 != nullptr && w.seg == 0) p.dh0[w.b * p.dim + w.c + c] = carry[c];
    }
  }
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

template <typename Tin, typename Tout, int C>
hipError_t run_fwd(const GlrParams &p, const GlrPlan &g, hipStream_t s) {
  const int64_t ct = (p.dim + kLanes * C - 1) / (kLanes * C);
  if (g.segs > 1)
    hipLaunchKernelGGL((glr_fwd_kernel<Tin, Tout, C, true>), dim3(static_cast<uint32_t>(p.batch * ct * (g.segs - 1))),
                       dim3(256), 0, s, p, g.segs, g.seg_tiles);
  hipLaunchKernelGGL((glr_fwd_kernel<Tin, Tout, C, false>), dim3(static_cast<uint32_t>(p.batch * ct * g.segs)), dim3(256), 0,
                     s, p, g.segs, g.seg_tiles);
  return hipGetLastError();
}

template <typename Tin, int C>
hipError_t run_bwd(const GlrBwdParams &p, const GlrPlan &g, hipStream_t s) {
  const int64_t ct = (p.dim + kLanes * C - 1) / (kLanes * C);
  if (p.batch > 0) {
    if (g.segs > 1)
      hipLaunchKernelGGL((glr_bwd_kernel<Tin, C, true>), dim3(static_cast<uint32_t>(p.batch * ct * (g.segs - 1))), dim3(256),
                         0, s, p, g.segs, g.seg_tiles);
    hipLaunchKernelGGL((glr_bwd_kernel<Tin, C, false>), dim3(static_cast<uint32_t>(p.batch * ct * g.segs)), dim3(256), 0, s,
                       p, g.segs, g.seg_tiles);
  }
  hipLaunchKernelGGL(glr_sum_kernel, blocks(p.dim, 256), dim3(256), 0, s, p.ws_dA, p.dA, p.batch * g.segs, p.dim);
  return hipGetLastError();
}

bool even(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }
bool even8(const void *p) { return reinterpret_cast<uintptr_t>(p) % 8 == 0; }

}  // namespace

GlrPlan glr_plan(int64_t batch, int64_t seqlen, int64_t dim) {
  // Workgroups of a whole sequence are enough from one per CU on; below that,
  // segments up to about three workgroups per CU (what fits at once).
  const int64_t tiles = (seqlen + T * kSubs - 1) / (T * kSubs), ct = (dim + kLanes - 1) / kLanes;
  const int64_t wide = batch * ((ct + 1) / 2);
  int64_t segs = 1;
  if (wide > 0 && wide < 256) segs = 768 / wide;
  if (segs > tiles) segs = tiles;
  if (segs > 64) segs = 64;
  GlrPlan g;
  g.seg_tiles = segs > 1 ? (tiles + segs - 1) / segs : (tiles > 0 ? tiles : 1);
  g.segs = static_cast<unsigned>(tiles > 0 ? (tiles + g.seg_tiles - 1) / g.seg_tiles : 1);
  return g;
}

hipError_t launch_glr(const GlrParams &p, const GlrPlan &g, int in_bf16, int out_bf16, hipStream_t s) {
  // Two channels per lane where every row of two starts on a dword.
  const bool pairs = p.dim % 2 == 0 && even(p.x) && even(p.rec) && even(p.inp) && even8(p.states) &&
                     (out_bf16 ? even(p.y) : even8(p.y));
  if (in_bf16 && out_bf16) return pairs ? run_fwd<uint16_t, uint16_t, 2>(p, g, s) : run_fwd<uint16_t, uint16_t, 1>(p, g, s);
  if (in_bf16) return pairs ? run_fwd<uint16_t, float, 2>(p, g, s) : run_fwd<uint16_t, float, 1>(p, g, s);
  return out_bf16 ? run_fwd<float, uint16_t, 1>(p, g, s) : run_fwd<float, float, 1>(p, g, s);
}

hipError_t launch_glr_step(const GlrParams &p, int in_bf16, int out_bf16, hipStream_t s) {
  const dim3 g = blocks(p.batch * p.dim, 256), t(256);
  if (in_bf16 && out_bf16) hipLaunchKernelGGL((glr_step_kernel<uint16_t, uint16_t>), g, t, 0, s, p);
  else if (in_bf16) hipLaunchKernelGGL((glr_step_kernel<uint16_t, float>), g, t, 0, s, p);
  else if (out_bf16) hipLaunchKernelGGL((glr_step_kernel<float, uint16_t>), g, t, 0, s, p);
  else hipLaunchKernelGGL((glr_step_kernel<float, float>), g, t, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_glr_bwd(const GlrBwdParams &p, const GlrPlan &g, int in_bf16, hipStream_t s) {
  const bool pairs = p.dim % 2 == 0 && even(p.x) && even(p.rec) && even(p.inp) && even(p.dy) && even8(p.states) &&
                     even(p.dx) && even(p.drec) && even(p.dinp);
  if (!in_bf16) return run_bwd<float, 1>(p, g, s);
  return pairs ? run_bwd<uint16_t, 2>(p, g, s) : run_bwd<uint16_t, 1>(p, g, s);
}

}  // namespace ssmb
