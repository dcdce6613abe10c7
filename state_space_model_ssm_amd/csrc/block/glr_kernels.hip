// Gated linear recurrence for gfx950: forward, backward and one step.
//
//   r = s(rec), i = s(inp), a = exp(A r), b = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + b_t i_t x_t
//
// A lane takes 16 steps of one channel, or of two that share a dword, in
// registers; a workgroup's tile is 128 steps by 32 lanes of channels (rows of
// 128 bytes).  A lane's steps are summed up as (product of a, end state from
// zero), the 8 summaries of a channel meet in LDS, the tile publishes its own
// summary, takes the state it starts with from its predecessors', and runs its
// steps: every tensor is read once, whatever the shape.  (Cutting the sequence
// into segments that a first launch sums up reads the inputs twice: 195 us
// against 106 for 1 x 32749 x 1536, and walking whole sequences with one
// workgroup per 64 channels leaves 320 workgroups for 4 x 5120 channels, at
// 2.3 TB/s against the 3.9 of enough tiles in flight.)  Bound by memory, inputs
// out of the caches: bfloat16, 4 x 4096 x 5120, forward 175 us, backward 293,
// both 3.9 TB/s; float32, 8 x 2048 x 1536, 92 and 134 us, 4.4 and 5.3 TB/s.
//
// Tiles of a channel block are grouped by 16 in time.  A tile waits for the
// state at its group's start and the summaries of the tiles before it in the
// group, and combines them in order; the group's last tile publishes the next
// group's start.  So a long sequence costs one wait per group, and the result
// does not depend on timing.  Tiles are numbered by a counter in the order in
// which workgroups start, first by time: a workgroup only waits for lower
// numbers, which have started, so the lowest unfinished one never waits.
// A published word carries its own sign of being there (it is not all ones,
// which the words are set to before), so no word has to be ordered against
// another and the caches need not be written back.
//
// 1 - a^2 is computed as 1 - exp(2 A r) without cancellation (one_minus_exp),
// since a is close to 1 in slow channels.
#include "block_internal.h"
#include "ssm_block.h"

namespace ssmb {
namespace {

// The smallest normal float: below it the reciprocal square root has no use.
constexpr float kSmallest = 0x1p-126f;

// 1 - exp(u) for u <= 0, where a = exp(u / 2) is at hand.  Above -0.4, where
// 1 - a^2 would cancel, -u times a polynomial fitted to expm1(u) / u there
// (relative error 6.2e-8, 1.5e-7 with its float32 roundings); below, 1 - a^2
// (1.3e-7 in its root).
__device__ __forceinline__ float one_minus_exp(float u, float a) {
  float p = fmaf(u, 0x1.ce7feep-8f, 0x1.51c052p-5f);
  p = fmaf(u, p, 0x1.5534a4p-3f);
  p = fmaf(u, p, 0x1.ffff2cp-2f);
  p = fmaf(u, p, 1.0f);
  return u > -0.4f ? -u * p : fmaf(-a, a, 1.0f);
}

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// The decay a and the weighted input u = b i x of one step.
__device__ __forceinline__ void gates(float x, float rec, float inp, float A, float &a, float &u) {
  const float r = sigmoid(rec);
  a = __builtin_amdgcn_exp2f(A * kLog2e * r);
  u = __builtin_amdgcn_sqrtf(one_minus_exp(2.0f * A * r, a)) * sigmoid(inp) * x;
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
  int sub, c;           // place in time within the tile; first channel
  int tiles, pos, k;    // tiles of a sequence; place in their order; the tile
  unsigned off;         // of the first of the lane's steps in a tile, in elements
  bool live;            // c is a channel (a pair never ends past dim: dim is even there)
  bool many;            // channel blocks: at least 64, so that few tiles of each are in flight
};

constexpr int kGroup = 16;                // tiles between two published states
constexpr unsigned kMissing = 0xffffffffu;  // a word not yet published
constexpr int kMostPolls = 1 << 22;       // some seconds: a wait that long would be a fault, and ends in NaN

// The workgroup's tile, from its set's counter (needed only if a sequence has
// more than one tile).  One tile per workgroup: workgroups that walk tiles and
// ask for the next number ahead hold numbers that others wait for, and took
// 206 us against 172 for the forward of 4 x 4096 x 5120.
template <int C, bool REVERSE>
__device__ __forceinline__ Place place(int64_t dim, int64_t seqlen, int64_t batch, const GlrChain &chain, unsigned &lds) {
  unsigned id = blockIdx.y * kGridWidth + blockIdx.x;
  const int tiles = static_cast<int>((seqlen + T * kSubs - 1) / (T * kSubs));
  const unsigned ct = static_cast<unsigned>((dim + kLanes * C - 1) / (kLanes * C)), rows = static_cast<unsigned>(batch) * ct;
  // Each round of ids begins a set later: workgroups go to the XCDs in turn, and
  // an XCD that kept the same few columns of 128 bytes would find them in as few
  // of its L2's channels (1 x 32749 x 1536: 125 us against 105).
  const unsigned sets = tiles > 1 ? glr_sets(rows) : 1, set = (id + id / sets) % sets;
  if (tiles > 1) {
    if (threadIdx.x == 0) lds = atomicAdd(chain.counter + set * (kGlrCounterBytes / 4), 1u);
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(lds);
  }
  Place w;
  const unsigned own = rows / sets, rest = set * own + id % own;  // rows of the set are adjacent
  w.pos = static_cast<int>(id / own);
  w.many = rows >= 64;
  w.tiles = tiles;
  w.k = REVERSE ? tiles - 1 - w.pos : w.pos;
  w.b = rest / ct;
  w.dim = dim;
  w.seqlen = seqlen;
  w.sub = threadIdx.x / kLanes;
  w.c = static_cast<int>(rest % ct) * kLanes * C + (threadIdx.x % kLanes) * C;
  w.live = w.c < dim;
  if (!w.live) w.c = static_cast<int>(dim) - C;
  w.off = static_cast<unsigned>(w.sub * T) * static_cast<unsigned>(dim) + w.c;
  return w;
}

// The compiler is not to keep what it computed from v: computing it again is
// cheaper than the registers.
template <typename R>
__device__ __forceinline__ void forget(R &v) {
  asm volatile("" : "+v"(v));
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

// Words that are read by other workgroups, at the scope of the whole GPU.
template <typename W>
__device__ __forceinline__ void publish(W *p, W v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W>
__device__ __forceinline__ W peek(const W *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W>
__device__ __forceinline__ W await(const W *p, W v) {  // v: what peek() saw
  for (int n = 0; v == static_cast<W>(~W{0}) && n < kMostPolls; ++n) {
    __builtin_amdgcn_s_sleep(2);
    v = peek(p);
  }
  return v;  // (all ones is a NaN)
}
__device__ __forceinline__ unsigned word(float v) {  // a NaN keeps its sign, and is not all ones
  const unsigned b = __float_as_uint(v);
  return v != v ? (b & 0x80000000u) | 0x7fc00000u : b;
}

struct Scratch {
  float subs[kSubs][kLanes][4];    // (product, end) of the lanes in time
  float tiles[kGroup][kLanes][4];  // and of the tiles before this one in its group
  float start[kLanes][2];          // state at the group's start
  unsigned number;
};

// What a thread fetches of the words a tile needs: the summaries of up to two
// of the tiles before it, looked at with the tile's loads, so that they are
// there when they are needed if they were published by then (4 x 4096 x 5120
// backward: 274 us against 282); and the place of the group's start.  With few
// channel blocks the tiles before have only just started too, and looking costs
// more than it finds (1 x 32749 x 1536 forward: 105 us against 101).
template <int C>
struct Words {
  const uint64_t *sums;
  const unsigned *starts;
  uint64_t sum[kGroup / kSubs][C];
  __device__ __forceinline__ void look(const GlrChain &chain, const Place &w) {
    const int before = w.pos % kGroup, group = w.pos / kGroup;
    sums = chain.sums + (w.b * w.tiles + w.pos - before) * w.dim + w.c;  // of the group's first tile
    starts = chain.starts + (w.b * ((w.tiles + kGroup - 1) / kGroup) + group) * w.dim + w.c;
    if (w.tiles == 1) return;
#pragma unroll
    for (int n = 0; n < kGroup / kSubs; ++n)
#pragma unroll
      for (int c = 0; c < C; ++c)
        sum[n][c] = w.many && w.sub + n * kSubs < before ? peek(sums + (w.sub + n * kSubs) * w.dim + c) : ~uint64_t{0};
  }
};

// Over stretch (p, e), then (q, f).
__device__ __forceinline__ void append(float &p, float &e, float q, float f) {
  e = after(q, e, f);
  p = both(p, q);
}

// The state this lane starts with, from all lanes' summaries prod, end, the
// tiles before, and `first`, the state the sequence starts with; `last` is the
// state after the tile (in the lanes sub = 0).
//
// The state at the group's start is what comes last, through a chain of one
// tile per group: everything else is summed up before it is waited for, and
// the group's last tile passes it on before it uses it.
template <int C, bool REVERSE>
__device__ __forceinline__ void join(Scratch &lds, const GlrChain &chain, const Place &w, const Words<C> &words,
                                     const float (&prod)[C], const float (&end)[C], const float (&first)[C],
                                     float (&start)[C], float (&last)[C]) {
  const int l = threadIdx.x % kLanes, before = w.pos % kGroup, group = w.pos / kGroup;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    lds.subs[w.sub][l][2 * c] = prod[c];
    lds.subs[w.sub][l][2 * c + 1] = end[c];
  }
  __syncthreads();
  // From the tile's start to this lane's, and to its end.
  float mine_p[C], mine_e[C], all_p[C], all_e[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    all_p[c] = 1.0f;
    all_e[c] = 0.0f;
  }
  constexpr int kAtOnce = C == 2 ? 4 : kSubs;  // reads in flight; eight by two channels cost a workgroup's registers
#pragma unroll kAtOnce
  for (int k = 0; k < kSubs; ++k) {
    const int sub = REVERSE ? kSubs - 1 - k : k;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (sub == w.sub) {
        mine_p[c] = all_p[c];
        mine_e[c] = all_e[c];
      }
      append(all_p[c], all_e[c], lds.subs[sub][l][2 * c], lds.subs[sub][l][2 * c + 1]);
    }
  }
  if (w.tiles > 1) {
    if (w.sub == 0 && w.live && before < kGroup - 1 && w.pos + 1 < w.tiles) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        publish(chain.sums + (w.b * w.tiles + w.pos) * w.dim + w.c + c,
                static_cast<uint64_t>(word(all_p[c])) | static_cast<uint64_t>(word(all_e[c])) << 32);
    }
#pragma unroll
    for (int n = 0; n < kGroup / kSubs; ++n) {
      const int m = w.sub + n * kSubs;
      if (m < before) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint64_t v = await(words.sums + m * w.dim + c, words.sum[n][c]);
          lds.tiles[m][l][2 * c] = __uint_as_float(static_cast<unsigned>(v));
          lds.tiles[m][l][2 * c + 1] = __uint_as_float(static_cast<unsigned>(v >> 32));
        }
      }
    }
    __syncthreads();
  }
  float p[C], e[C], s[C];  // from the group's start to the tile's
#pragma unroll
  for (int c = 0; c < C; ++c) {
    p[c] = 1.0f;
    e[c] = 0.0f;
    s[c] = first[c];
  }
#pragma unroll 4
  for (int m = 0; m < before; ++m)
#pragma unroll
    for (int c = 0; c < C; ++c) append(p[c], e[c], lds.tiles[m][l][2 * c], lds.tiles[m][l][2 * c + 1]);
  if (group > 0) {
    if (w.sub == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) s[c] = __uint_as_float(await(words.starts + c, peek(words.starts + c)));
    }
  }
  if (w.sub == 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      last[c] = after(all_p[c], after(p[c], s[c], e[c]), all_e[c]);
      if (before == kGroup - 1 && w.pos + 1 < w.tiles && w.live)
        publish(chain.starts + (w.b * ((w.tiles + kGroup - 1) / kGroup) + group + 1) * w.dim + w.c + c, word(last[c]));
      if (group > 0) lds.start[l][c] = s[c];
    }
  }
  if (group > 0) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = lds.start[l][c];
  }
#pragma unroll
  for (int c = 0; c < C; ++c) start[c] = after(mine_p[c], after(p[c], s[c], e[c]), mine_e[c]);
}

// All words missing, and the counters at 0.
__global__ void __launch_bounds__(256) glr_clear_kernel(uint4 *words, int64_t n, unsigned *counter) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  for (int64_t id = first; id < n; id += static_cast<int64_t>(gridDim.x) * 256)
    words[id] = make_uint4(kMissing, kMissing, kMissing, kMissing);
  if (first < kGlrSets) counter[first * (kGlrCounterBytes / 4)] = 0;
}

template <typename Tin, typename Tout, int C>
__global__ void __launch_bounds__(256, 4) glr_fwd_kernel(const GlrParams p) {
  __shared__ __align__(16) Scratch lds;
  const Place w = place<C, false>(p.dim, p.seqlen, p.batch, p.chain, lds.number);
  if (w.pos >= w.tiles) return;  // past the last, in a grid of two axes
  typename Raw<Tin, C>::type rx[T], rrec[T], rinp[T];
  load<Tin, C>(p.rec, w, w.k, rrec);
  load<Tin, C>(p.inp, w, w.k, rinp);
  load<Tin, C>(p.x, w, w.k, rx);
  Words<C> words;
  words.look(p.chain, w);
  const unsigned reset = reset_bits(load_reset(p.reset, w, w.k));
  float A[C], first[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    A[c] = p.A[w.c + c];
    first[c] = p.h0 == nullptr ? 0.0f : p.h0[w.b * p.dim + w.c + c];
  }
  const int64_t t0 = static_cast<int64_t>(w.k) * T * kSubs + w.sub * T;
  const int steps = p.seqlen - t0 < T ? static_cast<int>(p.seqlen - t0) : T;  // of this lane
  float a[T][C], u[T][C], prod[C], end[C], start[C], last[C];
#pragma unroll
  for (int j = 0; j < T; ++j) {
    float x[C], rec[C], inp[C];
    Raw<Tin, C>::get(rx[j], x);
    Raw<Tin, C>::get(rrec[j], rec);
    Raw<Tin, C>::get(rinp[j], inp);
#pragma unroll
    for (int c = 0; c < C; ++c) gates(x[c], rec[c], inp[c], A[c], a[j][c], u[j][c]);
    if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // bounds the registers of interleaved steps
  }
  if (w.k + 1 == w.tiles) {  // steps past the end change nothing
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
  // h_last may be h0: each wavefront has its h0 before the barrier that comes
  // before the tile's summary, so before the last tile can write.
#pragma unroll
  for (int c = 0; c < C; ++c) forget(first[c]);
  join<C, false>(lds, p.chain, w, words, prod, end, first, start, last);
  if (p.states != nullptr) {
    const int64_t nstate = (p.seqlen + T - 1) / T, row = static_cast<int64_t>(w.k) * kSubs;
    const __amdgpu_buffer_rsrc_t r = rows_of(p.states, w.b * nstate + row, nstate - row, kSubs, p.dim * 4);
    const unsigned at = (static_cast<unsigned>(w.sub) * static_cast<unsigned>(p.dim) + w.c) * 4;
    write(Raw<float, C>::put(start), r, w.live ? at : 0xfffffff0u);
  }
  Place to = w;
  forget(to.off);
  const __amdgpu_buffer_rsrc_t r = tile_of<Tout>(p.y, w, w.k);
#pragma unroll
  for (int j = 0; j < T; ++j) {
#pragma unroll
    for (int c = 0; c < C; ++c) start[c] = fmaf(a[j][c], resets && (reset >> j & 1) ? 0.0f : start[c], u[j][c]);
    write(Raw<Tout, C>::put(start), r, store_at<Tout>(to, j));
  }
  if (p.h_last != nullptr && w.k + 1 == w.tiles && w.live && w.sub == 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) p.h_last[w.b * p.dim + w.c + c] = last[c];
  }
}

// The backward of a tile needs a state per lane, which the forward saved, and
// the gradient that comes from later steps.  A first pass over the lane's
// steps takes a alone and sums up (product of a, what arrives before the
// lane); once joined, one pass back in time gives g, and one forward the state
// and every output, so each gate is computed once (r twice).
template <typename Tin, int C>
__global__ void __launch_bounds__(256, 3) glr_bwd_kernel(const GlrBwdParams p) {
  __shared__ __align__(16) Scratch lds;
  typedef typename Raw<Tin, C>::type raw;
  const Place w = place<C, true>(p.dim, p.seqlen, p.batch, p.chain, lds.number);
  if (w.pos >= w.tiles) return;  // past the last, in a grid of two axes
  raw rec[T], dy[T], x[T], inp[T];
  load<Tin, C>(p.rec, w, w.k, rec);
  load<Tin, C>(p.dy, w, w.k, dy);
  load<Tin, C>(p.x, w, w.k, x);
  load<Tin, C>(p.inp, w, w.k, inp);
  Words<C> words;
  words.look(p.chain, w);
  const unsigned reset = reset_bits(load_reset(p.reset, w, w.k));
  float A[C], first[C], dA[C], h[C];
  {
    const int64_t nstate = (p.seqlen + T - 1) / T, row = static_cast<int64_t>(w.k) * kSubs;
    const __amdgpu_buffer_rsrc_t r = rows_of(p.states, w.b * nstate + row, nstate - row, kSubs, p.dim * 4);
    const unsigned at = (static_cast<unsigned>(w.sub) * static_cast<unsigned>(p.dim) + w.c) * 4;
    Raw<float, C>::get(fetch<typename Raw<float, C>::type>(r, at), h);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    A[c] = p.A[w.c + c];
    first[c] = p.dh_last == nullptr ? 0.0f : p.dh_last[w.b * p.dim + w.c + c];
    dA[c] = 0.0f;
  }
  const int64_t t0 = static_cast<int64_t>(w.k) * T * kSubs + w.sub * T;
  const int steps = p.seqlen - t0 < T ? static_cast<int>(p.seqlen - t0) : T;  // of this lane
  float a[T][C], g[T][C], prod[C], end[C], start[C], last[C];
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
    for (int c = 0; c < C; ++c) a[j][c] = __builtin_amdgcn_exp2f(A[c] * kLog2e * sigmoid(r[c]));
    if (j % 4 == 0) __builtin_amdgcn_sched_barrier(0);  // bounds the registers of interleaved steps
  }
  if (w.k + 1 == w.tiles) {  // steps past the end change nothing
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
  join<C, true>(lds, p.chain, w, words, prod, end, first, start, last);
  Place to = w;
  forget(to.off);
  if constexpr (C == 2) {
#pragma unroll
    for (int j = 0; j < T; ++j) forget(rec[j]);
  }
#pragma unroll
  for (int j = T - 1; j >= 0; --j)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      g[j][c] += start[c];
      start[c] = (reset >> j & 1) ? 0.0f : a[j][c] * g[j][c];
    }
  if (w.k + 1 == w.tiles) {  // dh_last has passed the steps past the end: they add nothing to dA
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int c = 0; c < C; ++c) g[j][c] = j < steps ? g[j][c] : 0.0f;
  }
  const __amdgpu_buffer_rsrc_t rdx = tile_of<Tin>(p.dx, w, w.k), rdr = tile_of<Tin>(p.drec, w, w.k);
  const __amdgpu_buffer_rsrc_t rdi = tile_of<Tin>(p.dinp, w, w.k);
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
    const unsigned at = store_at<Tin>(to, j);
    write(Raw<Tin, C>::put(dx), rdx, at);
    write(Raw<Tin, C>::put(dr), rdr, at);
    write(Raw<Tin, C>::put(di), rdi, at);
    if (j % 2 == 1) __builtin_amdgcn_sched_barrier(0);
  }
  // dA over the lanes of a channel, in their order.
  __syncthreads();
  const int l = threadIdx.x % kLanes;
#pragma unroll
  for (int c = 0; c < C; ++c) lds.subs[w.sub][l][c] = dA[c];
  __syncthreads();
  if (!w.live || w.sub != 0) return;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float s = 0.0f;
    for (int sub = 0; sub < kSubs; ++sub) s += lds.subs[sub][l][c];
    p.ws_dA[(w.b * w.tiles + w.k) * p.dim + w.c + c] = s;
    if (p.dh0 != nullptr && w.k == 0) p.dh0[w.b * p.dim + w.c + c] = last[c];
  }
}

// dA: 16 threads share the terms of a channel, a workgroup has 64 channels.
__global__ void __launch_bounds__(1024) glr_sum_kernel(const float *part, float *dA, int64_t parts, int64_t dim) {
  __shared__ float lds[16][64];
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x % 64;
  const int k0 = threadIdx.x / 64;
  float s = 0.0f;
  if (c < dim) {
#pragma unroll 8
    for (int64_t k = k0; k < parts; k += 16) s += part[k * dim + c];
  }
  lds[k0][threadIdx.x % 64] = s;
  __syncthreads();
  if (k0 != 0 || c >= dim) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) s += lds[k][threadIdx.x];
  dA[c] = s;
}

// An empty sequence: the state passes through.
__global__ void __launch_bounds__(256) glr_pass_kernel(const float *from, float *to, int64_t n) {
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; id < n; id += static_cast<int64_t>(gridDim.x) * 256)
    to[id] = from != nullptr ? from[id] : 0.0f;
}

template <typename Tin, typename Tout>
__global__ void __launch_bounds__(256) glr_step_kernel(const GlrParams p) {
  const int64_t n = p.batch * p.dim;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; id < n; id += static_cast<int64_t>(gridDim.x) * 256) {
    float a, u;
    gates(ld(static_cast<const Tin *>(p.x), id), ld(static_cast<const Tin *>(p.rec), id),
          ld(static_cast<const Tin *>(p.inp), id), p.A[id % p.dim], a, u);
    const float h = fmaf(a, p.h0[id], u);
    p.h_last[id] = h;
    st(static_cast<Tout *>(p.y), id, h);
  }
}

// Workgroups for n items, `per` each; past 65536 they walk (see kGridWidth).
dim3 blocks(int64_t n, int64_t per) {
  const int64_t all = (n + per - 1) / per;
  return dim3(static_cast<uint32_t>(all < 65536 ? all : 65536));
}

// Tiles of all sequences, in workgroups.
template <int C>
int64_t all_tiles(int64_t batch, int64_t seqlen, int64_t dim) {
  return batch * ((dim + kLanes * C - 1) / (kLanes * C)) * ((seqlen + T * kSubs - 1) / (T * kSubs));
}

dim3 tile_grid(int64_t n) {
  if (n <= kGridWidth) return dim3(static_cast<uint32_t>(n));
  return dim3(kGridWidth, static_cast<uint32_t>((n + kGridWidth - 1) / kGridWidth));
}

void clear(const GlrChain &chain, int64_t seqlen, hipStream_t s) {
  if (seqlen <= T * kSubs) return;  // one tile per sequence: nothing is published
  hipLaunchKernelGGL(glr_clear_kernel, blocks(chain.bytes / 16, 256), dim3(256), 0, s, reinterpret_cast<uint4 *>(chain.sums),
                     chain.bytes / 16, chain.counter);
}

template <typename Tin, typename Tout, int C>
hipError_t run_fwd(const GlrParams &p, hipStream_t s) {
  const int64_t n = all_tiles<C>(p.batch, p.seqlen, p.dim);
  if (n > 0x7fffffff) return hipErrorInvalidValue;
  clear(p.chain, p.seqlen, s);
  hipLaunchKernelGGL((glr_fwd_kernel<Tin, Tout, C>), tile_grid(n), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename Tin, int C>
hipError_t run_bwd(const GlrBwdParams &p, hipStream_t s) {
  const int64_t n = all_tiles<C>(p.batch, p.seqlen, p.dim);
  if (n > 0x7fffffff) return hipErrorInvalidValue;
  clear(p.chain, p.seqlen, s);
  hipLaunchKernelGGL((glr_bwd_kernel<Tin, C>), tile_grid(n), dim3(256), 0, s, p);
  return hipGetLastError();
}

bool even(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }
bool even8(const void *p) { return reinterpret_cast<uintptr_t>(p) % 8 == 0; }

}  // namespace

size_t glr_chain_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  const int64_t tiles = (seqlen + T * kSubs - 1) / (T * kSubs);
  if (tiles <= 1) return 0;
  const int64_t sums = batch * tiles * dim * 8, starts = batch * ((tiles + kGroup - 1) / kGroup) * dim * 4;
  return static_cast<size_t>((sums + starts + 15) / 16 * 16);
}

GlrChain glr_chain(void *at, int64_t batch, int64_t seqlen, int64_t dim) {
  GlrChain c{};
  c.bytes = static_cast<int64_t>(glr_chain_bytes(batch, seqlen, dim));
  if (c.bytes == 0) return c;
  char *base = static_cast<char *>(at);
  c.counter = reinterpret_cast<unsigned *>(base);
  c.sums = reinterpret_cast<uint64_t *>(base + kGlrSets * kGlrCounterBytes);
  c.starts = reinterpret_cast<unsigned *>(c.sums + batch * ((seqlen + T * kSubs - 1) / (T * kSubs)) * dim);
  return c;
}

hipError_t launch_glr(const GlrParams &p, int in_bf16, int out_bf16, hipStream_t s) {
  if (p.seqlen == 0) {
    hipLaunchKernelGGL(glr_pass_kernel, blocks(p.batch * p.dim, 256), dim3(256), 0, s, p.h0, p.h_last, p.batch * p.dim);
    return hipGetLastError();
  }
  // Two channels per lane where every row of two starts on a dword.
  const bool pairs = p.dim % 2 == 0 && even(p.x) && even(p.rec) && even(p.inp) && even8(p.states) &&
                     (out_bf16 ? even(p.y) : even8(p.y));
  if (in_bf16 && out_bf16) return pairs ? run_fwd<uint16_t, uint16_t, 2>(p, s) : run_fwd<uint16_t, uint16_t, 1>(p, s);
  if (in_bf16) return pairs ? run_fwd<uint16_t, float, 2>(p, s) : run_fwd<uint16_t, float, 1>(p, s);
  return out_bf16 ? run_fwd<float, uint16_t, 1>(p, s) : run_fwd<float, float, 1>(p, s);
}

hipError_t launch_glr_step(const GlrParams &p, int in_bf16, int out_bf16, hipStream_t s) {
  const dim3 g = blocks(p.batch * p.dim, 256), t(256);
  if (in_bf16 && out_bf16) hipLaunchKernelGGL((glr_step_kernel<uint16_t, uint16_t>), g, t, 0, s, p);
  else if (in_bf16) hipLaunchKernelGGL((glr_step_kernel<uint16_t, float>), g, t, 0, s, p);
  else if (out_bf16) hipLaunchKernelGGL((glr_step_kernel<float, uint16_t>), g, t, 0, s, p);
  else hipLaunchKernelGGL((glr_step_kernel<float, float>), g, t, 0, s, p);
  return hipGetLastError();
}

int64_t glr_bwd_parts(int64_t batch, int64_t seqlen) { return batch * ((seqlen + T * kSubs - 1) / (T * kSubs)); }

hipError_t launch_glr_bwd(const GlrBwdParams &p, int in_bf16, hipStream_t s) {
  if (p.batch > 0 && p.seqlen > 0) {
    const bool pairs = p.dim % 2 == 0 && even(p.x) && even(p.rec) && even(p.inp) && even(p.dy) && even8(p.states) &&
                       even(p.dx) && even(p.drec) && even(p.dinp);
    const hipError_t e = !in_bf16 ? run_bwd<float, 1>(p, s) : pairs ? run_bwd<uint16_t, 2>(p, s) : run_bwd<uint16_t, 1>(p, s);
    if (e != hipSuccess) return e;
  } else if (p.batch > 0 && p.dh0 != nullptr) {
    hipLaunchKernelGGL(glr_pass_kernel, blocks(p.batch * p.dim, 256), dim3(256), 0, s, p.dh_last, p.dh0, p.batch * p.dim);
  }
  hipLaunchKernelGGL(glr_sum_kernel, blocks(p.dim, 64), dim3(1024), 0, s, p.ws_dA, p.dA, glr_bwd_parts(p.batch, p.seqlen),
                     p.dim);
  return hipGetLastError();
}

}  // namespace ssmb
