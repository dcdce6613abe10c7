// One token of sliding-window attention against a ring cache in e4m3 floats
// with a scale per block of 64 positions and head, and the ring's fill from a
// prompt, for gfx950.
//
// A block's scale is known only when its last position has come, and a value
// should be rounded once: so the block that is being filled stays in bfloat16,
// beside the sinks ("near"), and is stored in 8 bits, all at once, by the step
// that completes it.  The step is bound by memory like the one over a bfloat16
// ring, at half its bytes: a wavefront streams tiles of 8 KiB (a block of the
// ring, or 32 near positions; headdim 64: half) into LDS of its own, without
// registers or barriers.  e4m3 values become bfloat16, exactly, as they are
// read from LDS, keys along their elements and values transposed; the scales
// multiply the scores and the weights, in float32.  The weights enter the
// product in two parts (2^-16), as those over a bfloat16 ring do: the rest of
// the error is the cache's own rounding.  Heads that share a key head are the
// matrix instruction's 16 columns, 16 at a time (32 at a time, with half of
// them empty in groups of four, took 170 us where 16 took 95).
//
// Measured: 64 sequences, 32 heads of 128 on 8, windows of up to 4096 in 84 to
// 88 us a call, 4.6 to 4.8 TB/s of the cache's bytes, where a large copy reaches 4.8; 4
// sequences, 16 heads on 4, window 1024: 11 us, of a call's 12, all latency.
#include "block/swa_step.h"
#include "delta_internal.h"
#include "gdr_tile.h"

namespace ssmb {
namespace {

constexpr int kMaxSplits = 1024;
typedef __attribute__((ext_vector_type(2))) int i2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf2;

// Eight e4m3 bytes as an operand.
__device__ __forceinline__ bf8 widen(i2 v) {
  bf8 r;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const bf2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[k], 1.0f, false);
    const bf2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[k], 1.0f, true);
    r[4 * k] = lo[0];
    r[4 * k + 1] = lo[1];
    r[4 * k + 2] = hi[0];
    r[4 * k + 3] = hi[1];
  }
  return r;
}

// Place of 16-byte chunk c of row r in a ring tile in LDS, exchanged so that
// neighbouring rows' equal chunks lie on other banks.
template <int D>
__device__ __forceinline__ int chunk8(int r, int c) {
  if constexpr (D == 128) return c ^ ((r >> 1) & 7);
  else return c ^ ((r >> 2) & 3);
}

// Operand of keys 16 i .. (lane m), elements 32 a + 8g ..
template <int D>
__device__ __forceinline__ bf8 keys16(const u4 *tile, int i, int a, int lane) {
  typedef __attribute__((address_space(3))) const i2 lds8;
  const int r = 16 * i + (lane & 15), g = lane >> 4;
  return widen(*(lds8 *)(lds_at(tile) + r * D + chunk8<D>(r, 2 * a + (g >> 1)) * 16 + (g & 1) * 8));
}
// Operand of elements 16 e + m over keys 32 s .. in the order of a D result.
template <int D>
__device__ __forceinline__ bf8 values16(const u4 *tile, int s, int e, int lane) {
  typedef __attribute__((address_space(3))) i2 lds8;
  const int i = lane & 15, g = lane >> 4, k = i >> 1;  // lanes 2 k and 2 k + 1 read key k of the group's eight
  const int r = 32 * s + 16 * (k >> 2) + 4 * g + (k & 3);
  return widen(__builtin_amdgcn_ds_read_tr8_b64_v2i32((lds8 *)(lds_at(tile) + r * D + chunk8<D>(r, e) * 16 + (i & 1) * 8)));
}
// Start the copy of a block of the ring.
template <int D>
__device__ __forceinline__ void load_block(u4 *tile, const uint8_t *block, int lane) {
  const unsigned lds = __builtin_amdgcn_readfirstlane(lds_at(tile));
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const int id = k * 64 + lane, r = id / (D / 16);
    copy16(lds + k * 1024, block, static_cast<unsigned>(r * D + chunk8<D>(r, id % (D / 16)) * 16));
  }
}

// A block's scale. `top`: the largest |value|'s bits, NaN above all.
__device__ __forceinline__ float scale_of(unsigned top) { return __uint_as_float(top) / 448.0f; }
__device__ __forceinline__ float hold(float v) { return v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v; }
// Eight bfloat16 as bytes.  A true division: a product with the reciprocal
// would put quotients that lie between two bytes on either side.
__device__ __forceinline__ uint2 to_e4m3(const u4 &v, float scale) {
  const float s = scale != 0.0f ? scale : 1.0f;
  uint2 out;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int b = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const unsigned pair = v[2 * k + x];
      const float lo = hold(__uint_as_float(pair << 16) / s), hi = hold(__uint_as_float(pair & 0xffff0000u) / s);
      b = x != 0 ? __builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, b, true) : __builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, b, false);
    }
    (k != 0 ? out.y : out.x) = static_cast<unsigned>(b);
  }
  return out;
}
// The larger of the magnitudes' bits (NaN above infinity above all).
__device__ __forceinline__ unsigned top_of(unsigned top, const u4 &v) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const unsigned lo = v[k] << 16 & 0x7fff0000u, hi = v[k] & 0x7fff0000u;
    top = top > lo ? top : lo;
    top = top > hi ? top : hi;
  }
  return top;
}
__device__ __forceinline__ unsigned wave_top(unsigned top) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const unsigned other = __shfl_xor(top, d);
    top = top > other ? top : other;
  }
  return top;
}

// One wavefront stores 64 near positions, the last of them from the
// arguments, as a block of the ring.
template <int D>
__device__ __forceinline__ void store_block(const uint16_t *near, const uint16_t *own, uint8_t *block, float *scale, int lane) {
  constexpr int CH = D / 8;
  u4 v[CH];
  unsigned top = 0;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int id = k * 64 + lane, r = id / CH, c = id % CH;
    v[k] = *reinterpret_cast<const u4 *>((r == 63 ? own : near + r * D) + c * 8);
    top = top_of(top, v[k]);
  }
  const float s = scale_of(wave_top(top));
#pragma unroll
  for (int k = 0; k < CH; ++k) reinterpret_cast<uint2 *>(block)[k * 64 + lane] = to_e4m3(v[k], s);
  if (lane == 0) *scale = s;
}

// The value of the lane 16 away within its 32.
__device__ __forceinline__ float other_row(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float((threadIdx.x & 16) ? r[0] : r[1]);
}

// Weights as two operands whose sum they are to 2^-16: cut off after 8 bits, and
// what that leaves.  INF, where values may be infinities: held above 0, so that
// both times an infinity have its sign.  (Not with a block's bytes, which are
// not infinite: its scale is in the weights already, and the least that is held
// would be added to what may be smaller.)
template <bool INF>
__device__ __forceinline__ void two_parts(const f4v &lo, const f4v &hi, bf8 &cut, bf8 &rest) {
  u4 c;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = k < 2 ? lo[2 * (k % 2)] : hi[2 * (k % 2)], b = k < 2 ? lo[2 * (k % 2) + 1] : hi[2 * (k % 2) + 1];
    const unsigned ca = __float_as_uint(a) & 0xffff0000u, cb = __float_as_uint(b) & 0xffff0000u;
    c[k] = ca >> 16 | cb;
    const float ra = a - __uint_as_float(ca), rb = b - __uint_as_float(cb);
    rest[2 * k] = static_cast<__bf16>(INF ? fmaxf(ra, 0x1p-100f) : ra);
    rest[2 * k + 1] = static_cast<__bf16>(INF ? fmaxf(rb, 0x1p-100f) : rb);
  }
  cut = __builtin_bit_cast(bf8, c);
}

// Scores of 64 keys for the lane's head -> weights 2^(c2 s - top), with the
// running maximum and sum of this lane's quarter of the keys, and o, as
// to_weights() in swa_tile.h.
template <int NB>
__device__ __forceinline__ void weigh(f4v (&s)[4], float c2, f4v (&o)[NB], float &top, float &sum) {
  float m = s[0][0];
#pragma unroll
  for (int r = 1; r < 16; ++r) m = fmaxf(m, s[r / 4][r % 4]);
  m = fmaxf(m, other_row(m));
  m = fmaxf(m, other_half(m)) * c2;
  if (__any(m > top + kSlack)) {
    const float now = m > top + kSlack ? m : top;
    const float keep = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(top - now);
    sum *= keep;
#pragma unroll
    for (int e = 0; e < NB; ++e) o[e] *= keep;
    top = now;
  }
  const float off = top == -INFINITY ? 0.0f : top;
  float part[2] = {};
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    s[r / 4][r % 4] = __builtin_amdgcn_exp2f(fmaf(s[r / 4][r % 4], c2, -off));
    part[r & 1] += s[r / 4][r % 4];
  }
  sum += part[0] + part[1];
}

// Heads that share a key head, 16 at a time, as columns; NW wavefronts share the tiles.
template <int D, int NW>
__global__ void __launch_bounds__(64 * NW, 2) swa_q8_step_kernel(const SwaStepParams p, const SwaQ8Cache cache, unsigned splits,
                                                             unsigned qblocks) {
  constexpr int CH = D / 8, NB = D / 16, NS = D / 32, kNear = 32;
  constexpr int kCopies = D / 16;  // copies of 1 KiB per tile, of either kind
  __shared__ __align__(16) u4 lds[NW][2][kSwaBlock * D / 16];  // wavefront, K or V; in the end o, [16][D] float32
  __shared__ float tops[NW][16], sums[NW][16];
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned nkv = static_cast<unsigned>(p.nkv), group = static_cast<unsigned>(p.nheads) / nkv;
  // First a workgroup per (row, key head) that stores the near block in the
  // ring if it has become whole; then `splits` for each block of 16 heads.
  // (Beside those of their row, the ones that mostly have nothing to do would
  // all fall to the same XCDs: 100 sequences, 8 key heads of 128, window 1024,
  // 3 splits 66 us, now 46.)
  const unsigned rows = static_cast<unsigned>(p.batch) * nkv, each_row = splits * qblocks;
  const bool stores = blockIdx.x < rows;
  const unsigned id = stores ? blockIdx.x * each_row : blockIdx.x - rows, bc = id / each_row, rest = id % each_row;
  const unsigned split = rest % splits, qb = rest / splits;
  const int64_t b = bc / nkv, c = bc % nkv;
  const int g0 = qb * 16, heads = static_cast<int>(group) - g0 < 16 ? static_cast<int>(group) - g0 : 16;
  const int sinks = static_cast<int>(p.sinks), blocks = static_cast<int>(p.window / kSwaBlock);
  const int pos = p.pos[b] < 0 ? -1 : p.pos[b];
  // Of the positions behind the sinks, `spot` is the token's: blocks before
  // `now` are whole, and in the ring; place `off` of the near block is its own.
  const int spot = pos - sinks, now = spot >> 6, off = spot & 63;
  const int count = pos < sinks ? pos + 1 : sinks + off + 1, own = count - 1;  // near positions, the token the last
  const uint16_t *kn = p.k + b * p.k_batch + c * D, *vn = p.v + b * p.v_batch + c * D;
  uint16_t *near_k = cache.k_near + static_cast<int64_t>(bc) * (sinks + kSwaBlock) * D;
  uint16_t *near_v = cache.v_near + static_cast<int64_t>(bc) * (sinks + kSwaBlock) * D;
  if (stores) {
    if (pos < sinks || off != 63) return;
    // (No other workgroup reads the block of the ring that it replaces, nor writes what is near but the token's own place.)
    const int64_t to = static_cast<int64_t>(bc) * blocks + now % blocks;
    if (wave == 0)
      store_block<D>(near_k + static_cast<int64_t>(sinks) * D, kn, cache.k_ring + to * kSwaBlock * D, cache.k_scale + to, lane);
    else if (wave == 1)
      store_block<D>(near_v + static_cast<int64_t>(sinks) * D, vn, cache.v_ring + to * kSwaBlock * D, cache.v_scale + to, lane);
    return;
  }
  f4v o[NB] = {};
  float top = -INFINITY, sum = 0.0f;
  if (pos >= 0) {
    const int64_t ring = static_cast<int64_t>(bc) * p.window * D, scales = static_cast<int64_t>(bc) * blocks;
    const int near_tiles = (count + kNear - 1) / kNear;
    // Blocks of the ring that are seen: all whole ones, and of the one that
    // the near block will replace the places behind `off`.
    const int held = spot < 0 ? 0 : now < blocks ? now : blocks;
    const int old = now >= blocks ? now % blocks : -1;
    const int skip = old >= 0 && off == 63 ? old : blocks;  // it has no such places
    const int tiles = near_tiles + (skip < blocks ? held - 1 : held);
    const unsigned parts = splits * NW, part = split * NW + wave;
    const unsigned each = tiles / parts, more = tiles % parts;
    const int lo = static_cast<int>(each * part + (part < more ? part : more));
    const int hi = lo + static_cast<int>(each + (part < more ? 1 : 0));
    u4 *kt = lds[wave][0], *vt = lds[wave][1];
    const Lanes16 at = lanes16_of<D>(lane);
    auto block_of = [&](int i) { return i - near_tiles + (i - near_tiles >= skip ? 1 : 0); };
    auto load = [&](u4 *tile, const uint16_t *near, const uint8_t *bytes, int i) {
      if (i < near_tiles) load_tile<D, 64, kNear>(tile, near, D, i * kNear, own, lane);
      else load_block<D>(tile, bytes + ring + static_cast<int64_t>(block_of(i)) * kSwaBlock * D, lane);
    };
    if (lo < hi) {
      bf8 q[NS];
      const int row = m < heads ? m : 0;  // lanes past the group repeat its first head
      const u4 *src = reinterpret_cast<const u4 *>(p.q + b * p.q_batch + (c * group + g0 + row) * D);
#pragma unroll
      for (int a = 0; a < NS; ++a) {
        u4 v = src[4 * a + g];
        if (p.scale < 0.0f) v ^= 0x80008000u;  // a negative scale is taken as -q
        q[a] = __builtin_bit_cast(bf8, v);
      }
      const float c2 = fabsf(p.scale) * kLog2e;
      float k_scale = 0.0f, v_scale = 0.0f;  // lane l: those of tile i + l, for every 64th i
#pragma unroll 1
      for (int i = lo; i < hi; ++i) {
        if (((i - lo) & 63) == 0) {
          if (i == lo) {
            load(kt, near_k, cache.k_ring, i);
            load(vt, near_v, cache.v_ring, i);
          }
          const int mine = i + lane < hi ? i + lane : hi - 1;
          k_scale = mine < near_tiles ? 1.0f : cache.k_scale[scales + block_of(mine)];
          v_scale = mine < near_tiles ? 1.0f : cache.v_scale[scales + block_of(mine)];
        }
        const float ks = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(k_scale), (i - lo) & 63));
        const float vs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v_scale), (i - lo) & 63));
        const bool near = i < near_tiles;
        const int k0 = i * kNear;
        const bool has = near && own >= k0 && own < k0 + kNear;
        wait_tiles<kCopies>();  // the keys: all but the copies of the values
        f4v s[4] = {};
        if (near) {
          if (has) put_row<D>(kt, kn, own - k0, lane);
#pragma unroll
          for (int a = 0; a < NS; ++a)
#pragma unroll
            for (int x = 0; x < 2; ++x) s[x] = mfma16(row16<D>(lds_at(kt), x, a, at), q[a], s[x]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (k0 + 16 * x + 4 * g + r >= count) s[x][r] = -INFINITY;
            s[2][r] = s[3][r] = -INFINITY;
          }
        } else {
#pragma unroll
          for (int a = 0; a < NS; ++a)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[x] = mfma16(keys16<D>(kt, x, a, lane), q[a], s[x]);
          const int from = block_of(i) == old ? off : -1;
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (16 * x + 4 * g + r <= from) s[x][r] = -INFINITY;
        }
        wait_reads();
        if (i + 1 < hi) load(kt, near_k, cache.k_ring, i + 1);
        weigh(s, fmaxf(c2 * ks, 0x1p-100f), o, top, sum);
        if (i + 1 < hi) wait_tiles<kCopies>();  // the values: all but the copies of the next keys
        else wait_tiles<0>();
        if (near) {
          if (has) put_row<D>(vt, vn, own - k0, lane);
          // Rows behind the token repeat its slot, which may hold anything.
          for (int r = own + 1 - k0 + lane / CH; has && r < kNear; r += 64 / CH) vt[slot<D>(r, lane % CH)] = u4{};
          bf8 cut, left;
          two_parts<true>(s[0], s[1], cut, left);
#pragma unroll
          for (int e = 0; e < NB; ++e) {
            const bf8 v = elems16<D>(lds_at(vt), e, 0, lane);
            o[e] = mfma16(v, left, mfma16(v, cut, o[e]));
          }
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            bf8 cut, left;
            two_parts<false>(s[2 * x] * vs, s[2 * x + 1] * vs, cut, left);
#pragma unroll
            for (int e = 0; e < NB; ++e) {
              const bf8 v = values16<D>(vt, x, e, lane);
              o[e] = mfma16(v, left, mfma16(v, cut, o[e]));
            }
          }
        }
        wait_reads();
        if (i + 1 < hi) load(vt, near_v, cache.v_ring, i + 1);
        if (has && lane < CH) {  // the token takes its place
          reinterpret_cast<u4 *>(near_k + static_cast<int64_t>(own) * D)[lane] = reinterpret_cast<const u4 *>(kn)[lane];
          reinterpret_cast<u4 *>(near_v + static_cast<int64_t>(own) * D)[lane] = reinterpret_cast<const u4 *>(vn)[lane];
        }
      }
    }
    sum += other_row(sum);
    sum += other_half(sum);
  }
  // Join the wavefronts.
  float *mine = reinterpret_cast<float *>(lds[wave]);
#pragma unroll
  for (int e = 0; e < NB; ++e) *reinterpret_cast<f4v *>(mine + m * D + 16 * e + 4 * g) = o[e];
  if (g == 0) {
    tops[wave][m] = top;
    sums[wave][m] = sum;
  }
  __syncthreads();
  for (int i = tid; i < heads * D; i += 64 * NW) {
    const int row = i / D, e = i % D;
    float best = tops[0][row];
#pragma unroll
    for (int w = 1; w < NW; ++w) best = fmaxf(best, tops[w][row]);
    // (A share without a maximum holds zeros, or the NaN that all its scores were.)
    float acc = 0.0f, all = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = tops[w][row] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(tops[w][row] - best);
      acc = fmaf(f, reinterpret_cast<const float *>(lds[w])[row * D + e], acc);
      all = fmaf(f, sums[w][row], all);
    }
    const int64_t head = b * p.nheads + c * group + g0 + row;
    if (splits == 1) {
      st(p.y, head * D + e, all == 0.0f ? 0.0f : acc / all);
    } else {
      p.ws_o[(head * splits + split) * D + e] = acc;
      if (e == 0) {
        p.ws_stat[(head * splits + split) * 2] = best;
        p.ws_stat[(head * splits + split) * 2 + 1] = all;
      }
    }
  }
}

// Join the splits of a head.  The splits' factors, which all its elements take,
// are made first, by all threads; then 256 / D threads share an element.
template <int D>
__global__ void __launch_bounds__(256) swa_q8_join_kernel(const SwaStepParams p, int splits) {
  constexpr int NG = 256 / D;
  __shared__ float factor[kMaxSplits], best_of[4], all_of[4], sums[NG][D];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t head = blockIdx.x;
  const float *stat = p.ws_stat + head * splits * 2, *part = p.ws_o + head * splits * D;
  float best = -INFINITY, all = 0.0f;
  for (int k = tid; k < splits; k += 256) best = fmaxf(best, stat[2 * k]);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) best = fmaxf(best, __shfl_xor(best, d));
  if (lane == 0) best_of[w] = best;
  __syncthreads();
  best = fmaxf(fmaxf(best_of[0], best_of[1]), fmaxf(best_of[2], best_of[3]));
  for (int k = tid; k < splits; k += 256) {
    const float f = stat[2 * k] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(stat[2 * k] - best);
    factor[k] = f;
    all = fmaf(f, stat[2 * k + 1], all);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) all += __shfl_xor(all, d);
  if (lane == 0) all_of[w] = all;
  __syncthreads();
  const int e = tid % D, group = tid / D;
  float acc = 0.0f;
#pragma unroll 8
  for (int k = group; k < splits; k += NG) acc = fmaf(factor[k], part[static_cast<int64_t>(k) * D + e], acc);
  sums[group][e] = acc;
  __syncthreads();
  if (group != 0) return;
#pragma unroll
  for (int k = 1; k < NG; ++k) acc += sums[k][e];
  all = (all_of[0] + all_of[1]) + (all_of[2] + all_of[3]);
  st(p.y, head * D + e, all == 0.0f ? 0.0f : acc / all);
}

// A workgroup per (row, key head, block of the ring), and one for what is
// near.  Block r of the ring holds, of the `whole` complete blocks of the
// row's positions behind the sinks, the last whose number is r mod the ring's.
template <int D>
__global__ void __launch_bounds__(256) swa_q8_fill_kernel(const SwaParams p, const SwaQ8Cache cache) {
  constexpr int CH = D / 8, kEach = kSwaBlock * CH / 256;
  __shared__ unsigned tops[2][4];
  const int tid = threadIdx.x, blocks = static_cast<int>(p.window / kSwaBlock);
  const int64_t items = blocks + 1, all = p.batch * p.nkv * items;
  for (int64_t id = blockIdx.x; id < all; id += gridDim.x) {
    const int64_t r = id % items, bc = id / items, c = bc % p.nkv, b = bc / p.nkv;
    const int64_t n = row_length(p, b), behind = n > p.sinks ? n - p.sinks : 0, whole = behind / kSwaBlock;
    const uint16_t *src[2] = {p.k + b * p.k_batch + c * D, p.v + b * p.v_batch + c * D};
    const int64_t token[2] = {p.k_token, p.v_token};
    if (r == blocks) {
      const int64_t slots = p.sinks + kSwaBlock;
      uint16_t *near[2] = {cache.k_near + bc * slots * D, cache.v_near + bc * slots * D};
      for (int64_t i = tid; i < slots * CH; i += 256) {
        const int64_t s = i / CH, e = i % CH * 8, pos = s < p.sinks ? s : s + whole * kSwaBlock;
        if (pos < n)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            *reinterpret_cast<u4 *>(near[t] + s * D + e) = *reinterpret_cast<const u4 *>(src[t] + pos * token[t] + e);
      }
      continue;
    }
    if (r >= whole) continue;
    const int64_t pos = p.sinks + (r + (whole - 1 - r) / blocks * blocks) * kSwaBlock;
    // (All reads first: in turns with the maxima they took 58 us, not 45, for 8
    // prompts, a window of 4096 and 8 heads of 128; 4.5 TB/s.)
    u4 v[2][kEach];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int at = k * 256 + tid;
        v[t][k] = *reinterpret_cast<const u4 *>(src[t] + (pos + at / CH) * token[t] + at % CH * 8);
      }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      unsigned top = 0;
#pragma unroll
      for (int k = 0; k < kEach; ++k) top = top_of(top, v[t][k]);
      top = wave_top(top);
      if ((tid & 63) == 0) tops[t][tid >> 6] = top;
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      unsigned top = tops[t][0];
#pragma unroll
      for (int w = 1; w < 4; ++w) top = top > tops[t][w] ? top : tops[t][w];
      const float s = scale_of(top);
      uint2 *to = reinterpret_cast<uint2 *>((t == 0 ? cache.k_ring : cache.v_ring) + (bc * blocks + r) * kSwaBlock * D);
#pragma unroll
      for (int k = 0; k < kEach; ++k) to[k * 256 + tid] = to_e4m3(v[t][k], s);
      if (tid == 0) (t == 0 ? cache.k_scale : cache.v_scale)[bc * blocks + r] = s;
    }
    __syncthreads();
  }
}

}  // namespace

SwaQ8Plan swa_q8_plan(int64_t batch, int64_t nheads, int64_t nkv, int64_t window, int64_t sinks) {
  // As many workgroups as there is LDS for at once, two per CU, while a wavefront
  // has a tile; up to three tiles each it is as fast not to split, without the
  // join's launch.  32 heads on 8 of 128: 64 sequences, window 4096, 1 split 104
  // us, 2 and their join 110; 64, window 1024, 29 and 37; 4, window 4096, 16
  // splits 15, 18 (of a tile each) 18; 32, window 256, 1 split 9, 2 13.
  // Eight wavefronts, where a CU has one workgroup anyway, do so up to 24 tiles:
  // 8 sequences, window 1024, 12 us, 4 wavefronts and splits 14; 30, 18 and 27; 1
  // of 8 heads on 1, window 512, 8.7, 4 wavefronts alone 10.2.
  const int64_t rows = batch * nkv * ((nheads / nkv + 15) / 16), tiles = window / kSwaBlock + (sinks + kSwaBlock + 31) / 32;
  if (tiles <= 24 && rows <= 256) return {1, 8};
  if (tiles <= 12) return {1, 4};
  const int64_t want = (512 + rows - 1) / (rows > 0 ? rows : 1), most = (tiles + 3) / 4;
  const int64_t n = want < most ? want : most;
  return {static_cast<int>(n < kMaxSplits ? n : kMaxSplits), 4};
}

namespace {
template <int D>
void step(const SwaStepParams &p, const SwaQ8Cache &cache, const SwaQ8Plan &plan, hipStream_t s) {
  const unsigned qblocks = static_cast<unsigned>((p.nheads / p.nkv + 15) / 16), splits = static_cast<unsigned>(plan.splits);
  const dim3 g(static_cast<uint32_t>(p.batch * p.nkv * (qblocks * splits + 1)));
  if (plan.waves == 4) hipLaunchKernelGGL((swa_q8_step_kernel<D, 4>), g, dim3(256), 0, s, p, cache, splits, qblocks);
  else hipLaunchKernelGGL((swa_q8_step_kernel<D, 8>), g, dim3(512), 0, s, p, cache, splits, qblocks);
  if (splits > 1)
    hipLaunchKernelGGL((swa_q8_join_kernel<D>), dim3(static_cast<uint32_t>(p.batch * p.nheads)), dim3(256), 0, s, p, plan.splits);
}
}  // namespace

hipError_t launch_swa_q8_step(const SwaStepParams &p, const SwaQ8Cache &cache, const SwaQ8Plan &plan, hipStream_t s) {
  p.headdim == 64 ? step<64>(p, cache, plan, s) : step<128>(p, cache, plan, s);
  return hipGetLastError();
}

hipError_t launch_swa_q8_fill(const SwaParams &p, const SwaQ8Cache &cache, hipStream_t s) {
  const int64_t n = p.batch * p.nkv * (p.window / kSwaBlock + 1);
  if (n == 0) return hipSuccess;
  const dim3 g(static_cast<uint32_t>(n < kMaxGroups ? n : kMaxGroups));
  if (p.headdim == 64) hipLaunchKernelGGL((swa_q8_fill_kernel<64>), g, dim3(256), 0, s, p, cache);
  else hipLaunchKernelGGL((swa_q8_fill_kernel<128>), g, dim3(256), 0, s, p, cache);
  return hipGetLastError();
}

}  // namespace ssmb
