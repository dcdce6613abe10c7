// Tiles of the sliding-window attention kernels: 64 rows of one head in LDS,
// read as matrix-core operands along the head's elements (rows) or along the
// rows (transposed).
//
// v_mfma_f32_32x32x16_bf16, lane l with m = l % 32, h = l / 32: A holds row m,
// k = 8h .. 8h + 7; B column m, the same k; D column m, rows 8j + 4h + r in
// register 4j + r.  A sum over k does not care for its order as long as A and
// B agree, so where D becomes the next product's B (p and ds), k is counted
// as D's rows lie: element 4j + r of lane half h stands for row 8j + 4h + r of
// 16, and the A operand is read from LDS in that order.  No value crosses
// lanes between the two products.
#pragma once

#include "block_internal.h"

namespace ssmb {

typedef __attribute__((ext_vector_type(8))) __bf16 bf8;
typedef __attribute__((ext_vector_type(4))) __bf16 bf4;
typedef __attribute__((ext_vector_type(4))) short sh4;
typedef __attribute__((ext_vector_type(16))) float f16v;
typedef __attribute__((ext_vector_type(4))) unsigned int u4;

constexpr int kTile = 64;  // rows of a tile

__device__ __forceinline__ f16v mfma(bf8 a, bf8 b, f16v c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// LDS slot of 16-byte chunk c of row r.  Rows are a whole (D = 128) or half
// (D = 64) a turn of the 64 banks, so chunk c of all rows would share its
// banks; c is exchanged with a number made of the row instead.  16 rows in
// turn then fill the 16 slots of the banks (row reads), and so do the four rows
// by four chunks that 32 lanes of a transposed read take: that is why the
// row's lowest bits flip the chunk's highest.
template <int D>
__device__ __forceinline__ int slot(int r, int c) {
  if constexpr (D == 128) return r * 16 + (c ^ (((r & 3) << 2) | ((r >> 2) & 3)));
  else return r * 8 + (c ^ ((((r >> 1) & 1) << 2) | ((r >> 2) & 3)));
}

__device__ __forceinline__ unsigned lds_at(const void *p) {
  return static_cast<unsigned>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)(p)));
}

// Where a lane reads in a tile, in bytes.  The chunk's exchange is an
// exclusive or, so the other operands of a tile lie at one of these two
// addresses with constant bits flipped, plus whole rows: no register per
// operand.
struct Lanes {
  unsigned row, col;
};
template <int D>
__device__ __forceinline__ Lanes lanes_of(int lane) {
  const int i = lane & 15, g = (lane >> 4) & 1, h = lane >> 5;
  return {static_cast<unsigned>(slot<D>(lane & 31, h)) * 16,
          static_cast<unsigned>(slot<D>(4 * h + (i >> 2), g * 2 + ((i >> 1) & 1))) * 16 + (i & 1) * 8};
}

// Operand of rows base .. base + 31, elements 16 s + 8 h .. + 7.
template <int D>
__device__ __forceinline__ bf8 row_operand(const u4 *tile, int base, int s, const Lanes &l) {
  typedef __attribute__((address_space(3))) const u4 lds16;
  return __builtin_bit_cast(bf8, *(lds16 *)(((lds_at(tile) + l.row) ^ (32 * s)) + base * 2 * D));
}

// Operand of elements (columns) 32 db + lane % 32 over rows base .. base + 15
// (base a multiple of 16) in the order above: two transposing reads of 4 rows
// each, 8 rows apart (which flips bit 1 of the chunk's exchange).
template <int D>
__device__ __forceinline__ bf8 col_operand(const u4 *tile, int base, int db, const Lanes &l) {
  typedef __attribute__((address_space(3))) sh4 lds4;
  const unsigned at = (lds_at(tile) + l.col) ^ (64 * db);
  const sh4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(at + base * 2 * D));
  const sh4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)((at ^ 32) + (base + 8) * 2 * D));
  return __builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Registers 8 s .. 8 s + 7 of a D result as the B operand over its rows 16 s .. 16 s + 15.
__device__ __forceinline__ bf8 as_operand(const f16v &d, int s) {
  bf8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = static_cast<__bf16>(d[8 * s + e]);
  return v;
}

// What as_operand() rounded off, as an operand.
__device__ __forceinline__ bf8 left_over(const f16v &d, int s, bf8 rounded) {
  const u4 bits = __builtin_bit_cast(u4, rounded);
  bf8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = static_cast<__bf16>(d[8 * s + e] - __uint_as_float(e % 2 != 0 ? bits[e / 2] & 0xffff0000u : bits[e / 2] << 16));
  return v;
}

// Bits 15 and 31 are set where that half, a bfloat16, is an infinity or NaN.
__device__ __forceinline__ unsigned not_finite(unsigned x) { return (x & 0x7fff7fffu) + 0x00800080u; }

// 1.0 in the halves that equal those of `what`, that are NaN, or that are an
// infinity or NaN, 0 in the others.
__device__ __forceinline__ unsigned is_half(unsigned x, unsigned what) {
  const unsigned t = x ^ what, other = ((t & 0x7fff7fffu) + 0x7fff7fffu) | t;  // bits 15 and 31: not equal
  return ((~other >> 15) & 0x00010001u) * 0x3f80u;
}
__device__ __forceinline__ unsigned is_nan(unsigned x) {
  return ((((x & 0x7fff7fffu) + 0x007f007fu) >> 15) & 0x00010001u) * 0x3f80u;
}
__device__ __forceinline__ unsigned is_not_finite(unsigned x) { return ((not_finite(x) >> 15) & 0x00010001u) * 0x3f80u; }

// An operand with zeros for its infinities and NaN.
__device__ __forceinline__ bf8 only_finite(bf8 operand) {
  u4 v = __builtin_bit_cast(u4, operand);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] &= ~(((not_finite(v[k]) >> 15) & 0x00010001u) * 0xffffu);
  return __builtin_bit_cast(bf8, v);
}

// What the infinities and NaN of 16 NS rows of a tile, from row `base` on, add
// to the columns that see them: out[db] += vis * v over those elements alone.
// vis: 1 or 0 per row, in the order of as_operand().  NANS: each counts as a
// NaN, for factors that are NaN or 0 where the elements are not finite.
template <int D, int NS, bool NANS>
__device__ __forceinline__ void add_not_finite(const u4 *tile, int base, const bf8 (&vis)[NS], f16v (&out)[D / 32],
                                               const Lanes &at) {
#pragma unroll
  for (int db = 0; db < D / 32; ++db) {
    // (Not unrolled: this is rare, and must not cost the others registers.)
#pragma unroll 1
    for (int kind = NANS ? 2 : 0; kind < 3; ++kind) {  // +inf, -inf, NaN
      f16v count = {};
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        u4 v = __builtin_bit_cast(u4, col_operand<D>(tile, base + 16 * s, db, at));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (NANS) v[k] = is_not_finite(v[k]);
          else v[k] = kind == 2 ? is_nan(v[k]) : is_half(v[k], kind == 0 ? 0x7f807f80u : 0xff80ff80u);
        }
        count = mfma(__builtin_bit_cast(bf8, v), vis[s], count);
      }
      const float add = kind == 0 ? INFINITY : kind == 1 ? -INFINITY : NAN;
#pragma unroll
      for (int i = 0; i < 16; ++i) out[db][i] += count[i] > 0.0f ? add : 0.0f;
    }
  }
}

// The row that register i of a D result stands for in lane half h.
__device__ __forceinline__ constexpr int d_row(int i, int h) { return 8 * (i / 4) + 4 * h + i % 4; }

// Copy 16 bytes per lane from base + off to LDS, from `lds` on in lane order.
// The copy goes from memory to LDS without registers.  In asm, because the
// compiler would wait for it before any LDS read, of another buffer too:
// wait_tiles() waits for it.
__device__ __forceinline__ void copy16(unsigned lds, const void *base, unsigned off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void copy16(unsigned lds, const void *at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(at) : "memory", "m0");
}
// Start the copy of tile rows t0 .. t0 + ROWS - 1 of a strided tensor (p: row
// 0 of the head) into LDS, `NT` threads taking part; rows past `last` are read
// as row `last`, so nothing past a length is touched.  A wavefront's 64 pieces
// land in order, so the slots are permuted by the source address.
template <int D, int NT, int ROWS = kTile>
__device__ __forceinline__ void load_tile(u4 *tile, const uint16_t *p, int64_t token, int t0, int last, int tid) {
  constexpr int CH = D / 8;
  const uint16_t *base = p + t0 * token;
  const unsigned stride = static_cast<unsigned>(token) * 2;  // at most 2^25 bytes, so 63 rows fit 32 bits
  const unsigned lds = __builtin_amdgcn_readfirstlane(lds_at(tile) + (tid & ~63) * 16);
#pragma unroll
  for (int k = 0; k < ROWS * CH / NT; ++k) {
    const int id = k * NT + tid, r = id / CH;
    const int c = slot<D>(r, id % CH) - r * CH;  // slot() is its own inverse within a row
    copy16(lds + k * NT * 16, base, static_cast<unsigned>(r < last - t0 ? r : last - t0) * stride + c * 16);
  }
}

// The keys that some queries see, in one row: the sinks before the window,
// 0 .. first - 1, then the keys from `low` on.
struct KeyRow {
  int first, low;
  __device__ __forceinline__ int key(int v) const { return v < first ? v : v - first + low; }
};
__device__ __forceinline__ KeyRow key_row(int q0, int window, int sinks) {
  KeyRow k;
  k.low = q0 - window + 1 > 0 ? q0 - window + 1 : 0;
  k.first = sinks < k.low ? sinks : k.low;
  return k;
}

// Which places of such a row, c past v0 for this lane half, query t sees: those
// through the window count down from `ahead`, and sinks are the first ones (the
// keys before the window, or, where the window starts among the sinks, the
// first `own`).  Two comparisons with constants and a subtraction per place.
struct Seen {
  int ahead, own;
  unsigned window;
  __device__ __forceinline__ bool operator()(int c) const {
    return static_cast<unsigned>(ahead - c) < window || c < own;
  }
};
__device__ __forceinline__ Seen seen_by(const KeyRow &k, int t, int v0, int half, int window, int sinks) {
  const int own = k.first < k.low ? k.first : sinks < t + 1 ? sinks : t + 1;
  return {t - (v0 - k.first + k.low) - 4 * half, own - v0 - 4 * half, static_cast<unsigned>(window)};
}

// load_tile() for the places v0 .. v0 + 63 of such a row.
template <int D, int NT>
__device__ __forceinline__ void load_keys(u4 *tile, const uint16_t *p, int64_t token, const KeyRow &row, int v0, int last,
                                          int tid) {
  if (v0 >= row.first) {
    load_tile<D, NT>(tile, p, token, row.key(v0), last, tid);
    return;
  }
  constexpr int CH = D / 8;
  const unsigned lds = __builtin_amdgcn_readfirstlane(lds_at(tile) + (tid & ~63) * 16);
#pragma unroll
  for (int k = 0; k < kTile * CH / NT; ++k) {
    const int id = k * NT + tid, r = id / CH, j = row.key(v0 + r);
    const int c = slot<D>(r, id % CH) - r * CH;
    copy16(lds + k * NT * 16, p + (j < last ? j : last) * token + c * 8);
  }
}

// The same for one float of each of the rows t0 .. t0 + 63, by one wavefront.
__device__ __forceinline__ void load_stats(float *to, const float *p, int t0, int last, int lane) {
  const unsigned off = static_cast<unsigned>(lane < last - t0 ? lane : last - t0) * 4;
  const unsigned lds = __builtin_amdgcn_readfirstlane(lds_at(to));
  const float *base = p + t0;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}

// All but the last N copies this wavefront has started have landed.
template <int N = 0>
__device__ __forceinline__ void wait_tiles() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Order of N matrix products and the N LDS reads of their A operands in this
// block of code: six reads ahead of the products (left to itself the compiler
// keeps one ahead, and each product waits for LDS).
template <int N>
__device__ __forceinline__ void reads_ahead() {
  constexpr int kAhead = N < 12 ? N / 2 : 6;
  __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
  for (int i = 0; i < (N - kAhead) / 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
}

// Every LDS read this wavefront has started has its value: the copies that
// follow may overwrite what it read.
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ float other_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// The running maximum is raised (and what is summed so far scaled down) only
// when a score passes it by this factor's log2: weights stay below 2^8, which
// costs no precision in float32 or bfloat16.
constexpr float kSlack = 8.0f;

// Scores of 64 keys (rows) for the lane's query -> weights 2^(c2 s - top),
// with the running maximum `top` (in units of log2) raised where it must be,
// `sum` (of this lane's half of the keys) and o taken along.
template <int NB>
__device__ __forceinline__ void to_weights(f16v (&s)[2], float c2, f16v (&o)[NB], float &top, float &sum) {
  float m = s[0][0];
#pragma unroll
  for (int r = 1; r < 32; ++r) m = fmaxf(m, s[r / 16][r % 16]);
  m = fmaxf(m, other_half(m)) * c2;
  if (__any(m > top + kSlack)) {
    const float now = m > top + kSlack ? m : top;  // by each query for itself: no row's bits depend on another's
    const float keep = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(top - now);
    sum *= keep;
#pragma unroll
    for (int db = 0; db < NB; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[db][r] *= keep;
    top = now;
  }
  const float off = top == -INFINITY ? 0.0f : top;
  float part[2] = {};
#pragma unroll
  for (int blk = 0; blk < 2; ++blk)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[blk][r] = __builtin_amdgcn_exp2f(fmaf(s[blk][r], c2, -off));
      part[r & 1] += s[blk][r];
    }
  sum += part[0] + part[1];
}

__device__ __forceinline__ int row_length(const SwaParams &p, int64_t b) {
  if (p.lengths == nullptr) return static_cast<int>(p.seqlen);
  const int n = p.lengths[b], L = static_cast<int>(p.seqlen);
  return n < 0 ? 0 : n > L ? L : n;
}

// Workgroup number -> work number: the hardware deals workgroups out to the 8
// XCDs in turn, and each XCD has its own L2, in which neighbouring tiles of a
// head should find the same keys.  Work goes by key head, then batch row, so
// where the `groups` of both share out evenly each XCD gets a contiguous range
// with every row in it: unequal lengths leave no XCD idle (4 rows of up to 2048
// tokens, mean 0.63 of them, 32 heads on 8, window 512: forward 45 us, with row
// before head 64).  Else an XCD gets 8 neighbours of every 64, another 8 of the
// next 64 (3 such rows of 1500 tokens, 16 heads on 2: 28 -> 24 us).
__device__ __forceinline__ unsigned xcd_order(unsigned id, unsigned n, unsigned groups) {
  const unsigned x = id & 7, k = id >> 3;
  if (groups % 8 == 0) return x * (n >> 3) + k;
  return id < n / 64 * 64 ? k / 8 * 64 + (x + k / 8) % 8 * 8 + k % 8 : id;
}

// Most queries see a part of the window only, a later one more than an earlier
// one: longer work goes first, and is cut up more.
__host__ __device__ inline bool uneven(int64_t window, int64_t seqlen) { return 2 * window > seqlen; }

}  // namespace ssmb
