// Matrix-core operands of the gated delta rule's kernels.
//
// v_mfma_f32_16x16x32_bf16, lane l with m = l % 16, g = l / 16: A holds row m,
// k = 8g .. 8g + 7; B column m, the same k; D column m, rows 4g + r in
// register r.  Two D results, rows 0 .. 15 and 16 .. 31 of 32, become the next
// product's B without crossing lanes when k is counted in their order: element
// e of lane group g stands for row 16 (e / 4) + 4g + e % 4 of the 32, and A is
// read, or was stored, in that order ("D's order").  So a column of a chunk's
// products and of the state stays in its lanes from one chunk to the next:
// the state is a D result whose rows are key elements (32 a + 8g + 4x + r in
// register r of block 2a + x, which makes them B's plain order), the products
// of a chunk have the tokens as rows.
//
// A float32 factor enters a product as two bfloat16 parts that hold it to
// 2^-18 of its size, or three (2^-26); products of two such factors leave out
// the smallest term.  q, k, v and dy are bfloat16 already and enter as they are.
#pragma once

#include <type_traits>

#include "gdr_internal.h"
#include "block/swa_tile.h"

namespace ssmb {

typedef __attribute__((ext_vector_type(4))) float f4v;
typedef __attribute__((ext_vector_type(2))) unsigned int u2;

__device__ __forceinline__ f4v mfma16(bf8 a, bf8 b, f4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4v mfma_f32(float a, float b, f4v c) {  // 16x16x4: k = lane / 16
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Eight float32 values as an operand, and what that rounded off as another.
struct Parts {
  bf8 hi, lo;
};
__device__ __forceinline__ Parts parts(const f4v &a, const f4v &b) {
  Parts p;
#pragma unroll
  for (int e = 0; e < 8; ++e) p.hi[e] = static_cast<__bf16>(e < 4 ? a[e % 4] : b[e % 4]);
  const u4 bits = __builtin_bit_cast(u4, p.hi);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float up = __uint_as_float(e % 2 != 0 ? bits[e / 2] & 0xffff0000u : bits[e / 2] << 16);
    p.lo[e] = static_cast<__bf16>((e < 4 ? a[e % 4] : b[e % 4]) - up);
  }
  return p;
}

// And what that left off: 2^-27 of their size.
struct Parts3 : Parts {
  bf8 rest;
};
__device__ __forceinline__ Parts3 parts3(const f4v &a, const f4v &b) {
  Parts3 p;
  static_cast<Parts &>(p) = parts(a, b);
  const u4 hi = __builtin_bit_cast(u4, p.hi), lo = __builtin_bit_cast(u4, p.lo);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = __uint_as_float(e % 2 != 0 ? hi[e / 2] & 0xffff0000u : hi[e / 2] << 16);
    const float y = __uint_as_float(e % 2 != 0 ? lo[e / 2] & 0xffff0000u : lo[e / 2] << 16);
    p.rest[e] = static_cast<__bf16>((e < 4 ? a[e % 4] : b[e % 4]) - x - y);
  }
  return p;
}

// The first or second four of an operand.
__device__ __forceinline__ u2 half_of(bf8 v, int half) {
  const u4 bits = __builtin_bit_cast(u4, v);
  return half != 0 ? u2{bits[2], bits[3]} : u2{bits[0], bits[1]};
}

// c + a b for a factor in parts and an exact one, or two in parts.
__device__ __forceinline__ f4v mul_exact(bf8 a, const Parts &b, f4v c) { return mfma16(a, b.lo, mfma16(a, b.hi, c)); }
__device__ __forceinline__ f4v mul_parts(const Parts &a, const Parts &b, f4v c) {
  return mfma16(a.hi, b.hi, mfma16(a.hi, b.lo, mfma16(a.lo, b.hi, c)));
}
// With the third part: to 2^-26.
__device__ __forceinline__ f4v mul_exact(bf8 a, const Parts3 &b, f4v c) {
  return mfma16(a, b.hi, mfma16(a, b.lo, mfma16(a, b.rest, c)));
}
__device__ __forceinline__ f4v mul_parts(const Parts &a, const Parts3 &b, f4v c) {
  return mfma16(a.hi, b.hi, mfma16(a.hi, b.lo, mfma16(a.lo, b.hi, mfma16(a.hi, b.rest, mfma16(a.lo, b.lo, c)))));
}
__device__ __forceinline__ f4v mul_parts(const Parts3 &a, const Parts3 &b, f4v c) {
  return mul_parts(static_cast<const Parts &>(a), b, mfma16(a.rest, b.hi, c));
}
// As many parts as asked for.
template <bool THREE>
__device__ __forceinline__ auto split(const f4v &a, const f4v &b) {
  if constexpr (THREE) return parts3(a, b);
  else return parts(a, b);
}

// Where a lane reads in a tile of 64 rows of D elements laid out by slot<D>(),
// in bytes: as row operand (rows m, elements 8g ..), and for transposing reads
// of rows 4g .. 4g + 3 (elements 8 p .. of the tile's first 32, p = m % 4).
struct Lanes16 {
  unsigned row, col;
};
template <int D>
__device__ __forceinline__ Lanes16 lanes16_of(int lane) {
  const int m = lane & 15, g = lane >> 4;
  return {static_cast<unsigned>(slot<D>(m, g)) * 16, static_cast<unsigned>(slot<D>(4 * g + (m >> 2), m & 3)) * 16};
}

// Operand of rows 16 i .., elements 32 a + 8g ..
template <int D>
__device__ __forceinline__ bf8 row16(unsigned tile, int i, int a, const Lanes16 &at) {
  typedef __attribute__((address_space(3))) const u4 lds16;
  return __builtin_bit_cast(bf8, *(lds16 *)(((tile + at.row) ^ (64 * a)) + i * 32 * D));
}
// Transposed operand: rows are the elements of the state's block j (32 (j / 2)
// + 8 (m / 4) + 4 (j % 2) + m % 4), k the tile's rows 32 s .. in D's order.
template <int D>
__device__ __forceinline__ bf8 col16(unsigned tile, int j, int s, const Lanes16 &at) {
  typedef __attribute__((address_space(3))) sh4 lds4;
  const unsigned to = ((tile + at.col) ^ (64 * (j / 2))) + 8 * (j % 2) + s * 64 * D;
  const sh4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(to));
  const sh4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(to + 32 * D));
  return __builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
// The operand that was stored as fragment f of 1024 bytes.
__device__ __forceinline__ bf8 frag16(unsigned tile, int f, int lane) {
  typedef __attribute__((address_space(3))) const u4 lds16;
  return __builtin_bit_cast(bf8, *(lds16 *)(tile + f * 1024 + lane * 16));
}
// A D result in two parts, as operands left them in LDS (fragments of 32 rows,
// high and low part in turn; rows: tokens in D's order, or, PLAIN, key elements
// in plain order), turned round: lane m stands for row 16 i + m, its four
// values for columns 4g .. 4g + 3, half of an operand over 32 columns.
template <bool PLAIN>
__device__ __forceinline__ sh4 turned(unsigned from, int i, int part, int lane) {
  typedef __attribute__((address_space(3))) sh4 lds4;
  const int m = lane & 15, col = 4 * (lane >> 4) + (m >> 2), p = m & 3;
  const unsigned at = from + (i / 2) * 2048 + part * 1024 +
                      (PLAIN ? (16 * (2 * (i % 2) + (p >> 1)) + col) * 16 + (p & 1) * 8 : (16 * p + col) * 16 + (i % 2) * 8);
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(at));
}
// Both halves, of two column tiles.
template <bool PLAIN>
__device__ __forceinline__ bf8 turned(unsigned first, unsigned second, int i, int part, int lane) {
  return __builtin_bit_cast(bf8, __builtin_shufflevector(turned<PLAIN>(first, i, part, lane), turned<PLAIN>(second, i, part, lane),
                                                         0, 1, 2, 3, 4, 5, 6, 7));
}

// Fragment of a lower triangle: row block i (of 16), columns 32 s .., and of
// its transpose: row block j, columns 32 s .. (32 s + 31 >= 16 j).
__host__ __device__ constexpr int tri(int i, int s) { return i < 2 ? i : 2 * (i - 1) + s; }
__host__ __device__ constexpr int tri_t(int j, int s) { return j < 2 ? 2 * j + s : j + 2; }
// Operand of the transpose's row block j, columns 32 s .., of a triangle that lies as its own operands.
__device__ __forceinline__ bf8 tri_cols(unsigned from, int j, int s, int part, int lane) {
  typedef __attribute__((address_space(3))) sh4 lds4;
  const int m = lane & 15;
  const unsigned at = from + (16 * (m & 3) + 4 * (lane >> 4) + (m >> 2)) * 16 + (j % 2) * 8;
  const sh4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(at + (part * kGdrFrags + tri(2 * s, j / 2)) * 1024));
  const sh4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(at + (part * kGdrFrags + tri(2 * s + 1, j / 2)) * 1024));
  return __builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ f4v lds_f4(unsigned at) {
  typedef __attribute__((address_space(3))) const f4v lds16;
  return *(lds16 *)(at);
}

constexpr int kPairs = 2;  // wavefronts that carry the state, and as many beside them

// Call f with the wavefront's number (of 4) as a constant.  Each wavefront's
// products are straight code then: the compiler has left out the wait between a
// matrix product and a read of its result where a branch by a wavefront's
// number lay between them.  (tests/test_matrix_waits.py looks for that in every
// built library, over all paths.  Other branches by a wavefront's number, as in
// the backward's stores of triangles, have vector instructions that read the
// products before them, in the same straight code.)
template <typename F>
__device__ __forceinline__ void by_wave(int w, F &&f) {
  switch (w) {
    case 0: f(std::integral_constant<int, 0>{}); break;
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    default: f(std::integral_constant<int, 3>{}); break;
  }
}

// This wavefront's copies and stores are done, then all wavefronts meet.
__device__ __forceinline__ void arrive() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// All wavefronts meet, with what they have read and written in LDS.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// LDS slot of a tile of 64 rows of NC values.
template <int NC>
__device__ __forceinline__ int vslot(int r, int c) {
  if constexpr (NC == 32) return r * 4 + c;
  else return slot<NC>(r, c);
}
// Rows 16 i + 4g .. + 3 of column 16 ct + m of such a tile.
template <int NC>
__device__ __forceinline__ sh4 rows4(unsigned tile, int i, int ct, int lane) {
  typedef __attribute__((address_space(3))) sh4 lds4;
  const int m = lane & 15, r = 16 * i + 4 * (lane >> 4) + (m >> 2), piece = 4 * ct + (m & 3);
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(tile + vslot<NC>(r, piece >> 1) * 16 + (piece & 1) * 8));
}
typedef __attribute__((ext_vector_type(4))) int i4;
// A value that all lanes share, in scalar registers.  A memory instruction may
// read those five instructions after a vector instruction wrote them, which the
// compiler keeps to for its own, not for those in asm.
template <typename T>
__device__ __forceinline__ T *uniform(T *p) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  // (The builtin gives a signed int, which must not widen as one.)
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(at >> 32)));
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(at)));
  uint64_t u = static_cast<uint64_t>(hi) << 32 | lo;
  asm volatile("s_nop 4" : "+s"(u));
  return reinterpret_cast<T *>(u);
}
// A buffer resource: `bytes` from p.
__device__ __forceinline__ i4 resource(const void *p, unsigned bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  i4 r = {__builtin_amdgcn_readfirstlane(static_cast<int>(at)),
          __builtin_amdgcn_readfirstlane(static_cast<int>(at >> 32)) & 0xffff,
          __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00027000};
  asm volatile("s_nop 4" : "+s"(r));
  return r;
}
// Copies of 16 bytes per lane from memory to LDS (see copy16()), at a lane's
// offset plus one that all lanes share: few instructions per copy, for a
// wavefront that has its SIMD to itself is bound by how many it issues.
__device__ __forceinline__ void copy16(unsigned lds, const i4 &from, unsigned lane_off, unsigned off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(lane_off), "s"(from), "s"(off)
               : "memory", "m0");
}
// N KiB from `from` (this lane's 16 bytes at lane_off) to LDS, in order.
template <int N>
__device__ __forceinline__ void copy_kib(unsigned lds, const void *from, unsigned lane_off) {
  static_assert(N >= 1 && N <= 3, "the immediate offset");
  if constexpr (N == 1)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : : "s"(lds), "v"(lane_off), "s"(from) : "memory", "m0");
  else if constexpr (N == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\tglobal_load_lds_dwordx4 %1, %2 offset:1024"
                 :
                 : "s"(lds), "v"(lane_off), "s"(from)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\tglobal_load_lds_dwordx4 %1, %2 offset:1024"
                 "\n\tglobal_load_lds_dwordx4 %1, %2 offset:2048"
                 :
                 : "s"(lds), "v"(lane_off), "s"(from)
                 : "memory", "m0");
}
// A wavefront's share (of NW) of KIB KiB.
template <int KIB, int NW>
__device__ __forceinline__ void copy_share(unsigned lds, const char *from, int w, unsigned lane_off) {
  constexpr int kEach = (KIB + NW - 1) / NW, kLast = KIB - kEach * (NW - 1);
  static_assert(kLast > 0 && kLast <= kEach, "shares");
  lds = __builtin_amdgcn_readfirstlane(lds + w * kEach * 1024);
  from = uniform(from + w * kEach * 1024);
#pragma unroll
  for (int k = 0; k < kLast; k += 3) {
    constexpr int kRest = kLast % 3;
    if (k + 3 <= kLast) copy_kib<3>(lds + k * 1024, from + k * 1024, lane_off);
    else copy_kib<kRest != 0 ? kRest : 3>(lds + k * 1024, from + k * 1024, lane_off);
  }
  if constexpr (kEach > kLast) {
    if (w < NW - 1)
#pragma unroll
      for (int k = kLast; k < kEach; ++k) copy_kib<1>(lds + k * 1024, from + k * 1024, lane_off);
  }
}

// Copies of a tile of 64 rows of NC values, laid out by vslot<NC>(), by NT
// threads.  Rows a multiple of 16 apart have the same exchange of chunks, so a
// lane has one offset, or two, for all its pieces.
template <int NC, int NT>
struct TileCopy {
  static constexpr int kChunks = NC / 8, kRows = NT / kChunks, kOffsets = kRows >= 16 ? 1 : 16 / kRows;
  unsigned off[kOffsets], stride;  // in bytes
  __device__ __forceinline__ void init(int64_t token, int tid) {
    stride = static_cast<unsigned>(token) * 2;
#pragma unroll
    for (int q = 0; q < kOffsets; ++q) {
      const int r = q * kRows + tid / kChunks, c = tid % kChunks;
      off[q] = r * stride + (vslot<NC>(r, c) - r * kChunks) * 16;
    }
  }
  // p: the first of 64 rows, of which those past `last` are read as that one.
  __device__ __forceinline__ void start(u4 *tile, const uint16_t *p, int last, int tid) const {
    const unsigned lds = __builtin_amdgcn_readfirstlane(lds_at(tile) + (tid & ~63) * 16);
    if (last >= 63) {
      const i4 from = resource(p, 63 * stride + NC * 2);
#pragma unroll
      for (int k = 0; k < 64 / kRows; ++k)
        copy16(lds + k * NT * 16, from, off[k % kOffsets], __builtin_amdgcn_readfirstlane(k / kOffsets * (kOffsets * kRows) * stride));
    } else {
      p = uniform(p);
#pragma unroll
      for (int k = 0; k < 64 / kRows; ++k) {
        const int r = k * kRows + tid / kChunks, c = vslot<NC>(r, tid % kChunks) - r * kChunks;
        copy16(lds + k * NT * 16, p, static_cast<unsigned>(r < last ? r : last) * stride + c * 16);
      }
    }
  }
};

// Store D results (rows: tokens, this lane's column) of a chunk as bfloat16,
// `stride` bytes between tokens.  Rows behind `rows` are dropped.
struct RowStore {
  unsigned lane_off, stride;
  __device__ __forceinline__ void init(int64_t token, int lane) {
    stride = static_cast<unsigned>(token) * 2;
    lane_off = 4 * (lane >> 4) * stride + (lane & 15) * 2;
  }
  __device__ __forceinline__ void put(uint16_t *p, int rows, const f4v (&o)[4]) const {
    const auto to = __builtin_amdgcn_make_buffer_rsrc(uniform(p), 0, rows > 0 ? (static_cast<unsigned>(rows) - 1) * stride + 32 : 0, 0x00027000);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, static_cast<__bf16>(o[i][r])), to, lane_off, (16 * i + r) * stride, 0);
  }
};

// Operand of the elements 16 ct + m of a row-major tile, k its rows 32 s .. in D's order.
template <int D>
__device__ __forceinline__ bf8 elems16(unsigned tile, int ct, int s, int lane) {
  return __builtin_bit_cast(bf8, __builtin_shufflevector(rows4<D>(tile, 2 * s, ct, lane), rows4<D>(tile, 2 * s + 1, ct, lane), 0,
                                                         1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ float up(short v) {
  return __uint_as_float(static_cast<unsigned>(static_cast<uint16_t>(v)) << 16);
}

template <typename G>
__device__ __forceinline__ float gate(const void *p, int64_t i) { return ld(static_cast<const G *>(p), i); }

constexpr int kPitch = 68;  // floats between rows of 64 in LDS: 16-byte aligned, rows on other banks

// Row block J of a triangle's transpose, as fragments, from the triangle in LDS.
__device__ __forceinline__ void store_cols(const float *t, int J, u4 *to, int lane) {
  const int m = lane & 15, g = lane >> 4;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (2 * s + 1 < J) continue;
    f4v v[2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 32 * s + 16 * x + 4 * g + r;
        v[x][r] = i >= 16 * J + m ? t[i * kPitch + 16 * J + m] : 0.0f;
      }
    const Parts p = parts(v[0], v[1]);
    to[tri_t(J, s) * 64 + lane] = __builtin_bit_cast(u4, p.hi);
    to[(kGdrFrags + tri_t(J, s)) * 64 + lane] = __builtin_bit_cast(u4, p.lo);
  }
}

// A workgroup's head and column tile: the tiles of a head, which read the same
// keys and operands, 8 workgroups apart, so that they share an XCD's L2.
struct HeadTile {
  int64_t head;
  unsigned tile;
};
__device__ __forceinline__ HeadTile head_tile(unsigned id, unsigned heads, unsigned tiles) {
  const unsigned even = heads / 8 * 8;
  if (id < even * tiles) {
    const unsigned r = id % (8 * tiles);
    return {id / (8 * tiles) * 8 + r % 8, r / 8};
  }
  const unsigned r = id - even * tiles;
  return {even + r / tiles, r % tiles};
}

__device__ __forceinline__ int gdr_length(const int32_t *lengths, int64_t b, int64_t seqlen) {
  if (lengths == nullptr) return static_cast<int>(seqlen);
  const int n = lengths[b], L = static_cast<int>(seqlen);
  return n < 0 ? 0 : n > L ? L : n;
}

}  // namespace ssmb
