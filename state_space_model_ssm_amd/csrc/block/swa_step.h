// What the single-token attention kernels share: rows of a tile set from
// elsewhere, weights in two parts, and the joining of wavefronts and splits.
#pragma once

#include "swa_tile.h"

namespace ssmb {

// The token's own key or value, from the arguments, into row r of a tile.
template <int D>
__device__ __forceinline__ void put_row(u4 *tile, const uint16_t *src, int r, int lane) {
  if (lane < D / 8) tile[slot<D>(r, lane)] = reinterpret_cast<const u4 *>(src)[lane];
}

// Zeros in the rows from r on: they repeat the last slot, whose infinity, if it
// has one, would come out as 0 times itself.
template <int D>
__device__ __forceinline__ void clear_rows(u4 *tile, int r, int lane) {
  constexpr int CH = D / 8;
  for (int k = r + lane / CH; k < kTile; k += 64 / CH) tile[slot<D>(k, lane % CH)] = u4{};
}

// Weights (registers 8 s .. 8 s + 7 of a D result) as two operands whose sum
// they are to 2^-16: cut off after 8 bits, and what that leaves, which is held
// above 0, so that both times an infinity have its sign.
__device__ __forceinline__ void two_parts(const f16v &d, int s, bf8 &cut, bf8 &rest) {
  u4 c;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = d[8 * s + 2 * k], b = d[8 * s + 2 * k + 1];
    const unsigned ca = __float_as_uint(a) & 0xffff0000u, cb = __float_as_uint(b) & 0xffff0000u;
    c[k] = ca >> 16 | cb;
    rest[2 * k] = static_cast<__bf16>(fmaxf(a - __uint_as_float(ca), 0x1p-100f));
    rest[2 * k + 1] = static_cast<__bf16>(fmaxf(b - __uint_as_float(cb), 0x1p-100f));
  }
  cut = __builtin_bit_cast(bf8, c);
}

// Join the four wavefronts of a workgroup: o ([32][D] float32 each, in `lds`, a
// fourth per wavefront) and the running maxima and sums, for `heads` heads from
// number `first` on; y, or this split's share.
template <int D, size_t N>
__device__ __forceinline__ void join_waves(const SwaStepParams &p, u4 (&lds)[4][2][N], const f16v (&o)[D / 32], float top,
                                           float sum, float (&tops)[4][32], float (&sums)[4][32], int heads, int64_t first,
                                           unsigned splits, unsigned split) {
  static_assert(sizeof(lds[0]) >= 32 * D * sizeof(float), "o of a wavefront");
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  float *mine = reinterpret_cast<float *>(lds[wave]);
#pragma unroll
  for (int db = 0; db < D / 32; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<float4 *>(mine + (lane & 31) * D + 32 * db + 8 * g + 4 * half) =
          make_float4(o[db][4 * g], o[db][4 * g + 1], o[db][4 * g + 2], o[db][4 * g + 3]);
  if (half == 0) {
    tops[wave][lane] = top;
    sums[wave][lane] = sum;
  }
  __syncthreads();
  for (int i = tid; i < heads * D; i += 256) {
    const int row = i / D, e = i % D;
    float best = tops[0][row];
#pragma unroll
    for (int w = 1; w < 4; ++w) best = fmaxf(best, tops[w][row]);
    // (A share without a maximum holds zeros, or the NaN that all its scores were.)
    float acc = 0.0f, all = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = tops[w][row] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(tops[w][row] - best);
      acc = fmaf(f, reinterpret_cast<const float *>(lds[w])[row * D + e], acc);
      all = fmaf(f, sums[w][row], all);
    }
    const int64_t head = first + row;
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

// Join the splits of a head, a thread per element.
template <int D>
__global__ void __launch_bounds__(D) swa_join_kernel(const SwaStepParams p, int splits) {
  const int64_t head = blockIdx.x;
  const float *stat = p.ws_stat + head * splits * 2, *part = p.ws_o + head * splits * D + threadIdx.x;
  float best = -INFINITY, acc = 0.0f, all = 0.0f;
  for (int k = 0; k < splits; ++k) best = fmaxf(best, stat[2 * k]);
  for (int k = 0; k < splits; ++k) {
    const float f = stat[2 * k] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(stat[2 * k] - best);
    acc = fmaf(f, part[k * D], acc);
    all = fmaf(f, stat[2 * k + 1], all);
  }
  st(p.y, head * D + threadIdx.x, all == 0.0f ? 0.0f : acc / all);
}

}  // namespace ssmb
