// What the single-token attention kernels of both kinds of cache share.
#pragma once

#include "swa_tile.h"

namespace ssmb {

// The token's own key or value, from the arguments, into row r of a tile.
template <int D>
__device__ __forceinline__ void put_row(u4 *tile, const uint16_t *src, int r, int lane) {
  if (lane < D / 8) tile[slot<D>(r, lane)] = reinterpret_cast<const u4 *>(src)[lane];
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
