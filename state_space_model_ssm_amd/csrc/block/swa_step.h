// What the single-token attention kernels of both kinds of cache share: the
// token's own place in a tile.
#pragma once

#include "swa_tile.h"

namespace ssmb {

// The token's own key or value, from the arguments, into row r of a tile.
template <int D>
__device__ __forceinline__ void put_row(u4 *tile, const uint16_t *src, int r, int lane) {
  if (lane < D / 8) tile[slot<D>(r, lane)] = reinterpret_cast<const u4 *>(src)[lane];
}

}  // namespace ssmb
