// Reading single codes and norms of a packed tile (layout: include/gtq.h).
#pragma once

#include "gtq_internal.h"

namespace gtq {

// w bits (1..8) from bit `at` of a tile: at most two bytes.
__device__ __forceinline__ uint32_t tile_bits(const uint8_t* tile, int at, int w) {
  const int i = at >> 3, sh = at & 7;
  uint32_t v = tile[i];
  if (sh + w > 8) v |= (uint32_t)tile[i + 1] << 8;
  return (v >> sh) & ((1u << w) - 1);
}
// Key code of token j (0..63) at packed position pos (slot pos / 2) of width w > 0.
__device__ __forceinline__ uint32_t key_code(const uint8_t* tile, const HeadMeta& m, int j, int pos,
                                             int w) {
  return tile_bits(tile, 8 * m.slot_koff[pos >> 1] + (j & 7) * 16 * w + (2 * (j >> 3) + (pos & 1)) * w, w);
}
// Value code of token j, dim d of the rotated basis.
__device__ __forceinline__ uint32_t value_code(const uint8_t* tile, int kb, int vb, int j, int d) {
  const int p = ((d >> 4) * 8 + (d & 7)) * 4 + ((j & 7) >> 1);
  const int x = 8 * (j >> 4) + 4 * ((j >> 3) & 1) + 2 * ((d >> 3) & 1) + (j & 1);
  return tile_bits(tile, 8192 * kb + p * 32 * vb + x * vb, vb);
}
// Norm of token j in the row of 64 norms at byte `row` of a tile.
__device__ __forceinline__ float tile_norm(const uint8_t* tile, int row, int j) {
  return __half2float(*reinterpret_cast<const __half*>(tile + row + 2 * ((j & 7) * 8 + (j >> 3))));
}

}  // namespace gtq
