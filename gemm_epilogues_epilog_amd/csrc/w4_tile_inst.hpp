// Launchers of the 4-bit tile kernel, one unit per type (w4_tile_f16.hip, w4_tile_bf16.hip).
#pragma once

#include "w4_tile.hpp"

namespace gek {

template <int DT, bool GATED, class C>
const void* w4_tile_fn(bool g32, bool xd) {
  if (g32) return xd ? reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, C, true, true>)
                     : reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, C, true, false>);
  return xd ? reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, C, false, true>)
            : reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, C, false, false>);
}

// Tile `cfg` (gew4::W4Tiles) of one type.
template <int DT>
const void* w4_tile_pick(int cfg, bool gated, bool g32, bool xd) {
  using L = W4Tile<256, 256, 128, 64, 2>;
  using M = W4Tile<128, 128, 32, 64, 4>;
  using S = W4Tile<64, 128, 32, 64, 4>;
  switch (cfg) {
    case gew4::W4_L:   // (the other variants do not fit its registers, and choose() does not ask for them)
      if (g32 || !xd) return nullptr;
      return gated ? reinterpret_cast<const void*>(&w4_tile_kernel<DT, true, L, false, true>)
                   : reinterpret_cast<const void*>(&w4_tile_kernel<DT, false, L, false, true>);
    case gew4::W4_M: return gated ? w4_tile_fn<DT, true, M>(g32, xd) : w4_tile_fn<DT, false, M>(g32, xd);
    default: return gated ? w4_tile_fn<DT, true, S>(g32, xd) : w4_tile_fn<DT, false, S>(g32, xd);
  }
}

}  // namespace gek
