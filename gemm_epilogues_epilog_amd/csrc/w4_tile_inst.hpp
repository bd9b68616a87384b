// Launchers of the 4-bit tile kernel, one unit per type (w4_tile_f16.hip, w4_tile_bf16.hip).
#pragma once

#include "w4_tile.hpp"

namespace gek {

template <int DT, bool GATED, class C, int E>
const void* w4_tile_fn(bool xd) {
  return xd ? reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, C, E, true>)
            : reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, C, E, false>);
}
template <int DT, bool GATED, class C>
const void* w4_tile_fn(int e, bool xd) {
  return e == 4 ? w4_tile_fn<DT, GATED, C, 4>(xd) : e == 2 ? w4_tile_fn<DT, GATED, C, 2>(xd) : w4_tile_fn<DT, GATED, C, 1>(xd);
}
// The large tile: the other variants do not fit its registers, and choose() does not ask for them.
template <int DT, bool GATED, class C>
const void* w4_tile_large(int e, bool xd) {
  if (e == 4 || !xd) return nullptr;
  return e == 2 ? reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, C, 2, true>)
                : reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, C, 1, true>);
}

// Tile `cfg` (gew4::W4Tiles) of one type.
template <int DT>
const void* w4_tile_pick(int cfg, bool gated, int64_t group, bool xd) {
  using L = W4Tile<256, 256, 128, 64, 2, 1>;
  using M = W4Tile<128, 128, 32, 64, 4, 1>;
  using S = W4Tile<64, 128, 32, 64, 4, 2>;
  const int e = group == 32 ? 4 : group == 64 ? 2 : 1;
  switch (cfg) {
    case gew4::W4_L: return gated ? w4_tile_large<DT, true, L>(e, xd) : w4_tile_large<DT, false, L>(e, xd);
    case gew4::W4_M: return gated ? w4_tile_fn<DT, true, M>(e, xd) : w4_tile_fn<DT, false, M>(e, xd);
    default: return gated ? w4_tile_fn<DT, true, S>(e, xd) : w4_tile_fn<DT, false, S>(e, xd);
  }
}

}  // namespace gek
