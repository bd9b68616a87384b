// Launchers of the 4-bit tile kernels, one unit per type (w4_tile_f16.hip, w4_tile_bf16.hip).
#pragma once

#include "w4_large.hpp"
#include "w4_tile.hpp"

namespace gek {

template <int DT, bool GATED, int BM>
const void* w4_tile_fn(int e) {
  return e == 4   ? reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, BM, 4>)
         : e == 2 ? reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, BM, 2>)
                  : reinterpret_cast<const void*>(&w4_tile_kernel<DT, GATED, BM, 1>);
}
template <int DT, bool GATED, int BM>
const void* w4_large_fn(int e) {
  return e == 2 ? reinterpret_cast<const void*>(&w4_large_kernel<DT, GATED, BM, 2>)
                : reinterpret_cast<const void*>(&w4_large_kernel<DT, GATED, BM, 1>);
}

// Tile `cfg` (gew4::W4Tiles) of one type.
template <int DT>
const void* w4_tile_pick(int cfg, bool gated, int64_t group) {
  const int e = group == 32 ? 4 : group == 64 ? 2 : 1;
  switch (cfg) {
    case gew4::W4_L: return gated ? w4_large_fn<DT, true, 256>(e) : w4_large_fn<DT, false, 256>(e);
    case gew4::W4_L3: return gated ? w4_large_fn<DT, true, 192>(e) : w4_large_fn<DT, false, 192>(e);
    case gew4::W4_M: return gated ? w4_tile_fn<DT, true, 128>(e) : w4_tile_fn<DT, false, 128>(e);
    default: return gated ? w4_tile_fn<DT, true, 64>(e) : w4_tile_fn<DT, false, 64>(e);
  }
}

}  // namespace gek
