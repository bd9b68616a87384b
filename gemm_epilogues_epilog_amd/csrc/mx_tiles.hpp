// Kernel configurations of the microscaled product, shared by the host plan
// (mx_host.cpp, plain C++) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include "mx_format.hpp"

namespace gemx {

// Tile kernels: bm rows of X by bn rows of W, split over waves of 32 mb x 32 nb.
// Skinny kernels (stages 0): bm rows of X by bn rows of W, eight waves that split k.
struct MxTile {
  int bm, bn, mb, nb, stages;
  const char* name;
};
enum MxCfg { MX_L = 0, MX_M, MX_S64, MX_S32, MX_S16, MX_COUNT };
constexpr MxTile kMxTiles[MX_COUNT] = {
    {256, 256, 2, 4, 2, "L"}, {128, 128, 1, 4, 2, "M"},
    {64, 32, 0, 0, 0, "S64"}, {32, 32, 0, 0, 0, "S32"}, {16, 32, 0, 0, 0, "S16"},
};
constexpr bool mx_is_skinny(int c) { return c >= MX_S64; }
constexpr int mx_waves(const MxTile& t) { return t.stages ? (t.bm / 32 / t.mb) * (t.bn / 32 / t.nb) : 8; }
// k values of one LDS stage: 128 bytes of a row of X.
constexpr int mx_bk(int xfmt) { return xfmt == FP4 ? 256 : 128; }

// Split tiles: fp32 partial accumulators of one part, and the counters of arrived parts.
constexpr int kMxMaxSplit = 16;
constexpr int kMxCounters = 1024;   // one per split tile
constexpr size_t kMxCounterBytes = kMxCounters * 4;

}  // namespace gemx
