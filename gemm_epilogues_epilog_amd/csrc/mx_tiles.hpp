// Kernel configurations of the microscaled product, shared by the host plan
// (mx_host.cpp, plain C++) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include "mx_format.hpp"

namespace gemx {

// bm rows of X by bn rows of W per workgroup.
//   MX_L: persistent tile kernel, waves of 32 mb x 32 nb, two large stages: large products.
//   MX_R: ring kernel, one workgroup per tile, many small stages: a few dozen to a few
//     thousand rows. The larger tiles read less from the LDS and the L2 per product, the
//     smaller ones fill the compute units with fewer rows (1000 x 4096 x 4096, e4m3 X: 256
//     tiles of 128 x 128 take 19.7 us, 512 of 128 x 64 29, 64 of 256 x 256 42; 2000 rows: 128 x
//     256 32.7, 128 x 128 41, 256 x 256 47; 500 rows: 128 x 64 13.6, 128 x 128 18.9). Those
//     with mb 1 can share k between workgroups where the tiles are fewer than the compute
//     units.
//   MX_S16, MX_S16N: skinny kernel (stages 0), two to eight waves that split k and read W
//     straight into registers, sixteen rows at a time: few rows, or few per expert.
// kg: groups of waves, each with every kg-th k-tile (their sums are added through LDS).
struct MxTile {
  int bm, bn, mb, nb, stages, kg;
};
enum MxCfg { MX_L = 0, MX_R256, MX_R128W, MX_R128, MX_R64, MX_S16, MX_S16N, MX_COUNT };
constexpr MxTile kMxTiles[MX_COUNT] = {
    {256, 256, 2, 4, 2, 1}, {128, 256, 2, 2, 3, 1}, {128, 128, 1, 2, 4, 1}, {128, 64, 1, 2, 3, 2},
    {64, 64, 1, 1, 4, 2},   {16, 32, 0, 0, 0, 1},   {16, 16, 0, 0, 0, 1}};
constexpr bool mx_is_ring(int c) { return c >= MX_R256 && c <= MX_R64; }
constexpr int mx_waves(const MxTile& t) { return (t.bm / 32 / t.mb) * (t.bn / 32 / t.nb) * t.kg; }
constexpr int kMxSkinnyWaves = 8;   // at most
constexpr int kMxTailCfg = MX_R128W;   // quarters of the tile kernel's tiles, for its short last rounds
static_assert(kMxTiles[MX_L].bm == 2 * kMxTiles[kMxTailCfg].bm && kMxTiles[MX_L].bn == 2 * kMxTiles[kMxTailCfg].bn, "quarters");
// Tiles go down this many rows of tiles before the next column, so that neighbours share W and X
// in the L2.
constexpr int kMxGroupM = 8;
// k values of one LDS stage: 128 bytes of a row of X.
constexpr int mx_bk(int xfmt) { return xfmt == FP4 ? 256 : 128; }

// Split tiles: the counters of arrived parts, each in a cache line of its own (neighbours in
// one line queue for it), then the parts' fp32 accumulators.
constexpr int kMxMaxSplit = 16;
constexpr int kMxCounters = 512;
constexpr int kMxCounterStride = 64;   // words
constexpr size_t kMxCounterBytes = (size_t)kMxCounters * kMxCounterStride * 4;

}  // namespace gemx
