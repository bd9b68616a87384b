// Layout of 4-bit weights with group scales, shared by the host rules and the kernels.
//
// Rows lie in groups of 16 (a gated weight's two halves each padded to a multiple of 16), k in
// tiles of 128. A tile of 16 rows by 128 k is 1 KB, in the order in which a wave's 64 lanes feed
// v_mfma_f32_16x16x32: lane l has the 16 bytes at 16 l, row l % 16, and its dword j holds the
// eight k values 32 j + 8 (l / 16) .. + 7, the first four in the low halves of its bytes and the
// other four in the high halves, so that a wave loads a tile in one instruction of whole lines
// and a mask (with a shift) leaves bytes ready for conversion.
// Scales (16 bits) and zeros (a byte): [row group][group of k][16 rows].
#pragma once

#include <cstddef>
#include <cstdint>

namespace gew4 {

constexpr int kRows = 16;
constexpr int kTileK = 128;
constexpr int kTileBytes = 1024;

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// row groups of one half
constexpr int64_t row_groups(int64_t rows, int halves) { return ceil_div(rows / halves, kRows); }
constexpr int64_t k_tiles(int64_t k) { return ceil_div(k, kTileK); }
constexpr int64_t k_groups(int64_t k, int64_t group) { return ceil_div(k, group); }

// Tiles of the products: tokens by rows of W, and waves.
struct W4TileCfg {
  int bm, bn, waves;
};
enum W4Tiles { W4_L = 0, W4_L3, W4_M, W4_S, W4_COUNT };
constexpr W4TileCfg kTiles[W4_COUNT] = {{256, 256, 8}, {192, 256, 8}, {128, 128, 8}, {64, 128, 8}};

}  // namespace gew4
