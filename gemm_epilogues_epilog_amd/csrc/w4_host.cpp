// Rules declared in w4_host.hpp.
#include "w4_host.hpp"

namespace gew4h {

namespace {
bool known(ge_dtype_t d) { return d == GE_F32 || d == GE_F16 || d == GE_BF16; }
bool half_type(ge_dtype_t d) { return d == GE_F16 || d == GE_BF16; }
size_t esize(ge_dtype_t d) { return d == GE_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
}  // namespace

bool shape_ok(int64_t rows, int64_t k, int64_t group, int halves) {
  if (halves != 1 && halves != 2) return false;
  if (rows < 1 || rows > kMaxDim * halves || rows % halves || k < 1 || k > kMaxDim) return false;
  return group == 32 || group == 64 || (group >= 128 && group <= kMaxDim && group % 128 == 0);
}

size_t code_bytes(int64_t rows, int64_t k, int halves) {
  if (!shape_ok(rows, k, 128, halves)) return 0;
  return (size_t)(gew4::row_groups(rows, halves) * halves * gew4::k_tiles(k)) * gew4::kTileBytes;
}

size_t scale_count(int64_t rows, int64_t k, int64_t group, int halves) {
  if (!shape_ok(rows, k, group, halves)) return 0;
  return (size_t)(gew4::row_groups(rows, halves) * halves * gew4::k_groups(k, group)) * gew4::kRows;
}

ge_status_t check_weight(int64_t rows, int64_t k, int64_t group, int halves, const void* codes, const void* scales,
                         const void* zeros) {
  if (!shape_ok(rows, k, group, halves)) return GE_ERR_INVALID_VALUE;
  if (!codes || !scales || !zeros) return GE_ERR_NULL_POINTER;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(zeros, 16)) return GE_ERR_MISALIGNED;
  return GE_OK;
}

ge_status_t check_quantize(int64_t rows, int64_t k, ge_dtype_t src_dt, const void* src, int64_t ld, ge_dtype_t dt) {
  if (!known(src_dt) || !known(dt)) return GE_ERR_INVALID_VALUE;
  if (!half_type(dt)) return GE_ERR_NOT_SUPPORTED;
  if (rows > 1 && (ld < 0 || ld > (int64_t(1) << 40))) return GE_ERR_INVALID_VALUE;
  (void)k;
  if (!src) return GE_ERR_NULL_POINTER;
  return aligned(src, esize(src_dt)) ? GE_OK : GE_ERR_MISALIGNED;
}

ge_status_t check_dequantize(int64_t rows, int64_t k, ge_dtype_t dt, ge_dtype_t dst_dt, const void* dst, int64_t ld) {
  if (!known(dt) || !known(dst_dt)) return GE_ERR_INVALID_VALUE;
  if (!half_type(dt)) return GE_ERR_NOT_SUPPORTED;
  if (rows > 1 && (ld < k || ld > (int64_t(1) << 40))) return GE_ERR_INVALID_VALUE;
  if (!dst) return GE_ERR_NULL_POINTER;
  return aligned(dst, esize(dst_dt)) ? GE_OK : GE_ERR_MISALIGNED;
}

ge_status_t check_product(int64_t m, int64_t n, ge_dtype_t dt, ge_dtype_t out, const void* x, const void* bias,
                          ge_dtype_t vec, const void* D) {
  if (m < 0 || m > 0x7fffffff || !known(dt) || !known(out) || !known(vec)) return GE_ERR_INVALID_VALUE;
  if (!half_type(dt) || (out != dt && out != GE_F32) || (vec != dt && vec != GE_F32)) return GE_ERR_NOT_SUPPORTED;
  // at most 2^31 - 1 blocks of 16 x 16 values
  if (gew4::ceil_div(m, 16) * gew4::ceil_div(n, 16) > 0x7fffffff) return GE_ERR_NOT_SUPPORTED;
  if (m && (!x || !D)) return GE_ERR_NULL_POINTER;
  if (!aligned(x, 2) || !aligned(D, esize(out)) || !aligned(bias, esize(vec))) return GE_ERR_MISALIGNED;
  return GE_OK;
}

// By estimated time in microseconds, from measurements at 16 to 4000 tokens by 4096 x 4096 and below, 2 x
// 2752 x 2048 and 2 x 11008 x 4096:
//   skinny  start and joining 4, then 1.2 a round of workgroups; W from memory once per 64 tokens, and
//           X, which every row group reads for itself, at the 10 TB/s that the L2 caches gave (fewer
//           workgroups than compute units get their share): 7, 11, 18, 28 and 60 us for 16, 32, 64, 100
//           and 256 tokens by 4096 x 4096. X in pieces of less than 16 bytes: 2.5 times that;
//   tiles   start 2, a round of workgroups 2 and 128 k in 3.45 us (256 x 256), 2.9 (192 x 256), 1.15 (128
//           x 128) or 0.75 (64 x 128: 28 us for 100 tokens); groups of 64 and of 32 multiply the sums
//           more often.
int choose(int64_t m, int64_t n, int64_t k, int64_t group, bool gated, bool aligned, int cus) {
  if (m <= 16 || k < 8) return -1;   // (the tiles load eight k at a time)
  const int64_t rows = gated ? 2 * n : n;
  const double kt = (double)gew4::k_tiles(k);
  const int64_t step = m <= 32 ? 32 : 64, blocks = gew4::ceil_div(m, step);
  const double wgs = (double)gew4::ceil_div(n, 16) * (double)blocks, share = wgs < cus ? wgs / cus : 1.0;
  const double x = (double)m * (double)rows / 16 * (double)k * 2 / 10e6, w = (double)blocks * (double)rows * (double)k * 0.5 / 5e6;
  double best = (4.0 + 1.2 * (wgs / (share * cus) - 1.0) + (x + w) / share) * (aligned ? 1.0 : 2.5);
  int cfg = -1;
  const double per[gew4::W4_COUNT][3] = {{3.45, 4.1, 0.0}, {2.9, 3.6, 0.0}, {1.15, 1.55, 2.0}, {0.75, 0.87, 1.3}};
  const int e = group == 32 ? 2 : group == 64 ? 1 : 0;
  for (int c = 0; c < gew4::W4_COUNT; ++c) {
    if (c <= gew4::W4_L3 && (e == 2 || !aligned)) continue;   // (not instantiated)
    const int64_t tiles = gew4::ceil_div(m, gew4::kTiles[c].bm) * gew4::ceil_div(rows, gew4::kTiles[c].bn);
    const double t = 2.0 + (double)gew4::ceil_div(tiles, cus) * (2.0 + kt * per[c][e]);
    if (t < best) {
      best = t;
      cfg = c;
    }
  }
  return cfg;
}

}  // namespace gew4h
