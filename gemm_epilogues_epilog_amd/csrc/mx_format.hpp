// Microscaled operands: their layout in memory (host and device) and the device's
// conversions to and from them.
//
// A block of 32 consecutive k values of a row shares the scale 2^(s - 127) of one byte s;
// s = 255 stands for NaN. The elements are 4-bit e2m1 (two to a byte, even k in the low
// nibble) or 8-bit e4m3.
//
// Layout. The 32x32x64 scaled matrix product reads 16 bytes per lane: lane l takes row
// l % 32 of a group of 32 rows, and of its 64 k values 32 four-bit ones (those of half
// l / 32), or twice 16 eight-bit ones (at 16 (l / 32), and 32 further on). So a row group
// is kept as its 16-byte chunks of k in ascending order, each chunk for the 32 rows in
// turn: one operand of the instruction is 1 KB (2 KB) of consecutive memory, the copies to
// LDS are whole lines, and the reads from LDS are free of bank conflicts without a swizzle.
//   code byte of (r, k): ((r / 32) C + k / V) 512 + (r % 32) 16 + byte of k in its chunk,
//     V = 32 (e2m1) or 16 (e4m3) values per chunk, C = chunks of k padded to 256
//   scale byte of (r, k): ((r / 32) KT + k / 256) 256 + (k / 32 % 2) 128 + (r % 32) 4 + k / 64 % 4,
//     KT = k padded to 256, over 256: lane l's dword of a 256-k granule holds the scales of
//     its half's blocks, which the instruction picks a byte of.
// k is padded with zero codes and zero scales to a multiple of 256, rows to one of 32.
#pragma once

#include <cstddef>
#include <cstdint>

namespace gemx {

enum Fmt { FP4 = 0, FP8 = 1 };
constexpr int kBlock = 32;       // values that share a scale
constexpr int kRowGroup = 32;    // rows of a group
constexpr int kKPad = 256;       // k values of a scale granule
constexpr int kScaleGranule = 256;   // bytes: 32 rows x 8 blocks
constexpr int kScaleNaN = 255;

constexpr int64_t pad_to(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
constexpr int chunk_values(int fmt) { return fmt == FP4 ? 32 : 16; }
// bytes of one row group (32 rows over the padded k)
constexpr int64_t group_code_bytes(int fmt, int64_t k) { return pad_to(k, kKPad) / chunk_values(fmt) * 512; }
constexpr int64_t group_scale_bytes(int64_t k) { return pad_to(k, kKPad) / kKPad * kScaleGranule; }
constexpr int64_t row_groups(int64_t rows) { return (rows + kRowGroup - 1) / kRowGroup; }
constexpr int64_t code_bytes(int fmt, int64_t rows, int64_t k) { return row_groups(rows) * group_code_bytes(fmt, k); }
constexpr int64_t scale_bytes(int64_t rows, int64_t k) { return row_groups(rows) * group_scale_bytes(k); }

#if defined(__HIPCC__)

// The scale byte of a block whose largest magnitude is `a`: floor(log2 a) - emax + 127
// held to 0 .. 254 (emax 2 or 8), from the exponent bits; a subnormal or zero a gives 0;
// an infinite or NaN a gives 255. `a` is never negative.
__device__ __forceinline__ int scale_of(float a, int fmt) {
  const int e = (int)(__float_as_uint(a) >> 23);
  const int s = e - (fmt == FP4 ? 2 : 8);
  return e == 255 ? kScaleNaN : s > 0 ? s : 0;
}
// The larger of two magnitudes, NaN if either is: a block that holds a NaN has to say so,
// and the compare keeps a NaN that the max instruction would drop. On magnitudes the bit
// patterns order as the values do, with NaN above infinity.
__device__ __forceinline__ float amax2(float a, float b) {
  const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  return __uint_as_float(x > y ? x : y);
}
__device__ __forceinline__ float mag(float v) { return __uint_as_float(__float_as_uint(v) & 0x7fffffffu); }

// 1 / scale as a number: 2^(127 - s), normal for every s of 0 .. 254 but 254 itself
// (2^-127), which no finite block reaches (its s is at most 252).
__device__ __forceinline__ float inv_scale(int s) { return __uint_as_float((uint32_t)(254 - s) << 23); }
// The scale as the conversion instructions take it (they read the exponent field), and
// as a number (2^-127 is subnormal; 255 is NaN).
__device__ __forceinline__ float scale_value(int s) {
  return __uint_as_float(s == kScaleNaN ? 0x7fc00000u : s == 0 ? 0x00400000u : (uint32_t)s << 23);
}

// Eight values over their scale as e2m1, round to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t to_fp4x8(const float (&v)[8], int s) {
  const float sc = __uint_as_float((uint32_t)(s == kScaleNaN ? 127 : s) << 23);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], sc, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], sc, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], sc, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], sc, 3);
  return r;
}
// Four values over their scale as e4m3. Scaled first (exact but for results far below
// the smallest element, which round to zero either way) and held to +-448, since the
// conversion itself does not saturate in every mode.
__device__ __forceinline__ uint32_t to_fp8x4(float a, float b, float c, float d, int s) {
  const float f = inv_scale(s == kScaleNaN ? 127 : s);
  auto sat = [](float x) { return __builtin_amdgcn_fmed3f(x, -448.0f, 448.0f); };
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(sat(a * f), sat(b * f), r, 0);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(sat(c * f), sat(d * f), r, 1);
  return (uint32_t)r;
}

// The larger magnitude over a quad of lanes, in each of them.
__device__ __forceinline__ float amax_quad(float a) {
  const int x = __builtin_amdgcn_mov_dpp((int)__float_as_uint(a), 0xB1, 0xf, 0xf, true);   // lanes 1 0 3 2
  a = amax2(a, __uint_as_float((uint32_t)x));
  const int y = __builtin_amdgcn_mov_dpp((int)__float_as_uint(a), 0x4E, 0xf, 0xf, true);   // lanes 2 3 0 1
  return amax2(a, __uint_as_float((uint32_t)y));
}

#endif  // __HIPCC__

}  // namespace gemx
