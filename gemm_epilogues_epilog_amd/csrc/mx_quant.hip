// Conversion to and from microscaled operands (layout and arithmetic: mx_format.hpp), and
// packing of row-major codes into that layout.
//
// All four kernels work in tiles of 32 rows x 256 k, one workgroup of 256 lanes each: a
// tile's codes are 4 KB (e2m1) or 8 KB (e4m3) and its scales 256 bytes of consecutive
// memory, so they pass through LDS and move in whole lines, while the plain side moves in
// row pieces of 256 values. Bound by memory: one read and one write per value.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "gemm_epilog.h"
#include "kernels.hpp"
#include "mx_format.hpp"
#include "mx_host.hpp"

namespace gek {
namespace {

using namespace gemx;

// Eight values of type DT as they lie in memory.
template <int DT>
struct Raw8 {
  i32x4 v[DT == F32 ? 2 : 1];
  __device__ __forceinline__ float get(int e) const {
    if constexpr (DT == F32) return __int_as_float(v[e / 4][e % 4]);
    else return Tr<DT>::widen((uint16_t)((uint32_t)v[0][e / 2] >> (16 * (e & 1))));
  }
  // one by one, `step` elements apart, those from `n` on (n at least 1) repeating the last
  __device__ __forceinline__ void gather(const char* p, int64_t step, int n) {
    using U = std::conditional_t<DT == F32, uint32_t, uint16_t>;
    uint32_t x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = *reinterpret_cast<const U*>(p + min(e, n - 1) * step * (int64_t)sizeof(U));
    if constexpr (DT == F32) {
      __builtin_memcpy(v, x, 32);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[0][e] = (int)(x[2 * e] | x[2 * e + 1] << 16);
    }
  }
};
struct QuantArgs {
  const void* src;
  char* codes;
  char* scales;
  int64_t rows, k, row_stride, col_stride;   // strides in elements
  int64_t kt;                                // 256-k granules
};

// The tile's codes and scales from LDS to their place, 16 bytes a lane.
template <int FMT>
__device__ __forceinline__ void store_tile(const QuantArgs& a, int64_t rb, int64_t kt, const char* lc, const char* ls) {
  constexpr int CB = FMT == FP4 ? 4096 : 8192;
  char* dc = a.codes + (rb * a.kt + kt) * CB;
  char* ds = a.scales + (rb * a.kt + kt) * kScaleGranule;
#pragma unroll
  for (int i = 0; i < CB / 4096; ++i)
    reinterpret_cast<i32x4*>(dc)[i * 256 + threadIdx.x] = reinterpret_cast<const i32x4*>(lc)[i * 256 + threadIdx.x];
  if (threadIdx.x < 16) reinterpret_cast<i32x4*>(ds)[threadIdx.x] = reinterpret_cast<const i32x4*>(ls)[threadIdx.x];
}

// Rows contiguous along k (WIDE: 16-byte loads at the elements' alignment, which the memory
// pipe takes) or any strides. A lane takes 8 consecutive k of four rows; the four lanes of a
// quad share a block. Lanes past the operand read its last values again and put zeros in
// their place, so that no branch parts the loads of the rows.
// Bound by the memory: 16384 x 8192 bf16 to MXFP4 59 us (340 MB, 5.8 TB/s; with a branch
// around each row's load 66), 8192 x 8191 to MXFP8 36 (element by element 69).
template <int DT, int FMT, bool WIDE>
__global__ __launch_bounds__(256) void mx_quantize_rows_kernel(QuantArgs a) {
  __shared__ __attribute__((aligned(16))) char lc[FMT == FP4 ? 4096 : 8192];
  __shared__ __attribute__((aligned(16))) char ls[kScaleGranule];
  constexpr int ES = DT == F32 ? 4 : 2;
  const int64_t rb = blockIdx.x / a.kt, kt = blockIdx.x % a.kt;
  const int t = threadIdx.x, kk = (t & 31) * 8;
  const int64_t k0 = kt * kKPad + kk;
  const int left = (int)min((int64_t)8, a.k - k0);   // values of this lane (none past k)
  const int64_t from = min(k0, a.k - 1);
  Raw8<DT> raw[4];
  const auto at = [&](int i) {
    const int64_t row = min(rb * kRowGroup + i * 8 + (t >> 5), a.rows - 1);
    return static_cast<const char*>(a.src) + (row * a.row_stride + from * a.col_stride) * ES;
  };
  if (WIDE && left == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) __builtin_memcpy(raw[i].v, at(i), sizeof(raw[i].v));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i].gather(at(i), a.col_stride, max(left, 1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (t >> 5);
    const bool in = rb * kRowGroup + r < a.rows;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = in && e < left ? raw[i].get(e) : 0.0f;
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = amax2(m, mag(v[e]));
    const int s = scale_of(amax_quad(m), FMT);
    if constexpr (FMT == FP4) {
      *reinterpret_cast<uint32_t*>(lc + (kk / 32) * 512 + r * 16 + (kk % 32) / 2) = to_fp4x8(v, s);
    } else {
      const i32x2 c = {(int)to_fp8x4(v[0], v[1], v[2], v[3], s), (int)to_fp8x4(v[4], v[5], v[6], v[7], s)};
      *reinterpret_cast<i32x2*>(lc + (kk / 16) * 512 + r * 16 + kk % 16) = c;
    }
    const int b = kk / 32;
    if ((t & 3) == 0) ls[(b & 1) * 128 + r * 4 + b / 2] = (char)s;
  }
  __syncthreads();
  store_tile<FMT>(a, rb, kt, lc, ls);
}

// Rows that lie next to each other in memory (row_stride 1): a workgroup takes 128 rows by
// 256 k, each of its eight waves one block of 32 k; a lane takes two neighbouring rows, so
// a wave reads 128 rows of one k at a time (256 or 512 consecutive bytes). Bound by the
// memory: with the 32 reads of a lane in flight together 16384 x 8192 bf16 takes 81 us
// (5.0 TB/s read and written; with a branch between the reads 83). 1000 x 2048 f16 takes 6.9 us:
// 64 workgroups, bound by the latency of the reads.
constexpr int kColRows = 128;
template <int DT, int FMT>
__global__ __launch_bounds__(512) void mx_quantize_cols_kernel(QuantArgs a) {
  constexpr int CB = FMT == FP4 ? 4096 : 8192, G = kColRows / kRowGroup, ES = DT == F32 ? 4 : 2;
  __shared__ __attribute__((aligned(16))) char lc[G * CB];
  __shared__ __attribute__((aligned(16))) char ls[G * kScaleGranule];
  const int64_t tiles = (a.rows + kColRows - 1) / kColRows;
  const int64_t kt = blockIdx.x / tiles, row0 = blockIdx.x % tiles * kColRows;
  const int lane = threadIdx.x & 63, b = threadIdx.x >> 6, r = 2 * lane;
  const int64_t k0 = kt * kKPad + b * 32;
  const int left = (int)min((int64_t)32, a.k - k0);   // values of this block (none past k)
  // Lanes past the last row read the last two, and the k past the last one read it again, so
  // that no branch parts the loads; what they read is replaced by zeros. Row r + h is value
  // h + skip of the pair.
  const int64_t at = min(row0 + r, a.rows - 2);
  const int skip = (int)min((int64_t)2, row0 + r - at);
  struct Pair {   // two rows' values at one k, in whatever alignment
    char bytes[2 * ES];
  };
  Pair raw[32];
  const char* p = static_cast<const char*>(a.src) + (at + min(k0, a.k - 1) * a.col_stride) * ES;
#pragma unroll
  for (int e = 0; e < 32; ++e)
    __builtin_memcpy(&raw[e], p + min(e, max(left - 1, 0)) * a.col_stride * ES, 2 * ES);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[32];
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      float x[2];
      if constexpr (DT == F32) {
        __builtin_memcpy(x, raw[e].bytes, 8);
      } else {
        uint16_t u[2];
        __builtin_memcpy(u, raw[e].bytes, 4);
        x[0] = Tr<DT>::widen(u[0]);
        x[1] = Tr<DT>::widen(u[1]);
      }
      v[e] = e < left && h + skip < 2 ? (h + skip ? x[1] : x[0]) : 0.0f;
      m = amax2(m, mag(v[e]));
    }
    const int s = scale_of(m, FMT);
    char* d = lc + (r + h) / 32 * CB + (r + h) % 32 * 16;
    if constexpr (FMT == FP4) {
      i32x4 c;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float w[8] = {v[8 * q],     v[8 * q + 1], v[8 * q + 2], v[8 * q + 3],
                            v[8 * q + 4], v[8 * q + 5], v[8 * q + 6], v[8 * q + 7]};
        c[q] = (int)to_fp4x8(w, s);
      }
      *reinterpret_cast<i32x4*>(d + b * 512) = c;
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        i32x4 c;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          c[q] = (int)to_fp8x4(v[16 * j + 4 * q], v[16 * j + 4 * q + 1], v[16 * j + 4 * q + 2], v[16 * j + 4 * q + 3], s);
        *reinterpret_cast<i32x4*>(d + (2 * b + j) * 512) = c;
      }
    }
    ls[(r + h) / 32 * kScaleGranule + (b & 1) * 128 + (r + h) % 32 * 4 + b / 2] = (char)s;
  }
  __syncthreads();
  const int groups = (int)min((int64_t)G, row_groups(a.rows) - row0 / kRowGroup);
  for (int i = threadIdx.x; i < groups * (CB / 16); i += 512) {
    const int g = i / (CB / 16), o = i % (CB / 16);
    reinterpret_cast<i32x4*>(a.codes + ((row0 / kRowGroup + g) * a.kt + kt) * CB)[o] =
        reinterpret_cast<const i32x4*>(lc)[i];
  }
  for (int i = threadIdx.x; i < groups * 16; i += 512) {
    const int g = i / 16, o = i % 16;
    reinterpret_cast<i32x4*>(a.scales + ((row0 / kRowGroup + g) * a.kt + kt) * kScaleGranule)[o] =
        reinterpret_cast<const i32x4*>(ls)[i];
  }
}

struct DequantArgs {
  const char* codes;
  const char* scales;
  void* dst;
  int64_t rows, k, row_stride, kt;
};

// One lane writes 8 consecutive k of a row, in 16-byte stores at the elements' alignment, a
// row's last values one by one. Bound by the memory: MXFP8 16384 x 8192 to bf16 73 us
// (407 MB, 5.6 TB/s), 8192 x 8191 35 (element by element 95).
template <int DT, int FMT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(DequantArgs a) {
  constexpr int CB = FMT == FP4 ? 4096 : 8192;
  __shared__ __attribute__((aligned(16))) char lc[CB];
  __shared__ __attribute__((aligned(16))) char ls[kScaleGranule];
  const int64_t rb = blockIdx.x / a.kt, kt = blockIdx.x % a.kt;
  const int t = threadIdx.x;
  const char* sc = a.codes + (rb * a.kt + kt) * CB;
  const char* ss = a.scales + (rb * a.kt + kt) * kScaleGranule;
#pragma unroll
  for (int i = 0; i < CB / 4096; ++i)
    reinterpret_cast<i32x4*>(lc)[i * 256 + t] = reinterpret_cast<const i32x4*>(sc)[i * 256 + t];
  if (t < 16) reinterpret_cast<i32x4*>(ls)[t] = reinterpret_cast<const i32x4*>(ss)[t];
  __syncthreads();
  const int kk = (t & 31) * 8, b = kk / 32;
  const int64_t k0 = kt * kKPad + kk;
  if (k0 >= a.k) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (t >> 5);
    const int64_t row = rb * kRowGroup + r;
    if (row >= a.rows) break;
    const float f = scale_value((uint8_t)ls[(b & 1) * 128 + r * 4 + b / 2]);
    float v[8];
    if constexpr (FMT == FP4) {
      const uint32_t c = *reinterpret_cast<const uint32_t*>(lc + (kk / 32) * 512 + r * 16 + (kk % 32) / 2);
      const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
      const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
      v[0] = p0[0], v[1] = p0[1], v[2] = p1[0], v[3] = p1[1], v[4] = p2[0], v[5] = p2[1], v[6] = p3[0], v[7] = p3[1];
    } else {
      const i32x2 c = *reinterpret_cast<const i32x2*>(lc + (kk / 16) * 512 + r * 16 + kk % 16);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const auto p0 = __builtin_amdgcn_cvt_pk_f32_fp8(c[h], 0), p1 = __builtin_amdgcn_cvt_pk_f32_fp8(c[h], 1);
        v[4 * h] = p0[0], v[4 * h + 1] = p0[1], v[4 * h + 2] = p1[0], v[4 * h + 3] = p1[1];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= f;
    const int64_t at = row * a.row_stride + k0;
    char* d = static_cast<char*>(a.dst) + at * (DT == F32 ? 4 : 2);
    if (k0 + 8 <= a.k) {
      if constexpr (DT == F32) {
        __builtin_memcpy(d, v, 32);
      } else {
        i32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = (int)Tr<DT>::pack2(v[2 * e], v[2 * e + 1]);
        __builtin_memcpy(d, &o, 16);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k0 + e < a.k) store_vec(a.dst, DT, at + e, v[e]);
    }
  }
}

struct PackArgs {
  const uint8_t* src_codes;    // (rows, code_row) row-major
  const uint8_t* src_scales;   // (rows, ceil(k / 32)) row-major
  char* codes;
  char* scales;
  int64_t rows, k, kt, code_row;
  int fp4;
};

// Row-major codes and scales into the packed layout: one lane per block of 32 values.
// Runs once per weight, so it is kept simple: byte loads, no staging.
__global__ __launch_bounds__(256) void mx_pack_kernel(PackArgs a) {
  const int64_t rb = blockIdx.x / a.kt, kt = blockIdx.x % a.kt;
  const int r = threadIdx.x & 31, b = threadIdx.x >> 5;
  const int64_t row = rb * kRowGroup + r, k0 = kt * kKPad + b * 32, blk = k0 / 32;
  const bool in = row < a.rows && k0 < a.k;
  const int left = in ? (int)min((int64_t)32, a.k - k0) : 0;   // values of this block
  a.scales[(rb * a.kt + kt) * kScaleGranule + (b & 1) * 128 + r * 4 + b / 2] =
      in ? (char)a.src_scales[row * ((a.k + 31) / 32) + blk] : (char)0;
  if (a.fp4) {
    char* d = a.codes + (rb * a.kt + kt) * 4096 + b * 512 + r * 16;
    for (int e = 0; e < 16; ++e) {
      uint8_t c = 2 * e < left ? a.src_codes[row * a.code_row + k0 / 2 + e] : 0;
      if (2 * e + 1 >= left) c &= 15;   // an odd k's last byte holds one value
      d[e] = (char)c;
    }
  } else {
    char* d = a.codes + (rb * a.kt + kt) * 8192 + 2 * b * 512 + r * 16;
    for (int e = 0; e < 32; ++e) d[(e / 16) * 512 + e % 16] = e < left ? (char)a.src_codes[row * a.code_row + k0 + e] : 0;
  }
}

template <int DT, int FMT>
const void* quantize_fn(bool cols, bool wide) {
  if (cols) return reinterpret_cast<const void*>(&mx_quantize_cols_kernel<DT, FMT>);
  return wide ? reinterpret_cast<const void*>(&mx_quantize_rows_kernel<DT, FMT, true>)
              : reinterpret_cast<const void*>(&mx_quantize_rows_kernel<DT, FMT, false>);
}
template <int DT>
const void* quantize_fn(int fmt, bool cols, bool wide) {
  return fmt == FP4 ? quantize_fn<DT, FP4>(cols, wide) : quantize_fn<DT, FP8>(cols, wide);
}
template <int DT>
const void* dequantize_fn(int fmt) {
  return fmt == FP4 ? reinterpret_cast<const void*>(&mx_dequantize_kernel<DT, FP4>)
                    : reinterpret_cast<const void*>(&mx_dequantize_kernel<DT, FP8>);
}

}  // namespace
}  // namespace gek

extern "C" {

size_t gemm_epilog_mx_code_bytes(ge_mx_format_t fmt, int64_t rows, int64_t k) {
  return gemxh::shape_ok(rows, k) && gemxh::format_ok(fmt) ? (size_t)gemx::code_bytes(fmt, rows, k) : 0;
}

size_t gemm_epilog_mx_scale_bytes(int64_t rows, int64_t k) {
  return gemxh::shape_ok(rows, k) ? (size_t)gemx::scale_bytes(rows, k) : 0;
}

ge_status_t gemm_epilog_mx_quantize(int64_t rows, int64_t k, ge_dtype_t dt, const void* src, int64_t row_stride,
                                    int64_t col_stride, ge_mx_format_t fmt, void* codes, void* scales, void* stream) {
  if (ge_status_t st = gemxh::check_quantize(rows, k, dt, src, row_stride, col_stride, fmt, codes, scales); st != GE_OK)
    return st;
  if (rows == 0) return GE_OK;
  gek::QuantArgs a{src, static_cast<char*>(codes), static_cast<char*>(scales), rows, k, row_stride, col_stride,
                   gemx::pad_to(k, gemx::kKPad) / gemx::kKPad};
  // Rows next to each other (k strided) go to the kernel whose lanes run along the rows:
  // reading them along k would touch a line per value.
  const bool cols = col_stride != 1 && row_stride == 1 && rows > 1;
  const void* fn = dt == GE_F32   ? gek::quantize_fn<gek::F32>(fmt, cols, col_stride == 1)
                   : dt == GE_F16 ? gek::quantize_fn<gek::F16>(fmt, cols, col_stride == 1)
                                  : gek::quantize_fn<gek::BF16>(fmt, cols, col_stride == 1);
  void* params[] = {&a};
  const int64_t tiles = cols ? (rows + gek::kColRows - 1) / gek::kColRows : gemx::row_groups(rows);
  return hipLaunchKernel(fn, dim3((unsigned)(tiles * a.kt)), dim3(cols ? 512 : 256), params, 0,
                         static_cast<hipStream_t>(stream)) == hipSuccess
             ? GE_OK
             : GE_ERR_HIP;
}

ge_status_t gemm_epilog_mx_dequantize(int64_t rows, int64_t k, ge_mx_format_t fmt, const void* codes,
                                      const void* scales, ge_dtype_t dt, void* dst, int64_t row_stride, void* stream) {
  if (ge_status_t st = gemxh::check_dequantize(rows, k, fmt, codes, scales, dt, dst, row_stride); st != GE_OK) return st;
  if (rows == 0) return GE_OK;
  gek::DequantArgs a{static_cast<const char*>(codes), static_cast<const char*>(scales), dst, rows, k, row_stride,
                     gemx::pad_to(k, gemx::kKPad) / gemx::kKPad};
  const void* fn = dt == GE_F32   ? gek::dequantize_fn<gek::F32>(fmt)
                   : dt == GE_F16 ? gek::dequantize_fn<gek::F16>(fmt)
                                  : gek::dequantize_fn<gek::BF16>(fmt);
  void* params[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)(gemx::row_groups(rows) * a.kt)), dim3(256), params, 0,
                         static_cast<hipStream_t>(stream)) == hipSuccess
             ? GE_OK
             : GE_ERR_HIP;
}

ge_status_t gemm_epilog_mx_pack(int64_t rows, int64_t k, ge_mx_format_t fmt, const void* src_codes,
                                const void* src_scales, void* codes, void* scales, void* stream) {
  if (ge_status_t st = gemxh::check_pack(rows, k, fmt, src_codes, src_scales, codes, scales); st != GE_OK) return st;
  if (rows == 0) return GE_OK;
  gek::PackArgs a{static_cast<const uint8_t*>(src_codes), static_cast<const uint8_t*>(src_scales),
                  static_cast<char*>(codes), static_cast<char*>(scales), rows, k,
                  gemx::pad_to(k, gemx::kKPad) / gemx::kKPad, fmt == GE_MXFP4 ? (k + 1) / 2 : k, fmt == GE_MXFP4};
  void* params[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(&gek::mx_pack_kernel),
                         dim3((unsigned)(gemx::row_groups(rows) * a.kt)), dim3(256), params, 0,
                         static_cast<hipStream_t>(stream)) == hipSuccess
             ? GE_OK
             : GE_ERR_HIP;
}

}  // extern "C"
