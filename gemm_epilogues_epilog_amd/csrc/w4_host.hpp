// Host-side rules of 4-bit weights with group scales: sizes, argument checks, launches. Plain
// C++17 with no HIP call or header.
#pragma once

#include <cstddef>
#include <cstdint>

#include "gemm_epilog.h"
#include "w4_format.hpp"

namespace gew4h {

constexpr int64_t kMaxDim = 1 << 20;

bool shape_ok(int64_t rows, int64_t k, int64_t group, int halves);
size_t code_bytes(int64_t rows, int64_t k, int halves);
size_t scale_count(int64_t rows, int64_t k, int64_t group, int halves);   // and zeros

ge_status_t check_weight(int64_t rows, int64_t k, int64_t group, int halves, const void* codes, const void* scales,
                         const void* zeros);
ge_status_t check_quantize(int64_t rows, int64_t k, ge_dtype_t src_dt, const void* src, int64_t ld, ge_dtype_t dt);
ge_status_t check_dequantize(int64_t rows, int64_t k, ge_dtype_t dt, ge_dtype_t dst_dt, const void* dst, int64_t ld);
ge_status_t check_product(int64_t m, int64_t n, ge_dtype_t dt, ge_dtype_t out, const void* x, const void* bias,
                          ge_dtype_t vec, const void* D);

// The kernel of a product: a tile (gew4::W4Tiles), or -1 for the skinny kernel.
// aligned: X's rows are whole 16-byte chunks.
int choose(int64_t m, int64_t n, int64_t k, int64_t group, bool gated, bool aligned, int cus);

}  // namespace gew4h
