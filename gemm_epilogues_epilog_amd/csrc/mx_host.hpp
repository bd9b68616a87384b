// Host-side rules of the microscaled operators and of the norm: argument checks, the
// product's configuration choice and workspace. Plain C++17 with no HIP call or header,
// like plan_host.hpp.
#pragma once

#include <cstddef>
#include <cstdint>

#include "gemm_epilog.h"
#include "mx_format.hpp"

namespace gemxh {

bool format_ok(ge_mx_format_t f);
bool dtype_ok(ge_dtype_t d);
// rows 0 .. 2^31 - 1, k 1 .. 2^20, and few enough 32 x 256 tiles for one launch
bool shape_ok(int64_t rows, int64_t k);
size_t esize(ge_dtype_t d);

ge_status_t check_quantize(int64_t rows, int64_t k, ge_dtype_t dt, const void* src, int64_t row_stride,
                           int64_t col_stride, ge_mx_format_t fmt, const void* codes, const void* scales);
ge_status_t check_dequantize(int64_t rows, int64_t k, ge_mx_format_t fmt, const void* codes, const void* scales,
                             ge_dtype_t dt, const void* dst, int64_t row_stride);
ge_status_t check_pack(int64_t rows, int64_t k, ge_mx_format_t fmt, const void* src_codes, const void* src_scales,
                       const void* codes, const void* scales);

ge_status_t check_plan(int64_t n, int64_t k, int64_t experts, ge_mx_types_t t, ge_epilog_t ep);
// Pointers of an execute; `experts` 0 for one product.
ge_status_t check_execute(int64_t m, int64_t experts, ge_mx_types_t t, ge_epilog_t ep, const void* xc, const void* xs,
                          const void* wc, const void* ws, const void* bias, const void* offsets, const void* D,
                          const void* ds);

// The launch of one execute.
struct MxLaunch {
  int cfg = 0;               // gemx::MxCfg
  int tiles_m = 0, tiles_n = 0;   // grouped: the most tiles of rows there can be
  int splits = 1;
  int waves = 0;             // of a workgroup
  bool tail = false;         // a second launch takes (or may take, by expert) a short last round
  int64_t grid_x = 0, grid_y = 1, grid_z = 1;
};
MxLaunch choose(int64_t m, int64_t n, int64_t k, int64_t experts, ge_mx_types_t t, int cus);
// Workspace that covers every m: the split tiles' counters and partial sums.
size_t workspace_bytes(int64_t experts, int cus);

ge_status_t check_norm(int64_t rows, int64_t d, ge_dtype_t dt, const void* x, int64_t ldx, const void* residual,
                       int64_t ldr, const void* weight, ge_dtype_t wdt, float eps, const void* sum, int64_t lds,
                       const void* y, int64_t ldy, const void* codes, const void* scales);
ge_status_t check_norm_backward(int64_t rows, int64_t d, ge_dtype_t dt, const void* dy, int64_t lddy, const void* s,
                                int64_t lds, const void* weight, ge_dtype_t wdt, float eps, const void* dres,
                                int64_t lddr, const void* dx, int64_t lddx, const void* dw, const void* ws,
                                size_t ws_bytes);
constexpr int64_t kNormMaxD = 32768;
// LDS of a row slot's 8-bit rows in the norm's kernel, `walk` rows of `granules` 256-value
// granules: the rows' 16-byte chunks with an odd stride, then their scales. A workgroup's slots
// lie one after the other, each on 16 bytes.
constexpr int norm_stage_bytes(int granules, int walk) {
  return (int)gemx::pad_to(granules * (16 * (walk + 1) * 16 + 2 * walk * 4), 16);
}
// Workgroups of the backward (each adds up the weight gradient of its rows) and the
// workspace for their sums.
int64_t norm_backward_groups(int64_t rows, int64_t d);
size_t norm_workspace_bytes(int64_t rows, int64_t d);

}  // namespace gemxh
