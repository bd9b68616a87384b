// Host-side rules of the gated feed-forward block: argument checks, workspaces, the choice of
// kernels. Plain C++17 with no HIP call or header, like plan_host.hpp.
#pragma once

#include <cstddef>
#include <cstdint>

#include "gemm_epilog.h"
#include "plan_host.hpp"

namespace gegh {

constexpr int64_t kMaxDim = 1 << 20;
constexpr int64_t kMaxTokens = 0x7fffffff;
constexpr int64_t kMaxBackwardTokens = 1 << 24;   // k of the weights' gradients
constexpr int kCompute = 256;                     // compute units that workspaces are sized for

bool gate_ok(ge_gate_t a);
bool aligned(const void* p, size_t a);

ge_status_t check_forward(int64_t m, int64_t n, int64_t k, ge_dtype_t dt, ge_gate_t act, const void* x, const void* w,
                          const void* bias, ge_dtype_t vec, const void* h, const void* z);
ge_status_t check_down(int64_t m, int64_t d, int64_t n, ge_dtype_t dt, const void* h, const void* w, const void* y);
struct Backward {   // what a call of the backward wants, by its pointers
  const void *dy, *x, *w, *z, *h, *w_down, *dx, *dw, *dw_down, *dbias;
};
ge_status_t check_backward(int64_t m, int64_t n, int64_t k, int64_t d, ge_dtype_t dt, ge_gate_t act, const Backward& b,
                           ge_dtype_t vec, const void* ws, size_t ws_bytes);

// One product D (M, N) = A . B over K, dense operands in the storage orders of `lay` (bit 0: A
// stored (K, M), bit 1: B stored (N, K)): whether the 16-bit tile kernels take it (rows of whole
// 16-byte chunks).
bool fast_shape(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, int lay);
// Its configuration there, with the k loop split where that pays and `ws` bytes hold it.
ge_status_t fast_layout(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, int lay, int cus, size_t ws, geh::Layout* L);

// The general kernel: 128 x 128 tiles, or 64 x 64; and how many workgroups share a tile's k loop, as
// far as `ws` bytes hold their fp32 sums.
bool general_large(int64_t M, int64_t N, int cus);
int general_splits(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, size_t ws);

// The gated product X . W^T of (m, n) from 2 n rows, or (backward) dY . Wd with the activations'
// gradient, on the tile kernels.
ge_status_t gated_layout(int64_t m, int64_t n, int64_t k, ge_dtype_t dt, bool backward, int cus, geh::Layout* L);

// Whether X (m, k) . W^T with `rows` rows of W (gated: of both halves) goes to the kernel for few
// tokens.
bool skinny(int64_t m, int64_t rows, int64_t k, ge_dtype_t dt, bool gated, int cus);

// The kernel of X (m, k) . W^T with n columns (gated: of each half), where the pointers are on 16
// bytes or not; and of dY (m, d) . Wd with the activations' gradient.
enum class Kernel { kFew, kTiles, kGeneral };
Kernel forward_kernel(int64_t m, int64_t n, int64_t k, ge_dtype_t dt, bool gated, bool on16, int cus);
Kernel gradient_kernel(int64_t m, int64_t n, int64_t d, ge_dtype_t dt, bool on16);
// The general kernel's form for rows of fewer than 16 bytes.
bool general_narrow(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, int lay);

// Rows that one launch of any of these kernels takes, for n columns (gated: of each half): their
// workgroups have at least 16 values of the product for each lane.
int64_t launch_rows(int64_t n, bool gated);

// Column sums: ranges of rows summed side by side.
int64_t colsum_parts(int64_t m, int64_t cols);
// Rows of the sums of dZ's columns: from dH and Z, one for 16 rows or more; from any kernel of dZ at most.
int64_t dz_parts(int64_t m, int64_t n);
int64_t dz_sum_rows(int64_t m, int64_t n);

// The backward's workspace: dZ (m, 2 n), then dH in fp32 (written where the product and the
// activations' gradient are separate kernels, held for any: whether the tiles take them also depends
// on the pointers' alignment), then the flags of dX's split, beside them the column sums of dZ until
// they are added up, and after that what one product needs.
struct BackwardSpace {
  size_t dh, scratch, total;   // offsets; dZ is at 0
};
BackwardSpace backward_space(int64_t m, int64_t n, int64_t k, int64_t d, ge_dtype_t dt);

}  // namespace gegh
