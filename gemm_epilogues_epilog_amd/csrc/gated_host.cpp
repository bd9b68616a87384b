// Rules declared in gated_host.hpp.
#include "gated_host.hpp"

#include <algorithm>

#include "tiles.hpp"

namespace gegh {

namespace {
bool dtype_ok(ge_dtype_t d) { return d == GE_F32 || d == GE_F16 || d == GE_BF16; }
bool dim_ok(int64_t v) { return v >= 1 && v <= kMaxDim; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }
// every launch has at most 2^31 - 1 workgroups
bool grid_ok(int64_t rows, int64_t cols) { return cdiv(rows, 64) * cdiv(cols, 32) <= 0x7fffffff; }
}  // namespace

bool gate_ok(ge_gate_t a) { return a == GE_GATE_SILU || a == GE_GATE_GELU || a == GE_GATE_RELU; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

ge_status_t check_forward(int64_t m, int64_t n, int64_t k, ge_dtype_t dt, ge_gate_t act, const void* x, const void* w,
                          const void* bias, ge_dtype_t vec, const void* h, const void* z) {
  if (m < 0 || m > kMaxTokens || !dim_ok(n) || !dim_ok(k) || !dtype_ok(dt) || !gate_ok(act) || !dtype_ok(vec))
    return GE_ERR_INVALID_VALUE;
  if (vec != dt && vec != GE_F32) return GE_ERR_NOT_SUPPORTED;
  if (!grid_ok(m, n)) return GE_ERR_NOT_SUPPORTED;
  if (!w || (m && (!x || !h))) return GE_ERR_NULL_POINTER;
  const size_t es = geh::elem_size(dt);
  if (!aligned(x, es) || !aligned(w, es) || !aligned(h, es) || !aligned(z, es) || !aligned(bias, geh::elem_size(vec)))
    return GE_ERR_MISALIGNED;
  return GE_OK;
}

ge_status_t check_down(int64_t m, int64_t d, int64_t n, ge_dtype_t dt, const void* h, const void* w, const void* y) {
  if (m < 0 || m > kMaxTokens || !dim_ok(n) || !dim_ok(d) || !dtype_ok(dt)) return GE_ERR_INVALID_VALUE;
  if (!grid_ok(m, d)) return GE_ERR_NOT_SUPPORTED;
  if (!w || (m && (!h || !y))) return GE_ERR_NULL_POINTER;
  const size_t es = geh::elem_size(dt);
  if (!aligned(h, es) || !aligned(w, es) || !aligned(y, es)) return GE_ERR_MISALIGNED;
  return GE_OK;
}

ge_status_t check_backward(int64_t m, int64_t n, int64_t k, int64_t d, ge_dtype_t dt, ge_gate_t act, const Backward& b,
                           ge_dtype_t vec, const void* ws, size_t ws_bytes) {
  if (m < 0 || m > kMaxTokens || !dim_ok(n) || !dim_ok(k) || !dim_ok(d) || !dtype_ok(dt) || !gate_ok(act) ||
      !dtype_ok(vec))
    return GE_ERR_INVALID_VALUE;
  if (vec != dt && vec != GE_F32) return GE_ERR_NOT_SUPPORTED;
  if (m > kMaxBackwardTokens || !grid_ok(std::max(m, 2 * n), std::max({n, k, d}))) return GE_ERR_NOT_SUPPORTED;
  if (!b.w_down && d != n) return GE_ERR_INVALID_VALUE;   // dy is then the gradient of H itself
  if (m && (!b.dy || !b.z)) return GE_ERR_NULL_POINTER;
  if (b.dx && m && !b.w) return GE_ERR_NULL_POINTER;
  if (b.dw && m && !b.x) return GE_ERR_NULL_POINTER;
  if (b.dw_down && m && !b.h) return GE_ERR_NULL_POINTER;
  if (b.dw_down && !b.w_down) return GE_ERR_NULL_POINTER;
  const size_t es = geh::elem_size(dt);
  for (const void* p : {b.dy, b.x, b.w, b.z, b.h, b.w_down, b.dx, b.dw, b.dw_down})
    if (!aligned(p, es)) return GE_ERR_MISALIGNED;
  if (!aligned(b.dbias, geh::elem_size(vec)) || !aligned(ws, 256)) return GE_ERR_MISALIGNED;
  const size_t need = backward_space(m, n, k, d, dt).total;
  if (need && !ws) return GE_ERR_NULL_POINTER;
  if (ws_bytes < need) return GE_ERR_SCRATCH;
  return GE_OK;
}

bool fast_shape(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, int lay) {
  if (dt == GE_F32 || N % 8) return false;
  return (lay & 1 ? M : K) % 8 == 0 && (!(lay & 2) || K % 8 == 0);
}

ge_status_t fast_layout(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, int lay, int cus, size_t ws, geh::Layout* L) {
  const ge_dtypes_t t = {dt, dt, dt};
  const int cfg = geh::choose_cfg(M, N, K, dt, cus, lay);
  ge_status_t st = geh::make_layout(M, N, K, t, GE_EPILOG_NONE, lay, cus, cfg, true, true, L);
  if (st == GE_OK && L->ws_bytes > ws) st = geh::make_layout(M, N, K, t, GE_EPILOG_NONE, lay, cus, cfg, false, true, L);
  return st;
}

ge_status_t gated_layout(int64_t m, int64_t n, int64_t k, ge_dtype_t dt, bool backward, int cus, geh::Layout* L) {
  const ge_dtypes_t t = {dt, dt, dt};
  const int64_t cols = backward ? n : 2 * n;
  int cfg = geh::choose_cfg(m, cols, k, dt, cus, 2);   // (2: only configurations that take transposed operands)
  return geh::make_layout(m, cols, k, t, GE_EPILOG_NONE, 2, cus, cfg, false, cfg == gek::CFG_L, L);
}

int64_t colsum_parts(int64_t m, int64_t cols) {
  const int64_t across = cdiv(cols, 512);
  return std::max<int64_t>(1, std::min(cdiv(m, 32), cdiv(1024, across)));
}

BackwardSpace backward_space(int64_t m, int64_t n, int64_t k, int64_t d, ge_dtype_t dt) {
  BackwardSpace s = {0, 0, 0};
  if (m < 1 || m > kMaxBackwardTokens || !dim_ok(n) || !dim_ok(k) || !dim_ok(d) || !dtype_ok(dt)) return s;
  s.dh = align256((size_t)m * 2 * n * geh::elem_size(dt));
  s.scratch = s.dh + align256((size_t)m * n * 4);
  size_t most = (size_t)colsum_parts(m, 2 * n) * 2 * n * 4;
  geh::Layout L;
  if (fast_shape(m, k, 2 * n, dt, 0) && fast_layout(m, k, 2 * n, dt, 0, kCompute, ~(size_t)0, &L) == GE_OK)
    most = std::max(most, L.ws_bytes);
  s.total = s.scratch + align256(most);
  return s;
}

}  // namespace gegh
