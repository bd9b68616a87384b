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
  if (m && (!b.dy || (!b.z && (b.dx || b.dw || b.dbias)))) return GE_ERR_NULL_POINTER;
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

// The large tile where it gives every compute unit one.
bool general_large(int64_t M, int64_t N, int cus) { return cdiv(M, 128) * cdiv(N, 128) >= cus; }

// Parts of at least eight k-tiles of 128 bytes, so many that the tiles fill the compute units twice.
// Sized for kCompute of them, so that the result does not depend on the device.
int general_splits(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, size_t ws) {
  if (general_large(M, N, kCompute)) return 1;
  const int64_t kt = cdiv(K * (int64_t)geh::elem_size(dt), 128), tiles = cdiv(M, 64) * cdiv(N, 64);
  const int64_t s = std::min({kt / 8, cdiv(2 * kCompute, tiles), (int64_t)16});
  return s > 1 && (size_t)s * M * N * 4 <= ws ? (int)s : 1;
}

ge_status_t gated_layout(int64_t m, int64_t n, int64_t k, ge_dtype_t dt, bool backward, int cus, geh::Layout* L) {
  const ge_dtypes_t t = {dt, dt, dt};
  const int64_t cols = backward ? n : 2 * n;
  // (forward: the configurations for transposed operands; backward: those and the 192 and 128 x 256
  // tiles; the others' places are taken by the nearest, also where GE_TILE names a register-staged one)
  const int lay = backward ? 0 : 2;
  int cfg = geh::choose_cfg(m, cols, k, dt, cus, lay);
  if (cfg == gek::CFG_LH) cfg = gek::CFG_L;
  if (cfg == gek::CFG_LM4 || !gek::cfg_is_dtl(cfg)) cfg = gek::CFG_LM;
  return geh::make_layout(m, cols, k, t, GE_EPILOG_NONE, lay, cus, cfg, false, gek::cfg_can_persist(cfg), L);
}

// By estimated time in microseconds, fitted to 17 to 333 tokens by 2 x 1101 x 743, 1104 x 744, 1376 x
// 1024, 2752 x 1024, 4096 x 2048 and 11008 x 4096 and by their single halves (the kernel that is taken
// was at most 4 us, or an eighth, behind the other at any of them).
//   few tokens  a round of workgroups reads a block of tokens for every 16 rows (gated: 32) of W, at
//               8.5 TB/s (gated 5.6, as a workgroup waits for more); 16-bit types faster where
//               compute units stay idle, rows that are not whole 16-byte chunks slower. 64 tokens by 2
//               x 4096 x 2048: bf16 23 against 18, fp32 45 against 50;
//   tiles       128 x 128: W at 4.2 TB/s or half a microsecond per k-tile and round, whichever is
//               longer;
//   general     0.78 per 128 bytes of k in fp32 and 0.5 in 16 bits, 0.5 and 0.3 more for each further
//               tile of a compute unit.
bool skinny(int64_t m, int64_t rows, int64_t k, ge_dtype_t dt, bool gated, int cus) {
  if (m <= 16) return true;
  if (m > 65535) return false;   // (its grid, by far)
  const bool wide = dt == GE_F32;
  const double es = wide ? 4 : 2, w = (double)rows * k * es;
  const int64_t step = m <= 32 ? 32 : 64, wgs = cdiv(gated ? rows / 2 : rows, 16) * cdiv(m, step);
  const double rounds = wgs <= cus ? 1.0 : std::max(2.0, (double)wgs / cus);
  double rate = gated ? 5.6e6 : 8.5e6;
  if ((int64_t)(k * es) % 16) rate *= wide ? 0.7 : 0.4;
  else if (!wide) rate /= std::min(1.0, std::max(0.4, (double)wgs / cus));
  const double few = (wide ? 3.5 : 2.5) + rounds * (double)((gated ? 32 : 16) + step) * (double)k * es * cus / rate;
  double tiles;
  if (fast_shape(m, rows, k, dt, 2)) {
    tiles = 3.0 + std::max(w / 4.2e6, (double)(cdiv(cdiv(m, 128) * cdiv(rows, 128), cus) * cdiv(k, 64)) * 0.5);
  } else {
    const double more = (double)cdiv(cdiv(m, 64) * cdiv(rows, 64), cus) - 1.0;
    tiles = 3.0 + (double)cdiv((int64_t)(k * es), 128) * (wide ? 0.78 + 0.5 * more : 0.5 + 0.3 * more);
  }
  return few < tiles;
}

Kernel forward_kernel(int64_t m, int64_t n, int64_t k, ge_dtype_t dt, bool gated, bool on16, int cus) {
  if (skinny(m, gated ? 2 * n : n, k, dt, gated, cus)) return Kernel::kFew;
  return fast_shape(m, n, k, dt, 2) && on16 ? Kernel::kTiles : Kernel::kGeneral;
}

Kernel gradient_kernel(int64_t m, int64_t n, int64_t d, ge_dtype_t dt, bool on16) {
  return fast_shape(m, n, d, dt, 0) && on16 ? Kernel::kTiles : Kernel::kGeneral;
}

bool general_narrow(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, int lay) {
  const int64_t row_a = lay & 1 ? M : K, row_b = lay & 2 ? K : N;
  return std::min(row_a, row_b) * (int64_t)geh::elem_size(dt) < 16;
}

// (whole tiles of any of them: 256 rows)
int64_t launch_rows(int64_t n, bool gated) { return geh::rows_per_launch(256, 4 * cdiv(n, gated ? 32 : 64), 256); }

int64_t colsum_parts(int64_t m, int64_t cols) {
  const int64_t across = cdiv(cols, 512);
  if (m <= 128) return 1;   // (one kernel, 20 to 32 rows after each other in each of its four rows)
  return std::max<int64_t>(1, std::min(cdiv(m, 32), cdiv(1024, across)));
}

int64_t dz_parts(int64_t m, int64_t n) {
  if (m <= 32) return 1;   // (no second kernel)
  return std::max<int64_t>(1, std::min(cdiv(m, 16), cdiv(1024, cdiv(n, 512))));
}

// (the tiles: one for 32 rows at least, in whole tiles of 128)
int64_t dz_sum_rows(int64_t m, int64_t n) { return std::max(cdiv(m, 128) * 4, dz_parts(m, n)); }

BackwardSpace backward_space(int64_t m, int64_t n, int64_t k, int64_t d, ge_dtype_t dt) {
  BackwardSpace s = {0, 0, 0};
  if (m < 1 || m > kMaxBackwardTokens || !dim_ok(n) || !dim_ok(k) || !dim_ok(d) || !dtype_ok(dt)) return s;
  s.dh = align256((size_t)m * 2 * n * geh::elem_size(dt));
  s.scratch = s.dh + align256((size_t)m * n * 4);
  // sums of dZ, and of those (where they are too many for one kernel)
  const int64_t sums = dz_sum_rows(m, n);
  size_t most = geh::kSkFlagRegion + (size_t)(sums + colsum_parts(sums, 2 * n)) * 2 * n * 4;
  geh::Layout L;
  if (fast_shape(m, k, 2 * n, dt, 0) && fast_layout(m, k, 2 * n, dt, 0, kCompute, ~(size_t)0, &L) == GE_OK)
    most = std::max(most, L.ws_bytes);
  // sums of the general kernel's parts (also of 16-bit products whose pointers turn out unaligned)
  const int64_t prod[3][3] = {{m, k, 2 * n}, {2 * n, k, m}, {d, n, m}};
  for (const auto& q : prod) {
    const int parts = general_splits(q[0], q[1], q[2], dt, ~(size_t)0);
    if (parts > 1) most = std::max(most, (size_t)parts * q[0] * q[1] * 4);
  }
  s.total = s.scratch + align256(most);
  return s;
}

}  // namespace gegh
