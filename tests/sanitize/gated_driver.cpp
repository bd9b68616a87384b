// Exercises the host rules of the gated feed-forward block and of 4-bit weights (gated_host.cpp and
// w4_host.cpp with plan_host.cpp, which plans the products) under AddressSanitizer and
// UndefinedBehaviorSanitizer: built by tests/test_gated_host_sanitize.py with g++, host code only.
// Checks, over grids of sizes up to the limits:
//   * every product that the 16-bit tiles may take has a layout on any number of compute units,
//     within the workspace that it was given;
//   * the backward's workspace holds dZ, dH and what each of its products and the column sums ask
//     for, in parts on 256-byte borders, on devices of other sizes too;
//   * few tokens always go to their kernel, and more than its grid takes never;
//   * 4-bit weights: sizes of the layout, kernels that exist for the operands;
//   * argument rules at the ends of the supported ranges.
// Prints "ok (0 failures)" on success.
#include <algorithm>
#include <cstdio>

#include "gated_host.hpp"
#include "w4_host.hpp"

namespace {

int failures = 0;

void check(bool ok, const char* what, long long a = 0, long long b = 0, long long c = 0, long long d = 0) {
  if (!ok) {
    if (failures < 50) std::printf("FAIL %s %lld %lld %lld %lld\n", what, a, b, c, d);
    ++failures;
  }
}

const ge_dtype_t kTypes[] = {GE_F32, GE_F16, GE_BF16};
const int64_t kSizes[] = {1, 7, 8, 64, 72, 129, 520, 1000, 1101, 4096, 11008, 65544, 1 << 20};
const int64_t kTokens[] = {0, 1, 16, 17, 77, 128, 129, 333, 2048, 4100, 65536, 1 << 24, 0x7fffffff};
const int kCus[] = {1, 64, 256, 304};

void check_products() {
  for (ge_dtype_t dt : kTypes)
    for (int64_t m : kTokens)
      for (int64_t n : kSizes)
        for (int64_t k : kSizes)
          for (int lay : {0, 1, 2})
            for (int cus : kCus) {
              if (!m || !gegh::fast_shape(m, n, k, dt, lay)) continue;
              if ((m + 63) / 64 * ((n + 31) / 32) > 0x7fffffff) continue;
              geh::Layout L;
              for (size_t ws : {(size_t)0, (size_t)1 << 20, ~(size_t)0}) {
                check(gegh::fast_layout(m, n, k, dt, lay, cus, ws, &L) == GE_OK, "a layout", m, n, k, lay);
                check(L.ws_bytes <= ws && (L.sk_wgs == 0) == (L.ws_bytes == 0), "its workspace", m, n, k, cus);
              }
              const int64_t parts = gegh::general_splits(m, n, k, dt, (size_t)1 << 24);
              check(parts >= 1 && parts <= 16 && (parts == 1 || parts * m * n * 4 <= 1 << 24), "parts", m, n, k);
              if (lay < 2 && n <= 1 << 19)
                check(gegh::gated_layout(m, n, k, dt, lay == 0, cus, &L) == GE_OK && !L.sk_wgs, "a gated layout", m, n, k, lay);
            }
}

void check_space() {
  for (ge_dtype_t dt : kTypes)
    for (int64_t m : kTokens)
      for (int64_t n : kSizes)
        for (int64_t k : kSizes)
          for (int64_t d : kSizes) {
            const gegh::BackwardSpace s = gegh::backward_space(m, n, k, d, dt);
            if (m < 1 || m > gegh::kMaxBackwardTokens) {
              check(s.total == 0, "nothing to hold", m, n, k, d);
              continue;
            }
            const size_t es = dt == GE_F32 ? 4 : 2;
            check(s.dh % 256 == 0 && s.scratch % 256 == 0 && s.total % 256 == 0, "borders", m, n, k, d);
            check(s.dh >= (size_t)m * 2 * n * es && s.scratch >= s.dh + (size_t)m * n * 4, "dZ and dH", m, n, k, d);
            const size_t left = s.total - s.scratch;
            const int64_t parts = gegh::colsum_parts(m, 2 * n);
            check(parts >= 1 && parts <= 65535 && (size_t)parts * 2 * n * 4 <= left, "column sums", m, n, k, d);
            const int64_t p[3][3] = {{m, k, 2 * n}, {2 * n, k, m}, {d, n, m}};
            for (const auto& q : p)   // the parts that its size allows are the ones that were meant
              check(gegh::general_splits(q[0], q[1], q[2], dt, left) == gegh::general_splits(q[0], q[1], q[2], dt, ~(size_t)0),
                    "parts of a product", q[0], q[1], q[2]);
          }
}

void check_few() {
  for (ge_dtype_t dt : kTypes)
    for (int64_t n : kSizes)
      for (int64_t k : kSizes)
        for (bool gated : {false, true})
          for (int cus : kCus) {
            check(gegh::skinny(1, 2 * n, k, dt, gated, cus) && gegh::skinny(16, 2 * n, k, dt, gated, cus), "few", n, k);
            check(!gegh::skinny(65536, 2 * n, k, dt, gated, cus) && !gegh::skinny(0x7fffffff, 2 * n, k, dt, gated, cus), "many", n, k);
            gegh::skinny(100, 2 * n, k, dt, gated, cus);
          }
}

void check_gated_rules() {
  alignas(256) char buf[1024];
  const void *p = buf, *q = buf + 1;
  const ge_gate_t S = GE_GATE_SILU;
  const int64_t top = gegh::kMaxDim;
  check(gegh::check_forward(5, top, top, GE_BF16, S, p, p, nullptr, GE_F32, p, nullptr) == GE_OK, "largest sizes");
  check(gegh::check_forward(0, 1, 1, GE_F32, S, nullptr, p, nullptr, GE_F32, nullptr, nullptr) == GE_OK, "no tokens");
  check(gegh::check_forward(5, top + 1, 8, GE_BF16, S, p, p, nullptr, GE_F32, p, nullptr) == GE_ERR_INVALID_VALUE, "n");
  check(gegh::check_forward(5, 8, 0, GE_BF16, S, p, p, nullptr, GE_F32, p, nullptr) == GE_ERR_INVALID_VALUE, "k");
  check(gegh::check_forward(-1, 8, 8, GE_BF16, S, p, p, nullptr, GE_F32, p, nullptr) == GE_ERR_INVALID_VALUE, "m");
  check(gegh::check_forward(0x7fffffff, top, 8, GE_BF16, S, p, p, nullptr, GE_F32, p, nullptr) == GE_ERR_NOT_SUPPORTED, "grid");
  check(gegh::check_forward(5, 8, 8, GE_BF16, S, p, p, p, GE_F16, p, nullptr) == GE_ERR_NOT_SUPPORTED, "bias type");
  check(gegh::check_forward(5, 8, 8, GE_BF16, (ge_gate_t)9, p, p, p, GE_F32, p, nullptr) == GE_ERR_INVALID_VALUE, "activation");
  check(gegh::check_forward(5, 8, 8, GE_BF16, S, p, nullptr, p, GE_F32, p, nullptr) == GE_ERR_NULL_POINTER, "no w");
  check(gegh::check_forward(5, 8, 8, GE_BF16, S, q, p, p, GE_F32, p, nullptr) == GE_ERR_MISALIGNED, "x on one byte");
  check(gegh::check_down(5, 0, 8, GE_F32, p, p, p) == GE_ERR_INVALID_VALUE && gegh::check_down(5, 8, 8, GE_F32, p, p, q) == GE_ERR_MISALIGNED, "down");
  gegh::Backward b = {p, p, p, p, p, p, p, p, p, p};
  const size_t need = gegh::backward_space(5, 8, 8, 8, GE_F16).total;
  check(gegh::check_backward(5, 8, 8, 8, GE_F16, S, b, GE_F32, p, need) == GE_OK, "backward");
  check(gegh::check_backward(5, 8, 8, 8, GE_F16, S, b, GE_F32, p, need - 1) == GE_ERR_SCRATCH, "small workspace");
  check(gegh::check_backward(5, 8, 8, 8, GE_F16, S, b, GE_F32, nullptr, need) == GE_ERR_NULL_POINTER, "no workspace");
  check(gegh::check_backward(5, 8, 8, 8, GE_F16, S, b, GE_F32, buf + 16, need) == GE_ERR_MISALIGNED, "workspace");
  check(gegh::check_backward(gegh::kMaxBackwardTokens + 1, 8, 8, 8, GE_F16, S, b, GE_F32, p, ~(size_t)0) == GE_ERR_NOT_SUPPORTED, "tokens");
  check(gegh::check_backward(0, 8, 8, 8, GE_F16, S, b, GE_F32, nullptr, 0) == GE_OK, "no tokens back");
  b.w_down = nullptr;
  check(gegh::check_backward(5, 8, 8, 9, GE_F16, S, b, GE_F32, p, ~(size_t)0) == GE_ERR_INVALID_VALUE, "dH of another width");
  b.dw_down = nullptr;
  check(gegh::check_backward(5, 8, 8, 8, GE_F16, S, b, GE_F32, p, need) == GE_OK, "from dH");
}

void check_w4() {
  const int64_t top = gew4h::kMaxDim;
  for (int halves : {1, 2})
    for (int64_t rows : kSizes)
      for (int64_t k : kSizes)
        for (int64_t group : {32L, 64L, 128L, 384L, (long)top}) {
          if (rows % halves) continue;
          const int64_t rg = halves * ((rows / halves + 15) / 16);
          check(gew4h::code_bytes(rows, k, halves) == (size_t)(rg * ((k + 127) / 128) * 1024), "codes", rows, k, halves);
          check(gew4h::scale_count(rows, k, group, halves) == (size_t)(rg * ((k + group - 1) / group) * 16), "scales", rows, k, group);
        }
  for (int64_t group : {0L, 16L, 48L, 96L, 130L, -128L, (long)top + 128}) check(!gew4h::shape_ok(16, 128, group, 1), "group", group);
  check(!gew4h::shape_ok(3, 8, 32, 2) && !gew4h::shape_ok(0, 8, 32, 1) && !gew4h::shape_ok(8, 0, 32, 1), "shapes");
  check(!gew4h::shape_ok(top + 1, 8, 32, 1) && gew4h::shape_ok(2 * top, top, 32, 2) && !gew4h::shape_ok(8, 8, 32, 3), "limits");
  for (int64_t m : kTokens)
    for (int64_t n : kSizes)
      for (int64_t k : kSizes)
        for (int64_t group : {32, 64, 128, 1024})
          for (bool gated : {false, true})
            for (bool chunks : {false, true})
              for (int cus : kCus) {
                if (!m || (chunks && k % 8)) continue;
                const int c = gew4h::choose(m, n, k, group, gated, chunks, cus);
                check(c >= -1 && c < gew4::W4_COUNT, "kernel", m, n, k, c);
                check((c != gew4::W4_L && c != gew4::W4_L3) || (chunks && group >= 64), "the large tiles' operands", m, n, k, group);
                check(c < 0 || k >= 8, "rows of eight", m, n, k, c);
                check(m > 16 || c < 0, "few tokens", n, k, group, c);
              }
  alignas(16) char buf[64];
  check(gew4h::check_product(5, 8, GE_F32, GE_F32, buf, nullptr, GE_F32, buf) == GE_ERR_NOT_SUPPORTED, "f32 x");
  check(gew4h::check_product(0, 8, GE_F16, GE_F16, nullptr, nullptr, GE_F32, nullptr) == GE_OK, "no tokens");
  check(gew4h::check_product(5, 8, GE_F16, GE_BF16, buf, nullptr, GE_F32, buf) == GE_ERR_NOT_SUPPORTED, "out");
  check(gew4h::check_product(0x7fffffff, top, GE_F16, GE_F16, buf, nullptr, GE_F32, buf) == GE_ERR_NOT_SUPPORTED, "grid");
  check(gew4h::check_product(5, 8, GE_F16, GE_F16, buf + 1, nullptr, GE_F32, buf) == GE_ERR_MISALIGNED, "x on one byte");
  check(gew4h::check_weight(16, 128, 128, 1, buf + 8, buf, buf) == GE_ERR_MISALIGNED, "codes");
  check(gew4h::check_quantize(4, 8, GE_F32, buf, -1, GE_F16) == GE_ERR_INVALID_VALUE, "rows apart by less than nothing");
  check(gew4h::check_dequantize(4, 8, GE_F16, GE_F32, buf, 7) == GE_ERR_INVALID_VALUE, "rows over each other");
}

}  // namespace

int main() {
  check_products();
  check_space();
  check_few();
  check_gated_rules();
  check_w4();
  std::printf("%s (%d failures)\n", failures ? "FAILED" : "ok", failures);
  return failures != 0;
}
