// Exercises the host arithmetic of the microscaled operators and the norm (mx_host.cpp and
// the constexpr layout and tile tables that the kernels share) under AddressSanitizer and
// UndefinedBehaviorSanitizer: built by tests/test_mx_host_sanitize.py with g++, host code
// only. Checks:
//   * the norm's LDS stage: every row slot begins on 16 bytes (its chunks move 16 bytes at a
//     time), and a single row fits the LDS at every width.
// Prints "ok (0 failures)" on success.
#include <cstdio>

#include "mx_format.hpp"
#include "mx_host.hpp"
#include "mx_tiles.hpp"

namespace {

int failures = 0;

void check(bool ok, const char* what, long long a, long long b = 0, long long c = 0, long long d = 0) {
  if (!ok) {
    if (failures < 50) std::printf("FAIL %s %lld %lld %lld %lld\n", what, a, b, c, d);
    ++failures;
  }
}

void check_norm_stage() {
  for (int g = 1; g <= gemxh::kNormMaxD / gemx::kKPad; ++g)
    for (int walk = 1; walk <= 8; walk *= 2) {
      const int bytes = gemxh::norm_stage_bytes(g, walk), codes = g * 16 * (walk + 1) * 16;
      check(bytes % 16 == 0, "stage alignment", g, walk, bytes);
      check(bytes >= codes + g * 2 * walk * 4, "stage size", g, walk, bytes);
      if (walk == 1) check(bytes <= 80 * 1024, "a row's stage", g, walk, bytes);
    }
}

}  // namespace

int main() {
  check_norm_stage();
  std::printf("%s (%d failures)\n", failures ? "FAILED" : "ok", failures);
  return failures != 0;
}
