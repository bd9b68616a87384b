// Exercises the host arithmetic of the microscaled operators and the norm (mx_host.cpp and
// the constexpr layout and tile tables that the kernels share) under AddressSanitizer and
// UndefinedBehaviorSanitizer: built by tests/test_mx_host_sanitize.py with g++, host code
// only. Checks:
//   * the norm's LDS stage: every row slot begins on 16 bytes (its chunks move 16 bytes at a
//     time), and a single row fits the LDS at every width;
//   * sizes of the layout: whole 16-byte chunks that hold every value, 0 rows included;
//   * the product's launch over a grid of problems: tiles that cover the output, parts of k
//     that fit the device, the counters and the workspace, lane counts, and for products by
//     expert as many tiles of rows as any split of the rows over the experts takes;
//   * argument rules at the ends of the supported ranges, and the gradient's workspace.
// Prints "ok (0 failures)" on success.
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>

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

void check_layout() {
  for (int fmt : {(int)gemx::FP4, (int)gemx::FP8})
    for (int64_t rows : {0LL, 1LL, 31LL, 32LL, 33LL, 1000LL, (1LL << 29) - 32})
      for (int64_t k : {1LL, 31LL, 255LL, 256LL, 257LL, 11008LL, 1LL << 20}) {
        const int64_t c = gemx::code_bytes(fmt, rows, k), s = gemx::scale_bytes(rows, k);
        check(c % 16 == 0 && s % 16 == 0, "whole chunks", fmt, rows, k);
        check(c * (fmt == gemx::FP4 ? 2 : 1) >= rows * k && s >= rows * ((k + 31) / 32), "size", fmt, rows, k);
        check(rows || (!c && !s), "no rows", fmt, rows, k);
      }
}

// tiles of `bm` rows that a split of m rows over the experts takes
int64_t tiles_of(const std::vector<int64_t>& ends, int64_t bm) {
  int64_t lo = 0, t = 0;
  for (int64_t hi : ends) {
    if (hi > lo) t += (hi - (lo & ~int64_t(31)) + bm - 1) / bm;
    lo = std::max(lo, hi);
  }
  return t;
}

void check_choice(int64_t m, int64_t n, int64_t k, int64_t experts, ge_mx_types_t t, int cus) {
  using namespace gemx;
  if (gemxh::check_plan(n, k, experts, t, GE_EPILOG_NONE) != GE_OK) return;
  const gemxh::MxLaunch L = gemxh::choose(m, n, k, experts, t, cus);
  check(L.cfg >= 0 && L.cfg < MX_COUNT, "configuration", m, n, k, L.cfg);
  const MxTile& T = kMxTiles[L.cfg];
  const int64_t cols = t.d == GE_MX_D_MXFP8 ? pad_to(n, kKPad) : n;
  const int64_t lanes = L.grid_x * L.grid_y * L.grid_z * L.waves * 64;
  check(L.grid_x > 0 && L.grid_y > 0 && L.grid_z > 0 && L.grid_y <= 65535 && L.grid_z <= 65535, "grid", m, n, k, experts);
  check(lanes < (1LL << 32), "lanes", m, n, k, experts);
  check((int64_t)L.tiles_n * T.bn >= cols && (int64_t)(L.tiles_n - 1) * T.bn < cols, "columns", m, n, k, experts);
  check(L.splits >= 1 && L.splits <= kMxMaxSplit, "parts", m, n, k, L.splits);
  if (!T.stages) {   // skinny: a workgroup per expert and columns, or several
    check(L.tiles_m == (experts ? experts : 1) && L.splits == 1 && L.waves >= 2 && L.waves <= kMxSkinnyWaves, "skinny", m,
          n, k, L.waves);
    return;
  }
  check(L.waves == mx_waves(T), "waves", m, n, k, L.waves);
  const int64_t tiles = (int64_t)L.tiles_m * L.tiles_n;
  if (!experts) check((int64_t)L.tiles_m * T.bm >= m && (int64_t)(L.tiles_m - 1) * T.bm < m, "rows", m, n, k, L.tiles_m);
  check(L.grid_x == (L.cfg == MX_L ? std::min<int64_t>(tiles, cus) : tiles * L.splits), "workgroups", m, n, k, L.grid_x);
  if (L.splits > 1) {
    check(!experts && tiles <= kMxCounters && tiles * L.splits <= cus, "split tiles", m, n, k, L.splits);
    check(kMxCounterBytes + (size_t)(tiles * L.splits * T.bm * T.bn * 4) <= gemxh::workspace_bytes(experts, cus),
          "workspace", m, n, k, L.splits);
    check(L.splits <= pad_to(k, kKPad) / mx_bk((int)t.x), "a k-tile to each part", m, n, k, L.splits);
  }
  check(!L.tail || (L.cfg == MX_L && tiles > cus), "a second launch", m, n, k, L.cfg);
  if (experts) {
    std::mt19937_64 rng(m * 31 + experts);
    std::vector<int64_t> ends(experts);
    const auto fits = [&](const char* what) { check(tiles_of(ends, T.bm) <= L.tiles_m, what, m, experts, T.bm, L.tiles_m); };
    for (int64_t& e : ends) e = (int64_t)(rng() % (uint64_t)(m + 1));
    std::sort(ends.begin(), ends.end());
    fits("any split of the rows");
    for (int64_t e = 0; e < experts; ++e) ends[e] = std::min(m, e + 1);   // a row each, the last expert the rest
    ends[experts - 1] = m;
    fits("a row to each expert");
    for (int64_t e = 0; e < experts; ++e) ends[e] = std::min(m, 31 + e * (T.bm + 1));   // a row past a tile each
    ends[experts - 1] = m;
    fits("a row past a tile");
  }
}

void check_choices() {
  for (int64_t m : {1LL, 15LL, 16LL, 17LL, 33LL, 64LL, 100LL, 255LL, 300LL, 1000LL, 2200LL, 8192LL, 16001LL, 1LL << 20})
    for (int64_t n : {1LL, 96LL, 257LL, 1376LL, 4096LL, 16400LL, 1LL << 20})
      for (int64_t k : {1LL, 300LL, 2048LL, 4096LL, 11008LL, 1LL << 20})
        for (int64_t experts : {0LL, 1LL, 7LL, 64LL, 128LL, 300LL, 4096LL})
          for (ge_mx_format_t x : {GE_MXFP4, GE_MXFP8})
            for (ge_mx_out_t d : {GE_MX_D_F32, GE_MX_D_BF16, GE_MX_D_MXFP8})
              for (int cus : {256, 64, 1}) {
                // what fits the device's memory (an execute refuses launches of 2^32 lanes)
                const int64_t kp = gemx::pad_to(k, gemx::kKPad);
                if (m * n > (1LL << 37) || m * kp > (1LL << 38) || std::max<int64_t>(1, experts) * n * kp > (1LL << 39))
                  continue;
                check_choice(m, n, k, experts, ge_mx_types_t{x, d, GE_F32}, cus);
              }
}

void check_rules() {
  using namespace gemxh;
  void* p = reinterpret_cast<void*>(uintptr_t(1) << 20);
  check(shape_ok(0, 1) && shape_ok((1LL << 29) - 32, 256) && !shape_ok(1LL << 29, 256) && !shape_ok(1, (1LL << 20) + 1) &&
            !shape_ok(-1, 8) && !shape_ok(8, 0) && !shape_ok(1LL << 31, 1),
        "shapes", 0);
  const int64_t most = (1LL << 31) - 1;
  check(check_norm(most, 1, GE_BF16, p, 1, nullptr, 0, p, GE_F32, 0.0f, nullptr, 0, p, 1, nullptr, nullptr) == GE_OK,
        "norm of 2^31 - 1 rows", most);
  check(check_norm(most + 1, 1, GE_BF16, p, 1, nullptr, 0, p, GE_F32, 0.0f, nullptr, 0, p, 1, nullptr, nullptr) ==
            GE_ERR_INVALID_VALUE,
        "norm of 2^31 rows", most + 1);
  check(check_norm(most, kNormMaxD, GE_BF16, p, 0, nullptr, 0, p, GE_F32, 0.0f, nullptr, 0, nullptr, 0, p, p) ==
            GE_ERR_NOT_SUPPORTED,
        "8-bit result past the layout's tiles", most);
  for (int64_t rows : {0LL, 1LL, 3LL, 255LL, 2049LL, (long long)most})
    for (int64_t d : {1LL, 512LL, 513LL, 1024LL, 4096LL, 4097LL, 32768LL}) {
      const int64_t g = norm_backward_groups(rows, d);
      const size_t w = norm_workspace_bytes(rows, d);
      check(g <= rows && g <= 2048 && w == (size_t)g * (size_t)d * 4, "gradient's workspace", rows, d, g, (long long)w);
      if (rows)
        check(check_norm_backward(rows, d, GE_F16, p, 0, p, 0, p, GE_F16, 1e-6f, nullptr, 0, p, d, p, p, w - 1) ==
                  GE_ERR_SCRATCH,
              "a workspace too small", rows, d);
    }
  check(check_plan(1 << 20, 1 << 20, 0, ge_mx_types_t{GE_MXFP8, GE_MX_D_F32, GE_F32}, GE_EPILOG_NONE) ==
            GE_ERR_NOT_SUPPORTED,
        "a weight past the layout's tiles", 1 << 20);
}

}  // namespace

int main() {
  check_norm_stage();
  check_layout();
  check_choices();
  check_rules();
  std::printf("%s (%d failures)\n", failures ? "FAILED" : "ok", failures);
  return failures != 0;
}
