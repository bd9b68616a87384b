// Names the kernels that the host rules of the gated block and of 4-bit weights choose on 256 compute
// units, for 16-byte aligned operands: host code only, built by tests/test_gated_routes.py with g++.
// Reads lines of
//   forward m n k dt | down m d n dt | gradient m n d dt | product M N K dt lay |
//   w4 m n k group gated chunks
// (dt 0 f32, 1 f16, 2 bf16) and prints a name for each, and of
//   rows n gated | w4rows n gated tile
// and prints how many rows one launch takes, and of
//   sums m n k d dt
// and prints the rows of column sums that the kernels of dZ leave, and what the workspace has for them
// and for the sums of those, in rows.
#include <cstdio>
#include <cstring>

#include "gated_host.hpp"
#include "tiles.hpp"
#include "w4_host.hpp"

namespace {

constexpr int kCus = 256;

void tiles(const geh::Layout& L) {
  std::printf("%s%s%s\n", gek::kTiles[L.cfg].name, L.persist_grid ? " persistent" : "", L.sk_wgs ? " split" : "");
}

// The general kernel; lay 6: gated, of both halves.
void general(long M, long N, long K, ge_dtype_t dt, int lay, size_t ws) {
  if (gegh::general_narrow(M, N, K, dt, lay)) std::printf("general narrow");
  else std::printf(gegh::general_large(M, lay == 6 ? 2 * N : N, kCus) ? "general large" : "general small");
  const int parts = lay == 6 ? 1 : gegh::general_splits(M, N, K, dt, ws);
  if (parts > 1) std::printf(" %d parts", parts);
  std::printf("\n");
}

}  // namespace

int main() {
  char op[16];
  while (std::scanf("%15s", op) == 1) {
    geh::Layout L;
    long a, b, c, d, e, f;
    if (!std::strcmp(op, "w4")) {
      if (std::scanf("%ld %ld %ld %ld %ld %ld", &a, &b, &c, &d, &e, &f) != 6) return 1;
      const int cfg = gew4h::choose(a, b, c, d, e != 0, f != 0, kCus);
      if (cfg < 0) std::printf("few\n");
      else std::printf("%d x %d\n", gew4::kTiles[cfg].bm, gew4::kTiles[cfg].bn);
      continue;
    }
    if (!std::strcmp(op, "rows")) {
      if (std::scanf("%ld %ld", &a, &b) != 2) return 1;
      std::printf("%ld\n", (long)gegh::launch_rows(a, b != 0));
      continue;
    }
    if (!std::strcmp(op, "sums")) {
      if (std::scanf("%ld %ld %ld %ld %ld", &a, &b, &c, &d, &e) != 5) return 1;
      const gegh::BackwardSpace s = gegh::backward_space(a, b, c, d, (ge_dtype_t)e);
      long most = (long)gegh::dz_parts(a, b), used = most;
      for (int cus : {64, 256, 304})
        if (gegh::gradient_kernel(a, b, d, (ge_dtype_t)e, true) == gegh::Kernel::kTiles) {
          if (gegh::gated_layout(a, b, d, (ge_dtype_t)e, true, cus, &L) != GE_OK) return 1;
          const long rows = (long)L.tiles_m * (gek::kTiles[L.cfg].bm / gek::kTiles[L.cfg].wm), parts = (long)gegh::colsum_parts(rows, 2 * b);
          if (rows > most) most = rows;
          if (rows + (parts > 1 ? parts : 0) > used) used = rows + (parts > 1 ? parts : 0);
        }
      std::printf("%ld %ld %ld\n", most, used, (long)((s.total - s.scratch - geh::kSkFlagRegion) / (2 * b * 4)));
      continue;
    }
    if (!std::strcmp(op, "w4rows")) {
      if (std::scanf("%ld %ld %ld", &a, &b, &c) != 3) return 1;
      const gew4::W4TileCfg& T = gew4::kTiles[c];
      std::printf("%ld\n", (long)geh::rows_per_launch(T.bm, gew4::ceil_div(b ? 2 * a : a, T.bn), T.waves * 64));
      continue;
    }
    if (std::scanf("%ld %ld %ld %ld", &a, &b, &c, &d) != 4) return 1;
    const ge_dtype_t dt = (ge_dtype_t)d;
    const bool gated = !std::strcmp(op, "forward");
    if (gated || !std::strcmp(op, "down")) {
      const gegh::Kernel kernel = gegh::forward_kernel(a, b, c, dt, gated, true, kCus);
      if (kernel == gegh::Kernel::kFew) std::printf("few\n");
      else if (kernel == gegh::Kernel::kGeneral) general(a, b, c, dt, gated ? 6 : 2, 0);
      else if ((gated ? gegh::gated_layout(a, b, c, dt, false, kCus, &L) : gegh::fast_layout(a, b, c, dt, 2, kCus, 0, &L)) == GE_OK) tiles(L);
      else return 1;
    } else if (!std::strcmp(op, "gradient")) {
      if (gegh::gradient_kernel(a, b, c, dt, true) == gegh::Kernel::kGeneral) general(a, b, c, dt, 0, 0);
      else if (gegh::gated_layout(a, b, c, dt, true, kCus, &L) == GE_OK) tiles(L);
      else return 1;
    } else if (!std::strcmp(op, "product")) {
      if (std::scanf("%ld", &e) != 1) return 1;
      if (!gegh::fast_shape(a, b, c, dt, (int)e)) general(a, b, c, dt, (int)e, ~(size_t)0);
      else if (gegh::fast_layout(a, b, c, dt, (int)e, kCus, e ? 0 : ~(size_t)0, &L) == GE_OK) tiles(L);
      else return 1;
    } else {
      return 1;
    }
  }
  return 0;
}
