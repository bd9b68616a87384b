// Instances of the direct-to-LDS kernels with the gated block's epilogues (gated_epilogue.hpp).
//   GATED   X (m, k) . W^T, W (2 n, k): both operands k-major. The 256 x 256 tile holds 128 columns
//           of H; its waves are 64 x 128, so that each has 64 columns of the gate and the same 64 of
//           the up projection and H leaves in whole cache lines.
//   DGATED  dY (m, d) . Wd, Wd (d, n): B as stored.
#include "gated_tiles.hpp"
#include "gemm_dtl.hpp"
#include "launch.hpp"

namespace gek {
namespace {

template <int DT, int EP, int LAY, int BM, int BN, int WM, int WN, int ST, bool ILV, int CW>
hipError_t tile(const Args& a, int grid, hipStream_t s) {
  Args copy = a;
  void* params[] = {&copy};
  const void* fn = reinterpret_cast<const void*>(&gemm_dtl_kernel<DT, EP, BM, BN, WM, WN, 64, ST, ILV, CW, LAY>);
  if constexpr (BN == 256) {
    if (a.persist_grid > 0) {
      fn = reinterpret_cast<const void*>(
          &gemm_persist_kernel<DT, EP, BM, BN, WM, WN, 64, ST, CW, persist_pre((WM / 32) * (WN / 32)), LAY>);
      grid = a.persist_grid;
    }
  }
  return hipLaunchKernel(fn, dim3(grid), dim3((BM / WM) * (BN / WN) * 64), params, 0, s);
}

template <int DT>
LaunchFn pick_gated(int cfg) {
  switch (cfg) {
    case CFG_LM: return &tile<DT, GATED, 6, 128, 128, 32, 64, 2, false, 0>;
    case CFG_LMD: return &tile<DT, GATED, 6, 128, 128, 32, 64, 3, false, 0>;
    default: return &tile<DT, GATED, 6, 256, 256, 64, 128, 2, false, 4>;
  }
}
template <int DT>
LaunchFn pick_dgated(int cfg) {
  switch (cfg) {
    case CFG_L3: return &tile<DT, DGATED, 0, 192, 256, 96, 64, 2, true, 4>;
    case CFG_LW: return &tile<DT, DGATED, 0, 128, 256, 64, 64, 2, true, 4>;
    case CFG_LM: return &tile<DT, DGATED, 0, 128, 128, 32, 64, 2, false, 0>;
    case CFG_LMD: return &tile<DT, DGATED, 0, 128, 128, 32, 64, 3, false, 0>;
    default: return &tile<DT, DGATED, 0, 256, 256, 128, 64, 2, true, 4>;
  }
}

}  // namespace

LaunchFn get_launch_gated(int dt, bool backward, int cfg) {
  if (backward) return dt == F16 ? pick_dgated<F16>(cfg) : pick_dgated<BF16>(cfg);
  return dt == F16 ? pick_gated<F16>(cfg) : pick_gated<BF16>(cfg);
}

}  // namespace gek
