// The gated block's tile kernels (gated_tiles.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "kernels.hpp"

namespace gek {
using LaunchFn = hipError_t (*)(const Args&, int grid, hipStream_t);
// cfg: one of the configurations with kernels for transposed operands (cfg_has_layouts).
LaunchFn get_launch_gated(int dt, bool backward, int cfg);
}  // namespace gek
