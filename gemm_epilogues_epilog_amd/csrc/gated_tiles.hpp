// The gated block's tile kernels (gated_tiles.hip) and its kernel for few tokens (gated_skinny.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "kernels.hpp"

namespace gek {
using LaunchFn = hipError_t (*)(const Args&, int grid, hipStream_t);
// cfg: as gegh::gated_layout chooses it.
LaunchFn get_launch_gated(int dt, bool backward, int cfg);

// X . W^T of few tokens (gated_skinny.hpp), any type and alignment. At most 65535 groups of 64 tokens.
hipError_t launch_skinny(int64_t m, int64_t n, int64_t k, int dt, bool gated, int act, const void* x, const void* w,
                         const void* bias, int vec, void* D, void* Z, int cus, hipStream_t s);
}  // namespace gek
