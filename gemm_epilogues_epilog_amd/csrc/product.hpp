// The library's 16-bit product without an epilogue, for operators that plan per call.
#pragma once

#include <hip/hip_runtime.h>

#include "plan_host.hpp"

namespace gei {

// The current device's compute units; GE_ERR_NOT_SUPPORTED if it is not a gfx950. Asked of the
// driver once per device.
ge_status_t current_device(int* cus);

// D (m, n) = A . B of dense 16-bit operands in the storage orders of L, by the kernels of a plan
// with that layout. `ws`: L.ws_bytes of workspace, its flags cleared here unless they are already.
ge_status_t run_product(int64_t m, int n, int k, ge_dtype_t dt, const geh::Layout& L, const void* A, const void* B,
                        void* D, char* ws, bool cleared, hipStream_t s);

}  // namespace gei

namespace gek {
// out[i] = sum over t of partial[t][i], in a fixed order (defined in api.hip).
hipError_t launch_bgrad_reduce(const float* partial, int t, int64_t m, void* bgrad, int vec_dt, hipStream_t s);
}  // namespace gek
