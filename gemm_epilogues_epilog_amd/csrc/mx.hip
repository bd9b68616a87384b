// The microscaled product's plan, execute and free (kernels: mx_gemm.hpp, rules:
// mx_host.cpp).
#include <hip/hip_runtime.h>

#include <cstring>
#include <new>

#include "gemm_epilog.h"
#include "mx_gemm.hpp"
#include "mx_host.hpp"

struct ge_mx_plan {
  int64_t n, k, experts;
  ge_mx_types_t t;
  ge_epilog_t ep;
  int cus;
  void* ws;
  size_t ws_bytes;
};

namespace {

template <int XF, bool EXACT>
const void* kernel_of(int cfg) {
  using namespace gek;
  switch (cfg) {
    case MX_L: return reinterpret_cast<const void*>(&mx_tile_kernel<XF, MX_L, EXACT>);
    case MX_R256: return reinterpret_cast<const void*>(&mx_ring_kernel<XF, MX_R256, EXACT>);
    case MX_R128W: return reinterpret_cast<const void*>(&mx_ring_kernel<XF, MX_R128W, EXACT>);
    case MX_R128: return reinterpret_cast<const void*>(&mx_ring_kernel<XF, MX_R128, EXACT>);
    case MX_R64: return reinterpret_cast<const void*>(&mx_ring_kernel<XF, MX_R64, EXACT>);
    case MX_S16: return reinterpret_cast<const void*>(&mx_skinny_kernel<XF, 2>);
    case MX_S16N: return reinterpret_cast<const void*>(&mx_skinny_kernel<XF, 1>);
  }
  return nullptr;
}

// Zeroes the counters, on a stream of its own, and waits.
hipError_t clear_counters(void* p) {
  hipStream_t s = nullptr;
  hipError_t e = hipStreamCreateWithFlags(&s, hipStreamNonBlocking);
  if (e != hipSuccess) return e;
  e = hipMemsetAsync(p, 0, gemx::kMxCounterBytes, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  const hipError_t d = hipStreamDestroy(s);
  return e != hipSuccess ? e : d;
}

}  // namespace

extern "C" {

ge_status_t gemm_epilog_mx_plan(int64_t n, int64_t k, int64_t experts, ge_mx_types_t types, ge_epilog_t ep,
                                ge_mx_handle_t* out) {
  if (!out) return GE_ERR_NULL_POINTER;
  if (ge_status_t st = gemxh::check_plan(n, k, experts, types, ep); st != GE_OK) return st;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return GE_ERR_HIP;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GE_ERR_HIP;
  if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) return GE_ERR_NOT_SUPPORTED;
  ge_mx_plan* h = new (std::nothrow) ge_mx_plan();
  if (!h) return GE_ERR_ALLOC;
  h->n = n;
  h->k = k;
  h->experts = experts;
  h->t = types;
  h->ep = ep;
  h->cus = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 256;
  h->ws_bytes = gemxh::workspace_bytes(experts, h->cus);
  if (h->ws_bytes) {
    if (hipMalloc(&h->ws, h->ws_bytes) != hipSuccess) {
      delete h;
      return GE_ERR_ALLOC;
    }
    if (clear_counters(h->ws) != hipSuccess) {
      hipFree(h->ws);
      delete h;
      return GE_ERR_HIP;
    }
  }
  *out = h;
  return GE_OK;
}

ge_status_t gemm_epilog_mx_plan_info(int64_t n, int64_t k, int64_t experts, ge_mx_types_t types, ge_epilog_t ep,
                                     int64_t m, int compute_units, ge_mx_plan_info_t* info) {
  if (!info) return GE_ERR_NULL_POINTER;
  if (ge_status_t st = gemxh::check_plan(n, k, experts, types, ep); st != GE_OK) return st;
  if (m < 0 || m > 0x7fffffff || compute_units < 1 || compute_units > 4096) return GE_ERR_INVALID_VALUE;
  const gemxh::MxLaunch L = gemxh::choose(m, n, k, experts, types, compute_units);
  const gemx::MxTile& T = gemx::kMxTiles[L.cfg];
  info->tile_m = T.bm;
  info->tile_n = T.bn;
  info->waves = L.waves;
  info->stages = T.stages;
  info->splits = L.splits;
  info->tiles = m ? (int64_t)L.tiles_m * L.tiles_n : 0;
  info->workgroups = m ? L.grid_x * L.grid_y * L.grid_z : 0;
  info->workspace_bytes = gemxh::workspace_bytes(experts, compute_units);
  return GE_OK;
}

ge_status_t gemm_epilog_mx_execute(ge_mx_handle_t h, int64_t m, const void* x_codes, const void* x_scales,
                                   const void* w_codes, const void* w_scales, const void* bias, const void* offsets,
                                   void* D, void* d_scales, void* stream) {
  if (!h) return GE_ERR_NULL_POINTER;
  if (ge_status_t st = gemxh::check_execute(m, h->experts, h->t, h->ep, x_codes, x_scales, w_codes, w_scales, bias,
                                            offsets, D, d_scales);
      st != GE_OK)
    return st;
  if (m == 0) return GE_OK;
  const gemxh::MxLaunch L = gemxh::choose(m, h->n, h->k, h->experts, h->t, h->cus);
  gek::MxArgs a;
  a.xc = static_cast<const char*>(x_codes);
  a.xs = static_cast<const char*>(x_scales);
  a.wc = static_cast<const char*>(w_codes);
  a.ws = static_cast<const char*>(w_scales);
  a.bias = bias;
  a.offsets = h->experts ? static_cast<const int32_t*>(offsets) : nullptr;
  a.D = D;
  a.ds = static_cast<char*>(d_scales);
  a.counter = static_cast<uint32_t*>(h->ws);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(h->ws) + gemx::kMxCounterBytes);
  a.m = m;
  a.n = (int32_t)h->n;
  a.k = (int32_t)h->k;
  a.kt = (int32_t)(gemx::pad_to(h->k, gemx::kKPad) / gemx::kKPad);
  a.experts = (int32_t)h->experts;
  a.tiles_m = L.tiles_m;
  a.tiles_n = L.tiles_n;
  a.splits = L.splits;
  a.ep = (int32_t)h->ep;
  a.out = (int32_t)h->t.d;
  a.vec = (int32_t)h->t.vec;
  // a launch keeps its lane count below 2^32
  if (L.grid_x * L.grid_y * L.grid_z * L.waves * 64 >= (int64_t(1) << 32) || L.grid_y > 65535)
    return GE_ERR_NOT_SUPPORTED;
  const bool exact = h->t.d == GE_MX_D_F32 || h->t.d == GE_MX_D_MXFP8;   // see large_part (the skinny kernel always is)
  const auto launch = [&](int cfg, dim3 grid, int waves) {
    const void* fn = h->t.x == GE_MXFP4 ? kernel_of<gemx::FP4, false>(cfg)
                     : exact            ? kernel_of<gemx::FP8, true>(cfg)
                                        : kernel_of<gemx::FP8, false>(cfg);
    void* params[] = {&a};
    return hipLaunchKernel(fn, grid, dim3((unsigned)waves * 64), params, 0, static_cast<hipStream_t>(stream)) ==
           hipSuccess;
  };
  a.round = L.tail ? (int32_t)L.grid_x : 0;
  a.tail = 0;
  if (!launch(L.cfg, dim3((unsigned)L.grid_x, (unsigned)L.grid_y, (unsigned)L.grid_z), L.waves)) return GE_ERR_HIP;
  if (!L.tail) return GE_OK;
  a.tail = 1;
  return launch(gemx::kMxTailCfg, dim3((unsigned)(a.round / 4 * 4)), gemx::mx_waves(gemx::kMxTiles[gemx::kMxTailCfg]))
             ? GE_OK
             : GE_ERR_HIP;
}

ge_status_t gemm_epilog_mx_free(ge_mx_handle_t h) {
  if (!h) return GE_OK;
  ge_status_t st = GE_OK;
  if (h->ws && hipFree(h->ws) != hipSuccess) st = GE_ERR_HIP;
  delete h;
  return st;
}

}  // extern "C"
