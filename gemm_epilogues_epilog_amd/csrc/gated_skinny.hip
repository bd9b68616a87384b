// Launches of the gated block's kernel for few tokens.
#include "gated_skinny.hpp"

#include "gated_tiles.hpp"

namespace gek {
namespace {

template <int DT, bool GATED, bool VEC>
const void* of(int mt) {
  return mt == 1   ? reinterpret_cast<const void*>(&skinny_kernel<DT, GATED, 1, VEC>)
         : mt == 2 ? reinterpret_cast<const void*>(&skinny_kernel<DT, GATED, 2, VEC>)
                   : reinterpret_cast<const void*>(&skinny_kernel<DT, GATED, 4, VEC>);
}
template <int DT>
const void* of(bool gated, bool vec, int mt) {
  if (gated) return vec ? of<DT, true, true>(mt) : of<DT, true, false>(mt);
  return vec ? of<DT, false, true>(mt) : of<DT, false, false>(mt);
}

}  // namespace

hipError_t launch_skinny(int64_t m, int64_t n, int64_t k, int dt, bool gated, int act, const void* x, const void* w,
                         const void* bias, int vec, void* D, void* Z, int cus, hipStream_t s) {
  SkinnyArgs a;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.D = D;
  a.Z = Z;
  a.m = m;
  a.n = n;
  a.k = (int32_t)k;
  a.vec = vec;
  a.act = act;
  const int es = dt == F32 ? 4 : 2;
  const bool chunks = k * es % 16 == 0 && (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w)) % 16 == 0;
  const int mt = m <= 16 ? 1 : m <= 32 ? 2 : 4;
  const void* fn = dt == F32 ? of<F32>(gated, chunks, mt) : dt == F16 ? of<F16>(gated, chunks, mt) : of<BF16>(gated, chunks, mt);
  const dim3 grid((unsigned)((n + 15) / 16), (unsigned)((m + 16 * mt - 1) / (16 * mt)));
  // Waves of a workgroup: eight, or four where eight would not all be on the device at once
  const int nw = (int64_t)grid.x * grid.y * 8 > (int64_t)cus * (mt == 4 ? 8 : 16) ? 4 : 8;
  void* params[] = {&a};
  return hipLaunchKernel(fn, grid, dim3(nw * 64), params, (size_t)nw * (gated ? 2 : 1) * mt * 1024, s);
}

}  // namespace gek
