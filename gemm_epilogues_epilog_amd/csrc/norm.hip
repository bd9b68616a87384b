// Residual addition and root-mean-square norm, and its gradient.
//
//   s = round(x + residual)        (s = x without a residual)
//   r = 1 / sqrt(mean(s^2) + eps)
//   y = s r w, in the inputs' type, as e4m3 with a scale per 32 values, or both
// The norm sees s as it is stored, so the backward pass, which has only the stored s, works
// with the same numbers. Sums in fp32.
//   dx = r (g - h mean(g h)) + dresidual, g = dy w, h = s r;   dw = sum over rows of dy h
// The 8-bit result passes the gradient straight through.
//
// Bound by memory: a row stays in registers between its sums and its result, so each
// value is read once and written once.
#include <hip/hip_runtime.h>

#include "gemm_epilog.h"
#include "kernels.hpp"
#include "launch.hpp"
#include "mx_format.hpp"
#include "mx_host.hpp"

namespace gek {
namespace {

using namespace gemx;

struct NormArgs {
  const void* x;
  const void* res;
  const void* w;
  void* sum;
  void* y;
  char* codes;
  char* scales;
  int64_t rows, ldx, ldr, lds, ldy;
  int d, wdt;
  float eps;
};

// Eight values from element i on; the ones from `n` on (of this chunk) read as zero.
template <int DT, bool VEC>
__device__ __forceinline__ void load_chunk(const void* p, int64_t i, int n, float (&v)[8]) {
  if constexpr (VEC) {
    if constexpr (DT == F32) {
      const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
      const f32x4 a = q[0], b = q[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = a[e];
        v[4 + e] = b[e];
      }
    } else {
      const i32x4 a = *reinterpret_cast<const i32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = Tr<DT>::widen((uint16_t)((uint32_t)a[e / 2] >> (16 * (e & 1))));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? load_vec(p, DT, i + e) : 0.0f;
  }
}
template <int DT, bool VEC>
__device__ __forceinline__ void store_chunk(void* p, int64_t i, int n, const float (&v)[8]) {
  if constexpr (VEC) {
    if constexpr (DT == F32) {
      f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
      q[0] = f32x4{v[0], v[1], v[2], v[3]};
      q[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      i32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = (int)Tr<DT>::pack2(v[2 * e], v[2 * e + 1]);
      *reinterpret_cast<i32x4*>(static_cast<uint16_t*>(p) + i) = o;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) store_vec(p, DT, i + e, v[e]);
  }
}
// Weight values: of the row type or fp32.
template <int DT, bool VEC>
__device__ __forceinline__ void load_weight(const void* p, int wdt, int i, int n, float (&v)[8]) {
  if (DT == F32 || wdt != F32) load_chunk<DT, VEC>(p, i, n, v);
  else load_chunk<F32, VEC>(p, i, n, v);
}
template <int DT>
__device__ __forceinline__ float round_to(float v) {
  if constexpr (DT == F16) return (float)(_Float16)v;
  else if constexpr (DT == BF16) return (float)(__bf16)v;
  else return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
// Sum over the NT lanes of a row (waves added in order, the same in each of them).
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* red, int t) {
  v = wave_sum(v);
  if constexpr (NT > 64) {
    if ((t & 63) == 0) red[t >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v += red[i];
  }
  return v;
}

// NT lanes per row, C chunks of eight values per lane, WG / NT rows per workgroup.
constexpr int wg_of(int nt) { return nt > 256 ? nt : 256; }

template <int DT, int NT, int C, bool VEC>
__global__ __launch_bounds__(wg_of(NT)) void rms_norm_kernel(NormArgs a) {
  constexpr int RPW = wg_of(NT) / NT;
  __shared__ float red[16];
  const int t = threadIdx.x % NT, slot = threadIdx.x / NT;
  // With an 8-bit result the workgroups of 32 consecutive rows run on one XCD: their
  // 16-byte chunks share cache lines, which its L2 then joins.
  int64_t row;
  if (a.codes) {
    constexpr int Q = 32 / RPW;
    const int64_t x = blockIdx.x & 7, l = blockIdx.x >> 3;
    row = ((l / Q) * 8 + x) * 32 + (l % Q) * RPW + slot;
  } else {
    row = (int64_t)blockIdx.x * RPW + slot;
  }
  const bool in = row < a.rows;
  if (NT > 64 && RPW == 1 && !in) return;   // the whole workgroup
  const int64_t rr = in ? row : 0;
  float s[C][8], w[C][8];
  float sq = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * NT + t) * 8, n = a.d - i;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[c][e] = w[c][e] = 0.0f;
    if (n > 0) {
      load_chunk<DT, VEC>(a.x, rr * a.ldx + i, n, s[c]);
      if (a.res) {
        float q[8];
        load_chunk<DT, VEC>(a.res, rr * a.ldr + i, n, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[c][e] = round_to<DT>(s[c][e] + q[e]);
      }
      load_weight<DT, VEC>(a.w, a.wdt, i, n, w[c]);
      if (a.sum && in) store_chunk<DT, VEC>(a.sum, rr * a.lds + i, n, s[c]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sq = __builtin_fmaf(s[c][e], s[c][e], sq);
  }
  static_assert(NT == 64 || RPW == 1 || NT * RPW == 256, "");
  const float r = rsqrtf(row_sum<NT>(sq, red + slot * (NT / 64), t) / (float)a.d + a.eps);
  const int64_t granules = (a.d + kKPad - 1) / kKPad;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * NT + t) * 8, n = a.d - i;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = s[c][e] * r * w[c][e];
    if (a.y && in && n > 0) store_chunk<DT, VEC>(a.y, rr * a.ldy + i, n, y);
    if (a.codes) {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = amax2(m, mag(y[e]));
      const int sc = scale_of(amax_quad(m), FP8);
      if (in && i < granules * kKPad) {
        const i32x2 q = {(int)to_fp8x4(y[0], y[1], y[2], y[3], sc), (int)to_fp8x4(y[4], y[5], y[6], y[7], sc)};
        *reinterpret_cast<i32x2*>(a.codes + ((row >> 5) * granules * 16 + i / 16) * 512 + (row & 31) * 16 + i % 16) = q;
        if ((t & 3) == 0)
          a.scales[((row >> 5) * granules + i / kKPad) * kScaleGranule + ((i / 32) & 1) * 128 + (row & 31) * 4 +
                   (i / 64) % 4] = (char)sc;
      }
    }
  }
}

struct NormBwdArgs {
  const void* dy;
  const void* s;
  const void* w;
  const void* dres;
  void* dx;
  float* partial;   // [slots][d]
  int64_t rows, lddy, lds, lddr, lddx, slots;
  int d, wdt;
  float eps;
};

// Each row slot walks the rows with the stride of all slots and keeps its share of dw in
// registers; launch_bgrad_reduce then adds the slots in order (no atomics).
template <int DT, int NT, int C, bool VEC>
__global__ __launch_bounds__(wg_of(NT)) void rms_norm_backward_kernel(NormBwdArgs a) {
  constexpr int RPW = wg_of(NT) / NT, NWV = NT / 64;
  __shared__ float red[2][2][16];
  const int t = threadIdx.x % NT, slot = threadIdx.x / NT;
  const int64_t first = (int64_t)blockIdx.x * RPW + slot;
  float w[C][8], dw[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * NT + t) * 8, n = a.d - i;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[c][e] = dw[c][e] = 0.0f;
    if (n > 0) load_weight<DT, VEC>(a.w, a.wdt, i, n, w[c]);
  }
  // every slot of a workgroup takes the same number of steps (they share barriers)
  int par = 0;
  for (int64_t base = (int64_t)blockIdx.x * RPW; base < a.rows; base += a.slots, par ^= 1) {
    const int64_t row = base + slot;
    const bool in = row < a.rows;
    const int64_t rr = in ? row : 0;
    float s[C][8], g[C][8];
    float sq = 0.0f, dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * NT + t) * 8, n = a.d - i;
#pragma unroll
      for (int e = 0; e < 8; ++e) s[c][e] = g[c][e] = 0.0f;
      if (n > 0) {
        load_chunk<DT, VEC>(a.s, rr * a.lds + i, n, s[c]);
        load_chunk<DT, VEC>(a.dy, rr * a.lddy + i, n, g[c]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sq = __builtin_fmaf(s[c][e], s[c][e], sq);
        dot = __builtin_fmaf(g[c][e] * w[c][e], s[c][e], dot);
      }
    }
    sq = wave_sum(sq);
    dot = wave_sum(dot);
    if constexpr (NT > 64) {
      // two sets of words in turn, so that one barrier a row is enough
      if ((t & 63) == 0) {
        red[par][0][t >> 6] = sq;
        red[par][1][t >> 6] = dot;
      }
      __syncthreads();
      sq = dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NWV; ++i) {
        sq += red[par][0][i];
        dot += red[par][1][i];
      }
    }
    const float r = rsqrtf(sq / (float)a.d + a.eps);
    const float k = r * r * (dot / (float)a.d);   // h mean(g h) = s k
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * NT + t) * 8, n = a.d - i;
      if (n > 0 && in) {
        float o[8], q[8];
        if (a.dres) load_chunk<DT, VEC>(a.dres, rr * a.lddr + i, n, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[e] = r * (g[c][e] * w[c][e] - s[c][e] * k);
          if (a.dres) o[e] += q[e];
          dw[c][e] = __builtin_fmaf(g[c][e], s[c][e] * r, dw[c][e]);
        }
        store_chunk<DT, VEC>(a.dx, rr * a.lddx + i, n, o);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * NT + t) * 8, n = a.d - i;
    if (n > 0 && first < a.slots) {
      float* p = a.partial + first * a.d + i;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) p[e] = dw[c][e];
    }
  }
}

template <int DT, bool VEC>
const void* norm_fn(int d, int* nt) {
  auto pick = [&](int n, const void* f) {
    *nt = n;
    return f;
  };
#define GE_NORM(N, C) return pick(N, reinterpret_cast<const void*>(&rms_norm_kernel<DT, N, C, VEC>))
  if (d <= 512) GE_NORM(64, 1);
  if (d <= 1024) GE_NORM(64, 2);
  if (d <= 4096) GE_NORM(256, 2);
  if (d <= 8192) GE_NORM(512, 2);
  if (d <= 16384) GE_NORM(1024, 2);
  GE_NORM(1024, 4);
#undef GE_NORM
}
template <int DT, bool VEC>
const void* norm_bwd_fn(int d, int* nt) {
  auto pick = [&](int n, const void* f) {
    *nt = n;
    return f;
  };
#define GE_NORM(N, C) return pick(N, reinterpret_cast<const void*>(&rms_norm_backward_kernel<DT, N, C, VEC>))
  if (d <= 512) GE_NORM(64, 1);
  if (d <= 1024) GE_NORM(64, 2);
  if (d <= 4096) GE_NORM(256, 2);
  if (d <= 8192) GE_NORM(512, 2);
  if (d <= 16384) GE_NORM(1024, 2);
  GE_NORM(1024, 4);
#undef GE_NORM
}

bool lines(const void* p, int64_t ld, size_t e) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)e % 16 == 0;
}

}  // namespace
}  // namespace gek

extern "C" {

ge_status_t gemm_epilog_rms_norm(int64_t rows, int64_t d, ge_dtype_t dt, const void* x, int64_t ldx,
                                 const void* residual, int64_t ldr, const void* weight, ge_dtype_t wdt, float eps,
                                 void* sum, int64_t lds, void* y, int64_t ldy, void* codes, void* scales,
                                 void* stream) {
  if (ge_status_t st = gemxh::check_norm(rows, d, dt, x, ldx, residual, ldr, weight, wdt, eps, sum, lds, y, ldy, codes,
                                         scales);
      st != GE_OK)
    return st;
  if (rows == 0) return GE_OK;
  gek::NormArgs a{x,   residual, weight, sum, y,   static_cast<char*>(codes), static_cast<char*>(scales), rows, ldx,
                  ldr, lds,      ldy,    (int)d, (int)wdt, eps};
  const size_t e = gemxh::esize(dt);
  const bool vec = d % 8 == 0 && gek::lines(x, ldx, e) && gek::lines(residual, residual ? ldr : 0, e) &&
                   gek::lines(sum, sum ? lds : 0, e) && gek::lines(y, y ? ldy : 0, e) && gek::lines(weight, 0, e);
  int nt = 0;
  const void* fn = dt == GE_F32   ? (vec ? gek::norm_fn<gek::F32, true>(a.d, &nt) : gek::norm_fn<gek::F32, false>(a.d, &nt))
                   : dt == GE_F16 ? (vec ? gek::norm_fn<gek::F16, true>(a.d, &nt) : gek::norm_fn<gek::F16, false>(a.d, &nt))
                                  : (vec ? gek::norm_fn<gek::BF16, true>(a.d, &nt)
                                         : gek::norm_fn<gek::BF16, false>(a.d, &nt));
  const int wg = gek::wg_of(nt), rpw = wg / nt;
  int64_t grid = (rows + rpw - 1) / rpw;
  if (codes) grid = (gemx::row_groups(rows) + 7) / 8 * 8 * (32 / rpw);
  if (grid * wg >= (int64_t(1) << 32)) return GE_ERR_NOT_SUPPORTED;
  void* params[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3((unsigned)wg), params, 0, static_cast<hipStream_t>(stream)) ==
                 hipSuccess
             ? GE_OK
             : GE_ERR_HIP;
}

size_t gemm_epilog_rms_norm_workspace_bytes(int64_t rows, int64_t d) { return gemxh::norm_workspace_bytes(rows, d); }

ge_status_t gemm_epilog_rms_norm_backward(int64_t rows, int64_t d, ge_dtype_t dt, const void* dy, int64_t lddy,
                                          const void* s, int64_t lds, const void* weight, ge_dtype_t wdt, float eps,
                                          const void* dresidual, int64_t lddr, void* dx, int64_t lddx, void* dw,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  if (ge_status_t st = gemxh::check_norm_backward(rows, d, dt, dy, lddy, s, lds, weight, wdt, eps, dresidual, lddr, dx,
                                                  lddx, dw, workspace, workspace_bytes);
      st != GE_OK)
    return st;
  hipStream_t q = static_cast<hipStream_t>(stream);
  int64_t slots = 0;
  if (rows) {
    slots = gemxh::norm_backward_groups(rows, d);
    gek::NormBwdArgs a{dy,   s,    weight, dresidual, dx,    static_cast<float*>(workspace), rows, lddy, lds,
                       lddr, lddx, slots,  (int)d,    (int)wdt, eps};
    const size_t e = gemxh::esize(dt);
    const bool vec = d % 8 == 0 && gek::lines(dy, lddy, e) && gek::lines(s, lds, e) &&
                     gek::lines(dresidual, dresidual ? lddr : 0, e) && gek::lines(dx, lddx, e) &&
                     gek::lines(weight, 0, e);
    int nt = 0;
    const void* fn =
        dt == GE_F32 ? (vec ? gek::norm_bwd_fn<gek::F32, true>(a.d, &nt) : gek::norm_bwd_fn<gek::F32, false>(a.d, &nt))
        : dt == GE_F16
            ? (vec ? gek::norm_bwd_fn<gek::F16, true>(a.d, &nt) : gek::norm_bwd_fn<gek::F16, false>(a.d, &nt))
            : (vec ? gek::norm_bwd_fn<gek::BF16, true>(a.d, &nt) : gek::norm_bwd_fn<gek::BF16, false>(a.d, &nt));
    const int wg = gek::wg_of(nt), rpw = wg / nt;
    void* params[] = {&a};
    if (hipLaunchKernel(fn, dim3((unsigned)((slots + rpw - 1) / rpw)), dim3((unsigned)wg), params, 0, q) != hipSuccess)
      return GE_ERR_HIP;
  }
  return gek::launch_bgrad_reduce(static_cast<float*>(workspace), (int)slots, d, dw, (int)wdt, q) == hipSuccess
             ? GE_OK
             : GE_ERR_HIP;
}

}  // extern "C"
