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
// Bound by memory: a row stays in registers between its sums and its result, so each value is
// read once and written once. That holds up to 8192 values (the gradient of fp32 rows at any
// alignment spills 56 bytes a lane from 4096 on). Longer rows take 1024 lanes of 128 registers:
// with 16-byte aligned rows the forward still spills nothing, the gradient 148 to 244 bytes a lane
// from 16384 values on; at any other alignment the forward spills 36 to 156 bytes up to 16384 values
// and 276 to 708 above, the gradient 296 to 416 and 1040 to 1160. 4096 rows of bf16 with a residual, to
// bf16 and the gradient: 16384 values 109 and 116 us (4.9 and 4.7 TB/s), 16383 174 and 418, 32768
// 213 and 400, 32767 756 and 1789.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gemm_epilog.h"
#include "kernels.hpp"
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
  int walk;   // rows per slot
};

// Eight values from element i on as they lie in memory, and widened; the ones from `n` on
// (of this chunk; n at least 1) read as zero. VEC: 16-byte loads, n at least 8. Otherwise the
// same loads at the elements' alignment, which the memory pipe takes, and only a row's last
// chunk element by element, with no branch between those, so that they wait once (element
// by element with a branch each, 8192 x 8191 bf16 with a residual took 331 us, now 150, its
// gradient 346, now 173).
template <int DT, bool VEC>
struct Chunk {
  static constexpr int W = DT == F32 ? 2 : 1;
  i32x4 raw[W];
  __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
    const char* q = static_cast<const char*>(p) + i * (DT == F32 ? 4 : 2);
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < W; ++j) raw[j] = reinterpret_cast<const i32x4*>(q)[j];
    } else {
      if (n >= 8) {
        __builtin_memcpy(raw, q, sizeof(raw));
      } else {
        using U = std::conditional_t<DT == F32, uint32_t, uint16_t>;
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = reinterpret_cast<const U*>(q)[min(e, n - 1)];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? v[e] : 0u;
        if constexpr (DT == F32) {
          __builtin_memcpy(raw, v, sizeof(raw));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) raw[0][e] = (int)(v[2 * e] | v[2 * e + 1] << 16);
        }
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < W; ++j) raw[j] = i32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (DT == F32) return __int_as_float(raw[e / 4][e % 4]);
    else return Tr<DT>::widen((uint16_t)((uint32_t)raw[0][e / 2] >> (16 * (e & 1))));
  }
};
template <int DT, bool VEC>
__device__ __forceinline__ void store_chunk(void* p, int64_t i, int n, const float (&v)[8]) {
  if (VEC || n >= 8) {
    char* q = static_cast<char*>(p) + i * (DT == F32 ? 4 : 2);
    if constexpr (DT == F32) {
      if constexpr (VEC) q = static_cast<char*>(__builtin_assume_aligned(q, 16));
      __builtin_memcpy(q, v, 32);
    } else {
      i32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = (int)Tr<DT>::pack2(v[2 * e], v[2 * e + 1]);
      if constexpr (VEC) *reinterpret_cast<i32x4*>(q) = o;
      else __builtin_memcpy(q, &o, 16);
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
  if (DT == F32 || wdt != F32) {
    Chunk<DT, VEC> c;
    c.load(p, i, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c.get(e);
  } else {
    Chunk<F32, VEC> c;
    c.load(p, i, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c.get(e);
  }
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
// NT lanes per row, C chunks of eight values per lane, WG / NT rows side by side in a
// workgroup and a.walk rows one after the other per row slot: the weight is read once per
// slot, and the next row's loads are in flight while this one is summed and written.
// 16384 x 8192 bf16 with a residual: 189 us to MXFP8 (943 MB, 5.0 TB/s), 210 to bf16 (5.1),
// without a residual 104; 4096 x 4096 21 us (6.3 TB/s, the 256 MB cache helps).
constexpr int wg_of(int nt) { return nt > 64 ? nt : 256; }

template <int DT, int NT, int C, bool VEC>
__global__ __launch_bounds__(wg_of(NT)) void rms_norm_kernel(NormArgs a) {
  constexpr int RPW = wg_of(NT) / NT, NWV = NT / 64;
  static_assert(NT == 64 || RPW == 1, "rows that share a workgroup share no barrier");
  constexpr bool HOLD = NT * C <= 1024;   // registers for the next row and the weight (up to 8192 values)
  __shared__ float red[2][16];
  const int t = threadIdx.x % NT, slot = threadIdx.x / NT;
  int64_t row = ((int64_t)blockIdx.x * RPW + slot) * a.walk;
  const int64_t end = min(row + a.walk, a.rows);
  if (row >= end) return;   // the whole workgroup, or a wave that meets no barrier
  // An 8-bit result's rows are gathered in LDS: their 16-byte chunks lie 512 bytes apart in
  // memory, but those of neighbouring rows are neighbours, so a slot's rows leave together in
  // runs of 16 walk bytes (stored row by row the lines left the L2 half filled:
  // 16384 x 8192 took 206 to 320 us). Chunk c of the slot's row j is at (c (walk + 1) + j) 16
  // (the odd stride spreads the banks), scales of granule half g at (g walk + j) 4 after them.
  const int granules = (a.d + kKPad - 1) / kKPad, chunks = granules * 16;
  const int64_t row0 = row;
  extern __shared__ __attribute__((aligned(16))) char stage_all[];
  char* stage = stage_all + slot * gemxh::norm_stage_bytes(granules, a.walk);
  char* stage_s = stage + chunks * (a.walk + 1) * 16;
  Chunk<DT, VEC> x[C], res[C];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * NT + t) * 8, n = a.d - i;
      x[c].zero();
      res[c].zero();
      if (n > 0) {
        x[c].load(a.x, r * a.ldx + i, n);
        if (a.res) res[c].load(a.res, r * a.ldr + i, n);
      }
    }
  };
  float w[HOLD ? C : 1][8];
  auto weight = [&](int c, float (&v)[8]) {
    const int i = (c * NT + t) * 8, n = a.d - i;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    if (n > 0) load_weight<DT, VEC>(a.w, a.wdt, i, n, v);
  };
  if constexpr (HOLD) {
    load(row);
#pragma unroll
    for (int c = 0; c < C; ++c) weight(c, w[c]);
  }
  for (int par = 0; row < end; ++row, par ^= 1) {
    if constexpr (!HOLD) load(row);
    float s[C][8];
    float sq = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[c][e] = a.res ? round_to<DT>(x[c].get(e) + res[c].get(e)) : x[c].get(e);
        sq = __builtin_fmaf(s[c][e], s[c][e], sq);
      }
    if constexpr (HOLD) {
      if (row + 1 < end) load(row + 1);
    }
    if (a.sum) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = (c * NT + t) * 8, n = a.d - i;
        if (n > 0) store_chunk<DT, VEC>(a.sum, row * a.lds + i, n, s[c]);
      }
    }
    sq = wave_sum(sq);
    if constexpr (NT > 64) {
      // two sets of words in turn, so that one barrier a row is enough
      if ((t & 63) == 0) red[par][t >> 6] = sq;
      __syncthreads();
      sq = 0.0f;
#pragma unroll
      for (int i = 0; i < NWV; ++i) sq += red[par][i];
    }
    const float r = rsqrtf(sq / (float)a.d + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * NT + t) * 8, n = a.d - i;
      float y[8];
      if constexpr (!HOLD) weight(c, w[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = s[c][e] * r * w[HOLD ? c : 0][e];
      if (a.y && n > 0) store_chunk<DT, VEC>(a.y, row * a.ldy + i, n, y);
      if (a.codes) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = amax2(m, mag(y[e]));
        const int sc = scale_of(amax_quad(m), FP8);
        if (i < granules * kKPad) {
          const int j = (int)(row - row0);
          const i32x2 q = {(int)to_fp8x4(y[0], y[1], y[2], y[3], sc), (int)to_fp8x4(y[4], y[5], y[6], y[7], sc)};
          *reinterpret_cast<i32x2*>(stage + (i / 16 * (a.walk + 1) + j) * 16 + i % 16) = q;
          if ((t & 3) == 0) stage_s[((i / kKPad * 2 + ((i / 32) & 1)) * a.walk + j) * 4 + (i / 64) % 4] = (char)sc;
        }
      }
    }
  }
  if (a.codes) {
    if constexpr (NT > 64) __syncthreads();
    else __builtin_amdgcn_wave_barrier();
    const int rows = (int)(end - row0);
    char* dc = a.codes + (row0 >> 5) * chunks * 512 + (row0 & 31) * 16;
    for (int k = t; k < chunks * a.walk; k += NT) {
      const int c = k / a.walk, j = k % a.walk;
      if (j < rows)
        *reinterpret_cast<i32x4*>(dc + c * 512 + j * 16) =
            *reinterpret_cast<const i32x4*>(stage + (c * (a.walk + 1) + j) * 16);
    }
    char* ds = a.scales + (row0 >> 5) * granules * kScaleGranule + (row0 & 31) * 4;
    for (int k = t; k < granules * 2 * a.walk; k += NT) {
      const int g = k / a.walk, j = k % a.walk;
      if (j < rows) *reinterpret_cast<int*>(ds + g * 128 + j * 4) = *reinterpret_cast<const int*>(stage_s + k * 4);
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

// Each row slot walks the rows with the stride of all slots, the next row's loads in flight
// while this one is summed, and keeps its share of dw in registers; norm_dweight_kernel then
// adds the workgroups' sums in order (no atomics). With the gradient past
// the norm 8192 x 8192 bf16 takes 98 us (546 MB, 5.6 TB/s) and the second pass 4.6, 16384 x 8192
// 196 together (5.5 TB/s). More registers per lane (two chunks of the next row) spilled.
template <int DT, int NT, int C, bool VEC>
__global__ __launch_bounds__(wg_of(NT)) void rms_norm_backward_kernel(NormBwdArgs a) {
  constexpr int RPW = wg_of(NT) / NT, NWV = NT / 64;
  static_assert(NT == 64 || RPW == 1, "rows that share a workgroup share no barrier");
  constexpr bool HOLD = NT * C <= 1024;   // registers for the next row and the weight (up to 8192 values)
  __shared__ float red[2][2][16];
  const int t = threadIdx.x % NT, slot = threadIdx.x / NT;
  const int64_t first = (int64_t)blockIdx.x * RPW + slot;
  const bool active = first < a.slots;   // the last workgroup may have slots too many
  Chunk<DT, VEC> sc[C], gc[C], rc[C];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * NT + t) * 8, n = a.d - i;
      sc[c].zero();
      gc[c].zero();
      rc[c].zero();
      if (n > 0) {
        sc[c].load(a.s, r * a.lds + i, n);
        gc[c].load(a.dy, r * a.lddy + i, n);
        if (a.dres) rc[c].load(a.dres, r * a.lddr + i, n);
      }
    }
  };
  float w[HOLD ? C : 1][8], dw[C][8];
  auto weight = [&](int c, float (&v)[8]) {
    const int i = (c * NT + t) * 8, n = a.d - i;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    if (n > 0) load_weight<DT, VEC>(a.w, a.wdt, i, n, v);
  };
  if constexpr (HOLD) load(active ? first : 0);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (HOLD) weight(c, w[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[c][e] = 0.0f;
  }
  int par = 0;
  for (int64_t row = active ? first : a.rows; row < a.rows; row += a.slots, par ^= 1) {
    if constexpr (!HOLD) load(row);
    // this row's values move out of the way of the next row's
    Chunk<DT, VEC> s[C], g[C], o[C];
    float sq = 0.0f, dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s[c] = sc[c];
      g[c] = gc[c];
      o[c] = rc[c];
      if constexpr (!HOLD) weight(c, w[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sq = __builtin_fmaf(s[c].get(e), s[c].get(e), sq);
        dot = __builtin_fmaf(g[c].get(e) * w[HOLD ? c : 0][e], s[c].get(e), dot);
      }
    }
    if constexpr (HOLD) {
      if (row + a.slots < a.rows) load(row + a.slots);
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
      if (n > 0) {
        if constexpr (!HOLD) weight(c, w[0]);
        float dx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dx[e] = o[c].get(e) + r * (g[c].get(e) * w[HOLD ? c : 0][e] - s[c].get(e) * k);
          dw[c][e] = __builtin_fmaf(g[c].get(e), s[c].get(e) * r, dw[c][e]);
        }
        store_chunk<DT, VEC>(a.dx, row * a.lddx + i, n, dx);
      }
    }
  }
  // one row of sums per workgroup: the slots' sums are added in their order (a row per slot
  // left the second pass four times the work: 2272 x 148 f32 12.2 us, now 8.8)
  if constexpr (RPW > 1) {
    static_assert(C == 1, "a slot's row of sums");
    __shared__ float sums[RPW][NT * 8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[slot][t * 8 + e] = dw[0][e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += RPW * NT) {
      float v = sums[0][i];
#pragma unroll
      for (int q = 1; q < RPW; ++q) v += sums[q][i];
      a.partial[(int64_t)blockIdx.x * a.d + i] = v;
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * NT + t) * 8, n = a.d - i;
      if (n > 0) store_chunk<F32, VEC>(a.partial, first * a.d + i, n, dw[c]);   // VEC: d is a multiple of 8
    }
  }
}

// dw[i] = sum over t of partial[t][i]: 16 waves take 64 columns, each a run of the slots with
// 16 loads in flight, and their sums are added in wave order. (The bias gradient's second
// pass has four waves for this; here the columns are few and the slots many: 512 x 8192
// took 9.3 us with it.)
constexpr int kDwWaves = 16, kDwBatch = 16;
__global__ __launch_bounds__(64 * kDwWaves) void norm_dweight_kernel(const float* __restrict__ partial, int T, int d,
                                                                     void* dw, int wdt) {
  __shared__ float sums[kDwWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int i = blockIdx.x * 64 + lane;
  const int t0 = (int)((int64_t)T * w / kDwWaves), t1 = (int)((int64_t)T * (w + 1) / kDwWaves);
  float s = 0.0f;
  if (i < d) {
    for (int t = t0; t < t1; t += kDwBatch) {
      float v[kDwBatch];
#pragma unroll
      for (int j = 0; j < kDwBatch; ++j) v[j] = t + j < t1 ? partial[(int64_t)(t + j) * d + i] : 0.0f;
#pragma unroll
      for (int j = 0; j < kDwBatch; ++j) s += v[j];
    }
  }
  sums[w][lane] = s;
  __syncthreads();
  if (w == 0 && i < d) {
    float r = sums[0][lane];
#pragma unroll
    for (int q = 1; q < kDwWaves; ++q) r += sums[q][lane];
    store_vec(dw, wdt, i, r);
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
  if (d <= 1024) GE_NORM(128, 1);
  if (d <= 2048) GE_NORM(256, 1);
  if (d <= 4096) GE_NORM(512, 1);
  if (d <= 8192) GE_NORM(1024, 1);
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
                  ldr, lds,      ldy,    (int)d, (int)wdt, eps, 1};
  const size_t e = gemxh::esize(dt);
  const bool vec = d % 8 == 0 && gek::lines(x, ldx, e) && gek::lines(residual, residual ? ldr : 0, e) &&
                   gek::lines(sum, sum ? lds : 0, e) && gek::lines(y, y ? ldy : 0, e) && gek::lines(weight, 0, e);
  int nt = 0;
  const void* fn = dt == GE_F32   ? (vec ? gek::norm_fn<gek::F32, true>(a.d, &nt) : gek::norm_fn<gek::F32, false>(a.d, &nt))
                   : dt == GE_F16 ? (vec ? gek::norm_fn<gek::F16, true>(a.d, &nt) : gek::norm_fn<gek::F16, false>(a.d, &nt))
                                  : (vec ? gek::norm_fn<gek::BF16, true>(a.d, &nt)
                                         : gek::norm_fn<gek::BF16, false>(a.d, &nt));
  const int wg = gek::wg_of(nt), rpw = wg / nt;
  // rows one after the other: as many (up to 8) as leave the device 1024 workgroups and,
  // with an 8-bit result, as fit 76 KB of LDS (two workgroups per compute unit)
  const int granules = (int)((d + gemx::kKPad - 1) / gemx::kKPad);
  while (a.walk < 8 && rows >= (int64_t)1024 * rpw * a.walk * 2 &&
         (!codes || rpw * gemxh::norm_stage_bytes(granules, a.walk * 2) <= 76 * 1024))
    a.walk *= 2;
  const size_t stage = codes ? (size_t)rpw * gemxh::norm_stage_bytes(granules, a.walk) : 0;
  // a launch keeps its lane count below 2^32: more rows (5.4e8 narrow ones) take several, each
  // beginning on a row group of the 8-bit result
  const int64_t per = rpw * a.walk, most = ((int64_t(1) << 32) / wg - 1) * per / 32 * 32;
  const auto from = [](const void* p, int64_t bytes) {
    return p ? const_cast<char*>(static_cast<const char*>(p)) + bytes : nullptr;
  };
  for (int64_t r = 0; r < rows; r += most) {
    a.rows = std::min(rows - r, most);
    a.x = from(x, r * ldx * (int64_t)e);
    a.res = from(residual, r * ldr * (int64_t)e);
    a.sum = from(sum, r * lds * (int64_t)e);
    a.y = from(y, r * ldy * (int64_t)e);
    a.codes = from(codes, r / 32 * granules * 16 * 512);
    a.scales = from(scales, r / 32 * granules * gemx::kScaleGranule);
    void* params[] = {&a};
    if (hipLaunchKernel(fn, dim3((unsigned)((a.rows + per - 1) / per)), dim3((unsigned)wg), params, stage,
                        static_cast<hipStream_t>(stream)) != hipSuccess)
      return GE_ERR_HIP;
  }
  return GE_OK;
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
    slots = (slots + rpw - 1) / rpw;   // workgroups
    if (hipLaunchKernel(fn, dim3((unsigned)slots), dim3((unsigned)wg), params, 0, q) != hipSuccess)
      return GE_ERR_HIP;
  }
  const float* partial = static_cast<const float*>(workspace);
  int T = (int)slots, width = (int)d, wt = (int)wdt;
  void* params[] = {&partial, &T, &width, &dw, &wt};
  return hipLaunchKernel(reinterpret_cast<const void*>(&gek::norm_dweight_kernel), dim3((unsigned)((d + 63) / 64)),
                         dim3(64 * gek::kDwWaves), params, 0, q) == hipSuccess
             ? GE_OK
             : GE_ERR_HIP;
}

}  // extern "C"
