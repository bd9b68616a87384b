// 4-bit weights with group scales: entry points, and the kernels that make and undo them.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "product.hpp"
#include "w4.hpp"
#include "w4_host.hpp"

namespace gek {

const void* w4_tile_f16(int cfg, bool gated, int64_t group);    // w4_tile_f16.hip
const void* w4_tile_bf16(int cfg, bool gated, int64_t group);   // w4_tile_bf16.hip

namespace {

struct W4Weight {
  char* codes;
  uint16_t* scales;
  uint8_t* zeros;
  int64_t rows, k, kt, groups, group, rgs;   // rows and rgs: of a half
};

__device__ __forceinline__ uint16_t to_bits16(float v, int dt) {
  return dt == F16 ? (uint16_t)(Tr<F16>::pack2(v, v) & 0xffff) : (uint16_t)(Tr<BF16>::pack2(v, v) & 0xffff);
}
__device__ __forceinline__ float from_bits16(uint16_t v, int dt) {
  return dt == F16 ? Tr<F16>::widen(v) : Tr<BF16>::widen(v);
}

// The quotients of eight values and a scale, rounded to nearest even. 16-bit values: a product with
// the reciprocal rs, its mantissa rounded to 20 bits. A quotient of two 16-bit numbers lies on a
// border between two whole numbers or at least 2^-16 of itself away from it, and the product is
// within 2^-22 of the quotient: so borders come out exactly and nothing else reaches them. (The exact
// division took twice the instructions, which bound the kernel: 45 us at 11008 x 4096.) The exact
// division for fp32 values, and where the reciprocal overflows.
template <int SRC>
__device__ __forceinline__ void w4_quotients(const float (&v)[8], float s, float rs, float (&o)[8]) {
#pragma clang fp contract(off)
  if (SRC == F32 || __builtin_amdgcn_ballot_w64(!(rs <= 3.402823466e38f)) != 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = rintf(v[e] / s);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = fminf(fmaxf(v[e] * rs, -64.0f), 64.0f), c = y * 17.0f;   // (held: far outside of the codes either way)
      o[e] = rintf(c - (c - y));
    }
  }
}

// Rounds to a group's codes. A wave takes the tiles of one group (at most one tile holds several,
// NG): row l % 16, and in each tile the k values 32 j + 8 (l / 16) .. + 7. Groups past one tile
// (NG 0) are read twice, for the range and for the codes. Bound by memory: 11008 x 4096 bf16 25 us,
// 4.5 TB/s.
template <int SRC, int NG>
__global__ __launch_bounds__(256) void w4_quantize_kernel(const void* src, int64_t ld, W4Weight o, int dt, int symmetric,
                                                          int64_t first, int64_t units) {
  const int64_t unit = first + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int lane = threadIdx.x & 63, li = lane & 15, q = lane >> 4;
  const int64_t per = NG == 0 ? o.groups : o.kt;       // units of a row group
  const int64_t rg = unit / per, u = unit - rg * per;   // row group, counted over both halves
  const int64_t span = NG == 0 ? o.group / kTileK : 1;
  const int64_t ta = u * span, tb = ta + span < o.kt ? ta + span : o.kt;
  const int64_t half = rg / o.rgs, in = (rg - half * o.rgs) * kRows + li;
  const bool on = in < o.rows;
  const char* row = static_cast<const char*>(src) + (half * o.rows + (on ? in : 0)) * ld * Tr<SRC>::es;

  const auto read = [&](int64_t t, int j, float (&v)[8]) {
    constexpr int ES = Tr<SRC>::es, E = 16 / ES;
    const int64_t kp = t * kTileK + 32 * j + 8 * q;
    i32x4 raw[8 / E];
#pragma unroll
    for (int h = 0; h < 8 / E; ++h)
      raw[h] = kp + 8 <= o.k ? load16(row + (kp + h * E) * ES) : load_end<ES>(row, kp + h * E, o.k);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (SRC == F32) v[e] = __int_as_float(raw[e / 4][e % 4]);
      else v[e] = Tr<SRC>::widen((uint16_t)((uint32_t)raw[0][e / 2] >> (16 * (e & 1))));
    }
  };
  struct Group {
    float lo = 0.0f, hi = 0.0f, bad = 0.0f;   // bad: 0, or NaN once a value was not finite
    float s, rs, z;
    uint16_t bits;
  };
  const auto range = [&](Group& g, const float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g.lo = fminf(g.lo, v[e]);
      g.hi = fmaxf(g.hi, v[e]);
      g.bad = __builtin_fmaf(v[e], 0.0f, g.bad);
    }
  };
  // Scale and zero of a group from its range (of this lane's part; joined over the four quarters).
  const auto finish = [&](Group& g) {
#pragma unroll
    for (int d = 16; d < 64; d <<= 1) {
      g.lo = fminf(g.lo, __shfl_xor(g.lo, d));
      g.hi = fmaxf(g.hi, __shfl_xor(g.hi, d));
      g.bad += __shfl_xor(g.bad, d);
    }
    const double width = symmetric ? (double)fmaxf(-g.lo, g.hi) / 7.0 : ((double)g.hi - (double)g.lo) / 15.0;
    g.bits = g.bad != 0.0f ? (uint16_t)(dt == F16 ? 0x7e00 : 0x7fc0) : to_bits16((float)width, dt);
    g.s = from_bits16(g.bits, dt);
    g.rs = 1.0f / (g.s > 0.0f ? g.s : 1.0f);
    g.z = symmetric ? 8.0f : g.s > 0.0f ? (float)fmin(rint(-(double)g.lo / (double)g.s), 15.0) : 0.0f;
  };
  const auto encode = [&](const Group& g, const float (&v)[8], int64_t t, int j) {
    const int64_t left = on ? o.k - (t * kTileK + 32 * j + 8 * q) : 0;   // padding is zero
    float c[8];
    w4_quotients<SRC>(v, g.s, g.rs, c);
    uint32_t d = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      d |= (uint32_t)(g.s > 0.0f ? fminf(fmaxf(c[e] + g.z, 0.0f), 15.0f) : g.z) << (8 * (e % 4) + 4 * (e / 4));
    if (left < 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e >= left) d &= ~(15u << (8 * (e % 4) + 4 * (e / 4)));
    }
    return d;
  };
  const auto put = [&](const Group& g, int64_t at) {
    if (q == 0 && at < o.groups) {
      o.scales[(rg * o.groups + at) * kRows + li] = on ? g.bits : (uint16_t)0;
      o.zeros[(rg * o.groups + at) * kRows + li] = on ? (uint8_t)g.z : (uint8_t)0;
    }
  };

  if constexpr (NG > 0) {
    float v[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) read(ta, j, v[j]);
    i32x4 out;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      Group g;
#pragma unroll
      for (int j = 4 / NG * i; j < 4 / NG * (i + 1); ++j) range(g, v[j]);
      finish(g);
#pragma unroll
      for (int j = 4 / NG * i; j < 4 / NG * (i + 1); ++j) out[j] = (int)encode(g, v[j], ta, j);
      put(g, ta * NG + i);
    }
    *reinterpret_cast<i32x4*>(o.codes + (rg * o.kt + ta) * kTileBytes + lane * 16) = out;
  } else {
    Group g;
    float v[8];
    for (int64_t t = ta; t < tb; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        read(t, j, v);
        range(g, v);
      }
    finish(g);
    put(g, u);
    for (int64_t t = ta; t < tb; ++t) {
      i32x4 out;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        read(t, j, v);
        out[j] = (int)encode(g, v, t, j);
      }
      *reinterpret_cast<i32x4*>(o.codes + (rg * o.kt + t) * kTileBytes + lane * 16) = out;
    }
  }
}
template <int SRC>
const void* quantize_of(int64_t group) {
  return group == 32    ? reinterpret_cast<const void*>(&w4_quantize_kernel<SRC, 4>)
         : group == 64  ? reinterpret_cast<const void*>(&w4_quantize_kernel<SRC, 2>)
         : group == 128 ? reinterpret_cast<const void*>(&w4_quantize_kernel<SRC, 1>)
                        : reinterpret_cast<const void*>(&w4_quantize_kernel<SRC, 0>);
}

// Row-major codes, scales and zeros (null: all 8) into the layout; a wave per tile, and per 16
// rows' scales beside it. Once per weight of a checkpoint:
// 2 x 11008 x 4096 in 35 us.
__global__ __launch_bounds__(256) void w4_pack_kernel(const uint8_t* src, const uint16_t* scales, const uint8_t* zeros,
                                                      W4Weight o, int64_t first, int64_t units) {
  const int64_t unit = first + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int lane = threadIdx.x & 63, li = lane & 15, q = lane >> 4;
  const int64_t rg = unit / o.kt, t = unit - rg * o.kt;
  const int64_t half = rg / o.rgs, in = (rg - half * o.rgs) * kRows + li, row = half * o.rows + in;
  const bool on = in < o.rows;
  const int64_t width = (o.k + 1) / 2;
  i32x4 out = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t kp = t * kTileK + 32 * j + 8 * q;
    uint32_t d = 0, in4 = 0;
    const uint8_t* from = src + row * width + kp / 2;
    if (on && kp / 2 + 4 <= width) {
      __builtin_memcpy(&in4, from, 4);
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (on && kp / 2 + b < width) in4 |= (uint32_t)from[b] << (8 * b);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int64_t at = kp / 2 + b;   // holds k 2 at (low) and 2 at + 1 (high)
      uint32_t v = (in4 >> (8 * b)) & 255u;
      if (2 * at + 1 >= o.k) v &= 15u;
      const int e = 2 * b;   // element e and e + 1 of the dword
      d |= (v & 15u) << (8 * (e % 4) + 4 * (e / 4)) | (v >> 4) << (8 * ((e + 1) % 4) + 4 * ((e + 1) / 4));
    }
    out[j] = (int)d;
  }
  *reinterpret_cast<i32x4*>(o.codes + unit * kTileBytes + lane * 16) = out;
  // the groups that begin in this tile
  const int64_t ga = gew4::ceil_div(t * kTileK, o.group), gb = gew4::ceil_div((t + 1) * kTileK, o.group);
  const int64_t g = ga + q;
  if (g < gb && g < o.groups) {
    o.scales[(rg * o.groups + g) * kRows + li] = on ? scales[row * o.groups + g] : (uint16_t)0;
    o.zeros[(rg * o.groups + g) * kRows + li] = !on ? 0 : zeros ? zeros[row * o.groups + g] & 15 : 8;
  }
}

// (q - z) s, rounded to DT. A wave per tile, eight values at a time. Bound by memory: 11008 x 4096
// bf16 28 us, 4.0 TB/s; in 16 bits a lane's eight values leave in two stores of 8 bytes, and memory sees
// 10% more writes than the result has.
template <int DT>
__global__ __launch_bounds__(256) void w4_dequantize_kernel(W4Weight o, int sdt, void* dst, int64_t ld, int64_t first,
                                                            int64_t units) {
  const int64_t unit = first + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int lane = threadIdx.x & 63, li = lane & 15, q = lane >> 4;
  const int64_t rg = unit / o.kt, t = unit - rg * o.kt;
  const int64_t half = rg / o.rgs, in = (rg - half * o.rgs) * kRows + li, row = half * o.rows + in;
  const i32x4 c = *reinterpret_cast<const i32x4*>(o.codes + unit * kTileBytes + lane * 16);
  if (in >= o.rows) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t kp = t * kTileK + 32 * j + 8 * q;
    if (kp >= o.k) continue;
    const int64_t at = (rg * o.groups + kp / o.group) * kRows + li;
    const float s = from_bits16(o.scales[at], sdt), z = (float)o.zeros[at];
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = ((float)(((uint32_t)c[j] >> (8 * (e % 4) + 4 * (e / 4))) & 15u) - z) * s;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float u[4] = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
      store4<DT>(dst, row * ld + kp + 4 * h, o.k - kp - 4 * h, u);
    }
  }
}

W4Weight weight(int64_t rows, int64_t k, int64_t group, int halves, const void* codes, const void* scales,
                const void* zeros) {
  W4Weight w;
  w.codes = static_cast<char*>(const_cast<void*>(codes));
  w.scales = static_cast<uint16_t*>(const_cast<void*>(scales));
  w.zeros = static_cast<uint8_t*>(const_cast<void*>(zeros));
  w.rows = rows / halves;
  w.k = k;
  w.kt = gew4::k_tiles(k);
  w.group = group;
  w.groups = gew4::k_groups(k, group);
  w.rgs = gew4::row_groups(rows, halves);
  return w;
}

ge_status_t run(const void* fn, dim3 grid, int threads, size_t lds, void** params, void* stream) {
  return hipLaunchKernel(fn, grid, dim3(threads), params, lds, static_cast<hipStream_t>(stream)) == hipSuccess ? GE_OK
                                                                                                           : GE_ERR_HIP;
}

template <int DT, bool GATED, int MT, bool VEC, bool FEW>
const void* skinny_of(int64_t group) {
  return group == 32   ? reinterpret_cast<const void*>(&w4_skinny_kernel<DT, GATED, MT, 4, VEC, FEW>)
         : group == 64 ? reinterpret_cast<const void*>(&w4_skinny_kernel<DT, GATED, MT, 2, VEC, FEW>)
                       : reinterpret_cast<const void*>(&w4_skinny_kernel<DT, GATED, MT, 1, VEC, FEW>);
}
template <int DT, bool GATED, int MT>
const void* skinny_of(int64_t group, bool vec) {
  return vec ? skinny_of<DT, GATED, MT, true, false>(group) : skinny_of<DT, GATED, MT, false, false>(group);
}

template <int DT, bool GATED>
ge_status_t skinny(W4Args& a, bool vec, int cus, void* stream) {
  constexpr int NB = GATED ? 2 : 1;
  void* params[] = {&a};
  const int mt = a.m <= 16 ? 1 : a.m <= 32 ? 2 : 4;
  // Waves of a workgroup: as many as the device holds at once (16 to a compute unit, 12 and 8 with
  // more tokens), four at least: 1 x 4096 x 11008 takes 14.8, 9.9 and 8.1 us with 4, 8 and 16 waves in
  // 256 workgroups, 1 x 2 x 11008 x 4096 13.2, 15.5 and 16.7 in 688.
  const int64_t most = (int64_t)cus * (mt == 1 ? 16 : mt == 2 ? 12 : 8) / (a.rgs * gew4::ceil_div(a.m, 16 * mt));
  const int nw = mt == 1 && most >= 16 ? 16 : mt < 4 && most >= 8 ? 8 : 4;
  const void* fn = a.m <= 4 && vec ? skinny_of<DT, GATED, 1, true, true>(a.group)
                   : mt == 1 ? skinny_of<DT, GATED, 1>(a.group, vec)
                   : mt == 2 ? skinny_of<DT, GATED, 2>(a.group, vec)
                             : skinny_of<DT, GATED, 4>(a.group, vec);
  // (a launch has at most 65535 rows of workgroups)
  const int64_t step = (int64_t)65535 * 16 * mt, all = a.m;
  const char* x = static_cast<const char*>(a.x);
  char* d = static_cast<char*>(a.D);
  for (int64_t at = 0; at < all; at += step) {
    a.m = std::min(step, all - at);
    a.x = x + at * a.k * 2;
    a.D = d + at * a.n * (a.out == F32 ? 4 : 2);
    const dim3 grid((unsigned)a.rgs, (unsigned)gew4::ceil_div(a.m, 16 * mt));
    if (ge_status_t st = run(fn, grid, nw * 64, (size_t)nw * NB * mt * 1024, params, stream); st != GE_OK) return st;
  }
  return GE_OK;
}

ge_status_t tiled(W4Args& a, int cfg, ge_dtype_t dt, bool gated, void* stream) {
  const gew4::W4TileCfg& T = gew4::kTiles[cfg];
  W4Launch L;
  L.tiles_n = (int32_t)gew4::ceil_div(gated ? 2 * (int64_t)a.n : a.n, T.bn);
  L.group_m = 8;
  const void* fn = dt == GE_F16 ? w4_tile_f16(cfg, gated, a.group) : w4_tile_bf16(cfg, gated, a.group);
  const int64_t step = geh::rows_per_launch(T.bm, L.tiles_n, T.waves * 64), all = a.m;
  const char* x = static_cast<const char*>(a.x);
  char* d = static_cast<char*>(a.D);
  for (int64_t at = 0; at < all; at += step) {
    a.m = std::min(step, all - at);
    a.x = x + at * a.k * 2;
    a.D = d + at * a.n * (a.out == F32 ? 4 : 2);
    L.tiles_m = (int32_t)gew4::ceil_div(a.m, T.bm);
    void* params[] = {&a, &L};
    if (ge_status_t st = run(fn, dim3((unsigned)((int64_t)L.tiles_m * L.tiles_n)), T.waves * 64, 0, params, stream); st != GE_OK)
      return st;
  }
  return GE_OK;
}

ge_status_t multiply(int64_t m, int64_t n, int64_t k, int64_t group, ge_dtype_t dt, ge_dtype_t out, bool gated, int ep,
                     const void* x, const void* codes, const void* scales, const void* zeros, const void* bias,
                     ge_dtype_t vec, void* D, void* stream) {
  const W4Weight w = weight(gated ? 2 * n : n, k, group, gated ? 2 : 1, codes, scales, zeros);
  W4Args a;
  a.x = x;
  a.codes = w.codes;
  a.scales = w.scales;
  a.zeros = w.zeros;
  a.bias = bias;
  a.D = D;
  a.m = m;
  a.n = (int32_t)n;
  a.k = (int32_t)k;
  a.kt = (int32_t)w.kt;
  a.groups = (int32_t)w.groups;
  a.group = (int32_t)group;
  a.rgs = (int32_t)w.rgs;
  a.vec = (int32_t)vec;
  a.out = (int32_t)out;
  a.ep = ep;
  a.span = (int32_t)(group / gew4::kTileK);
  a.inv_span = a.span > 1 ? (uint32_t)(((uint64_t(1) << 32) + a.span - 1) / a.span) : 0u;
  const bool chunks = k % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  int cus = 0;
  if (ge_status_t st = gei::current_device(&cus); st != GE_OK) return st;
  if (const int cfg = gew4h::choose(m, n, k, group, gated, chunks, cus); cfg >= 0)
    return tiled(a, cfg, dt, gated, stream);
  if (dt == GE_F16) return gated ? skinny<F16, true>(a, chunks, cus, stream) : skinny<F16, false>(a, chunks, cus, stream);
  return gated ? skinny<BF16, true>(a, chunks, cus, stream) : skinny<BF16, false>(a, chunks, cus, stream);
}

// A kernel with a wave for each unit, four to a workgroup: units from `first` on, in launches of fewer
// than 2^32 lanes.
ge_status_t run_units(const void* fn, int64_t& first, int64_t units, void** params, void* stream) {
  const int64_t most = geh::rows_per_launch(4, 1, 256);
  for (first = 0; first < units; first += most)
    if (ge_status_t st = run(fn, dim3((unsigned)gew4::ceil_div(std::min(most, units - first), 4)), 256, 0, params, stream);
        st != GE_OK)
      return st;
  return GE_OK;
}

}  // namespace
}  // namespace gek

extern "C" {

size_t gemm_epilog_w4_code_bytes(int64_t rows, int64_t k, int halves) { return gew4h::code_bytes(rows, k, halves); }
size_t gemm_epilog_w4_scale_count(int64_t rows, int64_t k, int64_t group, int halves) {
  return gew4h::scale_count(rows, k, group, halves);
}

ge_status_t gemm_epilog_w4_quantize(int64_t rows, int64_t k, ge_dtype_t src_dt, const void* src, int64_t ld,
                                    int64_t group, int halves, int symmetric, ge_dtype_t dt, void* codes, void* scales,
                                    void* zeros, void* stream) {
  if (ge_status_t st = gew4h::check_weight(rows, k, group, halves, codes, scales, zeros); st != GE_OK) return st;
  if (ge_status_t st = gew4h::check_quantize(rows, k, src_dt, src, ld, dt); st != GE_OK) return st;
  int cus = 0;
  if (ge_status_t st = gei::current_device(&cus); st != GE_OK) return st;
  gek::W4Weight w = gek::weight(rows, k, group, halves, codes, scales, zeros);
  int64_t first = 0, units = w.rgs * halves * (group > gew4::kTileK ? w.groups : w.kt);
  int d = (int)dt, sym = symmetric != 0;
  void* params[] = {&src, &ld, &w, &d, &sym, &first, &units};
  const void* fn = src_dt == GE_F32   ? gek::quantize_of<gek::F32>(group)
                   : src_dt == GE_F16 ? gek::quantize_of<gek::F16>(group)
                                      : gek::quantize_of<gek::BF16>(group);
  return gek::run_units(fn, first, units, params, stream);
}

ge_status_t gemm_epilog_w4_pack(int64_t rows, int64_t k, int64_t group, int halves, const void* src_codes,
                                const void* src_scales, const void* src_zeros, void* codes, void* scales, void* zeros,
                                void* stream) {
  if (ge_status_t st = gew4h::check_weight(rows, k, group, halves, codes, scales, zeros); st != GE_OK) return st;
  if (!src_codes || !src_scales) return GE_ERR_NULL_POINTER;
  if (reinterpret_cast<uintptr_t>(src_scales) % 2) return GE_ERR_MISALIGNED;
  int cus = 0;
  if (ge_status_t st = gei::current_device(&cus); st != GE_OK) return st;
  gek::W4Weight w = gek::weight(rows, k, group, halves, codes, scales, zeros);
  int64_t first = 0, units = w.rgs * halves * w.kt;
  void* params[] = {&src_codes, &src_scales, &src_zeros, &w, &first, &units};
  return gek::run_units(reinterpret_cast<const void*>(&gek::w4_pack_kernel), first, units, params, stream);
}

ge_status_t gemm_epilog_w4_dequantize(int64_t rows, int64_t k, int64_t group, int halves, ge_dtype_t dt,
                                      const void* codes, const void* scales, const void* zeros, ge_dtype_t dst_dt,
                                      void* dst, int64_t ld, void* stream) {
  if (ge_status_t st = gew4h::check_weight(rows, k, group, halves, codes, scales, zeros); st != GE_OK) return st;
  if (ge_status_t st = gew4h::check_dequantize(rows, k, dt, dst_dt, dst, ld); st != GE_OK) return st;
  int cus = 0;
  if (ge_status_t st = gei::current_device(&cus); st != GE_OK) return st;
  gek::W4Weight w = gek::weight(rows, k, group, halves, codes, scales, zeros);
  int64_t first = 0, units = w.rgs * halves * w.kt;
  int d = (int)dt;
  void* params[] = {&w, &d, &dst, &ld, &first, &units};
  const void* fn = dst_dt == GE_F32   ? reinterpret_cast<const void*>(&gek::w4_dequantize_kernel<gek::F32>)
                   : dst_dt == GE_F16 ? reinterpret_cast<const void*>(&gek::w4_dequantize_kernel<gek::F16>)
                                      : reinterpret_cast<const void*>(&gek::w4_dequantize_kernel<gek::BF16>);
  return gek::run_units(fn, first, units, params, stream);
}

ge_status_t gemm_epilog_w4_matmul(int64_t m, int64_t n, int64_t k, int64_t group, ge_dtype_t dt, ge_dtype_t out,
                                  ge_epilog_t ep, const void* x, const void* codes, const void* scales,
                                  const void* zeros, const void* bias, ge_dtype_t vec, void* D, void* stream) {
  if (ge_status_t st = gew4h::check_weight(n, k, group, 1, codes, scales, zeros); st != GE_OK) return st;
  if (ep != GE_EPILOG_NONE && ep != GE_EPILOG_BIAS && ep != GE_EPILOG_RELU_BIAS && ep != GE_EPILOG_GELU_BIAS)
    return GE_ERR_NOT_SUPPORTED;
  if (ge_status_t st = gew4h::check_product(m, n, dt, out, x, bias, vec, D); st != GE_OK) return st;
  if (ep != GE_EPILOG_NONE && !bias) return GE_ERR_NULL_POINTER;
  if (m == 0) return GE_OK;
  return gek::multiply(m, n, k, group, dt, out, false, (int)ep, x, codes, scales, zeros,
                       ep == GE_EPILOG_NONE ? nullptr : bias, vec, D, stream);
}

ge_status_t gemm_epilog_w4_gated(int64_t m, int64_t n, int64_t k, int64_t group, ge_dtype_t dt, ge_gate_t act,
                                 const void* x, const void* codes, const void* scales, const void* zeros,
                                 const void* bias, ge_dtype_t vec, void* h, void* stream) {
  if (n < 1 || n > gew4h::kMaxDim) return GE_ERR_INVALID_VALUE;
  if (ge_status_t st = gew4h::check_weight(2 * n, k, group, 2, codes, scales, zeros); st != GE_OK) return st;
  if (act != GE_GATE_SILU && act != GE_GATE_GELU && act != GE_GATE_RELU) return GE_ERR_INVALID_VALUE;
  if (ge_status_t st = gew4h::check_product(m, n, dt, dt, x, bias, vec, h); st != GE_OK) return st;
  if (m == 0) return GE_OK;
  return gek::multiply(m, n, k, group, dt, dt, true, (int)act, x, codes, scales, zeros, bias, vec, h, stream);
}

}  // extern "C"
