// Products with 4-bit weights and group scales (layout: w4_format.hpp).
//
//   D[t][r] = sum over groups g of s[r][g] (sum over k in g of X[t][k] q[r][k] - z[r][g] sum of X[t][k])
// The codes 0 .. 15 go into the matrix instruction as they are, exact in 16 bits, and the group's
// fp32 sum is scaled once, so that no product sees a rounded weight. A code byte is e4m3's
// 2^-9 times its value (eight subnormals, then eight values of the same spacing), so one
// conversion with scale 2^9 turns two codes into two exact 16-bit numbers.
#pragma once

#include <type_traits>

#include "gated_general.hpp"
#include "w4_format.hpp"

namespace gek {

using gew4::kRows;
using gew4::kTileBytes;
using gew4::kTileK;

struct W4Args {
  const void* x;         // (m, k)
  const char* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  const void* bias;
  void* D;
  int64_t m;
  int32_t n, k;          // columns of D (gated: of H)
  int32_t kt, groups;    // k-tiles, groups of a row
  int32_t group;
  int32_t rgs;           // row groups (gated: of a half)
  int32_t vec, out;      // types of the bias and of D
  int32_t ep;            // Ep, or Gate
  int32_t vecx;          // X's rows are 16-byte aligned and whole 16-byte chunks
};

// Grid of the tile kernel.
struct W4Launch {
  int32_t tiles_m, tiles_n, group_m;
};

// The eight codes of a dword, in the order of k, as 16-bit numbers.
template <int DT>
__device__ __forceinline__ i32x4 w4_unpack(uint32_t w) {
  const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  if constexpr (DT == BF16) {
    return i32x4{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false)),
                 __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true)),
                 __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false)),
                 __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true))};
  } else {
    return i32x4{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, false)),
                 __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, true)),
                 __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, false)),
                 __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, true))};
  }
}

// 16 x 16 x 32: a holds 16 rows (lane l: row l % 16, k 8 (l / 16) .. + 7), b 16 columns likewise;
// lane l's result r is row 4 (l / 16) + r of column l % 16.
template <int DT>
__device__ __forceinline__ f32x4 mma16(i32x4 a, i32x4 b, f32x4 c) {
  if constexpr (DT == BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <int DT>
constexpr int kOnes = DT == BF16 ? 0x3f803f80 : 0x3c003c00;   // two 16-bit ones

__device__ __forceinline__ float act_ep(float v, int ep) {
  return ep == RELU_BIAS ? (v > 0.0f ? v : 0.0f) : ep == GELU_BIAS ? gelu_tanh(v) : v;
}

// A step of 128 k of the skinny kernel: codes, group scales and zeros of NB row groups, X of 16 MT
// tokens. NG groups to a step.
template <int NB, int MT, int NG>
struct W4Step {
  i32x4 w[NB], x[MT][4];
  i32x2 s[NB][NG];
  uint32_t z[NB][NG];
};

// Skinny kernel: a few tokens; bound by reading W once. A workgroup takes NB row groups (gated:
// the gate's and the up projection's) and 16 MT tokens; its waves take the steps of 128 k in
// turn and add their sums through LDS in wave order.
template <int DT, bool GATED, int FB, int MT, int NG>
__global__ __launch_bounds__(512, MT == 4 ? 2 : MT == 2 ? 3 : 4) void w4_skinny_kernel(W4Args p) {
  constexpr int NB = GATED ? 2 * FB : FB;
  using Step = W4Step<NB, MT, NG>;
  extern __shared__ __attribute__((aligned(16))) f32x4 red[];   // [wave][NB MT][64]
  const int nw = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, li = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rg0 = blockIdx.x * FB;
  const int64_t t0 = (int64_t)blockIdx.y * (16 * MT);

  // (row groups past the last one have an empty range: zeros, and no reads)
  __amdgpu_buffer_rsrc_t rc[NB], rs[NB], rz[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int in = rg0 + b % FB;
    const bool on = in < p.rgs;
    const int64_t rg = (on ? in : 0) + (b < FB ? 0 : (int64_t)p.rgs);
    rc[b] = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p.codes) + rg * p.kt * kTileBytes, 0, on ? p.kt * kTileBytes : 0, kBufDword3);
    rs[b] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p.scales) + rg * p.groups * kRows, 0, on ? p.groups * kRows * 2 : 0, kBufDword3);
    rz[b] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.zeros) + rg * p.groups * kRows, 0, on ? p.groups * kRows : 0, kBufDword3);
  }
  const char* xb = static_cast<const char*>(p.x) + t0 * p.k * 2;
  const __amdgpu_buffer_rsrc_t rx = rsrc(xb);

  const auto load = [&](Step& st, int t) {
#pragma unroll
    for (int b = 0; b < NB; ++b) st.w[b] = __builtin_amdgcn_raw_buffer_load_b128(rc[b], lane * 16, t * kTileBytes, 0);
    const int g0 = NG > 1 ? t * NG : (int)((uint32_t)(t * kTileK) / (uint32_t)p.group);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        st.s[b][g] = __builtin_amdgcn_raw_buffer_load_b64(rs[b], q * 8 + g * 32, g0 * 32, 0);
        st.z[b][g] = __builtin_amdgcn_raw_buffer_load_b32(rz[b], q * 4 + g * 16, g0 * 16, 0);
      }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const bool in = t0 + mt * 16 + li < p.m;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kp = t * kTileK + 32 * j + 8 * q;
        if (p.vecx) {
          const uint32_t off = in && kp < p.k ? (uint32_t)(((mt * 16 + li) * p.k + kp) * 2) : kOOB;
          st.x[mt][j] = __builtin_amdgcn_raw_buffer_load_b128(rx, off, 0, 0);
        } else {
          const int row = in ? mt * 16 + li : 0;   // (its column of the products is not stored)
          st.x[mt][j] = load_end<2>(xb + (int64_t)row * p.k * 2, kp, p.k);
        }
      }
    }
  };

  f32x4 acc[NB][MT];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[b][mt] = f32x4{0, 0, 0, 0};

  const auto multiply = [&](const Step& st) {
    const i32x4 ones = {kOnes<DT>, kOnes<DT>, kOnes<DT>, kOnes<DT>};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4 part[NB][MT], sx[MT];
#pragma unroll
      for (int j = 4 / NG * g; j < 4 / NG * (g + 1); ++j) {
        const bool first = j == 4 / NG * g;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) sx[mt] = mma16<DT>(ones, st.x[mt][j], first ? f32x4{0, 0, 0, 0} : sx[mt]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const i32x4 wq = w4_unpack<DT>((uint32_t)st.w[b][j]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            part[b][mt] = mma16<DT>(wq, st.x[mt][j], first ? f32x4{0, 0, 0, 0} : part[b][mt]);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float s = Tr<DT>::widen((uint16_t)((uint32_t)st.s[b][g][r / 2] >> (16 * (r & 1))));
          const float z = (float)((st.z[b][g] >> (8 * r)) & 255u);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            acc[b][mt][r] = __builtin_fmaf(s, __builtin_fmaf(-z, sx[mt][r], part[b][mt][r]), acc[b][mt][r]);
        }
    }
  };

  Step s0, s1;
  if (w < p.kt) load(s0, w);
  for (int t = w; t < p.kt; t += 2 * nw) {
    if (t + nw < p.kt) load(s1, t + nw);
    __builtin_amdgcn_sched_barrier(0);
    multiply(s0);
    if (t + nw >= p.kt) break;
    if (t + 2 * nw < p.kt) load(s0, t + 2 * nw);
    __builtin_amdgcn_sched_barrier(0);
    multiply(s1);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) red[((w * NB + b) * MT + mt) * 64 + lane] = acc[b][mt];
  __syncthreads();
  for (int i = threadIdx.x; i < FB * MT * 64; i += blockDim.x) {
    const int l = i & 63, mt = i / 64 % MT, b = i / 64 / MT;
    const auto total = [&](int blk) {
      f32x4 v = red[(blk * MT + mt) * 64 + l];
      for (int o = 1; o < nw; ++o) {
        const f32x4 u = red[((o * NB + blk) * MT + mt) * 64 + l];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += u[r];
      }
      return v;
    };
    const int64_t token = t0 + mt * 16 + (l & 15);
    const int col = (rg0 + b) * kRows + (l >> 4) * 4, left = p.n - col;
    if (token >= p.m || left <= 0) continue;
    f32x4 v = total(b);
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (p.bias && r < left) v[r] += load_vec(p.bias, p.vec, col + r);
      y[r] = v[r];
    }
    if constexpr (GATED) {
      f32x4 u = total(FB + b);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (p.bias && r < left) u[r] += load_vec(p.bias, p.vec, (int64_t)p.n + col + r);
      with_gate(p.ep, [&](auto a) {
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = gate_act<decltype(a)::value, false>(v[r]) * u[r];
      });
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = act_ep(v[r], p.ep);
    }
    if (p.out == F32) store4<F32>(p.D, token * p.n + col, left, y);
    else store4<DT>(p.D, token * p.n + col, left, y);
  }
}

}  // namespace gek
