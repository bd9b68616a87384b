// Products with 4-bit weights and group scales (layout: w4_format.hpp).
//
//   D[t][r] = sum over groups g of s[r][g] (sum over k in g of X[t][k] q[r][k] - z[r][g] sum of X[t][k])
// The codes 0 .. 15 go into the matrix instruction as they are, exact in 16 bits, and the group's
// fp32 sum is scaled once, so that no product sees a rounded weight. A code byte is e4m3's
// 2^-9 times its value (eight subnormals, then eight values of the same spacing), so one
// conversion with scale 2^9 turns two codes into two exact 16-bit numbers.
//
// Few tokens: a workgroup takes 16 rows of W (gated: 16 of each half) and up to 64 tokens; its waves
// share the k-tiles and add their sums through LDS in wave order. Bound by W's codes from memory, and
// by the start: 1 x 4096 x 11008 f16 7.6 us (3.1 TB/s; a kernel's start, the first reads and the joining
// are about 4), 1 x 2 x 11008 x 4096 bf16 11.4 (4.2 TB/s). Every byte comes once (23.9 and 47.4 MB by the
// counters). From 17 tokens on X, which every 16 rows read for themselves, bounds it: 32 and 64
// tokens by 4096 x 4096 take 11 and 18 us.
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
  int32_t span;          // groups of 128 and more: k-tiles of a group
  uint32_t inv_span;     // ceil(2^32 / span) (span > 1): t / span is the high half of t times it
};

template <int N, class F, int I = 0>
__device__ __forceinline__ void w4_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    w4_for<N, F, I + 1>(static_cast<F&&>(f));
  }
}

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

// v of another lane of the row of 16, by a DPP control.
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, true);
}
constexpr int kRowShl = 0x100, kRowRor = 0x120, kRowBcast = 0x150;   // lane i takes i + n, i - n, n

// A step of 128 k of the skinny kernel: codes of NB row groups and X of 16 MT tokens (XR loads).
template <int NB, int XR>
struct W4Step {
  i32x4 w[NB], x[XR];
};

// Skinny kernel: a few tokens; bound by reading W once, and beside that by the number of memory
// instructions. A workgroup takes a row group (gated: the gate's and the up projection's, NB) and 16
// MT tokens; its waves take the steps of 128 k in turn and add their sums through LDS in wave
// order. The next step is on its way during a step's products; with 33 tokens and more some of its
// registers do not fit and wait in scratch memory: 40 to 256 in a gated weight, up to 14 in another (204 with
// groups of 32 and 64 and unaligned bf16 X). NG: groups to a step. VEC: X's rows are whole, aligned 16-byte chunks. FEW: up to four
// tokens.
// Scales and zeros are loaded for 16 groups at a time, a group to each of the 16 lanes of a row
// (which need the same four scales, those of the rows 4 (l / 16) .. + 3 of the products), and
// handed to all of them as their turn comes. Of up to four tokens a lane loads a chunk of its own,
// and passes it on likewise: three memory instructions to a gated step of 2 KB instead of ten (one
// token by 2 x 11008 x 4096 from memory: 14.7 -> 13.2 us; 4096 x 11008 8.1).
template <int DT, bool GATED, int MT, int NG, bool VEC, bool FEW>
__global__ __launch_bounds__(MT == 1 ? 1024 : 512, MT == 4 ? 2 : MT == 2 ? 3 : 4) void w4_skinny_kernel(W4Args p) {
  constexpr int NB = GATED ? 2 : 1, XR = FEW ? 1 : 4 * MT, SPAN = 16 / NG;   // SPAN: steps of a load of scales
  static_assert(!FEW || (MT == 1 && VEC), "few tokens");
  using Step = W4Step<NB, XR>;
  extern __shared__ __attribute__((aligned(16))) f32x4 red[];   // [wave][NB MT][64]
  const int nw = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, li = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rg = blockIdx.x;
  const int64_t t0 = (int64_t)blockIdx.y * (16 * MT);

  __amdgpu_buffer_rsrc_t rc[NB], rs[NB], rz[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t in = rg + (b ? (int64_t)p.rgs : 0);
    rc[b] = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p.codes) + in * p.kt * kTileBytes, 0, p.kt * kTileBytes, kBufDword3);
    rs[b] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p.scales) + in * p.groups * kRows, 0, p.groups * kRows * 2, kBufDword3);
    rz[b] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.zeros) + in * p.groups * kRows, 0, p.groups * kRows, kBufDword3);
  }
  const char* xb = static_cast<const char*>(p.x) + t0 * p.k * 2;
  const __amdgpu_buffer_rsrc_t rx = rsrc(xb);
  uint32_t xo[MT];   // this lane's place in a step; of a token past the last one, out of range
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int row = FEW ? li & 3 : mt * 16 + li;
    xo[mt] = t0 + row < p.m ? (uint32_t)(row * p.k * 2 + (FEW ? (li >> 2) * 64 : 0) + q * 16) : kOOB;
  }

  const auto load = [&](Step& st, int tv) {
    // (the same in all lanes, which the compiler loses in the loop: offsets in vector registers
    // would cost each load a loop over the lanes)
    const int t = __builtin_amdgcn_readfirstlane(tv);
#pragma unroll
    for (int b = 0; b < NB; ++b) st.w[b] = __builtin_amdgcn_raw_buffer_load_b128(rc[b], lane * 16, t * kTileBytes, 0);
    const bool whole = (t + 1) * kTileK <= p.k;
    if constexpr (FEW) {
      const uint32_t off = whole || t * kTileK + (li >> 2) * 32 + 8 * q < p.k ? xo[0] : kOOB;
      st.x[0] = __builtin_amdgcn_raw_buffer_load_b128(rx, off, t * (2 * kTileK), 0);
    } else {
      if (VEC && whole) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st.x[mt * 4 + j] = __builtin_amdgcn_raw_buffer_load_b128(rx, xo[mt] + j * 64, t * (2 * kTileK), 0);
        return;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int kp = t * kTileK + 32 * j + 8 * q;
          if constexpr (VEC) {
            st.x[mt * 4 + j] = __builtin_amdgcn_raw_buffer_load_b128(rx, kp < p.k ? xo[mt] + j * 64 : kOOB, t * (2 * kTileK), 0);
          } else {
            // (tokens past the last one read the first: their columns of the products are not stored)
            const char* row = xb + (int64_t)(xo[mt] == kOOB ? 0 : mt * 16 + li) * p.k * 2;
            st.x[mt * 4 + j] = whole ? load16(row + (int64_t)kp * 2) : load_end<2>(row, kp, p.k);
          }
        }
      }
    }
  };
  // Scales and zeros of this wave's steps i .. i + SPAN - 1: those of group li % NG of step
  // i + li / NG in lane li.
  struct Scales {
    i32x2 s[NB];
    int z[NB];
  };
  const auto load_scales = [&](Scales& sc, int i) {
    const int t = w + (i + li / NG) * nw;
    const int g = NG > 1 ? t * NG + li % NG : p.span == 1 ? t : (int)__umulhi((uint32_t)t, p.inv_span);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      sc.s[b] = __builtin_amdgcn_raw_buffer_load_b64(rs[b], t < p.kt ? (uint32_t)(g * 32 + q * 8) : kOOB, 0, 0);
      sc.z[b] = __builtin_amdgcn_raw_buffer_load_b32(rz[b], t < p.kt ? (uint32_t)(g * 16 + q * 4) : kOOB, 0, 0);
    }
  };

  f32x4 acc[NB][MT];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[b][mt] = f32x4{0, 0, 0, 0};

  const auto multiply = [&](const Step& st, Scales& sc) {
    const i32x4 ones = {kOnes<DT>, kOnes<DT>, kOnes<DT>, kOnes<DT>};
    i32x4 x[4 * MT];
#pragma unroll
    for (int i = 0; i < 4 * MT; ++i) x[i] = st.x[FEW ? 0 : i];
    if constexpr (FEW) {   // chunk j of token l % 4 is in lane l + 4 j
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[1][e] = dpp<kRowShl + 4>(st.x[0][e]);
        x[2][e] = dpp<kRowShl + 8>(st.x[0][e]);
        x[3][e] = dpp<kRowShl + 12>(st.x[0][e]);
      }
    }
    w4_for<NG>([&](auto gtag) {
      constexpr int g = decltype(gtag)::value;
      f32x4 part[NB][MT], sx[MT];
#pragma unroll
      for (int j = 4 / NG * g; j < 4 / NG * (g + 1); ++j) {
        const bool first = j == 4 / NG * g;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) sx[mt] = mma16<DT>(ones, x[mt * 4 + j], first ? f32x4{0, 0, 0, 0} : sx[mt]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const i32x4 wq = w4_unpack<DT>((uint32_t)st.w[b][j]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            part[b][mt] = mma16<DT>(wq, x[mt * 4 + j], first ? f32x4{0, 0, 0, 0} : part[b][mt]);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const i32x2 s2 = {dpp<kRowBcast + g>(sc.s[b][0]), dpp<kRowBcast + g>(sc.s[b][1])};
        const uint32_t z4 = (uint32_t)dpp<kRowBcast + g>(sc.z[b]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float s = Tr<DT>::widen((uint16_t)((uint32_t)s2[r / 2] >> (16 * (r & 1))));
          const float z = (float)((z4 >> (8 * r)) & 255u);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            acc[b][mt][r] = __builtin_fmaf(s, __builtin_fmaf(-z, sx[mt][r], part[b][mt][r]), acc[b][mt][r]);
        }
      }
    });
    // the next step's groups to the first lanes
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      sc.s[b] = i32x2{dpp<kRowRor + 16 - NG>(sc.s[b][0]), dpp<kRowRor + 16 - NG>(sc.s[b][1])};
      sc.z[b] = dpp<kRowRor + 16 - NG>(sc.z[b]);
    }
  };

  const int steps = w < p.kt ? (p.kt - w + nw - 1) / nw : 0;   // of this wave
  Step s0, s1;
  Scales sc, ahead;
  if (steps > 0) {
    load_scales(ahead, 0);
    load(s0, w);
  }
  for (int i = 0; i < steps; i += 2) {
    if (i % SPAN == 0) {
      sc = ahead;
      if (i + SPAN < steps) load_scales(ahead, i + SPAN);
    }
    if (i + 1 < steps) load(s1, w + (i + 1) * nw);
    __builtin_amdgcn_sched_barrier(0);
    multiply(s0, sc);
    if (i + 1 >= steps) break;
    if (i + 2 < steps) load(s0, w + (i + 2) * nw);
    __builtin_amdgcn_sched_barrier(0);
    multiply(s1, sc);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) red[((w * NB + b) * MT + mt) * 64 + lane] = acc[b][mt];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * 64; i += blockDim.x) {
    const int l = i & 63, mt = i / 64;
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
    const int col = rg * kRows + (l >> 4) * 4, left = p.n - col;
    if (token >= p.m || left <= 0) continue;
    f32x4 v = total(0);
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (p.bias && r < left) v[r] += load_vec(p.bias, p.vec, col + r);
      y[r] = v[r];
    }
    if constexpr (GATED) {
      f32x4 u = total(1);
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
