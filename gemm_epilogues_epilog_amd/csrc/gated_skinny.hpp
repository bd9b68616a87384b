// Few tokens: X (m, k) by W^T, W (n, k) or a gated (2 n, k), bound by reading W once.
//
// A workgroup takes 16 rows of W (gated: of each half) and 16 MT tokens. Its waves take
// steps of 256 bytes of k in turn, stream W from memory straight into the registers that feed the
// 16 x 16 matrix instruction (lane l: row l % 16, the 16 bytes l / 16 of each 64), with the next
// step on its way during a step's products, and add their sums through LDS in wave order. (Gated,
// from 17 tokens on, two steps do not fit the registers: 4 to 28 of them go to scratch memory as they
// arrive, and with them the wave waits for those loads before the products; fp32 rows that are not whole
// 16-byte chunks from 33 tokens on 185.)
// W's rows at any alignment: 16-byte loads, the row's last ones moved back and shifted.
//
// One token by 2 x 11008 x 4096 bf16: 33 us in the kernel, 5.5 TB/s of W (every byte once: 183 MB by the
// counters). More tokens read X once per workgroup out of the L2 caches, and that is what bounds 17 to
// 64 of them (figures beside the rule that chooses, gated_host.cpp).
#pragma once

#include <type_traits>

#include "gated_general.hpp"

namespace gek {

struct SkinnyArgs {
  const void* x;
  const void* w;
  const void* bias;
  void* D;
  void* Z;        // gated: receives [G | U], or null
  int64_t m, n;   // n: columns of D (gated: half the rows of W)
  int32_t k;
  int32_t vec;    // type of bias
  int32_t act;
};

// 16 x 16 products of 16 bytes of k per lane.
template <int DT>
__device__ __forceinline__ f32x4 mma_skinny(i32x4 a, i32x4 b, f32x4 c) {
  if constexpr (DT == BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else if constexpr (DT == F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(a[e]), __int_as_float(b[e]), c, 0, 0, 0);
    return c;
  }
}

// VEC: rows are whole, aligned 16-byte chunks.
template <int DT, bool GATED, int MT, bool VEC>
__global__ __launch_bounds__(512, MT == 4 ? 2 : MT == 2 ? 3 : 4) void skinny_kernel(SkinnyArgs p) {
  constexpr int NB = GATED ? 2 : 1, ES = Tr<DT>::es, E = 16 / ES, STEP = 256 / ES;
  extern __shared__ __attribute__((aligned(16))) f32x4 red[];   // [wave][NB MT][64]
  const int nw = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, li = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * (16 * MT);
  const int steps = (p.k + STEP - 1) / STEP;
  const int64_t ldb = (int64_t)p.k * ES;

  // (rows past the last one read the last one again: their results are not stored)
  const char* wb[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) wb[b] = static_cast<const char*>(p.w) + ((b ? p.n : 0) + c0) * ldb;
  const int row = (int)(c0 + li < p.n ? li : p.n - 1 - c0);
  const char* xb = static_cast<const char*>(p.x) + t0 * ldb;
  __amdgpu_buffer_rsrc_t rw[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) rw[b] = rsrc(wb[b]);
  const __amdgpu_buffer_rsrc_t rx = rsrc(xb);
  const uint32_t w_off = (uint32_t)(row * ldb) + q * 16;

  struct Step {
    i32x4 w[NB][4], x[MT][4];
  };
  const auto load = [&](Step& s, int t) {
    if constexpr (!VEC) {
      if ((t + 1) * STEP <= p.k) {   // (a whole step needs no shifts)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int kp = t * STEP + j * (STEP / 4) + q * E;
#pragma unroll
          for (int b = 0; b < NB; ++b) s.w[b][j] = load16(wb[b] + row * ldb + (int64_t)kp * ES);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            s.x[mt][j] = load16(xb + (t0 + mt * 16 + li < p.m ? mt * 16 + li : 0) * ldb + (int64_t)kp * ES);
        }
        return;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kp = t * STEP + j * (STEP / 4) + q * E;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (VEC) s.w[b][j] = __builtin_amdgcn_raw_buffer_load_b128(rw[b], kp < p.k ? w_off + j * 64 : kOOB, t * 256, 0);
        else s.w[b][j] = load_end<ES>(wb[b] + row * ldb, kp, p.k);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const bool in = t0 + mt * 16 + li < p.m;
        if constexpr (VEC) {
          const uint32_t off = in && kp < p.k ? (uint32_t)((mt * 16 + li) * ldb) + kp * ES : kOOB;
          s.x[mt][j] = __builtin_amdgcn_raw_buffer_load_b128(rx, off, 0, 0);
        } else {
          s.x[mt][j] = load_end<ES>(xb + (in ? mt * 16 + li : 0) * ldb, kp, p.k);   // (as above)
        }
      }
    }
  };
  f32x4 acc[NB][MT];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[b][mt] = f32x4{0, 0, 0, 0};
  const auto multiply = [&](const Step& s) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[b][mt] = mma_skinny<DT>(s.w[b][j], s.x[mt][j], acc[b][mt]);
  };

  Step s0, s1;
  if (w < steps) load(s0, w);
  for (int t = w; t < steps; t += 2 * nw) {
    if (t + nw < steps) load(s1, t + nw);
    __builtin_amdgcn_sched_barrier(0);
    multiply(s0);
    if (t + nw >= steps) break;
    if (t + 2 * nw < steps) load(s0, t + 2 * nw);
    __builtin_amdgcn_sched_barrier(0);
    multiply(s1);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) red[((w * NB + b) * MT + mt) * 64 + lane] = acc[b][mt];
  __syncthreads();

  // result r of lane l: column 4 (l / 16) + r of the row group, token l % 16
  for (int i = threadIdx.x; i < MT * 64; i += blockDim.x) {
    const int l = i & 63, mt = i / 64;
    const int64_t token = t0 + mt * 16 + (l & 15), col = c0 + (l >> 4) * 4, left = p.n - col;
    if (token >= p.m || left <= 0) continue;
    float v[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      f32x4 sum = red[(b * MT + mt) * 64 + l];
      for (int o = 1; o < nw; ++o) {
        const f32x4 u = red[((o * NB + b) * MT + mt) * 64 + l];
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] += u[r];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
        v[b][r] = sum[r] + (p.bias && r < left ? load_vec(p.bias, p.vec, (b ? p.n : 0) + col + r) : 0.0f);
    }
    if constexpr (GATED) {
      float h[4];
      with_gate(p.act, [&](auto a) {
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = gate_act<decltype(a)::value, DT == F32>(v[0][r]) * v[1][r];
      });
      store4<DT>(p.D, token * p.n + col, left, h);
      if (p.Z) {
        store4<DT>(p.Z, token * 2 * p.n + col, left, v[0]);
        store4<DT>(p.Z, token * 2 * p.n + p.n + col, left, v[1]);
      }
    } else {
      store4<DT>(p.D, token * p.n + col, left, v[0]);
    }
  }
}

}  // namespace gek
