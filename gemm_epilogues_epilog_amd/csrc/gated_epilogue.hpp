// Epilogues of the gated feed-forward block on a wave's accumulators, through its LDS scratch:
//   GATED   the wave's WN tile columns are WN / 2 of the gate and the same WN / 2 of the up
//           projection (blocks a and a + NB / 2 hold the same columns): H = act(G) * U, and Z =
//           [G | U] if wanted;
//   DGATED  the accumulators are dH: with G and U read from Z, dZ = [dH U a'(G) | dH a(G)], and the
//           sums of its columns, for the bias, before its rounding.
// Lane l holds row l % 32 of a block, register r column 8 (r / 4) + 4 (l / 32) + r % 4 (kernels.hpp).
// 32 rows at a time go through 32 WN bytes (GATED) or 4 KB (DGATED) of scratch, so that memory
// sees 16 bytes a lane and whole pieces of rows.
//
// dZ leaves rounded to the operands' type, as the matrix instruction takes it in dX and dW: half a step
// of each term, independently, which adds as much to those gradients as their own rounding (root mean
// square error against 64 bits: bf16 2.35e-3 instead of 1.66e-3, fp16 2.95e-4 instead of 2.09e-4). Two
// 16-bit parts would keep fp32 and double two products of three.
//
// The product bounds both: 4096 x 2 x 11008 x 4096 bf16 592 us, 1250 TFLOP/s (the plain product with a
// bias and ReLU at 4096 x 11008 x 4096: 1230), its matrix unit busy 76% of the cycles; dZ at 2048 x
// 11008 x 4096 226 us in tiles of 192 x 256.
#pragma once

#include <type_traits>

#include "gated_math.hpp"
#include "tiles.hpp"

namespace gek {

// Scratch rows of C 16-bit values: 8-byte units, unit u of row r at u ^ swz(r), so that the 32
// rows of a half-wave's write spread over all banks; a 16-byte pair of units reads back at
// c ^ (swz / 2), its halves swapped where swz is odd.
template <int C>
struct GatedRows {
  static constexpr int RB = C * 2, LPR = RB / 16, RPI = 64 / LPR, NR = 32 / RPI;
  static_assert(C == 32 || C == 64, "row width");
  __device__ static __forceinline__ int swz(int row) { return C == 64 ? (row >> 1) & 15 : (row >> 2) & 7; }
  __device__ static __forceinline__ void put(char* scratch, int row, int unit, i32x2 v) {
    *reinterpret_cast<i32x2*>(scratch + row * RB + ((unit ^ swz(row)) << 3)) = v;
  }
  __device__ static __forceinline__ i32x4 get(const char* scratch, int row, int c) {
    const int s = swz(row);
    const i32x4 v = *reinterpret_cast<const i32x4*>(scratch + row * RB + ((c ^ (s >> 1)) << 4));
    return (s & 1) ? i32x4{v[2], v[3], v[0], v[1]} : v;
  }
};

// 32 rows from row m0 on of `scratch`, columns c0 .. c0 + C - 1 of a matrix with `ld` values to a
// row and `cols` columns from its base on.
template <int C>
__device__ __forceinline__ void gated_store(const char* scratch, void* base, int64_t m0, int64_t m, int64_t ld, int c0,
                                            int cols, int lane) {
  using L = GatedRows<C>;
  const __amdgpu_buffer_rsrc_t rd = rsrc(static_cast<char*>(base) + (m0 * ld + c0) * 2);
  const int c = lane % L::LPR;
  i32x4 v[L::NR];
#pragma unroll
  for (int i = 0; i < L::NR; ++i) v[i] = L::get(scratch, i * L::RPI + lane / L::LPR, c);
#pragma unroll
  for (int i = 0; i < L::NR; ++i) {
    const int row = i * L::RPI + lane / L::LPR;
    const bool ok = c0 + 8 * c < cols && m0 + row < m;
    const uint32_t off = ok ? (uint32_t)((row * ld + 8 * c) * 2) : kOOB;
    __builtin_amdgcn_raw_buffer_store_b128(v[i], rd, off, 0, 2 /* streamed, as D of the other epilogues */);
  }
}

// Adds the bias to a wave's sums. The columns' values go through the scratch as fp32, so that each
// lane reads the four of a register group at once (loading them straight from memory, by type,
// took the registers of the main loop: 203 spilled).
template <int MB, int NB>
__device__ __forceinline__ void gated_bias(const Args& p, f32x16 (&acc)[NB][MB], int h0, int lane, char* scratch) {
  constexpr int C = NB * 16;   // columns of each half
  float* v = reinterpret_cast<float*>(scratch);
  if (lane < C) {
    const int col = h0 + lane;
    v[lane] = col < p.n ? load_vec(p.bias, p.vec_dt, col) : 0.0f;
    v[C + lane] = col < p.n ? load_vec(p.bias, p.vec_dt, (int64_t)p.n + col) : 0.0f;
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int a = 0; a < NB; ++a)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(v + 32 * a + 8 * g + 4 * (lane >> 5));
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[a][b][4 * g + e] += u[e];
    }
  __builtin_amdgcn_wave_barrier();
}

// Block b of 32 rows; h0 is the wave's first column of H.
template <int DT, int MB, int NB>
__device__ __forceinline__ void gated_block(const Args& p, const f32x16 (&acc)[NB][MB], int b, int64_t m0, int h0, int lane,
                                            char* scratch) {
  using T = Tr<DT>;
  constexpr int NH = NB / 2, C = NH * 32;
  using L = GatedRows<C>;
  static_assert(NB % 2 == 0, "gate and up blocks");
  const int N = p.n, lrow = lane & 31, lhi = lane >> 5;
  m0 += 32 * b;
  const auto put = [&](int a, int g, const float (&v)[4]) {
    L::put(scratch, lrow, 8 * a + 2 * g + lhi, i32x2{(int)T::pack2(v[0], v[1]), (int)T::pack2(v[2], v[3])});
  };
  with_gate(p.act, [&](auto act) {
#pragma unroll
    for (int a = 0; a < NH; ++a)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h[e] = gate_act<decltype(act)::value, false>(acc[a][b][4 * g + e]) * acc[a + NH][b][4 * g + e];
        put(a, g, h);
      }
  });
  gated_store<C>(scratch, p.D, m0, p.m, N, h0, N, lane);
  if (p.z_out) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int a = 0; a < NH; ++a)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16& v = acc[a + half * NH][b];
          put(a, g, {v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]});
        }
      gated_store<C>(scratch, static_cast<char*>(p.z_out) + (int64_t)half * N * 2, m0, p.m, 2 * (int64_t)N, h0, N, lane);
    }
  }
}

// The whole wave tile of dH, 32 x 32 at a time; Z of the next block is on its way meanwhile. The
// first workgroup also clears the flags of the next product's split (every wave the same zeros):
// a launch less (77 x 1000 x 520 f16: 38.6 -> 37.6 us).
template <int DT, int MB, int NB>
__device__ __forceinline__ void dgated_tile(const Args& p, const f32x16 (&acc)[NB][MB], int64_t m0, int n0, int lane,
                                            char* scratch) {
  using T = Tr<DT>;
  const int N = p.n, lrow = lane & 31, lhi = lane >> 5;
  const int64_t ld = 2 * (int64_t)N;
  const int r16 = lane >> 2, c = lane & 3;   // this lane's row (and row + 16) and 8 columns in memory
  struct Z {
    i32x4 g[2], u[2];
  };
  const auto offset = [&](int b, int a, int h) {
    const int row = 16 * h + r16;
    const bool ok = m0 + 32 * b + row < p.m && n0 + 32 * a + 8 * c < N;
    return ok ? (uint32_t)((row * ld + 8 * c) * 2) : kOOB;
  };
  const auto load = [&](int i, Z& z) {
    const int b = i / NB, a = i % NB;
    const char* at = static_cast<const char*>(p.z) + ((m0 + 32 * b) * ld + n0 + 32 * a) * 2;
    const __amdgpu_buffer_rsrc_t rg = rsrc(at), ru = rsrc(at + (int64_t)N * 2);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      z.g[h] = __builtin_amdgcn_raw_buffer_load_b128(rg, offset(b, a, h), 0, 0);
      z.u[h] = __builtin_amdgcn_raw_buffer_load_b128(ru, offset(b, a, h), 0, 0);
    }
  };
  const auto swz = [](int row) { return (row ^ (row >> 3)) & 7; };   // 16-byte units of 128-byte rows
  float sum[NB] = {};   // of the column r16 of dG's eight, then of dU's, of this lane's chunk c
  Z z[2];
  load(0, z[0]);
  if (p.clear && blockIdx.x == 0)
    for (int i = lane; i < kSkFlagWords; i += 64) p.clear[i] = 0;
#pragma unroll
  for (int i = 0; i < MB * NB; ++i) {
    const int b = i / NB, a = i % NB;
    if (i + 1 < MB * NB) load(i + 1, z[(i + 1) & 1]);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x16& v = acc[a][b];
      *reinterpret_cast<f32x4*>(scratch + lrow * 128 + (((2 * g + lhi) ^ swz(lrow)) << 4)) =
          f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
    }
    char* at = static_cast<char*>(p.D) + ((m0 + 32 * b) * ld + n0 + 32 * a) * 2;
    const __amdgpu_buffer_rsrc_t rg = rsrc(at), ru = rsrc(at + (int64_t)N * 2);
    const Z& zi = z[i & 1];
    float t[16] = {};   // dG and dU of this lane's two rows
    with_gate(p.act, [&](auto act) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = m0 + 32 * b + 16 * h + r16 < p.m;   // (a row past the last one is NaN where Wd is)
        f32x4 d[2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
          d[q] = *reinterpret_cast<const f32x4*>(scratch + (16 * h + r16) * 128 + (((2 * c + q) ^ swz(16 * h + r16)) << 4));
        i32x4 og, ou;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float dg[2], du[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float gv = T::widen((uint16_t)((uint32_t)zi.g[h][w] >> (16 * e)));
            const float uv = T::widen((uint16_t)((uint32_t)zi.u[h][w] >> (16 * e)));
            const float dh = d[w / 2][2 * (w % 2) + e];
            float v, s;
            gate_slope<decltype(act)::value, false>(gv, v, s);
            dg[e] = dh * uv * s;
            du[e] = dh * v;
            t[2 * w + e] += in ? dg[e] : 0.0f;
            t[8 + 2 * w + e] += in ? du[e] : 0.0f;
          }
          og[w] = (int)T::pack2(dg[0], dg[1]);
          ou[w] = (int)T::pack2(du[0], du[1]);
        }
        __builtin_amdgcn_raw_buffer_store_b128(og, rg, offset(b, a, h), 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(ou, ru, offset(b, a, h), 0, 0);
      }
    });
    if (p.sums) {
      // the 16 lanes of the same columns: each step a lane hands half of its values to the lane that
      // keeps those, and takes its own, until it has one of all rows
#pragma unroll
      for (int h = 8; h > 0; h >>= 1) {
        const bool up = (r16 & h) != 0;
#pragma unroll
        for (int j = 0; j < h; ++j) {
          const float give = up ? t[j] : t[j + h];
          t[j] = (up ? t[j + h] : t[j]) + __shfl_xor(give, 4 * h);
        }
      }
      sum[a] += t[0];
      if (b == MB - 1 && n0 + 32 * a + 8 * c < N)
        p.sums[m0 / (32 * MB) * ld + (r16 & 8 ? N : 0) + n0 + 32 * a + 8 * c + (r16 & 7)] = sum[a];
    }
  }
}

}  // namespace gek
