// Tile kernel of the products with 4-bit weights (layout: w4_format.hpp): dozens to thousands of
// tokens.
//
// A workgroup computes BM tokens by 128 rows of W, in steps of 128 k ("pairs" of 64). Eight waves:
// four take 32 rows of W each (gated: 16 of the gate and the same 16 of the up projection), twice, for
// the even and the odd ones of a pair's eight products along k. A wave turns its own codes into the
// operand of v_mfma_f32_32x32x16 in registers, each code once in the workgroup, with no LDS between;
// lane l holds row l % 32 of W throughout: its codes, scales and sums. X is shared: it goes through
// registers into two LDS stages, with one barrier to a pair; X is loaded three pairs ahead of its use
// and W two, and no load stands behind a branch, so every wait leaves the younger ones on their way.
//
// What bounds it is instruction issue: turning eight codes into bf16 takes 19 vector instructions
// (f16: 11), and a group's factor one per sum, beside BM / 32 products. With W converted through LDS
// for both halves of the waves (w4_large.hpp's way) tiles of 128 x 128 took 156 us at 3000 x 4096 x
// 4096 bf16 (groups of 128) and 53 at 600 tokens, and tiles of 64 x 128 23 at 200 x 2 x 2752 x 2048 f16; in
// registers 137, 42 and 15.5.
//
// No weight is rounded: a scale s is split into a power of two p and f = s / p, and the operand is
// (q - z) p, exact in 16 bits. The sums are held in units of f: where a group of a row begins they
// are multiplied by the last group's f over the new one's (one fp32 multiplication per sum and
// group, no second set of sums), and by the last f at the end. p takes the whole exponent of s
// where (q - z) p stays a normal number, from 2^-14 to 2^11 in fp16 and 2^-126 to 2^124 in bf16, so f
// lies in [1, 2) but for scales out there: below 32 and 16, and not below 2^-10 and 2^-7 (subnormal
// scales). So the sums in units of f stay finite wherever the row's own stay below 2^120 (fp16: always).
#pragma once

#include "gemm_dtl.hpp"
#include "w4.hpp"

namespace gek {

// A scale in two: its power of two p (0 for 0, the scale itself if it is not finite), and f.
template <int DT>
__device__ __forceinline__ void w4_split(uint16_t bits, float& p, float& f) {
  const float s = Tr<DT>::widen(bits);
  const uint32_t e = __float_as_uint(s) & 0x7f800000u;
  constexpr uint32_t lo = (uint32_t)(127 - (DT == BF16 ? 126 : 14)) << 23, hi = (uint32_t)(127 + (DT == BF16 ? 124 : 11)) << 23;
  const uint32_t c = min(max(e, lo), hi);
  p = __uint_as_float(c);
  f = s * __uint_as_float((254u << 23) - c);
  if (s == 0.0f) {
    p = 0.0f;
    f = 1.0f;
  } else if (e == 0x7f800000u) {
    p = s;
    f = 1.0f;
  }
}

// p in a register's high half and z in its low byte. (p is a power of two, 0, or not finite: fp32
// with a 16-bit pattern.)
__device__ __forceinline__ uint32_t w4_pz(float p, uint32_t z) { return (__float_as_uint(p) & 0xffff0000u) | z; }

// The eight codes of a dword as (q - z) p, exact in 16 bits.
template <int DT>
__device__ __forceinline__ i32x4 w4_expand(uint32_t w, uint32_t pz) {
  const uint32_t h[2] = {w & 0x0f0f0f0fu, (w >> 4) & 0x0f0f0f0fu};
  const float p = __uint_as_float(pz & 0xffff0000u), nz = -(float)(pz & 0xffu) * p;
  i32x4 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (DT == F16) {
      typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
      const f16x2_t pp = {(_Float16)p, (_Float16)p}, zz = {(_Float16)nz, (_Float16)nz};
      const f16x2_t a = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(h[i], 512.0f, false));
      const f16x2_t b = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(h[i], 512.0f, true));
      o[2 * i] = __builtin_bit_cast(int, __builtin_elementwise_fma(a, pp, zz));
      o[2 * i + 1] = __builtin_bit_cast(int, __builtin_elementwise_fma(b, pp, zz));
    } else {
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(h[i], 512.0f, false);
      const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(h[i], 512.0f, true);
      o[2 * i] = (int)Tr<DT>::pack2(__builtin_fmaf(a[0], p, nz), __builtin_fmaf(a[1], p, nz));
      o[2 * i + 1] = (int)Tr<DT>::pack2(__builtin_fmaf(b[0], p, nz), __builtin_fmaf(b[1], p, nz));
    }
  }
  return o;
}

// Groups of a row in a pair: scales and zeros as loaded, and a pair's codes.
template <int E>
struct W4Raw {
  i32x4 c;
  uint32_t s[E], z[E];
};

// Epilogue of one 32 x 32 block (lane l: row l % 32 of W, register r: token 8 (r / 4) + 4 (l / 32) +
// r % 4) through 4 KB of fp32 scratch, so that a lane gets eight neighbouring columns of a token
// and memory sees whole pieces of rows at any alignment. Gated: columns 0 .. 15 are the gate's, 16 ..
// 31 the up projection's.
template <int DT, bool GATED>
__device__ __forceinline__ void w4_block(const W4Args& p, const f32x16& acc, int64_t m0, int64_t n0, int lane, char* scratch) {
  const int col = lane & 31, lhi = lane >> 5;
  const auto swz = [](int row) { return (row ^ (row >> 3)) & 7; };   // 16-byte units of 128-byte rows
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int row = 8 * (r / 4) + 4 * lhi + r % 4;
    *reinterpret_cast<float*>(scratch + row * 128 + (((col >> 2) ^ swz(row)) << 4) + (col & 3) * 4) = acc[r];
  }
  __builtin_amdgcn_wave_barrier();
  const auto get = [&](int row, int unit, float (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const f32x4 d = *reinterpret_cast<const f32x4*>(scratch + row * 128 + (((unit + u) ^ swz(row)) << 4));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * u + e] = d[e];
    }
  };
  constexpr int LPR = GATED ? 2 : 4, PASSES = GATED ? 1 : 2;   // lanes to a token
  const int c = lane % LPR;
  const int64_t at0 = n0 + 8 * c, left = p.n - at0;
  float bg[8], bu[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bg[e] = p.bias && e < left ? load_vec(p.bias, p.vec, at0 + e) : 0.0f;
    bu[e] = GATED && p.bias && e < left ? load_vec(p.bias, p.vec, p.n + at0 + e) : 0.0f;
  }
#pragma unroll
  for (int h = 0; h < PASSES; ++h) {
    const int row = h * (64 / LPR) + lane / LPR;
    const int64_t token = m0 + row;
    float y[8];
    get(row, 2 * c, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += bg[e];
    if constexpr (GATED) {
      float u[8];
      get(row, 4 + 2 * c, u);
      with_gate(p.ep, [&](auto act) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = gate_act<decltype(act)::value, false>(y[e]) * (u[e] + bu[e]);
      });
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = act_ep(y[e], p.ep);
    }
    if (token < p.m && left > 0) {
      const int64_t at = token * p.n + at0;
      const float y0[4] = {y[0], y[1], y[2], y[3]}, y1[4] = {y[4], y[5], y[6], y[7]};
      if (p.out == F32) {
        store4<F32>(p.D, at, left, y0);
        store4<F32>(p.D, at + 4, left - 4, y1);
      } else if (left >= 8) {
        const i32x4 o = {(int)Tr<DT>::pack2(y[0], y[1]), (int)Tr<DT>::pack2(y[2], y[3]), (int)Tr<DT>::pack2(y[4], y[5]),
                         (int)Tr<DT>::pack2(y[6], y[7])};
        __builtin_memcpy(static_cast<uint16_t*>(p.D) + at, &o, 16);
      } else {
        store4<DT>(p.D, at, left, y0);
        store4<DT>(p.D, at + 4, left - 4, y1);
      }
    }
  }
  __builtin_amdgcn_wave_barrier();
}

// E: groups of a row in a pair: 4 (of 32), 2 (of 64), 1 (of 128 and more). X's rows may have any
// alignment: the memory pipe takes 16-byte loads at it.
template <int DT, bool GATED, int BM, int E>
__global__ __launch_bounds__(512, 2) void w4_tile_kernel(W4Args p, W4Launch L) {
  constexpr int MB = BM / 32, XI = BM * 16 / 512, STAGE = BM * 256;
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wn = w & 3, kg = w >> 2;
  const int lrow = lane & 31, lhi = lane >> 5;
  int tm, tn;
  {
    Args r;
    r.tiles_m = L.tiles_m;
    r.tiles_n = L.tiles_n;
    r.group_m = L.group_m;
    raster(r, xcd_remap(blockIdx.x, L.tiles_m * L.tiles_n), tm, tn);
  }
  const int64_t m0 = (int64_t)tm * BM;
  const int n0 = tn * (GATED ? 64 : 128) + wn * (GATED ? 16 : 32);   // this wave's first column
  const int KP = p.kt;

  // ---- X: chunk i of a thread is chunk tid % 16 of row tid / 16 + 32 i of the pair ----
  // Every load happens (one that may not would turn the later waits into waits for all that are on
  // their way): past the last pair it is the last again, and where k ends in a chunk, or before it,
  // the row's last eight elements are loaded and moved down (k >= 8).
  const char* xb = static_cast<const char*>(p.x) + m0 * p.k * 2;
  const int over = max(0, (KP - 1) * 128 + (tid & 15) * 8 + 8 - p.k);   // of the last pair's chunk past k
  uint32_t x_off[XI];
  int x_lds[XI];
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int row = tid / 16 + 32 * i, c = tid & 15;
    const int at = (int)(m0 + row < p.m ? row : p.m - 1 - m0);   // (tokens past the last one are not stored)
    x_off[i] = (uint32_t)(at * (p.k * 2)) + c * 16;
    x_lds[i] = (c >> 3) * (BM * 128) + row * 128 + (((c & 7) ^ swz_a<128>(row)) << 4);
  }
  i32x4 xr[2][XI];
  auto load_x = [&](i32x4 (&r)[XI], int pair) {
    const char* at = xb + (int64_t)min(pair, KP - 1) * 256 - (pair < KP - 1 ? 0 : 2 * over);
#pragma unroll
    for (int i = 0; i < XI; ++i) r[i] = load16(at + x_off[i]);
  };
  auto store_x = [&](i32x4 (&r)[XI], int stage, int pair) {
    if (pair == KP - 1 && p.k % 128) {
#pragma unroll
      for (int i = 0; i < XI; ++i) r[i] = shift_down<2>(r[i], min(over, 8));
    }
#pragma unroll
    for (int i = 0; i < XI; ++i) *reinterpret_cast<i32x4*>(smem + stage * STAGE + x_lds[i]) = r[i];
  };

  // ---- W: this lane's row ----
  const int in = n0 / 16 + (GATED ? 0 : lrow >> 4);
  const int64_t rg = (in < p.rgs ? in : p.rgs - 1) + (GATED && lrow >= 16 ? (int64_t)p.rgs : 0);
  const char* cp = p.codes + rg * p.kt * kTileBytes + ((lane & 15) + 16 * (2 * kg + lhi)) * 16;
  const uint16_t* sp = p.scales + rg * p.groups * kRows + (lane & 15);
  const uint8_t* zp = p.zeros + rg * p.groups * kRows + (lane & 15);
  using Raw = W4Raw<E>;
  int group = 0, loaded = 0, begun = 0;   // (E 1) of the pair loaded next; pairs loaded, and used, of its group
  auto load_w = [&](Raw& d, int pair) {   // in order; past the last pair, the last one again
    d.c = *reinterpret_cast<const i32x4*>(cp + (int64_t)(pair < KP ? pair : KP - 1) * kTileBytes);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int g = min(E == 1 ? group : pair * E + e, p.groups - 1);
      d.s[e] = sp[(int64_t)g * kRows];
      d.z[e] = zp[(int64_t)g * kRows];
    }
    if (E == 1 && ++loaded == p.span) {
      loaded = 0;
      ++group;
    }
  };
  float f = 1.0f;   // of the group multiplied last

  // ---- fragments of X: own k-step i is step 2 i + kg of the pair ----
  const int rd = lrow * 128;
  auto read = [&](i32x4 (&fr)[MB], int stage, int i) {
    const int c = 2 * i + kg;   // 16-k step of the pair: chunks 2 (c % 4) and the next of half c / 4
    const char* at = smem + stage * STAGE + (c >> 2) * (BM * 128) + rd + (((2 * (c & 3) + lhi) ^ swz_a<128>(lrow)) << 4);
#pragma unroll
    for (int b = 0; b < MB; ++b) fr[b] = *reinterpret_cast<const i32x4*>(at + b * 32 * 128);
  };
  f32x16 acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = f32x16{};

  Raw raw[2];
  load_x(xr[1], 0);   // (in the loop's order, so that its waits hold here too)
  load_x(xr[0], 1);
  load_w(raw[0], 0);
  store_x(xr[1], 0, 0);
  load_x(xr[1], 2);
  load_w(raw[1], 1);
  wait_lgkmcnt<0>();
  barrier_only();

  auto pair_step = [&](auto utag, int P) {   // pair P, P % 2 == u
    constexpr int u = decltype(utag)::value;
    // the next pair to the other stage, later ones on their way
    const Raw now = raw[u];
    store_x(xr[u], u ^ 1, P + 1);
    load_x(xr[u], P + 3);
    load_w(raw[u], P + 2);
    // the groups' p, z and factors
    uint32_t pz[E];
    float ratio[E];
    const bool begins = E > 1 || begun == 0;
    if (E == 1 && ++begun == p.span) begun = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      uint32_t sb = now.s[e], zb = now.z[e];
      asm volatile("" : "+v"(sb), "+v"(zb));   // (or they are narrowed, and waited for, where they are loaded)
      float pw, fn;
      w4_split<DT>((uint16_t)sb, pw, fn);
      pz[e] = w4_pz(pw, zb);
      ratio[e] = begins ? f * __builtin_amdgcn_rcpf(fn) : 1.0f;
      f = begins ? fn : f;
    }
    i32x4 fr[2][MB];   // (the next step's beside this one's products)
    read(fr[0], u, 0);
    w4_for<4>([&](auto itag) {
      constexpr int i = decltype(itag)::value;
      if constexpr (i < 3) read(fr[(i + 1) & 1], u, i + 1);
      constexpr int e = E == 4 ? i : E == 2 ? i / 2 : 0;
      const i32x4 wf = w4_expand<DT>((uint32_t)now.c[i], pz[e]);
      if constexpr (E == 4 || (E == 2 && i % 2 == 0) || i == 0) {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[b][j] *= ratio[e];
      }
#pragma unroll
      for (int b = 0; b < MB; ++b) acc[b] = Tr<DT>::mma(fr[i & 1][b], wf, acc[b]);
    });
    wait_lgkmcnt<0>();   // reads of this stage, writes of the other
    barrier_only();
  };
  int P = 0;
  for (; P + 1 < KP; P += 2) {
    pair_step(std::integral_constant<int, 0>{}, P);
    pair_step(std::integral_constant<int, 1>{}, P + 1);
  }
  if (P < KP) pair_step(std::integral_constant<int, 0>{}, P);

  // ---- the sums of the two waves of the same rows: each finishes half of the tokens ----
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[b][j] *= f;
  constexpr int HB = MB / 2;
  f32x4* theirs = reinterpret_cast<f32x4*>(smem + ((kg ^ 1) * 4 + wn) * (HB * 4096)) + lane;
  char* mine = smem + w * (HB * 4096);
#pragma unroll
  for (int b = 0; b < HB; ++b)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = kg ? acc[b][4 * c + e] : acc[HB + b][4 * c + e];
      theirs[(b * 4 + c) * 64] = v;
    }
  __syncthreads();
  f32x16 sum[HB];
#pragma unroll
  for (int b = 0; b < HB; ++b)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const f32x4 v = reinterpret_cast<const f32x4*>(mine)[(b * 4 + c) * 64 + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[b][4 * c + e] = (kg ? acc[HB + b][4 * c + e] : acc[b][4 * c + e]) + v[e];
    }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int b = 0; b < HB; ++b)
    w4_block<DT, GATED>(p, sum[b], m0 + (kg * HB + b) * 32, n0, lane, mine);
}

}  // namespace gek
