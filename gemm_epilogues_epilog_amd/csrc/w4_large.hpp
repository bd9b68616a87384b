// Tile kernel of the products with 4-bit weights for thousands of tokens (layout: w4_format.hpp; the
// numbers (q - z) p and the units of the sums: w4_tile.hpp).
//
// A 256 x 256 or 192 x 256 tile of D, k in tiles of 64. X goes straight into LDS; W's codes go through registers,
// each once per workgroup, and lie in LDS as 16-bit numbers in the same k-major order. The two
// operands then meet in v_mfma_f32_32x32x16 as in the 16-bit kernels (gemm_dtl.hpp). A code is
// converted once per 256 tokens and a sum multiplied as often as in the smaller tiles, so this is
// the kernel where there is work for every compute unit. bf16 with groups of 128, tiles of 256, of 192
// and of 128 x 128: 3000 x 4096 x 4096 112, 107 and 136 us (groups of 64: 135, 121 and 159), 4096
// tokens 131, 186 and 187, 600 tokens 98, 86 and 44. X's rows are whole 16-byte chunks, and groups
// hold at least 64 (of 32 the factors do not fit the registers).
//
// The matrix unit is busy 37% of the cycles (192 x 256 at 3000 x 4096 x 4096, groups of 64): of the 4200 that
// a k-tile takes on a SIMD, 1540 are its two waves' products and about 1800 their vector instructions
// (conversions, and factors on the sums). All waves go through the same phases between two barriers,
// which leaves the rest to waiting.
//
// At the end of k-tile t every wave waits until its copies of X's tile t + 1 have landed and its
// reads of tile t and its writes of W's tile t + 1 are done; one barrier publishes tile t + 1 and
// releases tile t's stages, which X's tile t + 2 is copied into and, during the products of t + 1,
// W's tile t + 2 is converted into. Codes, scales and zeros come two k-tiles at a time, a pair
// ahead, through LDS as well (each wave its own), so that every wait in the loop is for copies
// whose number the kernel knows: registers loaded that early would be waited for by the compiler,
// which does not see the copies of X between them.
#pragma once

#include "w4_tile.hpp"

namespace gek {

template <int BM_>
struct W4Large {
  static constexpr int BM = BM_, BN = 256, WM = BM / 2, WN = 64;
  static constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN, NW = WAVES_M * WAVES_N, NT = NW * 64;
  static constexpr int MB = WM / 32, NB = WN / 32;
  static constexpr int X_BYTES = BM * 128, W_BYTES = BN * 128, OFF_W = 2 * X_BYTES;   // (two stages of each)
  static constexpr int XI = X_BYTES / 1024 / NW;      // copies of X per wave and k-tile
  static constexpr int RG = BN / 16 / NW;             // row groups that a wave converts
  static constexpr int CODES = RG * 1024 + 512;       // a pair's codes, scales and zeros of one wave
  static constexpr int OFF_R = OFF_W + 2 * W_BYTES;   // factors of the sums: [stage][BN]
  static constexpr int OFF_C = OFF_R + 2 * BN * 4;
  static constexpr int EPI = 8192;                    // epilogue bytes per wave (in the stages)
  static constexpr int LDS = OFF_C + NW * CODES;
  static_assert(X_BYTES % (1024 * NW) == 0 && WM % 32 == 0, "shares of a wave");
  static_assert(NW * EPI <= OFF_R && LDS <= 160 * 1024, "LDS");
};

// Waits whose place among the loads and copies the compiler keeps.
template <int N>
__device__ __forceinline__ void w4_wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}

// A pair of k-tiles of RG row groups, E groups of k to a row in it: codes, and of each group p and z
// and the factor that brings the sums into its units.
template <int RG, int E>
struct W4Codes {
  i32x4 c[RG];
  uint32_t pz[RG][E];
  float ratio[RG][E];
};

// 4 bytes per lane, as copy_to_lds_b128.
__device__ __forceinline__ void copy_to_lds_b32(const i32x4& srd, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(srd), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory", "m0");
}

// Epilogue: 32 x 32 blocks of sums through fp32 scratch (gated: one of the gate and one of the up
// projection), so that a lane gets eight neighbouring columns of a token and memory sees whole
// pieces of rows at any alignment.
template <int DT, bool GATED, class C>
__device__ __forceinline__ void w4_large_epilogue(const W4Args& p, const f32x16 (&acc)[C::NB][C::MB], int64_t m0, int n0,
                                                 int lane, char* scratch) {
  constexpr int NH = GATED ? C::NB / 2 : C::NB;
  const int lrow = lane & 31, lhi = lane >> 5, r16 = lane >> 2, c = lane & 3;
  const auto swz = [](int row) { return (row ^ (row >> 3)) & 7; };   // 16-byte units of 128-byte rows
  const auto put = [&](const f32x16& v, char* to) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<f32x4*>(to + lrow * 128 + (((2 * g + lhi) ^ swz(lrow)) << 4)) =
          f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
  };
  const auto get = [&](const char* from, int h, float (&v)[8]) {
    const int row = 16 * h + r16;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const f32x4 d = *reinterpret_cast<const f32x4*>(from + row * 128 + (((2 * c + u) ^ swz(row)) << 4));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * u + e] = d[e];
    }
  };
#pragma unroll
  for (int a = 0; a < NH; ++a) {
    const int64_t col = n0 + 32 * a + 8 * c, left = p.n - col;
    float bg[8], bu[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      bg[e] = p.bias && e < left ? load_vec(p.bias, p.vec, col + e) : 0.0f;
      bu[e] = GATED && p.bias && e < left ? load_vec(p.bias, p.vec, p.n + col + e) : 0.0f;
    }
#pragma unroll
    for (int b = 0; b < C::MB; ++b) {
      put(acc[a][b], scratch);
      if constexpr (GATED) put(acc[a + NH][b], scratch + 4096);
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t token = m0 + 32 * b + 16 * h + r16;
        float y[8];
        get(scratch, h, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += bg[e];
        if constexpr (GATED) {
          float u[8];
          get(scratch + 4096, h, u);
          with_gate(p.ep, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = gate_act<decltype(act)::value, false>(y[e]) * (u[e] + bu[e]);
          });
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = act_ep(y[e], p.ep);
        }
        if (token < p.m && left > 0) {
          const int64_t at = token * p.n + col;
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
  }
}

// E: groups of a row in a pair of k-tiles: 2 (of 64), 1 (of 128 and more).
template <int DT, bool GATED, int BM, int E>
__global__ __launch_bounds__(512, 2) void w4_large_kernel(W4Args p, W4Launch L) {
  using C = W4Large<BM>;
  constexpr int BN = C::BN, WM = C::WM, WN = C::WN, MB = C::MB, NB = C::NB, RG = C::RG, XI = C::XI;
  constexpr int NCODE = RG + 2, NMMA = MB * NB;
  static_assert(E == 1 || E == 2, "groups");
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w % C::WAVES_M, wn = w / C::WAVES_M;
  const int li = lane & 15, q = lane >> 4, lhi = lane >> 5;
  int tm, tn;
  {
    Args r;
    r.tiles_m = L.tiles_m;
    r.tiles_n = L.tiles_n;
    r.group_m = L.group_m;
    raster(r, xcd_remap(blockIdx.x, L.tiles_m * L.tiles_n), tm, tn);
  }
  const int64_t m0 = (int64_t)tm * BM;
  const int n0 = tn * (GATED ? BN / 2 : BN);
  const int KT = (p.k + 63) / 64, KT2 = (KT + 1) & ~1;
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_void*)smem;

  // ---- X ----
  uint32_t x_src[XI];
  int x_chunk[XI];
  const char* xb = static_cast<const char*>(p.x) + m0 * p.k * 2;
#pragma unroll
  for (int j = 0; j < XI; ++j) {
    const int row = (w * XI + j) * 8 + lane / 8;
    x_chunk[j] = (lane % 8) ^ swz_a<128>(row);
    x_src[j] = m0 + row < p.m ? (uint32_t)(row * p.k * 2 + x_chunk[j] * 16) : kOOB;
  }
  auto issue_x = [&](int t) {
    const int k0 = t * 64;
    // (a k-tile past the last one reads nothing: zeros)
    const i32x4 srd = make_srd(xb + (int64_t)k0 * 2, t < KT ? 0x7fffffffu : 0u);
    const bool tail = k0 + 64 > p.k;
#pragma unroll
    for (int j = 0; j < XI; ++j) {
      const uint32_t off = tail && k0 + x_chunk[j] * 8 >= p.k ? kOOB : x_src[j];
      copy_to_lds_b128(srd, off, lds + (t & 1) * C::X_BYTES + (w * XI + j) * 1024);
    }
  };

  // ---- W ----
  // Tile row groups of this wave: w RG .. + RG - 1; of a gated tile, pairs of groups alternate
  // between the halves, so that each wave column has 32 rows of both.
  const int first = w * RG;
  const int in0 = n0 / 16 + (GATED ? first / 4 * 2 + first % 2 : first);   // (RG of them follow each other)
  const int on = max(0, min(RG, p.rgs - in0));
  const int64_t rg0 = (on > 0 ? in0 : 0) + (GATED && first / 2 % 2 ? (int64_t)p.rgs : 0);
  const char* cb = p.codes + rg0 * p.kt * kTileBytes;
  const i32x4 srd_s = make_srd(p.scales + rg0 * p.groups * kRows), srd_z = make_srd(p.zeros + rg0 * p.groups * kRows);
  // this lane's dword of the scales and of the zeros: row group, entry, place
  const int s_r = lane / (8 * E), s_e = lane / 8 % E, z_r = lane / (4 * E), z_e = lane / 4 % E;
  const uint32_t s_off = s_r < on ? (uint32_t)(s_r * p.groups * 32 + lane % 8 * 4) : kOOB;
  const uint32_t z_off = z_r < on ? (uint32_t)(z_r * p.groups * 16 + lane % 4 * 4) : kOOB;
  const uint32_t lds_c = lds + C::OFF_C + w * C::CODES;
  // pairs to a group (E 1); the group of the pair copied next and its pairs copied; pairs read of theirs
  const int span = E == 1 ? p.group / 128 : 1;
  int next_group = 0, copied = 0, begun = 0;
  auto copy_w = [&](int pair) {   // k-tiles 2 pair and 2 pair + 1, in order
    const bool in = pair < p.kt;
#pragma unroll
    for (int r = 0; r < RG; ++r)
      copy_to_lds_b128(make_srd(cb + ((int64_t)r * p.kt + pair) * kTileBytes, in && r < on ? kTileBytes : 0u), lane * 16, lds_c + r * 1024);
    // group of this lane's dwords (E 1: the pairs of a group follow each other)
    const int gs = E == 1 ? next_group : pair * E + s_e, gz = E == 1 ? next_group : pair * E + z_e;
    copy_to_lds_b32(srd_s, gs < p.groups ? s_off + (s_off == kOOB ? 0u : gs * 32) : kOOB, lds_c + RG * 1024);
    copy_to_lds_b32(srd_z, gz < p.groups ? z_off + (z_off == kOOB ? 0u : gz * 16) : kOOB, lds_c + RG * 1024 + 256);
    if (E == 1 && ++copied == span) {
      copied = 0;
      ++next_group;
    }
  };
  using Codes = W4Codes<RG, E>;
  float f[RG];   // of the group read last
#pragma unroll
  for (int r = 0; r < RG; ++r) f[r] = 1.0f;
  auto read_w = [&](Codes& d, int pair) {
    const char* at = smem + C::OFF_C + w * C::CODES;
    // past the last pair, and inside a group of several, the units stay as they are
    bool in = 2 * pair < KT2;
    if (E == 1) {
      in = in && begun == 0;
      if (++begun == span) begun = 0;
    }
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      d.c[r] = *reinterpret_cast<const i32x4*>(at + r * 1024 + lane * 16);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float p, fn;
        w4_split<DT>(*reinterpret_cast<const uint16_t*>(at + RG * 1024 + ((r * E + e) * 16 + li) * 2), p, fn);
        d.pz[r][e] = w4_pz(p, *reinterpret_cast<const uint8_t*>(at + RG * 1024 + 256 + (r * E + e) * 16 + li));
        d.ratio[r][e] = in ? f[r] * __builtin_amdgcn_rcpf(fn) : 1.0f;
        f[r] = in ? fn : f[r];
      }
    }
  };
  // Converts dword i of this wave's 2 RG per k-tile into the stage of a k-tile of parity par: row
  // group i / 2, dword 2 par + i % 2. No branches, so that it runs among the products. (The four
  // lanes of a row write the same factor.)
  auto convert = [&](const Codes& d, auto ptag, auto itag) {
    constexpr int par = decltype(ptag)::value, i = decltype(itag)::value, r = i / 2, h = i % 2;
    constexpr int g = E == 2 ? par : 0;
    const int row = (w * RG + r) * 16 + li;   // of the tile
    char* st = smem + C::OFF_W + par * C::W_BYTES + row * 128;
    *reinterpret_cast<i32x4*>(st + (((4 * h + q) ^ swz_a<128>(row)) << 4)) = w4_expand<DT>((uint32_t)d.c[r][2 * par + h], d.pz[r][g]);
    if constexpr (h == 0 && (E == 2 || par == 0)) reinterpret_cast<float*>(smem + C::OFF_R)[par * BN + row] = d.ratio[r][g];
  };

  // ---- fragments ----
  int rd_x[4], rd_w[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int row = lane & 31, chunk = (s * 2 + lhi) ^ swz_a<128>(row);
    rd_x[s] = (wm * WM + row) * 128 + (chunk << 4);
    rd_w[s] = C::OFF_W + (wn * WN + row) * 128 + (chunk << 4);
  }
  f32x16 acc[NB][MB];
#pragma unroll
  for (int a = 0; a < NB; ++a)
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[a][b] = f32x16{};
  // Multiplies the sums by the factors of a k-tile of this parity.
  auto rescale = [&](int par) {
    const float* R = reinterpret_cast<const float*>(smem + C::OFF_R) + par * BN + wn * WN + 4 * lhi;
#pragma unroll
    for (int a = 0; a < NB; ++a) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(R + 32 * a + 8 * c);
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[a][b][4 * c + e] *= v[e];
      }
    }
  };
  struct Frag {
    i32x4 x[MB], w[NB];
  };
  auto read = [&](Frag& fr, auto ptag, int s) {
    constexpr int par = decltype(ptag)::value;
#pragma unroll
    for (int a = 0; a < NB; ++a)
      fr.w[a] = *reinterpret_cast<const i32x4*>(smem + par * C::W_BYTES + rd_w[s] + a * 32 * 128);
    const char* x = smem + par * C::X_BYTES;
#pragma unroll
    for (int b = 0; b < MB; ++b) fr.x[b] = *reinterpret_cast<const i32x4*>(x + rd_x[s] + b * 32 * 128);
  };

  constexpr std::integral_constant<int, 0> p0{};
  constexpr std::integral_constant<int, 1> p1{};
  Codes now;   // of the pair being converted
  copy_w(0);
  issue_x(0);
  issue_x(1);
  w4_wait_vm<0>();
  read_w(now, 0);
  w4_for<2 * RG>([&](auto i) { convert(now, p0, i); });
  w4_for<2 * RG>([&](auto i) { convert(now, p1, i); });
  wait_lgkmcnt<0>();
  barrier_only();
  copy_w(1);
  Frag fr[2];
  read(fr[0], p0, 0);

  // One k-step of k-tile t, t % 2 == u: reads of the next step's fragments, a part of the next
  // k-tile's (in the last step, of the next but one's) conversion, and with SCALE the factors, all
  // among the products.
  auto step = [&](auto utag, auto stag, auto scale_tag, int t) {
    constexpr int u = decltype(utag)::value, s = decltype(stag)::value;
    constexpr bool last = s == 3, SCALE = decltype(scale_tag)::value;
    constexpr std::integral_constant<int, u ^ 1> other{};
    if constexpr (SCALE) rescale(u);
    if constexpr (u == 1 && s == 0) {   // the pair read at the end of the last k-tile makes room
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      copy_w(t / 2 + 2);
    }
    constexpr int per = last ? 1 : (2 * RG + 1) / 3;
    if constexpr (last) {
      wait_lgkmcnt<0>();   // reads of k-tile t, writes of W's t + 1
      // X's t + 1 has landed, and for an even t the codes of the next pair
      w4_wait_vm<u * NCODE>();
      barrier_only();
      issue_x(t + 2);
      read(fr[0], other, 0);
      if constexpr (u == 0) read_w(now, t / 2 + 1);   // W's t + 2 begins a pair
      convert(now, utag, std::integral_constant<int, 0>{});
    } else {
      read(fr[(s + 1) & 1], utag, s + 1);
      constexpr int i0 = 1 + s * per, i1 = i0 + per < 2 * RG ? i0 + per : 2 * RG;
      w4_for<(i1 > i0 ? i1 - i0 : 0)>([&](auto i) { convert(now, other, std::integral_constant<int, i0 + decltype(i)::value>{}); });
    }
#pragma unroll
    for (int i = 0; i < NMMA; ++i)
      acc[i / MB][i % MB] = Tr<DT>::mma(fr[s & 1].w[i / MB], fr[s & 1].x[i % MB], acc[i / MB][i % MB]);
    // one product, then a read and a share of the rest (120 -> 115 us at 3000 x 4096 x 4096)
    w4_for<NMMA>([&](auto) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, (MB + NB + NMMA - 1) / NMMA, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, (per * 24 + NMMA - 1) / NMMA, 0);
    });
    __builtin_amdgcn_sched_barrier(0);
  };
  auto ktile = [&](auto utag, int t) {
    constexpr int u = decltype(utag)::value;
    w4_for<4>([&](auto stag) {
      // a group's factors, before its first products: with groups of 64 every tile, else every other
      // one (1 where no group begins: a branch around the multiplications would keep them from running
      // among the products)
      constexpr bool scale = decltype(stag)::value == 0 && (E == 2 || u == 0);
      step(utag, stag, std::integral_constant<bool, scale>{}, t);
    });
  };
  for (int t = 0; t < KT2; t += 2) {
    ktile(p0, t);
    ktile(p1, t + 1);
  }
  wait_vmcnt<0>();
  wait_lgkmcnt<0>();
  // the last groups' f of every row, and the stages to the epilogue
#pragma unroll
  for (int r = 0; r < RG; ++r)
    if (q == 0) reinterpret_cast<float*>(smem + C::OFF_R)[(w * RG + r) * 16 + li] = f[r];
  __syncthreads();
  rescale(0);
  w4_large_epilogue<DT, GATED, C>(p, acc, m0 + wm * WM, n0 + wn * (GATED ? WN / 2 : WN), lane, smem + w * C::EPI);
}

}  // namespace gek
