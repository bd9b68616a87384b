// General product kernel of the gated feed-forward operators: fp32, and 16-bit operands whose
// rows are not whole 16-byte chunks (odd sizes, any alignment).
//
// D = A . B over 128 x 128 or 64 x 64 tiles, operands in any of the storage orders below, copied
// through registers into two LDS buffers of "row = m or n, 128 bytes of k" whatever the order
// (mn-major operands are transposed in registers on the way). Every load is 16 bytes at the
// elements' alignment. At the end of a row the load is moved back to the row's last 16 bytes
// and its value shifted, so that nothing past a row is read and nothing branches per element;
// rows of fewer than 16 bytes are read one element at a time.
// fp32 runs v_mfma_f32_32x32x2 and is bound by it in large products (plain 8192^3 products by rocBLAS: 154 TFLOP/s):
// 2048 x 2 x 4096 x 2048 538 us, 128 TFLOP/s. 333 x 2 x 1101 x 743 takes 26 us, 0.8 per k-tile of
// 32, of which the products are 0.43: one wave a SIMD waits for LDS, for the stores of the next tile
// and for the barrier. Four k-tiles on their way, four groups of waves, and the next tile stored before
// the products changed nothing.
#pragma once

#include <type_traits>

#include "gated_math.hpp"

namespace gek {

struct GenArgs {
  const void* A;
  const void* B;
  const void* bias;
  void* D;
  void* Z;            // gated: receives [G | U] (m, 2 n), or null
  int64_t m, n, k;    // gated: n columns of D, 2 n rows of B
  int64_t lda, ldb, ldd;   // elements between stored rows
  int32_t vec;        // type of bias
  int32_t act;
  int32_t tiles_m, tiles_n;
};

// 16 bytes at any alignment.
__device__ __forceinline__ i32x4 load16(const void* p) {
  i32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
// v moved down by s elements (0 .. E), zeros from above.
template <int ES>
__device__ __forceinline__ i32x4 shift_down(i32x4 v, int s) {
  const int d = ES == 4 ? s : s >> 1;   // whole dwords
  if (d & 4) v = i32x4{0, 0, 0, 0};
  if (d & 2) v = i32x4{v[2], v[3], 0, 0};
  if (d & 1) v = i32x4{v[1], v[2], v[3], 0};
  if constexpr (ES == 2) {
    if (s & 1) {
      const uint32_t a = v[0], b = v[1], c = v[2], e = v[3];
      v = i32x4{(int)(a >> 16 | b << 16), (int)(b >> 16 | c << 16), (int)(c >> 16 | e << 16), (int)(e >> 16)};
    }
  }
  return v;
}
// Elements pos .. pos + E - 1 of a row of len elements (len >= 1), zeros past its end.
template <int ES>
__device__ __forceinline__ i32x4 load_end(const char* row, int64_t pos, int64_t len) {
  constexpr int E = 16 / ES;
  if (len >= E) {
    const int64_t a = pos < len - E ? pos : len - E, s = pos - a;
    return shift_down<ES>(load16(row + a * ES), (int)(s < E ? s : E));
  }
  i32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t i = pos + e;
    if (i < len) {
      if constexpr (ES == 4) v[e] = reinterpret_cast<const int*>(row)[i];
      else v[e / 2] |= (int)((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << (16 * (e & 1)));
    }
  }
  return v;
}

// One operand's tile: MN rows (or columns, mn-major) by BK k values, NT threads.
// HALVES (k-major): tile rows come from two halves of the stored rows, alternating by HW:
// HW rows of the first half, the same HW of the second, and so on.
// Every load happens, at the row's last 16 bytes where a chunk would pass its end, and is moved into
// place when it is stored: a load that may not happen would turn the waits for the loads before it
// into waits for all that are on their way. NARROW: rows of fewer than 16 bytes, element by element.
template <int ES, int MN, bool KMAJ, int NT, bool NARROW, int HW = 0>
struct GenOperand {
  static constexpr int E = 16 / ES, BK = kRowBytes / ES;
  static constexpr int LD = MN * 8 / NT;   // k-major: 16-byte chunks per thread
  static constexpr int NB = MN / E, R = NB * BK / NT;   // mn-major: one block of R k-rows by E columns per thread
  static_assert(KMAJ ? MN * 8 % NT == 0 : (R == 2 || R == 4) && NB * (BK / R) == NT, "tile split");
  static constexpr int REGS = KMAJ ? LD : R;

  const char* row[KMAJ ? LD : 1];   // k-major: this thread's rows; mn-major: its columns' first k
  int64_t ld, kdim;                 // (ld: bytes)
  int64_t col, len;                 // mn-major: first column and the number of columns
  struct Regs {
    i32x4 v[REGS];
  };

  __device__ static __forceinline__ int swz(int row) { return (row ^ (row >> 3)) & 7; }

  // mn0: first row / column; mndim, kdim the extents.
  __device__ __forceinline__ GenOperand(const char* X, int64_t ld_, int64_t mn0, int64_t mndim, int64_t kdim_, int t)
      : ld(ld_ * ES), kdim(kdim_), col(mn0 + t % NB * E), len(mndim) {
    if constexpr (KMAJ) {
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int r = (t + i * NT) >> 3;
        int64_t at;
        if constexpr (HW > 0) {
          const int64_t c = mn0 + r / (2 * HW) * HW + r % HW;
          at = (c < mndim ? c : mndim - 1) + (r / HW % 2 ? mndim : 0);
        } else {
          at = mn0 + r < mndim ? mn0 + r : mndim - 1;   // (rows past the last one are not stored)
        }
        row[i] = X + at * ld;
      }
    } else {
      row[0] = NARROW ? X : X + (col < mndim - E ? col : mndim - E) * ES;
    }
  }
  // Tile kt (of all k).
  __device__ __forceinline__ void load(Regs& reg, int64_t kt, int t) const {
    if constexpr (KMAJ) {
      const int64_t pos = kt * BK + (t & 7) * E;
#pragma unroll
      for (int i = 0; i < LD; ++i)
        reg.v[i] = NARROW ? load_end<ES>(row[i], pos, kdim) : load16(row[i] + (pos < kdim - E ? pos : kdim - E) * ES);
    } else {
      const int64_t kr = kt * BK + t / NB * R;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const char* p = row[0] + (kr + r < kdim ? kr + r : kdim - 1) * ld;
        reg.v[r] = NARROW ? load_end<ES>(p, col, len) : load16(p);
      }
    }
  }
  __device__ __forceinline__ void store(Regs& reg, char* lds, int64_t kt, int t) const {
    if constexpr (KMAJ) {
      if constexpr (!NARROW) {
        if ((kt + 1) * BK > kdim) {
          const int64_t over = kt * BK + (t & 7) * E + E - kdim;
#pragma unroll
          for (int i = 0; i < LD; ++i) reg.v[i] = shift_down<ES>(reg.v[i], (int)(over < 0 ? 0 : over < E ? over : E));
        }
      }
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int r = (t + i * NT) >> 3;
        *reinterpret_cast<i32x4*>(lds + r * kRowBytes + (((t & 7) ^ swz(r)) << 4)) = reg.v[i];
      }
    } else {
      const int64_t k0 = kt * BK + t / NB * R;
      if constexpr (!NARROW) {
        if (col - t % NB * E + MN > len) {
          const int64_t over = col + E - len;
#pragma unroll
          for (int r = 0; r < R; ++r) reg.v[r] = shift_down<ES>(reg.v[r], (int)(over < 0 ? 0 : over < E ? over : E));
        }
      }
      if ((kt + 1) * BK > kdim) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) reg.v[r][e] = k0 + r < kdim ? reg.v[r][e] : 0;
      }
      const int kb = t / NB * R * ES, chunk = kb >> 4, within = kb & 15;
#pragma unroll
      for (int c = 0; c < E; ++c) {
        const int r = t % NB * E + c;
        char* dst = lds + r * kRowBytes + ((chunk ^ swz(r)) << 4) + within;
        if constexpr (ES == 4) {
          if constexpr (R == 4) *reinterpret_cast<i32x4*>(dst) = i32x4{reg.v[0][c], reg.v[1][c], reg.v[2][c], reg.v[3][c]};
          else *reinterpret_cast<i32x2*>(dst) = i32x2{reg.v[0][c], reg.v[1][c]};
        } else {
          const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;
          const int lo = (int)__builtin_amdgcn_perm((uint32_t)reg.v[1][c >> 1], (uint32_t)reg.v[0][c >> 1], sel);
          if constexpr (R == 4)
            *reinterpret_cast<i32x2*>(dst) =
                i32x2{lo, (int)__builtin_amdgcn_perm((uint32_t)reg.v[3][c >> 1], (uint32_t)reg.v[2][c >> 1], sel)};
          else
            *reinterpret_cast<int*>(dst) = lo;
        }
      }
    }
  }
};

// v to elements i .. i + 3 of p, the first n of them.
template <int OUT>
__device__ __forceinline__ void store4(void* p, int64_t i, int64_t n, const float (&v)[4]) {
  if (n >= 4) {
    if constexpr (OUT == F32) {
      __builtin_memcpy(static_cast<float*>(p) + i, v, 16);
    } else {
      const i32x2 o = {(int)Tr<OUT>::pack2(v[0], v[1]), (int)Tr<OUT>::pack2(v[2], v[3])};
      __builtin_memcpy(static_cast<uint16_t*>(p) + i, &o, 8);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) store_vec(p, OUT, i + e, v[e]);
  }
}

// LAY bit 0: A stored (k, m); bit 1: B stored (n, k); bit 2 (with bit 1): gated, B (2 n, k).
// OUT: type of D. Waves of WM x 64, in KG groups that share the k-steps of every tile (their sums
// are added through LDS): the 64 x 64 tile has two, so that the few tiles of a small product still
// put a wave on every SIMD. gridDim.y workgroups share the k loop (not gated), each with its own D.
// Two k-tiles are on their way in registers while a third is multiplied.
template <int DT, int OUT, int LAY, int BM, int BN, int WM, int KG, bool NARROW>
__global__ __launch_bounds__((BM / WM) * (BN / 64) * KG * 64, 2) void gen_kernel(GenArgs p) {
  using T = Tr<DT>;
  constexpr bool TA = (LAY & 1) != 0, TB = (LAY & 2) != 0, GATED = (LAY & 4) != 0;
  constexpr int WN = 64, WAVES_M = BM / WM, WAVES = WAVES_M * (BN / WN), NT = WAVES * KG * 64, MB = WM / 32, NB = 2;
  constexpr int ES = T::es, BK = kRowBytes / ES, STAGE = (BM + BN) * kRowBytes, NS = 4 / KG;
  constexpr bool FINE = DT == F32;
  __shared__ __attribute__((aligned(16))) char lds[2 * STAGE];
  using OA = GenOperand<ES, BM, !TA, NT, NARROW>;
  using OB = GenOperand<ES, BN, TB, NT, NARROW, GATED ? 32 : 0>;
  struct Tile {
    typename OA::Regs a;
    typename OB::Regs b;
  } in[2];

  const int pos = xcd_remap(blockIdx.x, p.tiles_m * p.tiles_n);
  const int tm = __builtin_amdgcn_readfirstlane(pos % p.tiles_m), tn = __builtin_amdgcn_readfirstlane(pos / p.tiles_m);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * (GATED ? BN / 2 : BN);
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6), kg = w / WAVES, wt = w % WAVES;
  const int wm = wt % WAVES_M, wn = wt / WAVES_M, lrow = lane & 31, lhi = lane >> 5;
  const OA oa(static_cast<const char*>(p.A), p.lda, m0, p.m, p.k, t);
  const OB ob(static_cast<const char*>(p.B), p.ldb, n0, p.n, p.k, t);
  const int64_t KTA = (p.k + BK - 1) / BK;
  const int64_t kb = KTA * blockIdx.y / gridDim.y, KT = KTA * (blockIdx.y + 1) / gridDim.y - kb;

  f32x16 acc[NB][MB];
#pragma unroll
  for (int a = 0; a < NB; ++a)
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[a][b] = f32x16{};

  // The large tile's workgroups begin their k loops apart: rows lie a stride apart that may hit few of
  // the L2's channels, and many workgroups in step would all read those at once (2048 x 2 x 2752 x
  // 1024 fp32: 273 -> 236 us; with few workgroups, the small tile's, it costs 4%).
  const int64_t turn = BM == 128 && KT > 0 ? pos % KT : 0;
  const auto at = [&](int64_t kt) {   // (past the last tile the last one again)
    const int64_t i = (kt < KT ? kt : KT - 1) + turn;
    return kb + (i < KT ? i : i - KT);
  };
  const auto load = [&](Tile& v, int64_t kt) {
    oa.load(v.a, at(kt), t);
    ob.load(v.b, at(kt), t);
  };
  const auto store = [&](Tile& v, int64_t kt, int stage) {
    oa.store(v.a, lds + stage * STAGE, at(kt), t);
    ob.store(v.b, lds + stage * STAGE + BM * kRowBytes, at(kt), t);
  };
  const auto tile = [&](auto utag, int64_t kt) {   // kt % 2 == u: in stage u; its successor is in in[u ^ 1]
    constexpr int u = decltype(utag)::value;
    load(in[u], kt + 2);
    __builtin_amdgcn_sched_barrier(0);   // (the loads first)
    const char* sA = lds + u * STAGE + (wm * WM + lrow) * kRowBytes;
    const char* sB = lds + u * STAGE + (BM + wn * WN + lrow) * kRowBytes;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int chunk = 2 * (KG * s + kg) + lhi;
      i32x4 af[MB], bf[NB];
      // (the swizzle depends on the row's place in the tile: blocks of 32 rows, waves of 32 or 64)
#pragma unroll
      for (int b = 0; b < MB; ++b)
        af[b] = *reinterpret_cast<const i32x4*>(sA + b * 32 * kRowBytes + ((chunk ^ OA::swz(wm * WM + b * 32 + lrow)) << 4));
#pragma unroll
      for (int a = 0; a < NB; ++a)
        bf[a] = *reinterpret_cast<const i32x4*>(sB + a * 32 * kRowBytes + ((chunk ^ OB::swz(wn * WN + a * 32 + lrow)) << 4));
#pragma unroll
      for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[a][b] = T::mma(bf[a], af[b], acc[a][b]);
    }
    store(in[u ^ 1], kt + 1, u ^ 1);   // (past the last tile for nobody)
    __syncthreads();
  };
  if (KT > 0) {   // (a product over no tokens is zero)
    load(in[0], 0);
    load(in[1], 1);
    store(in[0], 0, 0);
    __syncthreads();
    int64_t kt = 0;
    for (; kt + 1 < KT; kt += 2) {
      tile(std::integral_constant<int, 0>{}, kt);
      tile(std::integral_constant<int, 1>{}, kt + 1);
    }
    if (kt < KT) tile(std::integral_constant<int, 0>{}, kt);
  }
  if constexpr (KG == 2) {
    static_assert(WAVES * MB * NB * 4096 <= 2 * STAGE, "sums of the second group of waves");
    f32x4* sums = reinterpret_cast<f32x4*>(lds) + wt * (MB * NB * 256) + lane;
    if (kg == 1) {
#pragma unroll
      for (int i = 0; i < MB * NB; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const f32x16& v = acc[i / MB][i % MB];
          sums[(i * 4 + c) * 64] = f32x4{v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]};
        }
    }
    __syncthreads();
    if (kg == 1) return;
#pragma unroll
    for (int i = 0; i < MB * NB; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const f32x4 v = sums[(i * 4 + c) * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i / MB][i % MB][4 * c + e] += v[e];
      }
  }
  char* const out = static_cast<char*>(p.D) + (int64_t)blockIdx.y * p.m * p.ldd * Tr<OUT>::es;

  // lane: row m0 + wm WM + 32 b + l % 32; register r: column 8 (r / 4) + 4 (l / 32) + r % 4 of a block
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int64_t row = m0 + wm * WM + 32 * b + lrow;
    if (row >= p.m) continue;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int in = 8 * g + 4 * lhi;
      if constexpr (GATED) {
        const int64_t col = n0 + wn * 32 + in, left = p.n - col;
        if (left <= 0) continue;
        float gv[4], uv[4], hv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          gv[e] = acc[0][b][4 * g + e];
          uv[e] = acc[1][b][4 * g + e];
          if (p.bias && e < left) {
            gv[e] += load_vec(p.bias, p.vec, col + e);
            uv[e] += load_vec(p.bias, p.vec, p.n + col + e);
          }
        }
        with_gate(p.act, [&](auto act) {
#pragma unroll
          for (int e = 0; e < 4; ++e) hv[e] = gate_act<decltype(act)::value, FINE>(gv[e]) * uv[e];
        });
        store4<OUT>(out, row * p.ldd + col, left, hv);
        if (p.Z) {
          store4<OUT>(p.Z, row * 2 * p.n + col, left, gv);
          store4<OUT>(p.Z, row * 2 * p.n + p.n + col, left, uv);
        }
      } else {
#pragma unroll
        for (int a = 0; a < NB; ++a) {
          const int64_t col = n0 + wn * WN + 32 * a + in, left = p.n - col;
          if (left <= 0) continue;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[a][b][4 * g + e];
          store4<OUT>(out, row * p.ldd + col, left, v);
        }
      }
    }
  }
}

}  // namespace gek
