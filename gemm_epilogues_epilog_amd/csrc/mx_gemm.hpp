// D = act(X W^T + bias) of microscaled operands (layout: mx_format.hpp): X (m, k) e4m3 or
// e2m1, W (n, k) e2m1, both along k, products and scales in the scaled matrix instruction
// with fp32 accumulators. Grouped form: rows of X sorted by expert, each expert with its
// own W and bias, its row range read on the device.
//
// The W fragment is the instruction's row operand and the X fragment its column operand,
// so a lane holds one row of D (a token) and its registers walk along n.
#pragma once

#include <type_traits>

#include "kernels.hpp"
#include "mx_format.hpp"
#include "mx_tiles.hpp"

namespace gek {

using namespace gemx;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void mx_lds_void;

enum MxOut { MX_OUT_F32 = 0, MX_OUT_F16 = 1, MX_OUT_BF16 = 2, MX_OUT_FP8 = 3 };

struct MxArgs {
  const char* xc;
  const char* xs;
  const char* wc;
  const char* ws;
  const void* bias;        // (n) or (experts, n), type vec; NULL without a bias
  const int32_t* offsets;  // (experts + 1) or NULL
  void* D;                 // (m, n), or e4m3 codes
  char* ds;                // scales of an e4m3 result
  float* partial;          // split tiles: parts' accumulators
  uint32_t* counter;       // split tiles: parts arrived
  int64_t m;
  int32_t n, k, kt;        // kt: 256-k granules
  int32_t experts;         // 0: one product
  int32_t tiles_m, tiles_n;
  int32_t splits;          // parts of the k loop
  int32_t ep, out, vec;
  int32_t round;           // tile kernel: its workgroups, if a short last round is left over
  int32_t tail;            // ring kernel: takes what the tile kernel left over
};

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Copies of the tile kernels: KB number PC of a row group's stage (lane l moves 16 bytes at
// 16 l of it), or its 256 bytes of scales, from srd.base + soff (uniform) on to LDS bytes
// `lds` on. An instruction's offset moves both its source and its LDS address. See
// copy_to_lds_b128 for the ordering rules.
template <int PC>
__device__ __forceinline__ void copy_kb_to_lds(const i32x4& srd, uint32_t lane16, int soff, uint32_t lds) {
  static_assert(PC >= 0 && PC < 4, "12-bit offsets");
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen offset:%4 lds"
               :
               : "v"(lane16), "s"(srd), "s"(soff), "s"(uniform(lds)), "n"(PC * 1024)
               : "memory", "m0");
}
// The scales of four row groups (256 bytes each, 16 lanes each) in one copy, by the waves with
// `on` set: the branch is inside the assembly, where the compiler cannot move products
// around it. Copies cost by the instruction here, whatever their size: one copy per row group
// took 6% of the whole product.
__device__ __forceinline__ void copy_scales_to_lds(const i32x4& srd, uint32_t voff, uint32_t lds, int on) {
  asm volatile(
      "s_cmp_eq_u32 %3, 0\n\ts_cbranch_scc1 .Lno_scales_%=\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %0, %1, 0 offen lds\n.Lno_scales_%=:"
      :
      : "v"(voff), "s"(srd), "s"(uniform(lds)), "s"(uniform(on))
      : "memory", "m0", "scc");
}

// act(v) by the run-time epilogue code (uniform).
__device__ __forceinline__ float mx_act(float v, int ep) {
  return ep == RELU_BIAS ? (v > 0.0f ? v : 0.0f) : ep == GELU_BIAS ? gelu_tanh(v) : v;
}

template <int N>
__device__ __forceinline__ void mx_act_n(float (&v)[N], int ep) {
  if (ep == RELU_BIAS) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] > 0.0f ? v[i] : 0.0f;
  } else if (ep == GELU_BIAS) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = gelu_tanh(v[i]);
  }
}

// The rows [lo, hi) of 64 experts from e0 on, one to a lane (lanes past the last expert get
// none). Offsets outside 0 .. m or that run backwards are held to an empty or valid range, and
// of that the rows up to `end`, the furthest end of the experts before, are taken off: a row
// has one expert, so no two workgroups write it, and there are at most as many tiles as the
// launch allows for. `end` moves on for the next 64. Ascending offsets need no look at the other lanes.
__device__ __forceinline__ void expert_rows(const MxArgs& p, int e0, int& end, int& lo, int& hi) {
  const int lane = threadIdx.x & 63, m = (int)p.m;
  int a = 0, b = 0;
  const bool in = e0 + lane < p.experts;
  if (in) {
    a = p.offsets[e0 + lane];
    b = p.offsets[e0 + lane + 1];
  }
  lo = min(max(a, 0), m);
  hi = max(min(b, m), lo);
  const int first = __builtin_amdgcn_readlane(lo, 0);
  if (__builtin_amdgcn_ballot_w64(b < a) == 0 && first >= end) {
    const int last = __builtin_amdgcn_readlane(hi, 63);
    if (last > first) end = last;
    return;
  }
  int top = hi > lo ? hi : 0;   // the furthest end up to this lane
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(top, d);
    if (lane >= d) top = max(top, up);
  }
  const int before = __shfl_up(top, 1);
  lo = max(lo, max(end, lane ? before : 0));
  hi = max(hi, lo);
  end = max(end, __builtin_amdgcn_readlane(top, 63));
}
// Expert e's alone, without a look at the ones before it.
__device__ __forceinline__ void offset_rows(const MxArgs& p, int e, int64_t& lo, int64_t& hi) {
  const int a = p.offsets[e], b = p.offsets[e + 1], m = (int)p.m;
  lo = min(max(a, 0), m);
  hi = max(min(b, m), (int)lo);
}
// The furthest end of the experts before e.
__device__ __forceinline__ int end_before(const MxArgs& p, int e) {
  int end = 0;
  for (int i = threadIdx.x & 63; i < e; i += 64) {
    int64_t lo, hi;
    offset_rows(p, i, lo, hi);
    if (hi > lo) end = max(end, (int)hi);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) end = max(end, __shfl_xor(end, d));
  return end;
}

// ---- finishing outputs ------------------------------------------------------------
// Eight consecutive finished values of row `row` from column c0 (a multiple of 8).
__device__ __forceinline__ void mx_store8(const MxArgs& p, int64_t row, int c0, const float (&v)[8]) {
  if (c0 >= p.n) return;
  const int64_t at = row * p.n + c0;
  if (c0 + 8 <= p.n) {   // 16 bytes at a time, at the elements' alignment
    if (p.out == MX_OUT_F32) {
      __builtin_memcpy(static_cast<float*>(p.D) + at, v, 32);
    } else {
      i32x4 o;
      if (p.out == MX_OUT_F16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = (int)Tr<F16>::pack2(v[2 * e], v[2 * e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = (int)Tr<BF16>::pack2(v[2 * e], v[2 * e + 1]);
      }
      __builtin_memcpy(static_cast<char*>(p.D) + at * 2, &o, 16);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c0 + e < p.n) store_vec(p.D, p.out, at + e, v[e]);
  }
}

// Sixteen e4m3 codes of row `row` from column c0 (a multiple of 16): one chunk.
__device__ __forceinline__ void mx_store_chunk(const MxArgs& p, int64_t row, int c0, i32x4 o) {
  const int64_t chunks = pad_to(p.n, kKPad) / 16;
  *reinterpret_cast<i32x4*>(static_cast<char*>(p.D) + ((row >> 5) * chunks + c0 / 16) * 512 + (row & 31) * 16) = o;
}
__device__ __forceinline__ void mx_store_scale(const MxArgs& p, int64_t row, int c0, int s) {
  const int64_t granules = pad_to(p.n, kKPad) / kKPad;
  p.ds[((row >> 5) * granules + c0 / kKPad) * kScaleGranule + ((c0 / 32) & 1) * 128 + (row & 31) * 4 +
       (c0 / 64) % 4] = (char)s;
}
// Bias of column c of expert e (0 past n, or without a bias).
__device__ __forceinline__ float mx_bias(const MxArgs& p, int e, int c) {
  return p.ep != NONE && c < p.n ? load_vec(p.bias, p.vec, (int64_t)e * p.n + c) : 0.0f;
}

// ---- tile kernel -------------------------------------------------------------------
// One workgroup computes bm x bn of D over its part of k. Copies go straight to LDS;
// all waves run the lockstep schedule: at the end of a k-tile every wave waits for its own
// copies of the next one, one barrier publishes it and releases the stage just read, and
// the next copies go there.
template <int XF, int CFG>
struct MxCfgT {
  static constexpr MxTile T = kMxTiles[CFG];
  static constexpr bool RING = mx_is_ring(CFG);
  static constexpr int MB = T.mb, NB = T.nb, STAGES = T.stages, KG = T.kg;
  static constexpr int WAVES_M = T.bm / 32 / MB, WAVES_N = T.bn / 32 / NB, NW = WAVES_M * WAVES_N;   // of a group
  static constexpr int BK = mx_bk(XF), KS = BK / 64;
  static constexpr int WRB = BK / 32 * 512;                // bytes of a W row group per stage
  static constexpr int XRB = BK / chunk_values(XF) * 512;  // and of an X row group (4096)
  static constexpr int W_BYTES = T.bn / 32 * WRB, X_BYTES = T.bm / 32 * XRB;
  // scales are copied four row groups at a time, by the first SWV waves
  static constexpr int SWW = (T.bn + 127) / 128, SWV = SWW + (T.bm + 127) / 128;
  static constexpr int OFF_X = W_BYTES, OFF_SW = OFF_X + X_BYTES, OFF_SX = OFF_SW + SWW * 1024;
  static constexpr int STAGE = OFF_SW + SWV * 1024;
  // copies per wave and stage: IW (IX) KB of W (X), PPW (PPX) of each of its GW (GX) row groups
  static constexpr int IW = W_BYTES / 1024 / NW, IX = X_BYTES / 1024 / NW;
  static constexpr int PW = WRB / 1024, PX = XRB / 1024;
  static constexpr int PPW = IW < PW ? IW : PW, PPX = IX < PX ? IX : PX, GW = IW / PPW, GX = IX / PPX;
  static constexpr int INST = IW + IX + 1;                 // with the copy of the scales
  // A copy after every STRIDE-th product from a k-tile's last step on: apart, so that the
  // waves do not queue for the memory pipe, but early enough to land before the next
  // barrier (8192^3: e2m1 X 170 -> 161 us at 2 on zeros, e4m3 X 272 -> 310).
  static constexpr int STRIDE = XF == FP4 ? 2 : 1;
  static constexpr int EPI = 32 * 32 * 2 + NB * 32 * 4;    // epilogue LDS per wave: 32 rows of 64 bytes, and bias
  // the persistent kernel's stages hold the next tile during the epilogue
  static constexpr int OFF_EPI = RING ? 0 : STAGES * STAGE;
  static constexpr int LDS = RING ? STAGES * KG * STAGE : OFF_EPI + NW * EPI;
  static constexpr int XR = XF == FP8 ? 2 : 1;             // 16-byte reads per X fragment
  static_assert(LDS <= 160 * 1024 && NW * EPI <= LDS && NW * (KG - 1) * MB * NB * 4096 <= LDS, "LDS");
  static_assert(IW >= 1 && IX >= 1 && IW * NW * 1024 == W_BYTES && IX * NW * 1024 == X_BYTES, "whole copies");
  static_assert(PW % PPW == 0 && PX % PPX == 0, "a wave's copies of a row group are consecutive");
  static_assert(SWV <= NW, "scale copies");
};

template <int XF, int MB, int NB>
struct MxFrags {
  i32x4 w[NB];
  i32x4 x[MB][XF == FP8 ? 2 : 1];
};

// One product of the k-step S of a scale dword (opsel picks its byte).
template <int XF, int S>
__device__ __forceinline__ f32x16 mx_mma(i32x4 w, const i32x4 (&x)[XF == FP8 ? 2 : 1], f32x16 c, int sw, int sx) {
  const i32x8 a = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
  if constexpr (XF == FP8) {
    const i32x8 b = {x[0][0], x[0][1], x[0][2], x[0][3], x[1][0], x[1][1], x[1][2], x[1][3]};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 0, S, sw, S, sx);
  } else {
    const i32x8 b = {x[0][0], x[0][1], x[0][2], x[0][3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, S, sw, S, sx);
  }
}

// Tile of this workgroup: expert, first row group (as a row), the rows to keep, column.
// Grouped: every expert's tiles start at the 32-row group that holds its first row (the
// rows of its neighbours in that group are computed and dropped), so that the copies stay
// whole lines; the launch has workgroups for the most tiles there can be, and the ones
// past the actual count leave at once.
struct MxPlace {
  int e, tn;
  int64_t row0, lo, hi;
};
// Tiles of BM rows over rows [lo, hi).
template <int BM>
__device__ __forceinline__ int expert_tiles(int lo, int hi) {
  return hi > lo ? (int)(((int64_t)hi - (lo & ~31) + BM - 1) / BM) : 0;
}
// TAIL 1: without the tiles of a short last round; 2: those only. A last round that fills at
// most a quarter of the device is left to smaller tiles in a launch of its own, which take
// under half its time (2200 x 7300 x 4096, 261 tiles on 256 units: e4m3 X to bf16 85 us, now
// 70, to fp32 158, now 119). The launch cannot know the tiles by expert: both kernels derive
// the same split from the offsets, and the second one costs 2 us where it has nothing to do.
template <int BM, int TAIL = 0>
__device__ __forceinline__ bool mx_place(const MxArgs& p, int id, bool remap, MxPlace& o) {
  int tiles_m = p.tiles_m;
  if (p.experts) {
    int total = 0, end = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
      int lo, hi;
      expert_rows(p, e0, end, lo, hi);
      int c = expert_tiles<BM>(lo, hi);
#pragma unroll
      for (int d = 32; d; d >>= 1) c += __shfl_xor(c, d);
      total += c;
    }
    tiles_m = __builtin_amdgcn_readfirstlane(total);
  }
  const int all = tiles_m * p.tiles_n;
  int G = all;
  if constexpr (TAIL != 0) {
    if (p.round > 0 && all > p.round && all % p.round <= p.round / 4) G -= all % p.round;
  }
  if (TAIL == 2) id += G;
  if (id >= (TAIL == 2 ? all : G)) return false;
  const int pos = remap ? xcd_remap(id, G) : id;   // each XCD takes a run of the order
  const int gsz = kMxGroupM * p.tiles_n;
  const int g = pos / gsz, first = g * kMxGroupM;
  const int rows = min(tiles_m - first, kMxGroupM);
  const int in = pos - g * gsz;
  const int tm = __builtin_amdgcn_readfirstlane(first + in % rows);
  o.tn = __builtin_amdgcn_readfirstlane(in / rows);
  if (!p.experts) {
    o.e = 0;
    o.row0 = (int64_t)tm * BM;
    o.lo = 0;
    o.hi = p.m;
    return true;
  }
  const int lane = threadIdx.x & 63;
  int base = 0, end = 0;
  for (int e0 = 0; e0 < p.experts; e0 += 64) {
    int lo, hi;
    expert_rows(p, e0, end, lo, hi);
    const int c = expert_tiles<BM>(lo, hi);
    int incl = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(incl, d);
      if (lane >= d) incl += up;
    }
    const uint64_t past = __builtin_amdgcn_ballot_w64(base + incl > tm);
    if (past) {
      const int f = __builtin_ctzll(past);
      o.e = e0 + f;
      const int t = tm - base - (__builtin_amdgcn_readlane(incl, f) - __builtin_amdgcn_readlane(c, f));
      o.lo = __builtin_amdgcn_readlane(lo, f);
      o.hi = __builtin_amdgcn_readlane(hi, f);
      o.row0 = (o.lo & ~(int64_t)31) + (int64_t)t * BM;
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// X's e4m3 values in two parts whose sum they are: the ones of at least 2 in magnitude, and
// the rest. The matrix unit adds the products of eight neighbouring elements aligned to the
// largest of them and drops what lies more than 13 bits below it (4 x 6 products span
// 21 bits). A block's largest value is in [256, 448]; products with the large part (2 ..
// 448 by 0.5 .. 6) span 13 bits, 14 where one of them reaches 2048, and those with the rest
// lose nothing, so two instructions keep what an fp32 sum keeps, where one leaves 1.3e-5
// of the result's norm (k = 4096, normal values with outlier channels). Results in 32 or 8
// bits take two. So does the skinny kernel, which waits for W (with one part and with two: one
// row by 11008 x 4096 9.5 and 9.9 us, 16 by 4096 x 4096 4.9 and 5.0, 512 rows over 64 experts
// of 2048 x 1024 15.8 and 16.9). 16-bit results of the tile and ring kernels, whose own
// rounding is 15 times as coarse in fp16 and 120 times in bf16, take one: two cost them 100 x
// 4096 x 11008 16.7 -> 23.2 us, 1000 x 4096 x 4096 22.6 -> 34, 8192^3 380 -> 645.
__device__ __forceinline__ i32x4 large_part(i32x4 x) {
  i32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // bit 6 of a byte is the exponent's top bit: selector 13 gives 0xff, 12 gives 0
    const uint32_t sel = (((uint32_t)x[i] >> 6) & 0x01010101u) | 0x0c0c0c0cu;
    r[i] = (int)((uint32_t)x[i] & __builtin_amdgcn_perm(0u, 0u, sel));
  }
  return r;
}

// f(0), f(1), .. f(N - 1) with constant arguments.
template <int N, int I = 0, class Fn>
__device__ __forceinline__ void static_for(Fn&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// ---- split k: the part that arrives last adds all parts in order and finishes --------
// Sums cross XCDs, whose L2 caches are not coherent: device-scope (sc1) accesses go to the
// memory side. A part's stores have completed before it counts itself; nobody waits, so
// no order of the workgroups can hang. Returns whether this workgroup finishes the tile.
template <class C>
__device__ __forceinline__ bool mx_join_parts(const MxArgs& p, const MxPlace& at, int part, int w, bool mine, int lane,
                                              f32x16 (&acc)[C::NB][C::MB], int* flag) {
  static_assert(C::MB == 1, "a wave's rows are one row group");
  const bool has_rows = mine && at.row0 + w % C::WAVES_M * 32 < p.m;   // others only take part in the barriers
  constexpr int NB = C::NB, MB = C::MB;
  constexpr int kDev = 16;
  constexpr int PART = C::NW * NB * MB * 16 * 64 * 4;
  const int tile_id = (int)(at.row0 / C::T.bm) * p.tiles_n + at.tn;
  char* slots = reinterpret_cast<char*>(p.partial) + (int64_t)tile_id * p.splits * PART;
  if (has_rows) {
    const __amdgpu_buffer_rsrc_t r = rsrc(slots + (int64_t)part * PART);
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const i32x4 v = {__float_as_int(acc[a][b][4 * g]), __float_as_int(acc[a][b][4 * g + 1]),
                           __float_as_int(acc[a][b][4 * g + 2]), __float_as_int(acc[a][b][4 * g + 3])};
          __builtin_amdgcn_raw_buffer_store_b128(v, r, (((w * NB + a) * MB + b) * 4 + g) * 1024 + lane * 16, 0, kDev);
        }
  }
  wait_vmcnt<0>();
  __syncthreads();
  if (threadIdx.x == 0)
    *flag = __hip_atomic_fetch_add(p.counter + tile_id * kMxCounterStride, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
              (uint32_t)p.splits - 1u;
  __syncthreads();
  if (!uniform(*flag)) return false;
  __syncthreads();   // the flag's LDS is the epilogue's
  if (threadIdx.x == 0) __hip_atomic_store(p.counter + tile_id * kMxCounterStride, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (!has_rows) return true;
  // four parts' loads in flight together: a trip to the memory side takes longer than the adds
  constexpr int Q = NB * MB * 4, G = 4;
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[q / 4 % NB][q / 4 / NB][q % 4 * 4 + e] = 0.0f;
  for (int s0 = 0; s0 < p.splits; s0 += G) {
    i32x4 v[G][Q];
#pragma unroll
    for (int s = 0; s < G; ++s) {
      if (s0 + s < p.splits) {
        const __amdgpu_buffer_rsrc_t r = rsrc(slots + (int64_t)(s0 + s) * PART);
#pragma unroll
        for (int q = 0; q < Q; ++q)
          v[s][q] = __builtin_amdgcn_raw_buffer_load_b128(
              r, (((w * NB + q / 4 % NB) * MB + q / 4 / NB) * 4 + q % 4) * 1024 + lane * 16, 0, kDev);
      } else {
#pragma unroll
        for (int q = 0; q < Q; ++q) v[s][q] = i32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int s = 0; s < G; ++s)
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[q / 4 % NB][q / 4 / NB][q % 4 * 4 + e] += __int_as_float(v[s][q][e]);
  }
  return true;
}

// ---- epilogue of a wave: 32 MB rows x 32 NB columns of sums to D -----------------------
// A lane holds, of one row, columns 8 g + 4 (l / 32) + 0 .. 3 of each 32-column block.
template <class C>
__device__ __forceinline__ void mx_epilogue(const MxArgs& p, const MxPlace& at, int wm, int c0w, int lane,
                                            const f32x16 (&acc)[C::NB][C::MB], const float* bias, char* scratch) {
  constexpr int NB = C::NB, MB = C::MB;
  const int lrow = lane & 31, lhi = lane >> 5;
  const int out = p.out;
  const int cpad = out == MX_OUT_FP8 ? (int)pad_to(p.n, kKPad) : p.n;
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int64_t r0 = at.row0 + (wm * MB + b) * 32;
    const int64_t row = r0 + lrow;
    const bool keep = row >= at.lo && row < at.hi;
#pragma unroll
    for (int a = 0; a < NB; ++a) {
      const int c = c0w + a * 32;
      if (c >= cpad) break;
      float v[16];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 bv = *reinterpret_cast<const f32x4*>(bias + a * 32 + 8 * g + 4 * lhi);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * g + e] = acc[a][b][4 * g + e] + bv[e];
      }
      mx_act_n(v, p.ep);
      if (out == MX_OUT_FP8) {
        // the other half-wave holds the rest of the block; two swaps of half-waves give
        // each lane 16 consecutive codes, a chunk
        if (c + 32 > p.n) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + 8 * (i / 4) + 4 * lhi + i % 4 >= p.n) v[i] = 0.0f;
        }
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = amax2(m, mag(v[i]));
        const uint32_t mu = __float_as_uint(m);
        const auto sm = __builtin_amdgcn_permlane32_swap(mu, mu, false, false);
        m = amax2(__uint_as_float(sm[0]), __uint_as_float(sm[1]));
        const int s = scale_of(m, FP8);
        uint32_t q[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) q[g] = to_fp8x4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3], s);
        const auto s0 = __builtin_amdgcn_permlane32_swap(q[0], q[2], false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(q[1], q[3], false, false);
        if (keep) {
          mx_store_chunk(p, row, c + 16 * lhi, i32x4{(int)s0[0], (int)s0[1], (int)s1[0], (int)s1[1]});
          if (lhi == 0) mx_store_scale(p, row, c, s);
        }
      } else if (out == MX_OUT_F32) {
        // 16 bytes a lane, at the elements' alignment; the line of a row's 32 columns fills
        // over four stores
        if (keep) {
          float* d = static_cast<float*>(p.D) + row * p.n + c + 4 * lhi;
          if (c + 32 <= p.n) {
#pragma unroll
            for (int g = 0; g < 4; ++g) __builtin_memcpy(d + 8 * g, v + 4 * g, 16);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c + 8 * (i / 4) + 4 * lhi + i % 4 < p.n) d[8 * (i / 4) + i % 4] = v[i];
          }
        }
      } else {
        // 16-bit: the block's 32 rows of 64 bytes through scratch, so that a store
        // instruction writes 64-byte row pieces. 8-byte unit u of row r sits at unit
        // u ^ (r & 7): the 32 lanes of a write, and the 16-byte reads, spread over all banks.
        i32x2* t = reinterpret_cast<i32x2*>(scratch) + lrow * 8;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const i32x2 u = out == MX_OUT_F16
                              ? i32x2{(int)Tr<F16>::pack2(v[4 * g], v[4 * g + 1]), (int)Tr<F16>::pack2(v[4 * g + 2], v[4 * g + 3])}
                              : i32x2{(int)Tr<BF16>::pack2(v[4 * g], v[4 * g + 1]), (int)Tr<BF16>::pack2(v[4 * g + 2], v[4 * g + 3])};
          t[(2 * g + lhi) ^ (lrow & 7)] = u;
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = i * 16 + (lane >> 2), cc = c + (lane & 3) * 8;
          const i32x2* q = reinterpret_cast<const i32x2*>(scratch) + r * 8;
          const i32x2 lo = q[(2 * (lane & 3)) ^ (r & 7)], hi = q[(2 * (lane & 3) + 1) ^ (r & 7)];
          const int64_t rw = r0 + r;
          if (rw >= at.lo && rw < at.hi && cc < p.n) {
            uint16_t* d = static_cast<uint16_t*>(p.D) + rw * p.n + cc;   // element-aligned
            const i32x4 o = {lo[0], lo[1], hi[0], hi[1]};
            if (cc + 8 <= p.n) {
              __builtin_memcpy(d, &o, 16);
            } else {
#pragma unroll
              for (int e = 0; e < 7; ++e)
                if (cc + e < p.n) d[e] = (uint16_t)((uint32_t)o[e / 2] >> (16 * (e & 1)));
            }
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
}

// The copies of one wave into one stage, issued one at a time.
template <class C>
struct MxCopies {
  i32x4 rw, rx, rs;
  int off_w[C::GW], off_x[C::GX];
  uint32_t lds_w, lds_x, lds_s;
  uint32_t voff_s;

  template <int J>
  __device__ __forceinline__ void issue(uint32_t lane16, int scales) const {
    constexpr int JX = J - C::IW, JS = JX - C::IX;
    if constexpr (JX < 0) copy_kb_to_lds<J % C::PPW>(rw, lane16, off_w[J / C::PPW], lds_w + J / C::PPW * C::WRB);
    else if constexpr (JS < 0) copy_kb_to_lds<JX % C::PPX>(rx, lane16, off_x[JX / C::PPX], lds_x + JX / C::PPX * C::XRB);
    else copy_scales_to_lds(rs, voff_s, lds_s, scales);
  }
  template <int J0, int J1>
  __device__ __forceinline__ void issue_range(uint32_t lane16, int scales) const {
    if constexpr (J0 < J1) {
      issue<J0>(lane16, scales);
      issue_range<J0 + 1, J1>(lane16, scales);
    }
  }
};

// Sources of a tile's copies: base addresses of its first row groups at its first k-tile, and
// this wave's row groups. Row groups past the operand's last one are read from the last
// one instead (their results are dropped), so every address is in range.
template <class C>
struct MxSrc {
  const char *wc, *xc, *sc;   // sc: scales of W (the first SWW waves) or X
  int off_w[C::GW], off_x[C::GX];
  uint32_t voff_s;            // of the lane's scales
  int KT;                     // k-tiles to copy; 0 for no tile

  __device__ __forceinline__ void set(const MxArgs& p, const MxPlace& at, int XF, int w, int lane, int kb, int nt) {
    const int64_t gw = group_code_bytes(FP4, p.k), gx = group_code_bytes(XF, p.k), gs = group_scale_bytes(p.k);
    const int64_t wrg = row_groups(p.n), xrg = row_groups(p.m);
    // a tile that only pads an 8-bit result reads W's last row group
    const int wg0 = (int)min((int64_t)at.tn * (C::T.bn / 32), wrg - 1);
    const int64_t xg0 = at.row0 / 32;
    const int wg_last = (int)(wrg - 1 - wg0);
    const int xg_last = (int)min((int64_t)C::T.bm / 32, xrg - 1 - xg0);
    wc = p.wc + (at.e * wrg + wg0) * gw + (int64_t)kb * C::WRB;
    xc = p.xc + xg0 * gx + (int64_t)kb * C::XRB;
#pragma unroll
    for (int j = 0; j < C::GW; ++j)
      off_w[j] = uniform((int)(min(w * C::IW / C::PW + j, wg_last) * gw) + w * C::IW % C::PW * 1024);
#pragma unroll
    for (int j = 0; j < C::GX; ++j)
      off_x[j] = uniform((int)(min(w * C::IX / C::PX + j, xg_last) * gx) + w * C::IX % C::PX * 1024);
    // wave w copies the scales of row groups 4 w .. 4 w + 3 of [W's, X's]
    const bool of_w = w < C::SWW;
    sc = of_w ? p.ws + (at.e * wrg + wg0) * gs : p.xs + xg0 * gs;
    const int g = (of_w ? 4 * w : 4 * (w - C::SWW)) + (lane >> 4);
    voff_s = (uint32_t)(min(g, of_w ? wg_last : xg_last) * gs) + (lane & 15) * 16;
    KT = nt;
  }
  // The copies of k-tile kt into the stage at LDS byte `dst`. K-tiles past the last one fill
  // it with zeros (an empty range: no memory traffic, and zero codes with zero scales add
  // nothing), so the loop has no branches and always runs over pairs of k-tiles.
  __device__ __forceinline__ MxCopies<C> at(int kt, int kb, int w, uint32_t dst) const {
    MxCopies<C> c;
    const uint32_t range = kt < KT ? 0x7fffffffu : 0u;
    c.rw = make_srd(wc + (int64_t)kt * C::WRB, range);
    c.rx = make_srd(xc + (int64_t)kt * C::XRB, range);
    c.rs = make_srd(sc + (int64_t)((kb + kt) * C::BK / kKPad) * kScaleGranule, range);
#pragma unroll
    for (int j = 0; j < C::GW; ++j) c.off_w[j] = off_w[j];
#pragma unroll
    for (int j = 0; j < C::GX; ++j) c.off_x[j] = off_x[j];
    c.lds_w = uniform(dst + w * C::IW * 1024);
    c.lds_x = uniform(dst + C::OFF_X + w * C::IX * 1024);
    c.voff_s = voff_s;
    c.lds_s = uniform(dst + C::OFF_SW + w * 1024);
    return c;
  }
};

// Persistent: gridDim.x workgroups walk the tile order with that stride, and the k loop runs
// on from one tile into the next: during a tile's last two k-tiles the copies fetch the
// next tile's first two, so its latency hides behind this tile's end and its epilogue, and
// the stores of D drain while the next tile computes. The epilogue has LDS of its own.
// Bound by the matrix unit: it sustains 6650 TFLOP/s (e2m1) and 3880 (e4m3 X) on random
// values in registers under the power limit, and 8192^3 runs at 4520 (243 us) and 3000
// (366 us; in two parts 669 us, twice the products at 3290). What e2m1 lacks is the LDS: a
// 256 x 256 tile of eight 64 x 128 waves reads 1.5 KB of fragments per product there, four
// waves of 128 x 128 a third less, but one wave per SIMD hides no wait (387 us).
template <int XF, int CFG, bool EXACT>
__global__ __launch_bounds__((MxCfgT<XF, CFG>::NW * 64), 2) void mx_tile_kernel(MxArgs p) {
  using C = MxCfgT<XF, CFG>;
  constexpr int MB = C::MB, NB = C::NB, KS = C::KS;
  constexpr int BM = C::T.bm, BN = C::T.bn;
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];

  int id = (int)blockIdx.x;
  MxPlace at;
  if (!mx_place<BM, 1>(p, id, true, at)) return;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w % C::WAVES_M, wn = w / C::WAVES_M;
  const uint32_t lds = (uint32_t)(uintptr_t)(mx_lds_void*)smem;
  const uint32_t lane16 = lane * 16;
  constexpr int kb = 0;
  const int KT = (int)(pad_to(p.k, kKPad) / C::BK);
  const int KT2 = (KT + 1) & ~1;
  MxSrc<C> src;
  src.set(p, at, XF, w, lane, kb, KT);
  const int scales = w < C::SWV;

  // ---- fragment reads ----
  using F = MxFrags<XF, MB, NB>;
  const char* rd_w = smem + wn * NB * C::WRB + lane * 16;
  const char* rd_x = smem + C::OFF_X + wm * MB * C::XRB + lane * 16;
  const char* rd_sw = smem + C::OFF_SW + wn * NB * kScaleGranule + lane * 4;
  const char* rd_sx = smem + C::OFF_SX + wm * MB * kScaleGranule + lane * 4;
  constexpr int PIECES = NB + MB * C::XR;
  auto piece = [&](int u, int s, int q, F& f) {   // u, s, q are constants once unrolled
    if (q < C::XR) f.x[0][q] = *reinterpret_cast<const i32x4*>(rd_x + u * C::STAGE + (s * C::XR + q) * 1024);
    else if (q < C::XR + NB)
      f.w[q - C::XR] = *reinterpret_cast<const i32x4*>(rd_w + u * C::STAGE + (q - C::XR) * C::WRB + s * 1024);
    else {
      const int b = (q - NB) / C::XR, h = (q - NB) % C::XR;
      f.x[b][h] = *reinterpret_cast<const i32x4*>(rd_x + u * C::STAGE + b * C::XRB + (s * C::XR + h) * 1024);
    }
  };
  int sw[NB], sx[MB];
  auto read_scales = [&](int u, int kt) {
    const int sh = XF == FP8 ? ((kb + kt) & 1) * 16 : 0;   // a 128-k stage uses half of the granule's bytes
#pragma unroll
    for (int a = 0; a < NB; ++a) sw[a] = *reinterpret_cast<const int*>(rd_sw + u * C::STAGE + a * kScaleGranule) >> sh;
#pragma unroll
    for (int b = 0; b < MB; ++b) sx[b] = *reinterpret_cast<const int*>(rd_sx + u * C::STAGE + b * kScaleGranule) >> sh;
  };

  f32x16 acc[NB][MB];
  F fr[2];
  constexpr int NMMA = MB * NB;
  static_assert(C::INST * C::STRIDE <= NMMA * KS, "copies of a stage between two barriers");
  MxCopies<C> cp;   // the stage being filled
  // k-tile kt (in stage u); then the copies go to k-tile `ckt` of `from`, one after each
  // product, so that no wave waits for the memory pipe while its SIMD's matrix unit idles;
  // the ones that do not fit into the last k-step follow in the next k-tile. Every k-tile
  // reads one k-step ahead, the tile's last one too: a branch around those reads costs more.
  auto tile = [&](auto u_tag, int kt, const MxSrc<C>& from, int ckt) {
    constexpr int u = decltype(u_tag)::value;
    auto step = [&](auto tag) {
      constexpr int s = decltype(tag)::value;
      constexpr bool last = s == KS - 1;
      constexpr int PER = (PIECES + NMMA - 1) / NMMA;
      constexpr int ru = last ? u ^ 1 : u, rs = last ? 0 : s + 1;
      F& f = fr[s & 1];
      i32x4 xl[MB][C::XR];
      if constexpr (last) {
        wait_lgkmcnt<0>();   // this wave's reads of stage u are done
        wait_vmcnt<0>();     // and its copies of the next k-tile have landed
        barrier_only();
        cp = from.at(ckt, kb, w, lds + u * C::STAGE);
      }
      auto slot = [&](auto itag) {
        constexpr int i = decltype(itag)::value;
        constexpr int a = i % NB, b = i / NB;
        if constexpr (EXACT) {
          if constexpr (a == 0) {
#pragma unroll
            for (int h = 0; h < C::XR; ++h) {
              xl[b][h] = large_part(f.x[b][h]);
#pragma unroll
              for (int e = 0; e < 4; ++e) f.x[b][h][e] ^= xl[b][h][e];
            }
          }
          acc[a][b] = mx_mma<XF, s>(f.w[a], xl[b], acc[a][b], sw[a], sx[b]);
        }
        acc[a][b] = mx_mma<XF, s>(f.w[a], f.x[b], acc[a][b], sw[a], sx[b]);
#pragma unroll
        for (int e = 0; e < PER; ++e)
          if (i * PER + e < PIECES) piece(ru, rs, i * PER + e, fr[(s & 1) ^ 1]);
        constexpr int j = (last ? 0 : (s + 1) * NMMA) + i;
        if constexpr (j % C::STRIDE == 0 && j / C::STRIDE < C::INST)
          cp.template issue<j / C::STRIDE>(lane16, scales);
        __builtin_amdgcn_sched_barrier(0);
      };
      static_for<NMMA>(slot);
      if constexpr (last) read_scales(ru, kt + 1);
    };
    static_for<KS>(step);
  };
  constexpr std::integral_constant<int, 0> u0{};
  constexpr std::integral_constant<int, 1> u1{};

  // prologue: the first tile's first two k-tiles in flight, the first complete
  // (of the second, the copies that a k-tile's last step issues)
  constexpr int EARLY = (NMMA + C::STRIDE - 1) / C::STRIDE < C::INST ? (NMMA + C::STRIDE - 1) / C::STRIDE : C::INST;
  cp = src.at(0, kb, w, lds);
  cp.template issue_range<0, C::INST>(lane16, scales);
  cp = src.at(1, kb, w, lds + C::STAGE);
  cp.template issue_range<0, EARLY>(lane16, scales);
  wait_vmcnt<EARLY - 1>();   // (a wave that copies no scales has one copy less in flight)
  barrier_only();

  float* bias = reinterpret_cast<float*>(smem + C::OFF_EPI + w * C::EPI);   // NB * 32 values
  char* scratch = reinterpret_cast<char*>(bias + NB * 32);
  for (;;) {
    // this tile's bias, in the epilogue's LDS (its last reads are behind the barriers of
    // the tile before)
    const int c0w = at.tn * BN + wn * NB * 32;
    float bv[NB / 2];
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) bv[i] = mx_bias(p, at.e, c0w + i * 64 + lane);
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int b = 0; b < MB; ++b) acc[a][b] = f32x16{};
#pragma unroll
    for (int q = 0; q < PIECES; ++q) piece(0, 0, q, fr[0]);
    read_scales(0, 0);

    for (int kt = 0; kt < KT2 - 2; kt += 2) {
      tile(u0, kt, src, kt + 2);
      tile(u1, kt + 1, src, kt + 3);
    }
    MxPlace next = at;
    id += (int)gridDim.x;
    const bool more = mx_place<BM, 1>(p, id, true, next);
    src.set(p, next, XF, w, lane, kb, more ? KT : 0);
    tile(u0, KT2 - 2, src, 0);
    tile(u1, KT2 - 1, src, 1);
    // the sums exist here: without this the compiler moves the last products into the
    // branches of the epilogue, next to their uses, and spills the fragments meanwhile
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int b = 0; b < MB; ++b) asm volatile("" : "+v"(acc[a][b]));

#pragma unroll
    for (int i = 0; i < NB / 2; ++i) bias[i * 64 + lane] = bv[i];
    __builtin_amdgcn_wave_barrier();
    mx_epilogue<C>(p, at, wm, c0w, lane, acc, bias, scratch);
    if (!more) break;
    at = next;
  }
  wait_vmcnt<0>();   // no copy may land in LDS that the next workgroup owns
}

// ---- ring kernel ---------------------------------------------------------------------
// Small tiles: bound by the latency and rate of the copies, not by the products. One
// workgroup per tile and part of k. KG groups of waves take the k-tiles in turn, each with a
// ring of STAGES stages of its own, so that the copies, LDS reads and products of one
// group fill the waits of the other; their sums are added through LDS at the end.
// Per round one barrier; the LDS reads of the next k-tile and the copies of a later one run
// beside the products of this one. A k-tile's time is its copies' and reads', 0.17 us
// (64 x 64) to 0.88 us (128 x 256) with e4m3 X, against 0.04 to 0.28 us of products. 100 x 4096 x
// 11008 takes 16.5 us with W from memory (W alone is 3.8 us of reading) and 15.2 with three W in
// turn, which the 256 MB cache holds; 1000 x 4096 x 4096 21 us (1600 TFLOP/s).
template <int XF, int CFG, bool EXACT>
__global__ __launch_bounds__((MxCfgT<XF, CFG>::NW * MxCfgT<XF, CFG>::KG * 64), 1) void mx_ring_kernel(MxArgs p) {
  using C = MxCfgT<XF, CFG>;
  constexpr int MB = C::MB, NB = C::NB, KS = C::KS, ST = C::STAGES, KG = C::KG;
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  // The parts of a tile run on one XCD (the XCDs start a launch's workgroups some
  // microseconds apart, and the last part to arrive finishes the tile).
  const int q = p.splits > 1 ? xcd_remap(blockIdx.x, gridDim.x) : (int)blockIdx.x;
  const int part = q % p.splits;
  MxPlace at;
  if (CFG == kMxTailCfg && p.tail) {
    // quarter q % 4 of a 256 x 256 tile
    constexpr MxTile L = kMxTiles[MX_L];
    if (!mx_place<L.bm, 2>(p, q / 4, false, at)) return;
    at.row0 += q % 2 * C::T.bm;
    at.tn = at.tn * 2 + q / 2 % 2;
    if (at.row0 >= at.hi || at.tn * C::T.bn >= (p.out == MX_OUT_FP8 ? (int)pad_to(p.n, kKPad) : p.n)) return;
  } else if (!mx_place<C::T.bm>(p, q / p.splits, p.splits == 1, at)) {
    return;
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wave % C::NW, kg = wave / C::NW;
  const int wm = w % C::WAVES_M, wn = w / C::WAVES_M;
  const uint32_t lds = (uint32_t)(uintptr_t)(mx_lds_void*)smem + kg * C::STAGE;
  const uint32_t lane16 = lane * 16;
  const int KTA = (int)(pad_to(p.k, kKPad) / C::BK);
  const int kb = (int)((int64_t)KTA * part / p.splits), KT = (int)((int64_t)KTA * (part + 1) / p.splits) - kb;
  MxSrc<C> src;
  src.set(p, at, XF, w, lane, kb, KT);
  const int scales = w < C::SWV;

  f32x16 acc[NB][MB];
#pragma unroll
  for (int a = 0; a < NB; ++a)
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[a][b] = f32x16{};
  // the fragments and scales of one k-tile
  struct Tile {
    MxFrags<XF, MB, NB> f[KS];
    int sw[NB], sx[MB];
  };
  auto read = [&](int u, int kt, Tile& t) {   // k-tile kt from stage u
    const char* st = smem + (u * KG + kg) * C::STAGE;
#pragma unroll
    for (int a = 0; a < NB; ++a)
      t.sw[a] = *reinterpret_cast<const int*>(st + C::OFF_SW + (wn * NB + a) * kScaleGranule + lane * 4);
#pragma unroll
    for (int b = 0; b < MB; ++b)
      t.sx[b] = *reinterpret_cast<const int*>(st + C::OFF_SX + (wm * MB + b) * kScaleGranule + lane * 4);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
#pragma unroll
      for (int a = 0; a < NB; ++a)
        t.f[s].w[a] = *reinterpret_cast<const i32x4*>(st + (wn * NB + a) * C::WRB + s * 1024 + lane * 16);
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int h = 0; h < C::XR; ++h)
          t.f[s].x[b][h] = *reinterpret_cast<const i32x4*>(st + C::OFF_X + (wm * MB + b) * C::XRB +
                                                           (s * C::XR + h) * 1024 + lane * 16);
    }
  };
  auto wait_copies = [&]() {   // all but the copies of the last ST - 2 k-tiles have landed
    if (scales) wait_vmcnt<(ST - 2) * C::INST>();
    else wait_vmcnt<(ST - 2) * (C::INST - 1)>();
  };
#pragma unroll
  for (int t = 0; t < ST - 1; ++t)
    src.at(t * KG + kg, kb, w, lds + t * KG * C::STAGE).template issue_range<0, C::INST>(lane16, scales);
  wait_copies();
  barrier_only();
  Tile tiles[2];
  read(0, kg, tiles[0]);
  src.at((ST - 1) * KG + kg, kb, w, lds + (ST - 1) * KG * C::STAGE).template issue_range<0, C::INST>(lane16, scales);

  // Round r: k-tile r KG + kg is in registers; the next one is read and the one ST rounds
  // ahead copied while its products run. K-tiles past the last one are zeros.
  const int R = (KT + KG - 1) / KG;
  int u = 0;   // stage of the round's k-tile
  auto round = [&](int r, Tile& now, Tile& next) {
    wait_copies();
    wait_lgkmcnt<0>();   // this wave's reads of stage u are done
    barrier_only();
    const int kt = r * KG + kg, un = u + 1 == ST ? 0 : u + 1;
    read(un, kt + KG, next);
    const int sh = XF == FP8 ? ((kb + kt) & 1) * 16 : 0;   // a 128-k stage uses half of the granule's bytes
#pragma unroll
    for (int a = 0; a < NB; ++a) now.sw[a] >>= sh;
#pragma unroll
    for (int b = 0; b < MB; ++b) now.sx[b] >>= sh;
    const MxCopies<C> cp = src.at(kt + ST * KG, kb, w, lds + u * KG * C::STAGE);
    static_for<KS>([&](auto stag) {
      constexpr int s = decltype(stag)::value;
      static_for<MB * NB>([&](auto itag) {
        constexpr int i = decltype(itag)::value, a = i % NB, b = i / NB, N = MB * NB * KS;
        if constexpr (EXACT) {
          i32x4 xl[C::XR];
#pragma unroll
          for (int h = 0; h < C::XR; ++h) {
            xl[h] = large_part(now.f[s].x[b][h]);
            if constexpr (a == NB - 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) now.f[s].x[b][h][e] ^= xl[h][e];
            }
          }
          acc[a][b] = mx_mma<XF, s>(now.f[s].w[a], xl, acc[a][b], now.sw[a], now.sx[b]);
          if constexpr (a == NB - 1) {
#pragma unroll
            for (int c = 0; c < NB; ++c)
              acc[c][b] = mx_mma<XF, s>(now.f[s].w[c], now.f[s].x[b], acc[c][b], now.sw[c], now.sx[b]);
          }
        } else {
          acc[a][b] = mx_mma<XF, s>(now.f[s].w[a], now.f[s].x[b], acc[a][b], now.sw[a], now.sx[b]);
        }
        constexpr int j = s * MB * NB + i;   // the copies spread over the products
        cp.template issue_range<j * C::INST / N, (j + 1) * C::INST / N>(lane16, scales);
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    u = un;
  };
  for (int r = 0; r < R; r += 2) {
    round(r, tiles[0], tiles[1]);
    round(r + 1, tiles[1], tiles[0]);
  }
  wait_vmcnt<0>();
  __syncthreads();   // every wave is done with the stages, whose LDS serves the rest

  if constexpr (KG > 1) {
    f32x4* red = reinterpret_cast<f32x4*>(smem);
    constexpr int Q = NB * MB * 4;
    if (kg > 0) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const f32x16& v = acc[q / 4 % NB][q / 4 / NB];
        red[(((kg - 1) * C::NW + w) * Q + q) * 64 + lane] =
            f32x4{v[q % 4 * 4], v[q % 4 * 4 + 1], v[q % 4 * 4 + 2], v[q % 4 * 4 + 3]};
      }
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int o = 0; o < KG - 1; ++o)
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const f32x4 v = red[((o * C::NW + w) * Q + q) * 64 + lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[q / 4 % NB][q / 4 / NB][q % 4 * 4 + e] += v[e];
        }
    }
    __syncthreads();
  }
  if constexpr (MB == 1) {   // (the configurations that split k)
    if (p.splits > 1 && !mx_join_parts<C>(p, at, part, w, kg == 0, lane, acc, reinterpret_cast<int*>(smem))) return;
  }
  if (kg != 0) return;
  float* bias = reinterpret_cast<float*>(smem + C::OFF_EPI + w * C::EPI);
  char* scratch = reinterpret_cast<char*>(bias + NB * 32);
  const int c0w = at.tn * C::T.bn + wn * NB * 32;
  if (lane < NB * 32) bias[lane] = mx_bias(p, at.e, c0w + lane);
  __builtin_amdgcn_wave_barrier();
  mx_epilogue<C>(p, at, wm, c0w, lane, acc, bias, scratch);
}

// ---- skinny kernel -----------------------------------------------------------------
// Few rows: bound by reading W once. A workgroup takes 16 FB rows of W and up to 16 rows
// of X at a time; its waves split k, stream W from memory straight into registers (16 bytes a
// lane, consecutive lines) and add their sums through LDS in wave order. 16x16x128
// products: lane l holds row l % 16 and the 32 k of quarter l / 16 of a 128-k step.
// Rows of X are addressed one by one, so an expert's rows may start anywhere.
// One row by W from memory: 32768 x 8192 29 us (4.9 TB/s of W), 11008 x 4096 10.1 us and
// 4096 x 11008 10.0 us (2.4 TB/s: the launch, the first reads and the joining of the waves take
// about 4 us); 48 rows over 32 experts of 1376 x 4096 16.4 us.
template <int XF, int S>
__device__ __forceinline__ f32x4 mx_mma16(i32x4 w, const i32x4 (&x)[XF == FP8 ? 2 : 1], f32x4 c, int sw, int sx) {
  const i32x8 a = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
  if constexpr (XF == FP8) {
    const i32x8 b = {x[0][0], x[0][1], x[0][2], x[0][3], x[1][0], x[1][1], x[1][2], x[1][3]};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 0, S, sw, S, sx);
  } else {
    const i32x8 b = {x[0][0], x[0][1], x[0][2], x[0][3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, S, sw, S, sx);
  }
}

// A step of 128 k; the next one's loads are on their way during its products. (Two or more steps
// at a time read sooner but take registers, and with them resident waves: 11008 x 4096 8.7 us
// at one, 10.4 at two, 13.6 at four; without the step ahead 8.9, and 32768 x 8192 28.3
// instead of 25.8.)
template <int XF, int FB>
struct MxStep {
  i32x4 w[FB], x[XF == FP8 ? 2 : 1];
  int sw[FB], sx;
};

constexpr uint32_t kPastRange = 0x7fffffffu;   // rsrc()'s range

template <int XF, int FB>
__global__ __launch_bounds__(512, 4) void mx_skinny_kernel(MxArgs p) {
  constexpr int XR = XF == FP8 ? 2 : 1;
  constexpr bool EXACT = XF == FP8;   // see large_part
  const int nw = blockDim.x >> 6;
  constexpr int ROW = FB * 16 + 4;   // floats per finished row
  __shared__ __attribute__((aligned(16))) f32x4 red[kMxSkinnyWaves][FB][64];
  __shared__ __attribute__((aligned(16))) float fin[16][ROW];
  const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = p.experts ? blockIdx.y : 0;
  int64_t lo = 0, hi = p.m;
  if (p.experts) offset_rows(p, e, lo, hi);
  const int c0 = blockIdx.x * (FB * 16), fg = c0 >> 5;   // first row of W, its row group
  const int64_t gw = group_code_bytes(FP4, p.k), gx = group_code_bytes(XF, p.k), gs = group_scale_bytes(p.k);
  const int64_t wrg = row_groups(p.n);
  const bool has_w = fg < wrg;   // columns past the last group only pad an e4m3 result
  const int steps = has_w ? p.kt * 2 : 0;
  const int s0 = steps * w / nw, s1 = steps * (w + 1) / nw;
  const __amdgpu_buffer_rsrc_t rw = rsrc(p.wc + (e * wrg + (has_w ? fg : 0)) * gw), rws = rsrc(p.ws + (e * wrg + (has_w ? fg : 0)) * gs);
  const uint32_t lw = g * 512 + (c0 % 32 + li) * 16, lws = (g & 1) * 128 + (c0 % 32 + li) * 4;
  // The first FB waves finish the sums, four columns a lane. Their bias is read here as it
  // lies (an fp32 value in two halves), so that nothing waits for it before the end; past n
  // and without a bias the range gives zeros.
  const bool finish = w < FB;
  const int vs = p.vec == F32 ? 4 : 2;
  uint16_t b_lo[4] = {}, b_hi[4] = {};
  if (finish) {
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(p.bias)) + (int64_t)e * p.n * vs, 0, p.ep != NONE ? p.n * vs : 0, kBufDword3);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = (c0 + w * 16 + 4 * g + j) * vs;
      b_lo[j] = __builtin_amdgcn_raw_buffer_load_b16(rb, at, 0, 0);
      b_hi[j] = __builtin_amdgcn_raw_buffer_load_b16(rb, at + 2, 0, 0);
    }
  }

  for (int64_t r0 = lo + (int64_t)blockIdx.z * 16; r0 < hi; r0 += (int64_t)gridDim.z * 16) {
    // Lanes past the last row read the first one again: a row of X is a column of the
    // products, and theirs is not stored.
    const int64_t rr = r0 + li < hi ? r0 + li : r0;
    const __amdgpu_buffer_rsrc_t rx = rsrc(p.xc + (r0 >> 5) * gx), rxs = rsrc(p.xs + (r0 >> 5) * gs);
    const int rg = (int)((rr >> 5) - (r0 >> 5));   // the rows lie in one row group or two
    const uint32_t lx = rg * (int)gx + (int)(rr & 31) * 16 + g * 512, lxs = rg * (int)gs + (int)(rr & 31) * 4 + (g & 1) * 128;
    f32x4 acc[FB];
#pragma unroll
    for (int f = 0; f < FB; ++f) acc[f] = f32x4{0, 0, 0, 0};
    const auto load = [&](MxStep<XF, FB>& b, int t) {
      // steps past the wave's last one lie past the buffers' range: zeros, and no reads
      const uint32_t past = t < s1 ? 0u : kPastRange, ts = past | (uint32_t)((t >> 1) * kScaleGranule);
#pragma unroll
      for (int f = 0; f < FB; ++f) {
        b.w[f] = __builtin_amdgcn_raw_buffer_load_b128(rw, lw + f * 256 + (past | (uint32_t)(t * 2048)), 0, 0);
        b.sw[f] = __builtin_amdgcn_raw_buffer_load_b32(rws, lws + f * 64 + ts, 0, 0);
      }
#pragma unroll
      for (int h = 0; h < XR; ++h)
        b.x[h] = __builtin_amdgcn_raw_buffer_load_b128(rx, lx + h * 2048 + (past | (uint32_t)(t * (2048 * XR))), 0, 0);
      b.sx = __builtin_amdgcn_raw_buffer_load_b32(rxs, lxs + ts, 0, 0);
    };
    const auto multiply = [&](const MxStep<XF, FB>& b, int t) {
      const int sh = 16 * (t & 1) + 8 * (g >> 1);   // byte of the scale dword: block 4 (t % 2) + g of the granule
      i32x4 xf[XR];
#pragma unroll
      for (int h = 0; h < XR; ++h) xf[h] = b.x[h];
      if constexpr (EXACT) {
        i32x4 xl[XR];
#pragma unroll
        for (int h = 0; h < XR; ++h) {
          xl[h] = large_part(xf[h]);
          xf[h] ^= xl[h];
        }
#pragma unroll
        for (int f = 0; f < FB; ++f) acc[f] = mx_mma16<XF, 0>(b.w[f], xl, acc[f], b.sw[f] >> sh, b.sx >> sh);
      }
#pragma unroll
      for (int f = 0; f < FB; ++f) acc[f] = mx_mma16<XF, 0>(b.w[f], xf, acc[f], b.sw[f] >> sh, b.sx >> sh);
    };
    MxStep<XF, FB> b0, b1;
    load(b0, s0);
    for (int s = s0; s < s1; s += 2) {
      load(b1, s + 1);
      __builtin_amdgcn_sched_barrier(0);   // the loads first
      multiply(b0, s);
      load(b0, s + 2);
      __builtin_amdgcn_sched_barrier(0);
      multiply(b1, s + 1);
    }
    // Rows that are an earlier expert's, by offsets that run backwards, were computed and are
    // dropped here; the first wave stores. (Looking here at the offsets before e takes 0.4 of
    // 18.9 us with 512 rows over 64 experts of 2048 x 1024; waiting for them before the products
    // took 0.8.)
    int off_a = 0, off_b = 0;
    if (w == 0 && lane < e) {
      off_a = p.offsets[lane];
      off_b = p.offsets[lane + 1];
    }
#pragma unroll
    for (int f = 0; f < FB; ++f) red[w][f][lane] = acc[f];
    __syncthreads();
    if (finish) {
      const int f = w, l = lane;
      f32x4 v = red[0][f][l];
#pragma unroll 4
      for (int i = 1; i < nw; ++i) {
        const f32x4 u = red[i][f][l];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += u[j];
      }
      const int c = f * 16 + 4 * (l >> 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float bias = p.vec == F32   ? __uint_as_float(b_lo[j] | (uint32_t)b_hi[j] << 16)
                           : p.vec == F16 ? Tr<F16>::widen(b_lo[j])
                                          : Tr<BF16>::widen(b_lo[j]);
        const int col = c0 + c + j;
        const float y = mx_act(v[j] + bias, p.ep);
        fin[l & 15][c + j] = col < p.n ? y : 0.0f;
      }
    }
    __syncthreads();
    int own = 0;   // the first row to keep
    if (w == 0) {
      bool back = off_b < off_a;
      for (int i = lane + 64; i < e; i += 64) back |= p.offsets[i + 1] < p.offsets[i];
      if (__builtin_amdgcn_ballot_w64(back)) own = end_before(p, e);
    }
    if (FB == 2 && p.out == MX_OUT_FP8) {
      if (threadIdx.x < 16 && r0 + threadIdx.x < hi && r0 + threadIdx.x >= own) {
        const int t = threadIdx.x;
        float m = 0.0f;
        for (int c = 0; c < 32; ++c) m = amax2(m, mag(fin[t][c]));
        const int s = scale_of(m, FP8);
        for (int h = 0; h < 2; ++h) {
          const float* v = fin[t] + 16 * h;
          i32x4 o;
#pragma unroll
          for (int q = 0; q < 4; ++q) o[q] = (int)to_fp8x4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3], s);
          mx_store_chunk(p, r0 + t, c0 + 16 * h, o);
        }
        mx_store_scale(p, r0 + t, c0, s);
      }
    } else {
      const int t = threadIdx.x / (FB * 2), c = threadIdx.x % (FB * 2) * 8;
      if (t < 16 && r0 + t < hi && r0 + t >= own) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fin[t][c + j];
        mx_store8(p, r0 + t, c0 + c, v);
      }
    }
    __syncthreads();
  }
}

}  // namespace gek
