#include "mx_host.hpp"

#include <algorithm>
#include <cmath>

#include "mx_tiles.hpp"

namespace gemxh {

namespace {
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxK = int64_t(1) << 20;
// a launch of 256 lanes per tile keeps its lane count below 2^32
constexpr int64_t kMaxTiles = (int64_t(1) << 24) - 1;
bool has_bias(ge_epilog_t ep) { return ep != GE_EPILOG_NONE; }
}  // namespace

bool format_ok(ge_mx_format_t f) { return f == GE_MXFP4 || f == GE_MXFP8; }
bool dtype_ok(ge_dtype_t d) { return d == GE_F32 || d == GE_F16 || d == GE_BF16; }
size_t esize(ge_dtype_t d) { return d == GE_F32 ? 4 : 2; }
bool shape_ok(int64_t rows, int64_t k) {
  return rows >= 0 && rows <= kMaxRows && k >= 1 && k <= kMaxK &&
         gemx::row_groups(rows) * (gemx::pad_to(k, gemx::kKPad) / gemx::kKPad) <= kMaxTiles;
}

ge_status_t check_quantize(int64_t rows, int64_t k, ge_dtype_t dt, const void* src, int64_t row_stride,
                           int64_t col_stride, ge_mx_format_t fmt, const void* codes, const void* scales) {
  if (!format_ok(fmt) || !dtype_ok(dt) || !shape_ok(rows, k) || row_stride < 0 || col_stride < 0)
    return GE_ERR_INVALID_VALUE;
  if (rows == 0) return GE_OK;
  if (!src || !codes || !scales) return GE_ERR_NULL_POINTER;
  if (!aligned(src, esize(dt)) || !aligned(codes, 16) || !aligned(scales, 16)) return GE_ERR_MISALIGNED;
  return GE_OK;
}

ge_status_t check_dequantize(int64_t rows, int64_t k, ge_mx_format_t fmt, const void* codes, const void* scales,
                             ge_dtype_t dt, const void* dst, int64_t row_stride) {
  if (!format_ok(fmt) || !dtype_ok(dt) || !shape_ok(rows, k) || row_stride < (rows > 1 ? k : 0))
    return GE_ERR_INVALID_VALUE;
  if (rows == 0) return GE_OK;
  if (!dst || !codes || !scales) return GE_ERR_NULL_POINTER;
  if (!aligned(dst, esize(dt)) || !aligned(codes, 16) || !aligned(scales, 16)) return GE_ERR_MISALIGNED;
  return GE_OK;
}

ge_status_t check_pack(int64_t rows, int64_t k, ge_mx_format_t fmt, const void* src_codes, const void* src_scales,
                       const void* codes, const void* scales) {
  if (!format_ok(fmt) || !shape_ok(rows, k)) return GE_ERR_INVALID_VALUE;
  if (rows == 0) return GE_OK;
  if (!src_codes || !src_scales || !codes || !scales) return GE_ERR_NULL_POINTER;
  if (!aligned(codes, 16) || !aligned(scales, 16)) return GE_ERR_MISALIGNED;
  return GE_OK;
}

ge_status_t check_plan(int64_t n, int64_t k, int64_t experts, ge_mx_types_t t, ge_epilog_t ep) {
  if (n < 1 || n > kMaxK || k < 1 || k > kMaxK || experts < 0 || experts > 4096) return GE_ERR_INVALID_VALUE;
  if (!format_ok(t.x) || !dtype_ok(t.vec)) return GE_ERR_INVALID_VALUE;
  if (t.d != GE_MX_D_F32 && t.d != GE_MX_D_F16 && t.d != GE_MX_D_BF16 && t.d != GE_MX_D_MXFP8)
    return GE_ERR_INVALID_VALUE;
  switch (ep) {
    case GE_EPILOG_NONE:
    case GE_EPILOG_BIAS:
    case GE_EPILOG_RELU_BIAS:
    case GE_EPILOG_GELU_BIAS: break;
    case GE_EPILOG_RELU_AUX_BIAS:
    case GE_EPILOG_DRELU_BGRAD:
    case GE_EPILOG_RELU_BIAS_UNFUSED:
    case GE_EPILOG_DRELU_BGRAD_UNFUSED: return GE_ERR_NOT_SUPPORTED;
    default: return GE_ERR_INVALID_VALUE;
  }
  // the bias has D's type or fp32 (any type beside an 8-bit D)
  if (t.d != GE_MX_D_MXFP8 && t.vec != GE_F32 && (int)t.vec != (int)t.d) return GE_ERR_NOT_SUPPORTED;
  if (!shape_ok(n, k)) return GE_ERR_NOT_SUPPORTED;
  return GE_OK;
}

ge_status_t check_execute(int64_t m, int64_t experts, ge_mx_types_t t, ge_epilog_t ep, const void* xc, const void* xs,
                          const void* wc, const void* ws, const void* bias, const void* offsets, const void* D,
                          const void* ds) {
  if (m < 0 || m > kMaxRows) return GE_ERR_INVALID_VALUE;
  if (m == 0) return GE_OK;
  if (!xc || !xs || !wc || !ws || !D || (has_bias(ep) && !bias) || (experts && !offsets) ||
      (t.d == GE_MX_D_MXFP8 && !ds))
    return GE_ERR_NULL_POINTER;
  if (!aligned(xc, 16) || !aligned(xs, 16) || !aligned(wc, 16) || !aligned(ws, 16) ||
      (has_bias(ep) && !aligned(bias, esize(t.vec))) || (experts && !aligned(offsets, 4)) ||
      !aligned(D, t.d == GE_MX_D_MXFP8 ? 16 : t.d == GE_MX_D_F32 ? 4 : 2))
    return GE_ERR_MISALIGNED;
  return GE_OK;
}

// Estimated microseconds of each configuration; the least wins. The constants come from
// measurements (X e2m1; e4m3; e4m3 in two parts); `experts` products are estimated with three
// experts in four used, and half a tile of each left empty. (At the tile counts the launches
// have to allow for, 2000 rows over 8 experts of 2752 x 4096 to MXFP8 took 77 us, with the
// estimate 52; 11559 over 32 of 495 x 1792 44 and 32.)
MxLaunch choose(int64_t m, int64_t n, int64_t k, int64_t experts, ge_mx_types_t t, int cus) {
  using namespace gemx;
  MxLaunch L;
  const int64_t cols = t.d == GE_MX_D_MXFP8 ? pad_to(n, kKPad) : n;   // an 8-bit D is written with its padding
  const int64_t groups = experts ? experts : 1;
  const auto over = [](int64_t a, int64_t b) { return (a + b - 1) / b; };

  // Skinny kernel: the workgroups' work over the device, or one workgroup's way through its
  // rows, sixteen at a time, whichever is longer.
  double best;
  {
    const int64_t steps = pad_to(k, kKPad) / 128, sixteens = std::max<int64_t>(1, over(m, 16));
    // 16 columns each where 32 leave compute units idle (4096 x 11008, one row: 11.2 us, 9.0)
    L.cfg = t.d != GE_MX_D_MXFP8 && over(cols, 32) * groups < cus ? MX_S16N : MX_S16;
    L.tiles_n = (int)over(cols, kMxTiles[L.cfg].bn);
    L.tiles_m = (int)groups;
    L.grid_x = L.tiles_n;
    L.grid_y = groups;
    // Workgroups that share an expert's rows: two, as a skewed router gives some experts
    // several times the even share (m 320, n 1148, k 192, 16 experts: 8.4 us, one workgroup
    // 10.7, eight 9.7; 512 x 2048 x 1024 over 64: 23.2, 21.0 and 26.5), more where the
    // device has room.
    L.grid_z = std::min<int64_t>({sixteens, 64, std::max<int64_t>(experts ? 2 : 1, 2 * cus / (L.grid_x * groups))});
    // Waves by the 128-k steps there are: with workgroups to spare six or eight steps to each,
    // as a wave's start costs as much as some steps (32 experts of 1376 x 4096, 48 rows: two
    // waves 12.1 us, four 11.8, eight 12.8; 64 of 2048 x 1024, 512 rows: 15, 19, 36; 6144 x
    // 4096, one row: 7.6, 6.0, 6.4); otherwise two, to have the reads of k on their way
    // together (4096 x 11008, one row: 15, 10.6, 9.0).
    const int64_t wgs = L.grid_x * groups * L.grid_z;
    L.waves = (int)std::max<int64_t>(
        2, std::min<int64_t>(kMxSkinnyWaves, steps / (wgs > 4 * cus ? 8 : wgs > cus ? 6 : 2)));
    const double work = 1.0 + 0.36e-3 * (double)over(cols, 32) * ((double)m / 16 + 0.5 * (double)groups) * (double)steps;
    // (an expert may have four times the even share)
    const int64_t most = experts ? std::min(sixteens, over(4 * sixteens, groups)) : sixteens;
    const double way = (double)over(most, L.grid_z) * (1.0 + 0.5 * (double)over(steps, L.waves));
    best = 2.0 + std::max(work, way);
  }

  // Tile kernels: rounds of workgroups over the compute units, each so many k-tiles and a
  // fixed part (start, epilogue, joining parts of k).
  static constexpr double kPerTile[5][3] = {
      {1.55, 1.2, 2.1}, {1.2, 0.88, 1.6}, {0.58, 0.48, 0.87}, {0.34, 0.26, 0.42}, {0.19, 0.17, 0.33}};
  static constexpr double kFixed[5] = {5.0, 5.6, 5.8, 5.5, 4.6};
  const int kind = t.x == GE_MXFP4 ? 0 : (t.d == GE_MX_D_F32 || t.d == GE_MX_D_MXFP8) ? 2 : 1;
  const int64_t kt = pad_to(k, kKPad) / mx_bk((int)t.x);
  for (int cfg = MX_L; cfg <= MX_R64; ++cfg) {
    const MxTile& T = kMxTiles[cfg];
    const int64_t tm = experts ? (m + 31 * experts) / T.bm + experts : over(m, T.bm);   // at most
    const int64_t tn = over(cols, T.bn), tiles = tm * tn;
    const double used = std::max((double)m / T.bm + 0.5 * (double)experts, 0.75 * (double)experts) * (double)tn;
    const int most = T.mb > 1 || experts || tiles > kMxCounters
                         ? 1
                         : (int)std::max<int64_t>(1, std::min<int64_t>({cus / std::max<int64_t>(1, tiles), kt / 2, kMxMaxSplit}));
    const auto round_us = [&](int c, int s) { return (double)over(kt, s) * kPerTile[c][kind] + kFixed[c]; };
    // a short last round of large tiles goes to smaller ones (by expert it may)
    const int64_t rest = tiles % cus;
    const bool tail = cfg == MX_L && tiles > cus && (experts || (rest > 0 && rest <= cus / 4));
    for (int s = 1; s <= most; ++s) {
      double us;
      if (experts) {
        // (large tiles: a short last round is cut short, and part empty ones multiply fewer rows)
        us = cfg == MX_L ? std::max(1.0, used / cus + 0.3) * 0.85 * round_us(cfg, 1) + 4.0
                         : std::ceil(used / cus) * round_us(cfg, 1);
      } else {
        us = tail ? (double)(tiles / cus) * round_us(cfg, 1) + round_us(kMxTailCfg, 1) + 3.0
                  : (double)over(tiles * s, cus) * round_us(cfg, s);
      }
      us += cfg == MX_L ? 7.0 : s > 1 ? 1.0 * s : 0.0;
      if (us < best) {
        best = us;
        L = MxLaunch();
        L.cfg = cfg;
        L.tiles_m = (int)tm;
        L.tiles_n = (int)tn;
        L.splits = s;
        L.waves = mx_waves(T);
        L.tail = tail;
        // the persistent kernel: one workgroup per compute unit
        L.grid_x = cfg == MX_L ? std::min<int64_t>(tiles, cus) : tiles * s;
      }
    }
  }
  return L;
}

size_t workspace_bytes(int64_t experts, int cus) {
  using namespace gemx;
  if (experts) return 0;
  // split tiles times parts stay within one workgroup per compute unit
  return kMxCounterBytes + (size_t)cus * kMxTiles[MX_R128W].bm * kMxTiles[MX_R128W].bn * 4;   // the largest tile that splits
}

// ---- norm ---------------------------------------------------------------------------
namespace {
ge_status_t norm_common(int64_t rows, int64_t d, ge_dtype_t dt, ge_dtype_t wdt, float eps) {
  if (rows < 0 || rows > kMaxRows || d < 1 || !dtype_ok(dt) || !dtype_ok(wdt) || !(eps >= 0.0f) || std::isinf(eps))
    return GE_ERR_INVALID_VALUE;
  if (d > kNormMaxD || (wdt != GE_F32 && wdt != dt)) return GE_ERR_NOT_SUPPORTED;
  return GE_OK;
}
bool ld_ok(int64_t ld, int64_t rows, int64_t d) { return rows <= 1 || ld >= d; }
}  // namespace

ge_status_t check_norm(int64_t rows, int64_t d, ge_dtype_t dt, const void* x, int64_t ldx, const void* residual,
                       int64_t ldr, const void* weight, ge_dtype_t wdt, float eps, const void* sum, int64_t lds,
                       const void* y, int64_t ldy, const void* codes, const void* scales) {
  if (ge_status_t st = norm_common(rows, d, dt, wdt, eps); st != GE_OK) return st;
  // inputs may repeat a row (stride 0), outputs may not overlap
  if (ldx < 0 || (residual && ldr < 0) || (sum && !ld_ok(lds, rows, d)) || (y && !ld_ok(ldy, rows, d)))
    return GE_ERR_INVALID_VALUE;
  if (codes && !shape_ok(rows, d)) return GE_ERR_NOT_SUPPORTED;
  if (rows == 0) return GE_OK;
  if (!x || !weight || (!y && !codes) || (residual && !sum) || !codes != !scales) return GE_ERR_NULL_POINTER;
  const size_t e = esize(dt);
  if (!aligned(x, e) || !aligned(residual, e) || !aligned(weight, esize(wdt)) || !aligned(sum, e) || !aligned(y, e) ||
      !aligned(codes, 16) || !aligned(scales, 16))
    return GE_ERR_MISALIGNED;
  return GE_OK;
}

ge_status_t check_norm_backward(int64_t rows, int64_t d, ge_dtype_t dt, const void* dy, int64_t lddy, const void* s,
                                int64_t lds, const void* weight, ge_dtype_t wdt, float eps, const void* dres,
                                int64_t lddr, const void* dx, int64_t lddx, const void* dw, const void* ws,
                                size_t ws_bytes) {
  if (ge_status_t st = norm_common(rows, d, dt, wdt, eps); st != GE_OK) return st;
  if (lddy < 0 || lds < 0 || (dres && lddr < 0) || !ld_ok(lddx, rows, d)) return GE_ERR_INVALID_VALUE;
  if (!dw || !weight || (rows && (!dy || !s || !dx || !ws))) return GE_ERR_NULL_POINTER;
  const size_t e = esize(dt);
  if (!aligned(dy, e) || !aligned(s, e) || !aligned(weight, esize(wdt)) || !aligned(dres, e) || !aligned(dx, e) ||
      !aligned(dw, esize(wdt)) || !aligned(ws, 16))
    return GE_ERR_MISALIGNED;
  if (ws_bytes < norm_workspace_bytes(rows, d)) return GE_ERR_SCRATCH;
  return GE_OK;
}

int64_t norm_backward_groups(int64_t rows, int64_t d) {
  // Row slots: enough to fill the device, few enough to keep the second pass short (16384 x
  // 512, where four slots share a workgroup and its row of sums: 16.4 us at 2048, 18.7 at
  // 1024, 17.8 at 4096; 16384 x 1024: 30 at 1024, 34 at 2048, 37 at 512; 4096 x 4096: 26 at 512,
  // 32 at 1024; 16384 x 8192: 196 at 256, 203 at 512)
  return std::min<int64_t>(rows, d <= 512 ? 2048 : d <= 1024 ? 1024 : d <= 4096 ? 512 : 256);
}
size_t norm_workspace_bytes(int64_t rows, int64_t d) {
  if (rows <= 0 || d < 1) return 0;
  return (size_t)norm_backward_groups(rows, d) * (size_t)d * 4;
}

}  // namespace gemxh
