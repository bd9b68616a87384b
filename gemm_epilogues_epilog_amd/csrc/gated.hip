// The gated feed-forward block: entry points and small kernels.
//   H = act(G) * U, [G | U] = X W^T + bias;  Y = H Wd^T
//   dH = dY Wd;  dG = dH U a'(G), dU = dH a(G);  dX = dZ W, dW = dZ^T X, dWd = dY^T H
// with dZ = [dG | dU], so that both projections' products are one.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "gated_general.hpp"
#include "gated_host.hpp"
#include "gated_tiles.hpp"
#include "product.hpp"
#include "tiles.hpp"

namespace gek {
namespace {

// Eight values of a row of len from pos on (zeros past its end), widened. FLAT (rows of at least
// eight): without a branch, so that several are on their way at once.
template <int DT, bool FLAT = false>
__device__ __forceinline__ void load8(const void* row, int64_t pos, int64_t len, float (&v)[8]) {
  constexpr int ES = Tr<DT>::es, E = 16 / ES;
  const char* p = static_cast<const char*>(row);
  i32x4 raw[8 / E];
#pragma unroll
  for (int j = 0; j < 8 / E; ++j) {
    if constexpr (FLAT) {
      const int64_t to = pos + j * E, a = to < len - E ? to : len - E;
      raw[j] = shift_down<ES>(load16(p + a * ES), (int)(to - a < E ? to - a : E));
    } else {
      raw[j] = pos + 8 <= len ? load16(p + (pos + j * E) * ES) : load_end<ES>(p, pos + j * E, len);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (DT == F32) v[e] = __int_as_float(raw[e / 4][e % 4]);
    else v[e] = Tr<DT>::widen((uint16_t)((uint32_t)raw[0][e / 2] >> (16 * (e & 1))));
  }
}
template <int DT>
__device__ __forceinline__ void store8(void* row, int64_t pos, int64_t len, const float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float q[4] = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    store4<DT>(row, pos + 4 * h, len - pos - 4 * h, q);
  }
}

// dZ from dH and Z, eight columns a thread, where the product's kernel does not do it (fp32, unaligned
// rows, or dH given). Bound by memory: reads dH and Z, writes dZ.
template <int DT, int DH>
__global__ __launch_bounds__(256) void dz_kernel(const void* dh, const void* z, void* dz, int64_t m, int64_t n, int act) {
  constexpr int64_t es = Tr<DT>::es;
  const int cpr = (int)((n + 7) / 8);   // chunks of a row
  const int64_t first = (int64_t)blockIdx.x * 256, row0 = first / cpr;
  const int at = (int)(first - row0 * cpr) + threadIdx.x;
  const int64_t row = row0 + at / cpr, pos = (int64_t)(at % cpr) * 8;
  if (row >= m) return;
  float d[8], g[8], u[8], dg[8], du[8];
  load8<DH>(static_cast<const char*>(dh) + row * n * Tr<DH>::es, pos, n, d);
  const char* zr = static_cast<const char*>(z) + row * 2 * n * es;
  load8<DT>(zr, pos, n, g);
  load8<DT>(zr + n * es, pos, n, u);
  with_gate(act, [&](auto a) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v, s;
      gate_slope<decltype(a)::value, DT == F32>(g[e], v, s);
      dg[e] = d[e] * u[e] * s;
      du[e] = d[e] * v;
    }
  });
  char* o = static_cast<char*>(dz) + row * 2 * n * es;
  store8<DT>(o, pos, n, dg);
  store8<DT>(o + n * es, pos, n, du);
}

// The four rows' sums of a workgroup, V values for each of 64 lanes, in order.
template <int V>
__device__ __forceinline__ float four_rows(const float (&sums)[4][64][V + 1], int c, int e) {
  return ((sums[0][c][e] + sums[1][c][e]) + sums[2][c][e]) + sums[3][c][e];
}

// dz_kernel with partial[part][2 n], or with one part out[2 n] of type vec: sums of dZ's columns over the
// part's rows, before its rounding, in a fixed order: four rows side by side, each in ascending order, then
// those four in order. Bound by memory: 2048 x 11008 bf16 40 us, 5.6 TB/s (dz_kernel, which has more
// workgroups, 34).
template <int DT, int DH>
__global__ __launch_bounds__(256) void dz_sums_kernel(const void* dh, const void* z, void* dz, int64_t m, int64_t n,
                                                      int act, float* partial, void* out, int vec) {
  constexpr int64_t es = Tr<DT>::es;
  constexpr int U = 4;
  __shared__ float sums[4][64][17];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t pos = ((int64_t)blockIdx.x * 64 + c) * 8;
  const int64_t r0 = m * blockIdx.y / gridDim.y, r1 = m * (blockIdx.y + 1) / gridDim.y;
  float sg[8] = {}, su[8] = {};
  if (pos < n) {
    const auto add = [&](auto a, auto flat) {
      constexpr bool FLAT = decltype(flat)::value;
      for (int64_t r = r0 + q; r < r1; r += 4 * U) {
        float d[U][8], g[U][8], u[U][8];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int64_t at = r + 4 * i < r1 ? r + 4 * i : r;
          load8<DH, FLAT>(static_cast<const char*>(dh) + at * n * Tr<DH>::es, pos, n, d[i]);
          load8<DT, FLAT>(static_cast<const char*>(z) + at * 2 * n * es, pos, n, g[i]);
          load8<DT, FLAT>(static_cast<const char*>(z) + (at * 2 + 1) * n * es, pos, n, u[i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const bool in = r + 4 * i < r1;
          float dg[8], du[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float v, s;
            gate_slope<decltype(a)::value, DT == F32>(g[i][e], v, s);
            dg[e] = d[i][e] * u[i][e] * s;
            du[e] = d[i][e] * v;
            sg[e] += in ? dg[e] : 0.0f;
            su[e] += in ? du[e] : 0.0f;
          }
          if (in) {
            char* o = static_cast<char*>(dz) + (r + 4 * i) * 2 * n * es;
            store8<DT>(o, pos, n, dg);
            store8<DT>(o + n * es, pos, n, du);
          }
        }
      }
    };
    with_gate(act, [&](auto a) {
      if (n >= 8) add(a, std::true_type{});
      else add(a, std::false_type{});
    });
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    sums[q][c][e] = sg[e];
    sums[q][c][8 + e] = su[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 1024; i += 256) {
    const int64_t col = (int64_t)blockIdx.x * 512 + i % 512;
    if (col < n) {
      const float v = four_rows<16>(sums, i % 512 / 8, i / 512 * 8 + i % 8);
      const int64_t to = i / 512 * n + col;
      if (gridDim.y == 1) store_vec(out, vec, to, v);
      else partial[(int64_t)blockIdx.y * 2 * n + to] = v;
    }
  }
}

// The same of a dense (m, cols) matrix in fp32, cols a multiple of 8; with few rows bound by its start
// (4 us).
__global__ __launch_bounds__(256) void colsum_kernel(const float* x, int64_t m, int64_t cols, float* partial, void* out,
                                                     int vec) {
  constexpr int U = 4;
  __shared__ float sums[4][64][9];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t pos = ((int64_t)blockIdx.x * 64 + c) * 8;
  const int64_t r0 = m * blockIdx.y / gridDim.y, r1 = m * (blockIdx.y + 1) / gridDim.y;
  float s[8] = {};
  if (pos < cols) {
    for (int64_t r = r0 + q; r < r1; r += 4 * U) {
      float v[U][8];
#pragma unroll
      for (int i = 0; i < U; ++i) __builtin_memcpy(v[i], x + (r + 4 * i < r1 ? r + 4 * i : r) * cols + pos, 32);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += r + 4 * i < r1 ? v[i][e] : 0.0f;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[q][c][e] = s[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int64_t col = (int64_t)blockIdx.x * 512 + i;
    if (col < cols) {
      const float v = four_rows<8>(sums, i / 8, i % 8);
      if (gridDim.y == 1) store_vec(out, vec, col, v);
      else partial[(int64_t)blockIdx.y * cols + col] = v;
    }
  }
}

template <int DT, int OUT, int LAY>
const void* gen_of(bool large, bool narrow) {
  return narrow  ? reinterpret_cast<const void*>(&gen_kernel<DT, OUT, LAY, 64, 64, 32, 2, true>)
         : large ? reinterpret_cast<const void*>(&gen_kernel<DT, OUT, LAY, 128, 128, 64, 1, false>)
                 : reinterpret_cast<const void*>(&gen_kernel<DT, OUT, LAY, 64, 64, 32, 2, false>);
}
// (fp32 results of 16-bit operands: dH, and the sums of a shared k loop, which dX, dW and dWd have)
template <int DT>
const void* gen_kernel_of(int lay, bool f32_out, bool large, bool narrow) {
  switch (lay) {
    case 0: return f32_out ? gen_of<DT, F32, 0>(large, narrow) : gen_of<DT, DT, 0>(large, narrow);
    case 1: return f32_out ? gen_of<DT, F32, 1>(large, narrow) : gen_of<DT, DT, 1>(large, narrow);
    case 2: return gen_of<DT, DT, 2>(large, narrow);
    default: return gen_of<DT, DT, 6>(large, narrow);
  }
}

hipError_t launch(const void* fn, dim3 grid, int threads, void** params, hipStream_t s) {
  return hipLaunchKernel(fn, grid, dim3(threads), params, 0, s);
}

// The general kernel. lay 6: gated, N columns of D from 2 N rows of B. splits: workgroups that share
// a tile's k loop, D then that many matrices of sums.
hipError_t general(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, int lay, const void* A, const void* B, void* D,
                   bool f32_out, int splits, const void* bias, int vec, int act, void* Z, int cus, hipStream_t s) {
  GenArgs a;
  a.A = A;
  a.B = B;
  a.bias = bias;
  a.D = D;
  a.Z = Z;
  a.m = M;
  a.n = N;
  a.k = K;
  a.lda = lay & 1 ? M : K;
  a.ldb = lay & 2 ? K : N;
  a.ldd = N;
  a.vec = vec;
  a.act = act;
  // the large tile where it gives every compute unit one
  const auto tiles = [&](int t) { return (M + t - 1) / t * ((N + (lay == 6 ? t / 2 : t) - 1) / (lay == 6 ? t / 2 : t)); };
  const bool narrow = gegh::general_narrow(M, N, K, dt, lay);
  const bool large = !narrow && gegh::general_large(M, lay == 6 ? 2 * N : N, cus);
  const int t = large ? 128 : 64;
  a.tiles_m = (int)((M + t - 1) / t);
  a.tiles_n = (int)(tiles(t) / a.tiles_m);
  const void* fn = dt == GE_F32   ? gen_kernel_of<F32>(lay, f32_out, large, narrow)
                   : dt == GE_F16 ? gen_kernel_of<F16>(lay, f32_out, large, narrow)
                                  : gen_kernel_of<BF16>(lay, f32_out, large, narrow);
  void* params[] = {&a};
  return launch(fn, dim3((unsigned)tiles(t), (unsigned)splits), 256, params, s);
}

bool fast_product(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, int lay, const void* A, const void* B, const void* D) {
  return K > 0 && gegh::fast_shape(M, N, K, dt, lay) && gegh::aligned(A, 16) && gegh::aligned(B, 16) && gegh::aligned(D, 16);
}

// D (M, N) of type dt = A . B; `ws` for the k loop's split, its flags cleared already or not.
ge_status_t product(int64_t M, int64_t N, int64_t K, ge_dtype_t dt, int lay, const void* A, const void* B, void* D,
                    char* ws, size_t ws_bytes, bool cleared, int cus, hipStream_t s) {
  if (fast_product(M, N, K, dt, lay, A, B, D)) {
    geh::Layout L;
    if (ge_status_t st = gegh::fast_layout(M, N, K, dt, lay, cus, lay ? 0 : ws_bytes, &L); st != GE_OK) return st;
    return gei::run_product(M, (int)N, (int)K, dt, L, A, B, D, ws, cleared, s);
  }
  const int splits = gegh::general_splits(M, N, K, dt, ws_bytes);
  if (splits == 1)
    return general(M, N, K, dt, lay, A, B, D, false, 1, nullptr, F32, 0, nullptr, cus, s) == hipSuccess ? GE_OK : GE_ERR_HIP;
  if (general(M, N, K, dt, lay, A, B, ws, true, splits, nullptr, F32, 0, nullptr, cus, s) != hipSuccess) return GE_ERR_HIP;
  return launch_bgrad_reduce(reinterpret_cast<float*>(ws), splits, M * N, D, (int)dt, s) == hipSuccess ? GE_OK : GE_ERR_HIP;
}

// The tile kernels with the gated epilogues: H (and Z) of X and W, or dZ of dY, Wd and Z.
ge_status_t gated_tiles(int64_t m, int64_t n, int64_t k, ge_dtype_t dt, bool backward, int act, const void* A,
                        const void* B, const void* bias, int vec, const void* z, void* D, void* z_out, uint32_t* clear,
                        float* sums, int64_t* sum_rows, int cus, hipStream_t s) {
  geh::Layout L;
  if (ge_status_t st = gegh::gated_layout(m, n, k, dt, backward, cus, &L); st != GE_OK) return st;
  Args a = {};
  a.A = A;
  a.B = B;
  a.bias = bias;
  a.D = D;
  a.m = m;
  a.n = (int32_t)n;
  a.k = (int32_t)k;
  a.vec_dt = vec;
  a.tiles_m = L.tiles_m;
  a.tiles_n = L.tiles_n;
  a.group_m = L.group_m;
  a.dp_tiles = L.dp_tiles;
  a.persist_grid = L.persist_grid;
  a.act = act;
  a.z = z;
  a.z_out = z_out;
  a.clear = clear;
  a.sums = sums;
  if (sums) *sum_rows = (int64_t)L.tiles_m * (kTiles[L.cfg].bm / kTiles[L.cfg].wm);
  return get_launch_gated((int)dt, backward, L.cfg)(a, L.tiles_m * L.tiles_n, s) == hipSuccess ? GE_OK : GE_ERR_HIP;
}

// out[cols] of type vec from `rows` rows of sums; what lies behind them is scratch.
ge_status_t add_sums(float* sums, int64_t rows, int64_t cols, void* out, ge_dtype_t vec, hipStream_t s) {
  const int parts = rows ? (int)gegh::colsum_parts(rows, cols) : 0;
  float* partial = sums + rows * cols;
  int v = (int)vec;
  if (parts) {
    void* params[] = {&sums, &rows, &cols, &partial, &out, &v};
    if (launch(reinterpret_cast<const void*>(&colsum_kernel), dim3((unsigned)((cols + 511) / 512), parts), 256, params, s) != hipSuccess)
      return GE_ERR_HIP;
    if (parts == 1) return GE_OK;
  }
  return launch_bgrad_reduce(partial, parts, cols, out, v, s) == hipSuccess ? GE_OK : GE_ERR_HIP;
}

template <int DT>
const void* dz_sums_of(bool f32_dh) {
  return f32_dh ? reinterpret_cast<const void*>(&dz_sums_kernel<DT, F32>) : reinterpret_cast<const void*>(&dz_sums_kernel<DT, DT>);
}
// dZ from dH and Z, and out[2 n] of type vec: its column sums, by way of `partial`.
ge_status_t dz_sums(const void* dh, bool f32_dh, const void* z, void* dz, int64_t m, int64_t n, ge_dtype_t dt, int act, void* out,
                    ge_dtype_t vec, float* partial, hipStream_t s) {
  const int parts = (int)gegh::dz_parts(m, n);
  const void* fn = dt == GE_F32 ? dz_sums_of<F32>(f32_dh) : dt == GE_F16 ? dz_sums_of<F16>(f32_dh) : dz_sums_of<BF16>(f32_dh);
  int v = (int)vec;
  void* params[] = {&dh, &z, &dz, &m, &n, &act, &partial, &out, &v};
  if (launch(fn, dim3((unsigned)((n + 511) / 512), parts), 256, params, s) != hipSuccess) return GE_ERR_HIP;
  if (parts == 1) return GE_OK;
  return launch_bgrad_reduce(partial, parts, 2 * n, out, v, s) == hipSuccess ? GE_OK : GE_ERR_HIP;
}

ge_status_t status(hipError_t e) { return e == hipSuccess ? GE_OK : GE_ERR_HIP; }
const void* at(const void* p, int64_t bytes) { return p ? static_cast<const char*>(p) + bytes : nullptr; }
void* at(void* p, int64_t bytes) { return p ? static_cast<char*>(p) + bytes : nullptr; }

// The rows of one launch.
ge_status_t forward_rows(int64_t m, int64_t n, int64_t k, ge_dtype_t dt, ge_gate_t act, const void* x, const void* w,
                         const void* bias, ge_dtype_t vec, void* h, void* z, int cus, hipStream_t s) {
  const bool on16 = gegh::aligned(x, 16) && gegh::aligned(w, 16) && gegh::aligned(h, 16) && gegh::aligned(z, 16);
  switch (gegh::forward_kernel(m, n, k, dt, true, on16, cus)) {
    case gegh::Kernel::kFew:
      return status(launch_skinny(m, n, k, (int)dt, true, (int)act, x, w, bias, (int)vec, h, z, cus, s));
    case gegh::Kernel::kTiles:
      return gated_tiles(m, n, k, dt, false, (int)act, x, w, bias, (int)vec, nullptr, h, z, nullptr, nullptr, nullptr, cus, s);
    default:
      return status(general(m, n, k, dt, 6, x, w, h, false, 1, bias, (int)vec, (int)act, z, cus, s));
  }
}
ge_status_t down_rows(int64_t m, int64_t d, int64_t n, ge_dtype_t dt, const void* h, const void* w_down, void* y, int cus,
                      hipStream_t s) {
  if (gegh::forward_kernel(m, d, n, dt, false, false, cus) == gegh::Kernel::kFew)
    return status(launch_skinny(m, d, n, (int)dt, false, 0, h, w_down, nullptr, 0, y, nullptr, cus, s));
  return product(m, d, n, dt, 2, h, w_down, y, nullptr, 0, false, cus, s);
}

template <int DT>
const void* dz_of(bool f32_dh) {
  return f32_dh ? reinterpret_cast<const void*>(&dz_kernel<DT, F32>) : reinterpret_cast<const void*>(&dz_kernel<DT, DT>);
}

}  // namespace
}  // namespace gek

extern "C" {

ge_status_t gemm_epilog_gated_forward(int64_t m, int64_t n, int64_t k, ge_dtype_t dt, ge_gate_t act, const void* x,
                                      const void* w, const void* bias, ge_dtype_t vec, void* h, void* z, void* stream) {
  if (ge_status_t st = gegh::check_forward(m, n, k, dt, act, x, w, bias, vec, h, z); st != GE_OK) return st;
  if (m == 0) return GE_OK;
  int cus = 0;
  if (ge_status_t st = gei::current_device(&cus); st != GE_OK) return st;
  const int64_t most = gegh::launch_rows(n, true), row = (int64_t)geh::elem_size(dt);
  for (int64_t r = 0; r < m; r += most)
    if (ge_status_t st = gek::forward_rows(std::min(most, m - r), n, k, dt, act, gek::at(x, r * k * row), w, bias, vec,
                                           gek::at(h, r * n * row), gek::at(z, r * 2 * n * row), cus,
                                           static_cast<hipStream_t>(stream));
        st != GE_OK)
      return st;
  return GE_OK;
}

ge_status_t gemm_epilog_gated_down(int64_t m, int64_t d, int64_t n, ge_dtype_t dt, const void* h, const void* w_down,
                                   void* y, void* stream) {
  if (ge_status_t st = gegh::check_down(m, d, n, dt, h, w_down, y); st != GE_OK) return st;
  if (m == 0) return GE_OK;
  int cus = 0;
  if (ge_status_t st = gei::current_device(&cus); st != GE_OK) return st;
  const int64_t most = gegh::launch_rows(d, false), row = (int64_t)geh::elem_size(dt);
  for (int64_t r = 0; r < m; r += most)
    if (ge_status_t st = gek::down_rows(std::min(most, m - r), d, n, dt, gek::at(h, r * n * row), w_down,
                                        gek::at(y, r * d * row), cus, static_cast<hipStream_t>(stream));
        st != GE_OK)
      return st;
  return GE_OK;
}

size_t gemm_epilog_gated_workspace_bytes(int64_t m, int64_t n, int64_t k, int64_t d, ge_dtype_t dt) {
  return gegh::backward_space(m, n, k, d, dt).total;
}

ge_status_t gemm_epilog_gated_backward(int64_t m, int64_t n, int64_t k, int64_t d, ge_dtype_t dt, ge_gate_t act,
                                       const void* dy, const void* x, const void* w, const void* z, const void* h,
                                       const void* w_down, void* dx, void* dw, void* dw_down, void* dbias,
                                       ge_dtype_t vec, void* workspace, size_t workspace_bytes, void* stream) {
  const gegh::Backward b = {dy, x, w, z, h, w_down, dx, dw, dw_down, dbias};
  if (ge_status_t st = gegh::check_backward(m, n, k, d, dt, act, b, vec, workspace, workspace_bytes); st != GE_OK)
    return st;
  int cus = 0;
  if (ge_status_t st = gei::current_device(&cus); st != GE_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const gegh::BackwardSpace at = gegh::backward_space(m, n, k, d, dt);
  char* ws = static_cast<char*>(workspace);
  char* dz = ws;
  char* scratch = ws + at.scratch;
  const size_t scratch_bytes = workspace_bytes - at.scratch;   // (m = 0: nothing, and nothing is needed)

  if (m > 0 && (dx || dw || dbias)) {   // (dw_down needs neither dZ nor Z)
    const void* dh = dy;
    bool f32 = false;
    uint32_t* flags = nullptr;   // of a split of dX's product
    if (dx && gek::fast_product(m, k, 2 * n, dt, 0, dz, w, dx)) {
      geh::Layout L;
      if (ge_status_t st = gegh::fast_layout(m, k, 2 * n, dt, 0, cus, scratch_bytes, &L); st != GE_OK) return st;
      if (L.sk_wgs) flags = reinterpret_cast<uint32_t*>(scratch + L.off_sk_flag);
    }
    float* sums = reinterpret_cast<float*>(scratch + geh::kSkFlagRegion);   // (beside the flags)
    const bool on16 = gegh::aligned(dy, 16) && gegh::aligned(w_down, 16) && gegh::aligned(z, 16);
    if (w_down && gegh::gradient_kernel(m, n, d, dt, on16) == gegh::Kernel::kTiles) {
      int64_t sum_rows = 0;
      if (ge_status_t st = gek::gated_tiles(m, n, d, dt, true, (int)act, dy, w_down, nullptr, 0, z, dz, nullptr, flags,
                                            dbias ? sums : nullptr, &sum_rows, cus, s);
          st != GE_OK)
        return st;
      if (dbias)
        if (ge_status_t st = gek::add_sums(sums, sum_rows, 2 * n, dbias, vec, s); st != GE_OK) return st;
      dh = nullptr;
    } else if (w_down) {
      dh = ws + at.dh;
      f32 = true;
      if (gek::general(m, n, d, dt, 0, dy, w_down, ws + at.dh, true, 1, nullptr, 0, 0, nullptr, cus, s) != hipSuccess)
        return GE_ERR_HIP;
    }
    if (dh && dbias) {
      if (ge_status_t st = gek::dz_sums(dh, f32, z, dz, m, n, dt, (int)act, dbias, vec, sums, s); st != GE_OK) return st;
    } else if (dh) {
      const void* fn = dt == GE_F32   ? gek::dz_of<gek::F32>(f32)
                       : dt == GE_F16 ? gek::dz_of<gek::F16>(f32)
                                      : gek::dz_of<gek::BF16>(f32);
      int a = (int)act;
      void* params[] = {&dh, &z, &dz, &m, &n, &a};
      const int64_t chunks = m * ((n + 7) / 8);
      if (gek::launch(fn, dim3((unsigned)((chunks + 255) / 256)), 256, params, s) != hipSuccess) return GE_ERR_HIP;
    }
    if (dx)
      if (ge_status_t st = gek::product(m, k, 2 * n, dt, 0, dz, w, dx, scratch, scratch_bytes, !dh, cus, s); st != GE_OK)
        return st;
  }
  if (dw)
    if (ge_status_t st = gek::product(2 * n, k, m, dt, 1, dz, x, dw, scratch, scratch_bytes, false, cus, s); st != GE_OK) return st;
  if (dw_down)
    if (ge_status_t st = gek::product(d, n, m, dt, 1, dy, h, dw_down, scratch, scratch_bytes, false, cus, s); st != GE_OK) return st;
  if (dbias && m == 0)
    if (ge_status_t st = gek::add_sums(nullptr, 0, 2 * n, dbias, vec, s); st != GE_OK) return st;
  return GE_OK;
}

}  // extern "C"
