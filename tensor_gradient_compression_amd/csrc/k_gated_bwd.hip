// Gated linear layer: the gradients of x and of the weights from dg and du (k_gated.hip),
// dx = dg Wg + du Wu and dWg = dg^T x, dWu = du^T x, and the biases' from sums over rows.
//
// The operands lie as they are used elsewhere: the weights by rows of hidden, which dx sums
// over, and dg, du and x by rows, which the weights' gradients sum over. All of these come from
// LDS through the transposing reads, and no transposed copy is made.
// The weights' gradients are few tiles and a long sum (over all rows): it is split over
// workgroups, whose fp32 sums a second kernel joins in their order.
#include "gated.h"

namespace tg {

namespace {

// splits of a sum over k of `tiles` tiles: enough workgroups for every CU, and at least 512
// values of k each
int splits_of(int64_t tiles, int64_t k, int tile) {
  const int64_t want = tile == 0 ? 256 : 512;
  int64_t s = want / (tiles > 0 ? tiles : 1);
  if (s > k / 512) s = k / 512;
  if (s > 64) s = 64;
  return s < 1 ? 1 : (int)s;
}
int64_t tiles_of(int64_t ni, int64_t nj, int tile) {
  const int64_t b = tile == 0 ? 256 : tile == 1 ? 128 : 64;
  return ((ni + b - 1) / b) * ((nj + b - 1) / b);
}
// a tile for a product that may be split
int tile_of(int64_t ni, int64_t nj, int64_t k) {
  const int64_t big = tiles_of(ni, nj, 0), mid = tiles_of(ni, nj, 1);
  if (ni >= 256 && nj >= 256 && big * (k / 512 < 64 ? k / 512 : 64) >= 256) return 0;
  if (ni >= 128 && nj >= 128 && mid * (k / 512 < 64 ? k / 512 : 64) >= 128) return 1;
  return big >= 200 ? 0 : mid >= 200 ? 1 : 2;
}
// values of k of each split, whole stages
int64_t split_size(int64_t k, int splits) { return ((k + splits - 1) / splits + 63) / 64 * 64; }

// 4 sums to row m, columns n.. of a result of `cols` columns, or to a split's
template <typename T>
__device__ __forceinline__ void leave(T* out, float* partial, int64_t m, uint32_t n, uint32_t cols, f32x4 c) {
  const int k = (int)(cols - n < 4 ? cols - n : 4);
  if (partial) {
    store4(partial + m * cols + n, (const float*)&c, k, (cols & 3) == 0);
  } else {
    T v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = from_f32<T>(c[e]);
    store4(out + m * cols + n, v, k, (cols & 3) == 0 && ((uintptr_t)out & (4 * sizeof(T) - 1)) == 0);
  }
}

// dx: one sum over the gate's and the other weight's hidden values (65536 x 256 x 1024 in bf16: 95 us, 720
// TFLOP/s, one tile a CU that waits for 268 MB of dg and du; 8192 x 4096 x 8192: 966 us, 1138).
template <class S, int DT>
__global__ void __launch_bounds__(S::THREADS, 2) k_gated_dx(const GatedDx a, const int64_t size) {
  using G = GatedType<DT>;
  using T = typename G::T;
  extern __shared__ char lds_raw[];
  TG_LDS char* const lds = (TG_LDS char*)lds_raw;
  const uint32_t nj = (a.in + S::BN - 1) / S::BN, ni = (uint32_t)((a.rows + S::BM - 1) / S::BM);
  uint32_t ti, tj;
  tile_at(xcd_order(blockIdx.x, gridDim.x), ni, nj, ti, tj);
  const int64_t row0 = (int64_t)ti * S::BM, k0 = (int64_t)blockIdx.y * size;
  const uint32_t n0 = tj * S::BN, pad = gated_pad(a.hidden);
  const int64_t k = (int64_t)a.hidden - k0 < size ? (int64_t)a.hidden - k0 : size;   // zeros behind in dg and du
  MmSums<S> sums;
  mm_tile<S, G::MM, false, true, false>(
      sums, lds,
      [&](int s, MmOperand& g, MmOperand& w, MmOperand&) {
        // the parts' products of dg Wg, then those of du Wu
        const int up = s >= G::SEGS, q = up ? s - G::SEGS : s;
        GatedParts p = a.grads;
        p.p = (const char*)p.p + (up ? (size_t)pad * 2 : 0);
        p.len = pad;
        g = gated_operand<G::SEGS>(p, GATED_PART_A, q, k0, false);
        w = gated_operand<G::SEGS>(up ? a.wu : a.wg, GATED_PART_B, q, k0, true);
      },
      2 * G::SEGS, k, row0, n0, a.grads.stride, a.wg.stride);
  const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  float* const part = a.partial ? a.partial + (int64_t)blockIdx.y * a.rows * a.in : nullptr;
#pragma unroll
  for (int i = 0; i < S::FM; ++i) {
    const int64_t m = row0 + (wm * S::FM + i) * 16 + (lane & 15);
#pragma unroll
    for (int j = 0; j < S::FN; ++j) {
      const uint32_t n = n0 + (wn * S::FN + j) * 16 + (lane >> 4) * 4;
      if (m < a.rows && n < a.in) leave((T*)a.dx, part, m, n, a.in, sums.c[i][j]);
    }
  }
}

// dWg and dWu (65536 x 256 x 1024 in bf16: 92 us in 32 splits; 8192 x 4096 x 8192: 1063 us, 1034 TFLOP/s,
// where a library's product of two crossed operands reaches 1112).
template <class S, int DT>
__global__ void __launch_bounds__(S::THREADS, 2) k_gated_dw(const GatedDw a, const int64_t size) {
  using G = GatedType<DT>;
  using T = typename G::T;
  extern __shared__ char lds_raw[];
  TG_LDS char* const lds = (TG_LDS char*)lds_raw;
  const uint32_t pad = gated_pad(a.hidden);
  const uint32_t nj = (a.in + S::BN - 1) / S::BN, ni = (2 * pad + S::BM - 1) / S::BM;
  uint32_t ti, tj;
  tile_at(xcd_order(blockIdx.x, gridDim.x), ni, nj, ti, tj);
  const uint32_t f0 = ti * S::BM, n0 = tj * S::BN;
  const int64_t k0 = (int64_t)blockIdx.y * size, k = a.rows - k0 < size ? a.rows - k0 : size;
  MmSums<S> sums;
  mm_tile<S, G::MM, true, true, false>(
      sums, lds,
      [&](int s, MmOperand& g, MmOperand& x, MmOperand&) {
        g = gated_operand<G::SEGS>(a.grads, GATED_PART_A, s, k0, true);
        x = gated_operand<G::SEGS>(a.x, GATED_PART_B, s, k0, true);
      },
      G::SEGS, k, f0, n0, a.grads.stride, a.x.stride);
  const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  float* const part = a.partial ? a.partial + (int64_t)blockIdx.y * 2 * a.hidden * a.in : nullptr;
#pragma unroll
  for (int i = 0; i < S::FM; ++i) {
    uint32_t f = f0 + (wm * S::FM + i) * 16 + (lane & 15);
    const bool up = f >= pad;
    if (up) f -= pad;
#pragma unroll
    for (int j = 0; j < S::FN; ++j) {
      const uint32_t n = n0 + (wn * S::FN + j) * 16 + (lane >> 4) * 4;
      if (f >= a.hidden || n >= a.in) continue;
      leave((T*)(up ? a.dwu : a.dwg), part ? part + (up ? (int64_t)a.hidden * a.in : 0) : nullptr, f, n, a.in, sums.c[i][j]);
    }
  }
}

// out[v] = the sum of the n values v of `rows` rows, in their order; the values from `half` on
// go to out2 (32 rows of 524288: 14 us, 4.7 TB/s)
template <typename T>
__global__ void __launch_bounds__(256) k_gated_join(const float* p, int64_t rows, int64_t pitch, int64_t n, T* out,
                                                    T* out2, int64_t half, int64_t half_at) {
  const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (v >= n) return;
  const int64_t at = v < half ? v : v - half + half_at;
  float s = 0.0f;
  int64_t r = 0;
  for (; r + 8 <= rows; r += 8) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = p[(r + e) * pitch + at];
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[e];
  }
  for (; r < rows; ++r) s += p[r * pitch + at];
  if (v < half) out[v] = from_f32<T>(s);
  else out2[v - half] = from_f32<T>(s);
}
// The same for few columns and many rows: a workgroup takes 16 columns, 16 threads each
// (1024 rows of 2048: 7 us).
template <typename T>
__global__ void __launch_bounds__(256) k_gated_join_rows(const float* p, int64_t rows, int64_t pitch, int64_t n, T* out,
                                                         T* out2, int64_t half, int64_t half_at) {
  __shared__ float sums[16][17];
  const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int64_t v = (int64_t)blockIdx.x * 16 + c;
  const int64_t at = v < half ? v : v - half + half_at;
  float s = 0.0f;
  if (v < n) {
    int64_t r = q;
    for (; r + 7 * 16 < rows; r += 8 * 16) {   // eight loads under way
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = p[(r + e * 16) * pitch + at];
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x[e];
    }
    for (; r < rows; r += 16) s += p[r * pitch + at];
  }
  sums[q][c] = s;
  __syncthreads();
  if (q == 0 && v < n) {
    for (int i = 1; i < 16; ++i) s += sums[i][c];
    if (v < half) out[v] = from_f32<T>(s);
    else out2[v - half] = from_f32<T>(s);
  }
}

template <class S, class K, class A>
hipError_t launch_tiles(K* k, int64_t tiles, int splits, int64_t size, const A& a, hipStream_t s) {
  if (tiles > 0x7FFFFFFF / S::THREADS) return hipErrorInvalidValue;
  const hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS_BYTES);
  if (e != hipSuccess) return e;
  k<<<dim3((uint32_t)tiles, (uint32_t)splits), S::THREADS, S::LDS_BYTES, s>>>(a, size);
  return hipGetLastError();
}

using Big = MmBig;
using Mid = MmMid;
using Small = MmSmall;

template <int DT>
hipError_t dx_type(const GatedDx& a, hipStream_t s) {
  const int t = tile_of(a.rows, a.in, a.hidden), n = gated_dx_splits(a.rows, a.in, a.hidden);
  const int64_t tiles = tiles_of(a.rows, a.in, t), size = split_size(a.hidden, n);
  hipError_t e = t == 0   ? launch_tiles<Big>(k_gated_dx<Big, DT>, tiles, n, size, a, s)
                 : t == 1 ? launch_tiles<Mid>(k_gated_dx<Mid, DT>, tiles, n, size, a, s)
                          : launch_tiles<Small>(k_gated_dx<Small, DT>, tiles, n, size, a, s);
  if (e != hipSuccess || n == 1) return e;
  using T = typename GatedType<DT>::T;
  const int64_t v = a.rows * a.in;
  if ((v + 255) / 256 > 0x7FFFFFFF / 256) return hipErrorInvalidValue;
  k_gated_join<T><<<(uint32_t)((v + 255) / 256), 256, 0, s>>>(a.partial, n, v, v, (T*)a.dx, (T*)a.dx, v, 0);
  return hipGetLastError();
}

template <int DT>
hipError_t dw_type(const GatedDw& a, hipStream_t s) {
  using T = typename GatedType<DT>::T;
  const uint32_t pad = gated_pad(a.hidden);
  const int t = tile_of(2 * (int64_t)pad, a.in, a.rows), n = gated_dw_splits(a.rows, a.in, a.hidden);
  const int64_t tiles = tiles_of(2 * (int64_t)pad, a.in, t), size = split_size(a.rows, n);
  hipError_t e = !a.dwg   ? hipSuccess
                 : t == 0 ? launch_tiles<Big>(k_gated_dw<Big, DT>, tiles, n, size, a, s)
                 : t == 1 ? launch_tiles<Mid>(k_gated_dw<Mid, DT>, tiles, n, size, a, s)
                          : launch_tiles<Small>(k_gated_dw<Small, DT>, tiles, n, size, a, s);
  if (e == hipSuccess && a.dwg && n > 1) {
    const int64_t v = 2 * (int64_t)a.hidden * a.in;
    if ((v + 255) / 256 > 0x7FFFFFFF / 256) return hipErrorInvalidValue;
    k_gated_join<T><<<(uint32_t)((v + 255) / 256), 256, 0, s>>>(a.partial, n, v, v, (T*)a.dwg, (T*)a.dwu, v / 2, v / 2);
    e = hipGetLastError();
  }
  if (e == hipSuccess && a.dbg) {
    const int64_t v = 2 * (int64_t)a.hidden;
    k_gated_join_rows<T><<<(uint32_t)((v + 15) / 16), 256, 0, s>>>(a.row_sums, a.sum_rows, 2 * (int64_t)pad, v, (T*)a.dbg,
                                                                 (T*)a.dbu, a.hidden, pad);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

int gated_dx_splits(int64_t rows, uint32_t in, uint32_t hidden) {
  const int t = tile_of(rows, in, hidden);
  const int n = splits_of(tiles_of(rows, in, t), hidden, t);
  // none of them empty
  return (int)((hidden + split_size(hidden, n) - 1) / split_size(hidden, n));
}
int gated_dw_splits(int64_t rows, uint32_t in, uint32_t hidden) {
  const int64_t f = 2 * (int64_t)gated_pad(hidden);
  const int t = tile_of(f, in, rows), n = splits_of(tiles_of(f, in, t), rows, t);
  if (rows < 1) return 1;
  return (int)((rows + split_size(rows, n) - 1) / split_size(rows, n));
}

hipError_t launch_gated_dx(const GatedDx& a, hipStream_t s) {
  return a.dt == DT_F32 ? dx_type<DT_F32>(a, s) : a.dt == DT_F16 ? dx_type<DT_F16>(a, s) : dx_type<DT_BF16>(a, s);
}
hipError_t launch_gated_dw(const GatedDw& a, hipStream_t s) {
  return a.dt == DT_F32 ? dw_type<DT_F32>(a, s) : a.dt == DT_F16 ? dw_type<DT_F16>(a, s) : dw_type<DT_BF16>(a, s);
}

}  // namespace tg
