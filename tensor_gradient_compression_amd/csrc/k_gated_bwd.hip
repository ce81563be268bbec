// Gated linear layer: the gradients of x and of the weights from dg and du (k_gated.hip),
// dx = dg Wg + du Wu and dWg = dg^T x, dWu = du^T x, and the biases' from sums over rows.
//
// The operands lie as they are used elsewhere: the weights by rows of hidden, which dx sums
// over, and dg, du and x by rows, which the weights' gradients sum over. All of these come from
// LDS through the transposing reads, and no transposed copy is made.
// The weights' gradients are few tiles and a long sum (over all rows): it is split over
// workgroups, whose fp32 sums a second kernel joins in their order, or the last workgroup of a tile
// where the tiles are small.
#include "gated.h"

namespace tg {

namespace {

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

// A product of ni x nj with a sum over k in `segs` segments. Splits: enough workgroups for every CU,
// with 512 values of k each at least; a 64 x 64 tile's are counted and joined by its last workgroup up to
// 8 (1000 x 333 x 444 in fp32: dx, 96 tiles, 23.7 us by one workgroup a tile and 23.0 by five; dw, 84
// tiles, 23.2 and 19.9), more are left to the second kernel, which reads them on all CUs.
GatedWay way_of(int64_t ni, int64_t nj, int64_t k, int segs) {
  GatedWay w{tile_of(ni, nj, k), 1, false, 0};
  const int64_t tiles = tiles_of(ni, nj, w.tile);
  auto most = [&](int64_t s, int64_t limit) { return s < 1 ? 1 : s < limit ? s : limit; };
  if (w.tile == 2) {
    int64_t s = most(MM_MOST_SPLIT / (tiles > 0 ? tiles : 1), k * segs / 512);
    s = most(s, (k + 63) / 64);
    if (s > 1 && s <= MM_MOST_SPLITS) {
      w.counted = true;
      w.splits = (int)s;
      w.bytes = mm_split_bytes(tiles, s, 64);
      w.tile = 4;
      return w;
    }
    if (tiles > 256) w.tile = 4;
  }
  const int64_t s = most(most((w.tile == 0 ? 256 : 512) / (tiles > 0 ? tiles : 1), k / 512), 64);
  // none of them empty
  w.splits = k < 1 ? 1 : (int)((k + split_size(k, (int)s) - 1) / split_size(k, (int)s));
  return w;
}

// The rows lo..hi - 1 of a tile, which are rows `row0`.. of a result of `cols` columns (or of a split's,
// in fp32), from column n0 on.
template <typename T, class S>
__device__ __forceinline__ void leave_as(const MmSums<S>& sums, T* out, int64_t row0, int64_t lo, int64_t hi, uint32_t n0,
                                         uint32_t cols) {
  const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
  const int r = wave / S::WN * S::FM * 16 + (lane & 15);
  const uint32_t c = wave % S::WN * S::FN * 16 + (lane >> 4) * 4;
  const MmWindow to(out + row0 * cols + n0);
  const bool wide = (cols & 3) == 0 && ((uintptr_t)out & (4 * sizeof(T) - 1)) == 0;
#pragma unroll
  for (int i = 0; i < S::FM; ++i) {
    const bool row = r + i * 16 >= lo && r + i * 16 < hi;
    const uint32_t at = ((uint32_t)(r + i * 16 - (int)lo) * cols + c) * sizeof(T);
#pragma unroll
    for (int j = 0; j < S::FN; ++j) {
      const uint32_t n = n0 + c + j * 16, all = j * 16 * sizeof(T);
      alignas(16) T v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = from_f32<T>(sums.c[i][j][e]);
      if constexpr (sizeof(T) == 4) {
        if (wide) to.store16(*(const u32x4*)v, row && n < cols, at, all);
        else
#pragma unroll
          for (int e = 0; e < 4; ++e) to.store4(__builtin_bit_cast(uint32_t, v[e]), row && n + e < cols, at + e * 4, all);
      } else {
        if (wide) to.store8(*(const u32x2*)v, row && n < cols, at, all);
        else
#pragma unroll
          for (int e = 0; e < 4; ++e) to.store2(__builtin_bit_cast(uint16_t, v[e]), row && n + e < cols, at + e * 2, all);
      }
    }
  }
}
template <typename T, class S>
__device__ __forceinline__ void leave(const MmSums<S>& sums, T* out, float* partial, int64_t row0, int64_t lo, int64_t hi,
                                      uint32_t n0, uint32_t cols) {
  if (partial) leave_as(sums, partial, row0, lo, hi, n0, cols);
  else leave_as(sums, out, row0, lo, hi, n0, cols);
}

// dx: one sum over the gate's and the other weight's hidden values (65536 x 256 x 1024 in bf16: 84 us, 820
// TFLOP/s, one tile a CU that waits for 268 MB of dg and du; 8192 x 4096 x 8192: 907 us, 1212).
template <class S, int DT>
__global__ void __launch_bounds__(S::THREADS, 2) k_gated_dx(const GatedDx a, const int64_t size) {
  using G = GatedType<DT>;
  using T = typename G::T;
  extern __shared__ char lds_raw[];
  TG_LDS char* const lds = (TG_LDS char*)lds_raw;
  const uint32_t nj = (a.in + S::BN - 1) / S::BN, ni = (uint32_t)((a.rows + S::BM - 1) / S::BM);
  uint32_t ti, tj;
  tile_at(xcd_order(blockIdx.x, gridDim.x), ni, nj, ti, tj);
  constexpr bool NEAR = S::MODE == MM_AHEAD;
  const uint32_t split = NEAR && a.way.counted ? blockIdx.y : 0, splits = NEAR && a.way.counted ? gridDim.y : 1;
  const int64_t row0 = (int64_t)ti * S::BM, k0 = splits > 1 ? 0 : (int64_t)blockIdx.y * size;
  const uint32_t n0 = tj * S::BN, pad = gated_pad(a.hidden);
  const int segs = G::SEGS == 1 ? a.parts : G::SEGS;
  const int64_t k = (int64_t)a.hidden - k0 < size ? (int64_t)a.hidden - k0 : size;   // zeros behind in dg and du
  MmSums<S> sums;
  mm_tile<S, G::MM, false, true, false>(
      sums, lds,
      [&](int s, MmOperand& g, MmOperand& w, MmOperand&) {
        // the parts' products of dg Wg, then those of du Wu
        const int up = s >= segs, q = up ? s - segs : s;
        GatedParts p = a.grads;
        p.p = (const char*)p.p + (up ? (size_t)pad * 2 : 0);
        p.len = pad;
        g = gated_grad_operand<G::SEGS>(p, a.parts, q, k0, false);
        w = gated_operand<G::SEGS>(up ? a.wu : a.wg, GATED_PART_B, q, k0, true);
      },
      2 * segs, k, row0, n0, a.grads.stride, a.wg.stride, split, splits);
  if (NEAR && !whole_sums(sums, (uint32_t*)a.sums, ti * nj + tj, split, splits, lds)) return;
  float* const part = a.way.counted || a.way.splits == 1 ? nullptr : (float*)a.sums + (int64_t)blockIdx.y * a.rows * a.in;
  leave(sums, (T*)a.dx, part, row0, 0, a.rows - row0, n0, a.in);
}

// dWg and dWu (65536 x 256 x 1024 in bf16: 93 us in 32 splits; 8192 x 4096 x 8192: 948 us, 1160 TFLOP/s,
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
  constexpr bool NEAR = S::MODE == MM_AHEAD;
  const uint32_t split = NEAR && a.way.counted ? blockIdx.y : 0, splits = NEAR && a.way.counted ? gridDim.y : 1;
  const int64_t k0 = splits > 1 ? 0 : (int64_t)blockIdx.y * size, k = a.rows - k0 < size ? a.rows - k0 : size;
  MmSums<S> sums;
  mm_tile<S, G::MM, true, true, false>(
      sums, lds,
      [&](int s, MmOperand& g, MmOperand& x, MmOperand&) {
        g = gated_grad_operand<G::SEGS>(a.grads, a.parts, s, k0, true);
        x = gated_operand<G::SEGS>(a.x, GATED_PART_B, s, k0, true);
      },
      G::SEGS == 1 ? a.parts : G::SEGS, k, f0, n0, a.grads.stride, a.x.stride, split, splits);
  if (NEAR && !whole_sums(sums, (uint32_t*)a.sums, ti * nj + tj, split, splits, lds)) return;
  const int64_t each = (int64_t)a.hidden * a.in;
  float* const part = a.way.counted || a.way.splits == 1 ? nullptr : (float*)a.sums + (int64_t)blockIdx.y * 2 * each;
  if (f0 < a.hidden) leave(sums, (T*)a.dwg, part, f0, 0, (int64_t)a.hidden - f0, n0, a.in);
  const int64_t up = (int64_t)pad - f0;      // the tile's row where the other weight's begin
  if (up < S::BM)
    leave(sums, (T*)a.dwu, part ? part + each : nullptr, up < 0 ? -up : 0, up < 0 ? 0 : up, up + a.hidden, n0, a.in);
}

// out[v] = the sum of the n values v of `rows` rows, in their order; the values from `half` on
// go to out2 (32 rows of 524288: 11.5 us, 5.8 TB/s from the last-level cache)
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
// (1024 rows of 2048: 7.5 us).
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
  if (tiles > kMostThreads / S::THREADS) return hipErrorInvalidValue;
  const hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS_BYTES);
  if (e != hipSuccess) return e;
  k<<<dim3((uint32_t)tiles, (uint32_t)splits), S::THREADS, S::LDS_BYTES, s>>>(a, size);
  return hipGetLastError();
}

using Big = MmBig;
using Mid = MmMid;
using Small = MmSmall;
using Near = MmNear;

template <int DT>
hipError_t dx_type(const GatedDx& a, hipStream_t s) {
  const int t = a.way.tile, n = a.way.splits;
  const int64_t tiles = tiles_of(a.rows, a.in, t), size = a.way.counted ? a.hidden : split_size(a.hidden, n);
  hipError_t e = t == 0   ? launch_tiles<Big>(k_gated_dx<Big, DT>, tiles, n, size, a, s)
                 : t == 1 ? launch_tiles<Mid>(k_gated_dx<Mid, DT>, tiles, n, size, a, s)
                 : t == 2 ? launch_tiles<Small>(k_gated_dx<Small, DT>, tiles, n, size, a, s)
                          : launch_tiles<Near>(k_gated_dx<Near, DT>, tiles, n, size, a, s);
  if (e != hipSuccess || n == 1 || a.way.counted) return e;
  using T = typename GatedType<DT>::T;
  const int64_t v = a.rows * a.in;
  if ((v + 255) / 256 > kMostThreads / 256) return hipErrorInvalidValue;
  k_gated_join<T><<<(uint32_t)((v + 255) / 256), 256, 0, s>>>((const float*)a.sums, n, v, v, (T*)a.dx, (T*)a.dx, v, 0);
  return hipGetLastError();
}

template <int DT>
hipError_t dw_type(const GatedDw& a, hipStream_t s) {
  using T = typename GatedType<DT>::T;
  const uint32_t pad = gated_pad(a.hidden);
  const int t = a.way.tile, n = a.way.splits;
  const int64_t tiles = tiles_of(2 * (int64_t)pad, a.in, t), size = a.way.counted ? a.rows : split_size(a.rows, n);
  hipError_t e = !a.dwg   ? hipSuccess
                 : t == 0 ? launch_tiles<Big>(k_gated_dw<Big, DT>, tiles, n, size, a, s)
                 : t == 1 ? launch_tiles<Mid>(k_gated_dw<Mid, DT>, tiles, n, size, a, s)
                 : t == 2 ? launch_tiles<Small>(k_gated_dw<Small, DT>, tiles, n, size, a, s)
                          : launch_tiles<Near>(k_gated_dw<Near, DT>, tiles, n, size, a, s);
  if (e == hipSuccess && a.dwg && n > 1 && !a.way.counted) {
    const int64_t v = 2 * (int64_t)a.hidden * a.in;
    if ((v + 255) / 256 > kMostThreads / 256) return hipErrorInvalidValue;
    k_gated_join<T><<<(uint32_t)((v + 255) / 256), 256, 0, s>>>((const float*)a.sums, n, v, v, (T*)a.dwg, (T*)a.dwu, v / 2,
                                                                v / 2);
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

GatedWay gated_dx_way(int64_t rows, uint32_t in, uint32_t hidden, int parts) {
  GatedWay w = way_of(rows, in, hidden, 2 * gated_grad_segs(parts));
  if (w.splits > 1 && !w.counted) w.bytes = (size_t)w.splits * rows * in * 4;
  return w;
}
GatedWay gated_dw_way(int64_t rows, uint32_t in, uint32_t hidden, int parts) {
  GatedWay w = way_of(2 * (int64_t)gated_pad(hidden), in, rows, gated_grad_segs(parts));
  if (w.splits > 1 && !w.counted) w.bytes = (size_t)w.splits * 2 * hidden * in * 4;
  return w;
}

hipError_t launch_gated_dx(const GatedDx& a, hipStream_t s) {
  return a.dt == DT_F32 ? dx_type<DT_F32>(a, s) : a.dt == DT_F16 ? dx_type<DT_F16>(a, s) : dx_type<DT_BF16>(a, s);
}
hipError_t launch_gated_dw(const GatedDw& a, hipStream_t s) {
  return a.dt == DT_F32 ? dw_type<DT_F32>(a, s) : a.dt == DT_F16 ? dw_type<DT_F16>(a, s) : dw_type<DT_BF16>(a, s);
}

}  // namespace tg
