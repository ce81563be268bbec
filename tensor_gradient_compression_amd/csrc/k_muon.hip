// Newton-Schulz orthogonalisation of matrices, and the Muon step around it.
//
//   X = U / (|U| + eps);  `steps` times  A = X X^T,  B = b A + c A A,  X = a X + B X
// with the products on the side that has fewer rows (a tall matrix: A = X^T X, X = a X + X B),
// so that every singular value s of X goes through s (a + b s^2 + c s^4) and ends near 1.
//
// What the numbers need. The products are matrix instructions on fp16 (11 bits) with fp32 sums;
// X is bounded by its norm, so a power of two fixes the range. Small singular values grow by up
// to a^steps (485 for the usual 3.4445^5), and with them every rounding of X: with X in 16 bits
// alone the result is 2e-1 (bf16) or 4e-2 (fp16) of its norm off for a matrix of 16 strong
// directions and 1% of noise. Therefore
//   * X is carried in two fp16 parts (22 bits), and the linear term a X takes both. What the
//     upper part's rounding does to the products is not amplified: B's weight in a direction
//     falls with the square of its singular value;
//   * the diagonals of A and B stay fp32 vectors beside the matrices, whose diagonals are zero:
//     with D = diag(A), A A = D D + D O + O D + O O, and B X = diag(B) X + B' X. Near the end A
//     is the identity with little beside it, and the rounding of the large entries is gone.
// That leaves 3e-4 to 2e-3 of the result's norm on the spectra tried (a bf16 result is rounded by
// 1.7e-3); most of it is the lower part of X that B X leaves out. For fp32 and fp16 results the products take both parts of X, A and B
// (three products of parts; 3e-7 to 1e-5), which is `exact` here.
//
// What bounds it: matrix instructions for large matrices (8192 x 8192 in bf16: 12.0 ms; B X at 1115
// TFLOP/s, and A and A A, whose 528 tiles are three rounds of 256 with 16 tiles in the last, at 820); launches for middle ones (two, and three for every step; 777 x 2051 in fp16
// 325 us, in bf16 191); small ones are k_muon_small.hip's. All matrices of a handle share every launch.
// Of the symmetric products only the tiles on and below the diagonal are formed.
#include "muon.h"
#include "muon_common.h"

namespace tg {

static_assert(sizeof(NsCommon) + sizeof(MuonFirst) + sizeof(MuonTable) + sizeof(NsParts) <= 4096, "kernel arguments");

namespace {

constexpr uint32_t kPartsA = 0x001, kPartsB = 0x010;   // lower upper, upper lower, upper upper

__device__ __forceinline__ void workgroup_sum(double s, double* out) {
  __shared__ double w[4];
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) *out = (w[0] + w[1]) + (w[2] + w[3]);
}

// A chunk of a matrix: f(row, column, n) for pieces of 8 values of a line, n of them inside (zeros are
// what lines are padded with).
template <class F>
__device__ __forceinline__ void each_piece(const NsMat& m, uint32_t chunk, const F& f) {
  const uint32_t pieces = m.ldx / 8;
  const uint64_t first = (uint64_t)chunk * (MUON_CHUNK / 8), row0 = first / pieces;
  const uint32_t skip = (uint32_t)(first - row0 * pieces);
#pragma unroll
  for (uint32_t q = 0; q < MUON_CHUNK / 8 / 256; ++q) {
    const uint32_t at = skip + q * 256 + threadIdx.x, down = at / pieces, k = (at - down * pieces) * 8;
    const uint64_t row = row0 + down;
    if (row < m.rows) f((uint32_t)row, k, k >= m.cols ? 0 : m.cols - k < 8 ? m.cols - k : 8);
  }
}
// 8 values from p on, of which n are there (zeros behind)
template <typename T>
__device__ __forceinline__ void load_piece(const T* p, uint32_t n, float* v) {
  T raw[8] = {};
  if (n == 8) {
    load_values<8>(p, raw);
  } else {
#pragma unroll
    for (uint32_t e = 0; e < 7; ++e)
      if (e < n) raw[e] = p[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = to_f32(raw[e]);
}

// New momentum, and the sums of squares of the update: memory's (75M values of bf16 gradients 143 us,
// 5.3 TB/s). The update itself is formed again by the next pass, which costs a gradient's bytes where
// keeping it would cost four, twice.
__global__ void __launch_bounds__(256) k_muon_first(const NsCommon c, const MuonFirst f, const MuonTable t,
                                                    const NsParts p) {
  if (blockIdx.x == 0 && threadIdx.x < f.tensors) {
    f.w[f.first_tensor + threadIdx.x] = t.w[threadIdx.x];
    f.g[f.first_tensor + threadIdx.x] = t.g[threadIdx.x];
  }
  if (left_out(c)) return;
  const float coef = c.clip ? c.clip[1] : 1.0f;
  NsMat m;
  uint32_t chunk, none;
  my_part(c, p, blockIdx.x, m, chunk, none);
  double s = 0.0;
  with_type(m.gdt, [&](auto zero) {
    using T = decltype(zero);
    const T* const g = (const T*)t.g[m.tensor - f.first_tensor] + m.elem;
    float* const mom = f.momentum + m.state;
    each_piece(m, chunk, [&](uint32_t r, uint32_t k, uint32_t n) {
      const uint64_t o = (uint64_t)r * m.cols + k;
      float v[8], w[8];
      load_piece(g + o, n, v);
      load_piece(mom + o, n, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] *= coef;
        w[e] = f.mu * w[e] + f.nu * v[e];
        const double u = updated(v[e], w[e], f);
        s += u * u;
      }
      if (n == 8) {
        store_values<8>(mom + o, w);
      } else {
#pragma unroll
        for (uint32_t e = 0; e < 7; ++e)
          if (e < n) mom[o + e] = w[e];
      }
    });
  });
  workgroup_sum(s, (double*)(c.ws + m.sums) + chunk);
}

// Sums of squares of matrices given as they are (777 x 2051 in fp16: 5.2 us).
__global__ void __launch_bounds__(256) k_ns_norm(const NsCommon c, const NsSource f, const NsParts p) {
  NsMat m;
  uint32_t chunk, none;
  const uint32_t mat = my_part(c, p, blockIdx.x, m, chunk, none);
  double s = 0.0;
  with_type(m.gdt, [&](auto zero) {
    using T = decltype(zero);
    const T* const x = (const T*)f.x + mat * f.matrix_stride;
    each_piece(m, chunk, [&](uint32_t r, uint32_t k, uint32_t n) {
      float v[8];
      load_piece(x + r * f.row_stride + k, n, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += (double)v[e] * v[e];
    });
  });
  workgroup_sum(s, (double*)(c.ws + m.sums) + chunk);
}

// counters for whole_sums()
__device__ __forceinline__ void clear_counters(const NsCommon& c) {
  if (blockIdx.x || !c.counters) return;
  for (uint32_t i = threadIdx.x; i < MM_MOST_SPLIT; i += 256) c.counters[i] = 0;
}

// X's factor, by every workgroup from all sums of the matrix in their order
__device__ __forceinline__ NsScale start_scale(const NsCommon& c, const NsMat& m, double eps) {
  __shared__ double total;
  double s = 0.0;
  const double* const sums = (const double*)(c.ws + m.sums);
  for (uint32_t i = threadIdx.x; i < m.chunks; i += 256) s += sums[i];
  workgroup_sum(s, &total);
  __syncthreads();
  return NsScale(total, eps);
}

// 8 values of a line of X in their parts
__device__ __forceinline__ void write_x(const NsCommon& c, const NsMat& m, uint32_t r, uint32_t k, const float* v,
                                        const NsScale& scale) {
  _Float16* const hi = (_Float16*)(c.ws + m.x) + (uint64_t)r * m.ldx + k;
  _Float16 h[8], l[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) two_parts(scale(v[e]), h[e], l[e]);
  *(uint4*)hi = *(const uint4*)h;
  *(uint4*)(hi + (uint64_t)m.rows * m.ldx) = *(const uint4*)l;
}

// X in its parts from the update: memory's (75M values of bf16 gradients 145 us, 5.2 TB/s).
__global__ void __launch_bounds__(256) k_muon_start(const NsCommon c, const MuonFirst f, const double eps, const NsParts p) {
  if (left_out(c)) return;
  clear_counters(c);
  const float coef = c.clip ? c.clip[1] : 1.0f;
  NsMat m;
  uint32_t chunk, none;
  my_part(c, p, blockIdx.x, m, chunk, none);
  const NsScale scale = start_scale(c, m, eps);
  with_type(m.gdt, [&](auto zero) {
    using T = decltype(zero);
    const T* const g = (const T*)f.g[m.tensor] + m.elem;
    const float* const mom = f.momentum + m.state;
    each_piece(m, chunk, [&](uint32_t r, uint32_t k, uint32_t n) {
      const uint64_t o = (uint64_t)r * m.cols + k;
      float v[8], w[8];
      load_piece(mom + o, n, w);
      if (f.nesterov) {
        load_piece(g + o, n, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = updated(v[e] * coef, w[e], f);
      }
      write_x(c, m, r, k, w, scale);
    });
  });
}

__global__ void __launch_bounds__(256) k_ns_start(const NsCommon c, const NsSource f, const double eps, const NsParts p) {
  clear_counters(c);
  NsMat m;
  uint32_t chunk, none;
  const uint32_t mat = my_part(c, p, blockIdx.x, m, chunk, none);
  const NsScale scale = start_scale(c, m, eps);
  with_type(m.gdt, [&](auto zero) {
    using T = decltype(zero);
    const T* const x = (const T*)f.x + mat * f.matrix_stride;
    each_piece(m, chunk, [&](uint32_t r, uint32_t k, uint32_t n) {
      float v[8];
      load_piece(x + r * f.row_stride + k, n, v);
      write_x(c, m, r, k, v, scale);
    });
  });
}

// The part of segment s of a matrix in fp16 parts.
__device__ __forceinline__ MmOperand ns_operand(const NsCommon& c, const NsMat& m, uint64_t at, uint32_t lines, uint32_t ld,
                                                uint32_t parts, int s) {
  MmOperand o;
  const uint32_t part = m.exact ? (parts >> (4 * s)) & 3u : 0u;
  o.p = c.ws + at + (uint64_t)part * lines * ld * 2;
  o.lines = lines;
  o.len = o.stride = ld;
  return o;
}

// The tile and the split of this workgroup: a tile's are neighbours.
__device__ __forceinline__ void my_split(const NsParts& p, uint32_t& tile, uint32_t& split) {
  const uint32_t t = xcd_order(blockIdx.x, gridDim.x);
  tile = t / p.splits;
  split = t - tile * p.splits;
}

__device__ __forceinline__ uint32_t whole8(uint32_t n) { return (n + 7u) & ~7u; }

// Where this lane's sums are: four columns of a row in each block.
template <class S>
struct Place {
  uint32_t r, c;                    // of the first block, in the tile
  int wi, wj;                       // its wave's first block
  __device__ __forceinline__ Place() {
    const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
    wi = wave / S::WN * S::FM;
    wj = wave % S::WN * S::FN;
    r = wi * 16 + (lane & 15);
    c = wj * 16 + (lane >> 4) * 4;
  }
};

// f(i, j, what load(i, j) gave) for all blocks. Some blocks' loads go out before the first of
// their stores, which the compiler would not let them pass: waits for memory one after another, and
// branches around every access, were most of an epilogue (a sum over 768 by 128 x 128 tiles: 9 of 19 us).
template <class S, class V, class Load, class F>
__device__ __forceinline__ void each_block(const Load& load, const F& f) {
  constexpr int BLOCKS = sizeof(V) > 32 ? 4 : sizeof(V) > 16 ? 8 : 16;
  constexpr int ROWS = S::FM * S::FN > BLOCKS ? BLOCKS / S::FN : S::FM;
  static_assert(S::FM % ROWS == 0, "whole groups");
#pragma unroll
  for (int g = 0; g < S::FM; g += ROWS) {
    V v[ROWS][S::FN];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) v[i][j] = load(g + i, j);
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) f(g + i, j, v[i][j]);
  }
}
struct Nothing {};
// four values in their parts
struct Four {
  u32x2 h, l;
  __device__ __forceinline__ void get(float* v) const {
    _Float16 a[4], b[4];
    __builtin_memcpy(a, &h, 8);
    __builtin_memcpy(b, &l, 8);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)a[e] + (float)b[e];
  }
};

// A symmetric matrix around the tile at (i0, j0), and its other half.
struct Symmetric {
  MmWindow hi, lo, mirrored_hi, mirrored_lo;
  __device__ __forceinline__ Symmetric(const NsCommon& c, const NsMat& m, uint64_t at, uint32_t i0, uint32_t j0)
      : hi(c.ws + at + ((uint64_t)i0 * m.ldm + j0) * 2), lo(c.ws + at + ((uint64_t)m.m * m.ldm + (uint64_t)i0 * m.ldm + j0) * 2),
        mirrored_hi(c.ws + at + ((uint64_t)j0 * m.ldm + i0) * 2),
        mirrored_lo(c.ws + at + ((uint64_t)m.m * m.ldm + (uint64_t)j0 * m.ldm + i0) * 2) {}
};

// v (four columns under NS_M, of block (bi, bj)) to a symmetric matrix, and to its other half. The
// rows from m to ldm are only the other half's padding.
template <class S>
__device__ __forceinline__ void write_symmetric(const NsMat& m, const Symmetric& to, const Place<S>& at, uint32_t i0,
                                                uint32_t j0, int bi, int bj, const float* v) {
  _Float16 h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) two_parts(v[e], h[e], l[e]);
  const uint32_t i = i0 + at.r + bi * 16, j = j0 + at.c + bj * 16;
  const bool in = i < m.m && j < m.ldm;
  const uint32_t lane = (at.r * m.ldm + at.c) * 2, all = (bi * 16 * m.ldm + bj * 16) * 2;
  to.hi.store8(*(const u32x2*)h, in, lane, all);
  if (m.exact) to.lo.store8(*(const u32x2*)l, in, lane, all);
  if (i0 == j0) return;
  const uint32_t mlane = (at.c * m.ldm + at.r) * 2, mall = (bj * 16 * m.ldm + bi * 16) * 2;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool min = i < m.ldm && j + e < m.m;
    to.mirrored_hi.store2(__builtin_bit_cast(uint16_t, h[e]), min, mlane + e * m.ldm * 2, mall);
    if (m.exact) to.mirrored_lo.store2(__builtin_bit_cast(uint16_t, l[e]), min, mlane + e * m.ldm * 2, mall);
  }
}

// The entries of block (bi, bj) on the diagonal: f(row, e) in the lanes that hold one.
template <class S, class F>
__device__ __forceinline__ void on_diagonal(const NsMat& m, const Place<S>& at, uint32_t i0, uint32_t j0, int bi, int bj, const F& f) {
  if (i0 != j0 || at.wi + bi != at.wj + bj) return;   // all lanes alike
  const uint32_t i = i0 + at.r + bi * 16, e = (at.r & 15) - (at.c & 15);
  if (e < 4 && i < m.m) f(i, e);
}
__device__ __forceinline__ float pick(const float* v, uint32_t e) { return e == 0 ? v[0] : e == 1 ? v[1] : e == 2 ? v[2] : v[3]; }

// A = X X^T (X^T X): its diagonal, and the rest under NS_M. Both operands are X, by its rows or across
// them. Matrix instructions' and LDS's (18 of 1024 x 4096: 112 us, 690 TFLOP/s on 180 tiles; 8192 x 8192
// 669, 820), latency's with few tiles (777 x 2051, three products in five splits: 20 us).
template <class S>
__global__ void __launch_bounds__(S::THREADS, 2) k_ns_gram(const NsCommon c, const int at, const NsParts p) {
  extern __shared__ char lds_raw[];
  if (left_out(c)) return;
  NsMat m;
  uint32_t ti, tj, tile, split;
  my_split(p, tile, split);
  my_part(c, p, tile, m, ti, tj);
  const uint32_t i0 = ti * S::BM, j0 = tj * S::BN;
  const uint64_t from = at ? m.y : m.x;
  MmSums<S> sums;
  const uint32_t splits = S::MODE == MM_TURNS ? 1 : p.splits;
  auto source = [&](int s, MmOperand& a, MmOperand& b, MmOperand&) {
    a = ns_operand(c, m, from, m.rows, m.ldx, kPartsA, s);
    b = ns_operand(c, m, from, m.rows, m.ldx, kPartsB, s);
  };
  const int nseg = m.exact ? 3 : 1;
  if (m.rows <= m.cols)
    mm_tile<S, DT_F16, false, false, false>(sums, (TG_LDS char*)lds_raw, source, nseg, whole8(m.cols), i0, j0, m.ldx, m.ldx, split,
                                           splits);
  else
    mm_tile<S, DT_F16, true, true, false>(sums, (TG_LDS char*)lds_raw, source, nseg, m.rows, i0, j0, m.ldx, m.ldx, split, splits);
  if (S::MODE != MM_TURNS && !whole_sums(sums, c.counters, tile, split, p.splits, (TG_LDS char*)lds_raw)) return;
  float* const diag = (float*)(c.ws + m.da);
  const Place<S> at_tile;
  const Symmetric to(c, m, m.a, i0, j0);
  each_block<S, Nothing>([](int, int) { return Nothing{}; }, [&](int bi, int bj, Nothing) {
    const f32x4 v = sums.c[bi][bj];
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = i0 + at_tile.r + bi * 16 < m.m && j0 + at_tile.c + bj * 16 + e < m.m ? v[e] * (NS_M / (NS_X * NS_X)) : 0.0f;
    on_diagonal(m, at_tile, i0, j0, bi, bj, [&](uint32_t i, uint32_t d) {
      diag[i] = pick(o, d) * (1.0f / NS_M);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = d == (uint32_t)e ? 0.0f : o[e];
    });
    write_symmetric(m, to, at_tile, i0, j0, bi, bj, o);
  });
}

// B = b A + c A A from A off its diagonal, O: A A = D D + D O + O D + O O, so that the products
// see only O. As k_ns_gram (18 of 1024: 51 us; 8192: 668).
template <class S>
__global__ void __launch_bounds__(S::THREADS, 2) k_ns_poly(const NsCommon c, const NsParts p) {
  extern __shared__ char lds_raw[];
  if (left_out(c)) return;
  NsMat m;
  uint32_t ti, tj, tile, split;
  my_split(p, tile, split);
  my_part(c, p, tile, m, ti, tj);
  const uint32_t i0 = ti * S::BM, j0 = tj * S::BN;
  MmSums<S> sums;
  const uint32_t splits = S::MODE == MM_TURNS ? 1 : p.splits;
  mm_tile<S, DT_F16, false, false, false>(
      sums, (TG_LDS char*)lds_raw,
      [&](int s, MmOperand& a, MmOperand& b, MmOperand&) {
        a = ns_operand(c, m, m.a, m.m, m.ldm, kPartsA, s);
        b = ns_operand(c, m, m.a, m.m, m.ldm, kPartsB, s);
      },
      m.exact ? 3 : 1, whole8(m.m), i0, j0, m.ldm, m.ldm, split, splits);
  if (S::MODE != MM_TURNS && !whole_sums(sums, c.counters, tile, split, p.splits, (TG_LDS char*)lds_raw)) return;
  float* const db = (float*)(c.ws + m.db);
  const Place<S> at;
  const Symmetric from(c, m, m.a, i0, j0), to(c, m, m.b, i0, j0);
  const MmWindow da_i((const float*)(c.ws + m.da) + i0), da_j((const float*)(c.ws + m.da) + j0);
  float di[S::FM];
  f32x4 dj[S::FN];                      // behind the m-th anything
#pragma unroll
  for (int i = 0; i < S::FM; ++i) di[i] = __uint_as_float(da_i.load4(i0 + at.r + i * 16 < m.m, at.r * 4, i * 64));
#pragma unroll
  for (int j = 0; j < S::FN; ++j) dj[j] = __builtin_bit_cast(f32x4, da_j.load16(j0 + at.c + j * 16 < m.ldm, at.c * 4, j * 64));
  auto load = [&](int bi, int bj) {
    const bool in = i0 + at.r + bi * 16 < m.m && j0 + at.c + bj * 16 < m.ldm;
    const uint32_t lane = (at.r * m.ldm + at.c) * 2, all = (bi * 16 * m.ldm + bj * 16) * 2;
    Four x = {};
    x.h = from.hi.load8(in, lane, all);
    if (m.exact) x.l = from.lo.load8(in, lane, all);
    return x;
  };
  each_block<S, Four>(load, [&](int bi, int bj, const Four& old) {
    const f32x4 v = sums.c[bi][bj];
    float x[4], o[4];
    old.get(x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float q = v[e] * (1.0f / (NS_M * NS_M)), y = x[e] * (1.0f / NS_M);
      const float b = (c.cb * y + c.cc * (q + (di[bi] + dj[bj][e]) * y)) * NS_M;
      o[e] = i0 + at.r + bi * 16 < m.m && j0 + at.c + bj * 16 + e < m.m ? b : 0.0f;
    }
    on_diagonal(m, at, i0, j0, bi, bj, [&](uint32_t i, uint32_t d) {
      const float q[4] = {v[0], v[1], v[2], v[3]};
      db[i] = c.cb * di[bi] + c.cc * (di[bi] * di[bi] + pick(q, d) * (1.0f / (NS_M * NS_M)));
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = d == (uint32_t)e ? 0.0f : o[e];
    });
    write_symmetric(m, to, at, i0, j0, bi, bj, o);
  });
}

// X = a X + B X (a X + X B), with B's diagonal in fp32 and X's parts read and written where the sums
// are: 8 bytes a value of reading and writing after the products, which is half of the time where sums are
// short (18 of 1024 x 4096: 309 us, 154 GFLOP and 600 MB; 8192 x 8192: 986, 1115 TFLOP/s). The last one
// writes the result, or the weights.
template <class S>
__global__ void __launch_bounds__(S::THREADS, 2) k_ns_apply(const NsCommon c, const int at, const NsLast last, const NsParts p) {
  extern __shared__ char lds_raw[];
  if (left_out(c)) return;
  NsMat m;
  uint32_t ti, tj, tile, split;
  my_split(p, tile, split);
  const uint32_t mat = my_part(c, p, tile, m, ti, tj);
  const uint32_t i0 = ti * S::BM, j0 = tj * S::BN;
  const uint64_t from = at ? m.y : m.x;
  const bool wide = m.rows <= m.cols;
  MmSums<S> sums;
  const uint32_t splits = S::MODE == MM_TURNS ? 1 : p.splits;
  const int nseg = m.exact ? 3 : 1;
  if (wide)
    mm_tile<S, DT_F16, false, true, false>(
        sums, (TG_LDS char*)lds_raw,
        [&](int s, MmOperand& a, MmOperand& b, MmOperand&) {
          a = ns_operand(c, m, m.b, m.m, m.ldm, kPartsA, s);
          b = ns_operand(c, m, from, m.rows, m.ldx, kPartsB, s);
        },
        nseg, m.m, i0, j0, m.ldm, m.ldx, split, splits);
  else
    mm_tile<S, DT_F16, false, false, false>(
        sums, (TG_LDS char*)lds_raw,
        [&](int s, MmOperand& a, MmOperand& b, MmOperand&) {
          a = ns_operand(c, m, from, m.rows, m.ldx, kPartsA, s);
          b = ns_operand(c, m, m.b, m.m, m.ldm, kPartsB, s);
        },
        nseg, whole8(m.cols), i0, j0, m.ldx, m.ldm, split, splits);
  if (S::MODE != MM_TURNS && !whole_sums(sums, c.counters, tile, split, p.splits, (TG_LDS char*)lds_raw)) return;
  const float step = (float)(last.lr * m.scale), decay = (float)(1.0 - last.lr * m.wd);
  const Place<S> place;
  const uint64_t first = ((uint64_t)i0 * m.ldx + j0) * 2, part = (uint64_t)m.rows * m.ldx * 2;
  const MmWindow xh(c.ws + from + first), xl(c.ws + from + part + first);
  // diag(B) of a row, or of the columns (behind the m-th anything)
  const MmWindow db((const float*)(c.ws + m.db) + (wide ? i0 : j0));
  float di[S::FM];
  f32x4 dj[S::FN];
#pragma unroll
  for (int i = 0; i < S::FM; ++i)
    di[i] = c.ca + __uint_as_float(db.load4(wide && i0 + place.r + i * 16 < m.m, place.r * 4, i * 64));
#pragma unroll
  for (int j = 0; j < S::FN; ++j)
    dj[j] = __builtin_bit_cast(f32x4, db.load16(!wide && j0 + place.c + j * 16 < m.ldm, place.c * 4, j * 64));
  auto row = [&](int bi) { return i0 + place.r + bi * 16; };
  auto col = [&](int bj) { return j0 + place.c + bj * 16; };
  const uint32_t lane = (place.r * m.ldx + place.c) * 2;
  auto all = [&](int bi, int bj) { return (bi * 16 * m.ldx + bj * 16) * 2; };
  auto load = [&](int bi, int bj) {
    const bool in = row(bi) < m.rows && col(bj) < m.ldx;
    return Four{xh.load8(in, lane, all(bi, bj)), xl.load8(in, lane, all(bi, bj))};
  };
  auto next = [&](int bi, int bj, const Four& old, float* r) {   // under NS_X
    float was[4];
    old.get(was);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      r[e] = col(bj) + e < m.cols ? (di[bi] + dj[bj][e]) * was[e] + sums.c[bi][bj][e] * (1.0f / NS_M) : 0.0f;
  };
  if (!last.last) {
    char* const to = c.ws + (at ? m.x : m.y) + first;
    const MmWindow nh(to), nl(to + part);
    each_block<S, Four>(load, [&](int bi, int bj, const Four& old) {
      float r[4];
      next(bi, bj, old, r);
      _Float16 h[4], l[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) two_parts(r[e], h[e], l[e]);
      const bool in = row(bi) < m.rows && col(bj) < m.ldx;
      nh.store8(*(const u32x2*)h, in, lane, all(bi, bj));
      nl.store8(*(const u32x2*)l, in, lane, all(bi, bj));
    });
    return;
  }
  void* const out = last.w ? last.w[m.tensor] : last.out;
  const uint64_t elem = last.w ? m.elem : (uint64_t)mat * m.rows * m.cols;
  with_type(m.wdt, [&](auto zero) {
    using T = decltype(zero);
    struct Weight {
      Four old;
      T y[4];
    };
    T* const to = (T*)out + elem;
    auto both = [&](int bi, int bj) {
      Weight w{load(bi, bj), {}};
      const uint32_t i = row(bi), j = col(bj);
      if (!last.w || i >= m.rows || j >= m.cols) return w;
      const T* const y = to + (uint64_t)i * m.cols + j;
      if (j + 4 <= m.cols) {
        load_values<4>(y, w.y);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (j + e < m.cols) w.y[e] = y[e];
      }
      return w;
    };
    each_block<S, Weight>(both, [&](int bi, int bj, const Weight& w) {
      const uint32_t i = row(bi), j = col(bj);
      if (i >= m.rows || j >= m.cols) return;
      T* const o = to + (uint64_t)i * m.cols + j;
      float r[4];
      next(bi, bj, w.old, r);
      T y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = r[e] * (1.0f / NS_X);
        y[e] = from_f32<T>(last.w ? to_f32(w.y[e]) * decay - step * x : x);
      }
      if (j + 4 <= m.cols) {
        store_values<4>(o, y);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (j + e < m.cols) o[e] = y[e];
      }
    });
  });
}

template <class S, class K, class... A>
hipError_t launch_shape(K* k, uint32_t n, uint32_t splits, hipStream_t s, const A&... a) {
  if (n == 0) return hipSuccess;
  n *= splits;
  if (n > 0x7FFFFFFFu / S::THREADS) return hipErrorInvalidValue;
  const hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS_BYTES);
  if (e != hipSuccess) return e;
  k<<<n, S::THREADS, S::LDS_BYTES, s>>>(a...);
  return hipGetLastError();
}
using Big = MmBig;
using Mid = MmMid;
using Deep = MmDeep;
using Small = MmNear;

}  // namespace

hipError_t launch_muon_first(const NsCommon& c, const MuonFirst& f, const MuonTable& t, const NsParts& p, uint32_t n,
                             hipStream_t s) {
  if (n == 0) return hipSuccess;
  k_muon_first<<<n, 256, 0, s>>>(c, f, t, p);
  return hipGetLastError();
}
hipError_t launch_muon_start(const NsCommon& c, const MuonFirst& f, double eps, const NsParts& p, uint32_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  k_muon_start<<<n, 256, 0, s>>>(c, f, eps, p);
  return hipGetLastError();
}
hipError_t launch_ns_norm(const NsCommon& c, const NsSource& f, const NsParts& p, uint32_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  k_ns_norm<<<n, 256, 0, s>>>(c, f, p);
  return hipGetLastError();
}
hipError_t launch_ns_start(const NsCommon& c, const NsSource& f, double eps, const NsParts& p, uint32_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  k_ns_start<<<n, 256, 0, s>>>(c, f, eps, p);
  return hipGetLastError();
}
hipError_t launch_ns_gram(const NsCommon& c, int at, int tile, const NsParts& p, uint32_t n, hipStream_t s) {
  return tile == 0   ? launch_shape<Big>(k_ns_gram<Big>, n, p.splits, s, c, at, p)
         : tile == 1 ? launch_shape<Mid>(k_ns_gram<Mid>, n, p.splits, s, c, at, p)
         : tile == 3 ? launch_shape<Deep>(k_ns_gram<Deep>, n, p.splits, s, c, at, p)
                     : launch_shape<Small>(k_ns_gram<Small>, n, p.splits, s, c, at, p);
}
hipError_t launch_ns_poly(const NsCommon& c, int tile, const NsParts& p, uint32_t n, hipStream_t s) {
  return tile == 0   ? launch_shape<Big>(k_ns_poly<Big>, n, p.splits, s, c, p)
         : tile == 1 ? launch_shape<Mid>(k_ns_poly<Mid>, n, p.splits, s, c, p)
         : tile == 3 ? launch_shape<Deep>(k_ns_poly<Deep>, n, p.splits, s, c, p)
                     : launch_shape<Small>(k_ns_poly<Small>, n, p.splits, s, c, p);
}
hipError_t launch_ns_apply(const NsCommon& c, int at, int tile, const NsLast& l, const NsParts& p, uint32_t n,
                           hipStream_t s) {
  return tile == 0   ? launch_shape<Big>(k_ns_apply<Big>, n, p.splits, s, c, at, l, p)
         : tile == 1 ? launch_shape<Mid>(k_ns_apply<Mid>, n, p.splits, s, c, at, l, p)
         : tile == 3 ? launch_shape<Deep>(k_ns_apply<Deep>, n, p.splits, s, c, at, l, p)
                     : launch_shape<Small>(k_ns_apply<Small>, n, p.splits, s, c, at, l, p);
}

}  // namespace tg
