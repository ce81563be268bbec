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
// What bounds it: matrix instructions for large matrices, launches (two, and three for every
// step) for middle ones; small ones are k_muon_small.hip's. All matrices of a handle share every
// launch.
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

// A chunk of a matrix: f(row, column, n) for pieces of 8 values of a line, n of them inside.
template <class F>
__device__ __forceinline__ void each_piece(const NsMat& m, uint32_t chunk, const F& f) {
  const uint32_t pieces = m.ldx / 8;
  const uint64_t first = (uint64_t)chunk * (MUON_CHUNK / 8), row0 = first / pieces;
  const uint32_t skip = (uint32_t)(first - row0 * pieces);
#pragma unroll
  for (uint32_t q = 0; q < MUON_CHUNK / 8 / 256; ++q) {
    const uint32_t at = skip + q * 256 + threadIdx.x, down = at / pieces, k = (at - down * pieces) * 8;
    const uint64_t row = row0 + down;
    if (row < m.rows) f((uint32_t)row, k, m.cols - k < 8 ? m.cols - k : 8);
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

// 2^12 / (|U| + eps), by every workgroup from all sums of the matrix in their order
__device__ __forceinline__ float start_scale(const NsCommon& c, const NsMat& m, double eps) {
  __shared__ double total;
  double s = 0.0;
  const double* const sums = (const double*)(c.ws + m.sums);
  for (uint32_t i = threadIdx.x; i < m.chunks; i += 256) s += sums[i];
  workgroup_sum(s, &total);
  __syncthreads();
  return (float)((double)NS_X / (__builtin_sqrt(total) + eps));
}

// 8 values of a line of X in their parts
__device__ __forceinline__ void write_x(const NsCommon& c, const NsMat& m, uint32_t r, uint32_t k, const float* v, float scale) {
  _Float16* const hi = (_Float16*)(c.ws + m.x) + (uint64_t)r * m.ldx + k;
  _Float16 h[8], l[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) two_parts(v[e] * scale, h[e], l[e]);
  *(uint4*)hi = *(const uint4*)h;
  *(uint4*)(hi + (uint64_t)m.rows * m.ldx) = *(const uint4*)l;
}

__global__ void __launch_bounds__(256) k_muon_start(const NsCommon c, const MuonFirst f, const double eps, const NsParts p) {
  if (left_out(c)) return;
  const float coef = c.clip ? c.clip[1] : 1.0f;
  NsMat m;
  uint32_t chunk, none;
  my_part(c, p, blockIdx.x, m, chunk, none);
  const float scale = start_scale(c, m, eps);
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
  NsMat m;
  uint32_t chunk, none;
  const uint32_t mat = my_part(c, p, blockIdx.x, m, chunk, none);
  const float scale = start_scale(c, m, eps);
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

// the four columns that a lane holds of block (i, j)
template <class S, class F>
__device__ __forceinline__ void each_four(const MmSums<S>& sums, uint32_t i0, uint32_t j0, const F& f) {
  const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
#pragma unroll
  for (int i = 0; i < S::FM; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j)
      f(i0 + (wm * S::FM + i) * 16 + (lane & 15), j0 + (wn * S::FN + j) * 16 + (lane >> 4) * 4, sums.c[i][j]);
}

// v (four columns of row i, under NS_M) to a symmetric matrix, and to its other half. The rows
// from m to ldm are only the other half's padding.
__device__ __forceinline__ void write_symmetric(const NsCommon& c, const NsMat& m, uint64_t at, uint32_t i, uint32_t j,
                                                bool mirror, const float* v) {
  _Float16* const hi = (_Float16*)(c.ws + at);
  const uint64_t part = (uint64_t)m.m * m.ldm;
  _Float16 h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) two_parts(v[e], h[e], l[e]);
  if (i < m.m && j < m.ldm) {
    *(uint2*)(hi + (uint64_t)i * m.ldm + j) = *(const uint2*)h;
    if (m.exact) *(uint2*)(hi + part + (uint64_t)i * m.ldm + j) = *(const uint2*)l;
  }
  if (mirror) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < m.m) {
        hi[(uint64_t)(j + e) * m.ldm + i] = h[e];
        if (m.exact) hi[part + (uint64_t)(j + e) * m.ldm + i] = l[e];
      }
  }
}

template <class S>
__global__ void __launch_bounds__(S::THREADS, 2) k_ns_gram(const NsCommon c, const int at, const NsParts p) {
  extern __shared__ char lds_raw[];
  if (left_out(c)) return;
  NsMat m;
  uint32_t ti, tj;
  my_part(c, p, xcd_order(blockIdx.x, gridDim.x), m, ti, tj);
  const uint32_t i0 = ti * S::BM, j0 = tj * S::BN;
  const uint64_t from = at ? m.y : m.x;
  MmSums<S> sums;
  auto source = [&](int s, MmOperand& a, MmOperand& b, MmOperand&) {
    a = ns_operand(c, m, from, m.rows, m.ldx, kPartsA, s);
    b = ns_operand(c, m, from, m.rows, m.ldx, kPartsB, s);
  };
  const int nseg = m.exact ? 3 : 1;
  if (m.rows <= m.cols)
    mm_tile<S, DT_F16, false, false, false>(sums, (TG_LDS char*)lds_raw, source, nseg, m.ldx, i0, j0, m.ldx, m.ldx);
  else
    mm_tile<S, DT_F16, true, true, false>(sums, (TG_LDS char*)lds_raw, source, nseg, m.rows, i0, j0, m.ldx, m.ldx);
  float* const diag = (float*)(c.ws + m.da);
  each_four(sums, i0, j0, [&](uint32_t i, uint32_t j, f32x4 v) {
    if (i >= m.ldm) return;
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[e] * (1.0f / (NS_X * NS_X));
      const bool in = i < m.m && j + e < m.m;
      if (in && i == j + e) diag[i] = x;
      o[e] = in && i != j + e ? x * NS_M : 0.0f;
    }
    write_symmetric(c, m, m.a, i, j, ti != tj, o);
  });
}

template <class S>
__global__ void __launch_bounds__(S::THREADS, 2) k_ns_poly(const NsCommon c, const NsParts p) {
  extern __shared__ char lds_raw[];
  if (left_out(c)) return;
  NsMat m;
  uint32_t ti, tj;
  my_part(c, p, xcd_order(blockIdx.x, gridDim.x), m, ti, tj);
  const uint32_t i0 = ti * S::BM, j0 = tj * S::BN;
  MmSums<S> sums;
  mm_tile<S, DT_F16, false, false, false>(
      sums, (TG_LDS char*)lds_raw,
      [&](int s, MmOperand& a, MmOperand& b, MmOperand&) {
        a = ns_operand(c, m, m.a, m.m, m.ldm, kPartsA, s);
        b = ns_operand(c, m, m.a, m.m, m.ldm, kPartsB, s);
      },
      m.exact ? 3 : 1, m.ldm, i0, j0, m.ldm, m.ldm);
  const float* const da = (const float*)(c.ws + m.da);
  float* const db = (float*)(c.ws + m.db);
  const _Float16* const oh = (const _Float16*)(c.ws + m.a);
  const uint64_t part = (uint64_t)m.m * m.ldm;
  each_four(sums, i0, j0, [&](uint32_t i, uint32_t j, f32x4 v) {
    if (i >= m.ldm || j >= m.ldm) return;
    _Float16 h[4] = {}, l[4] = {};
    float di = 0.0f;
    if (i < m.m) {
      *(uint2*)h = *(const uint2*)(oh + (uint64_t)i * m.ldm + j);
      if (m.exact) *(uint2*)l = *(const uint2*)(oh + part + (uint64_t)i * m.ldm + j);
      di = da[i];
    }
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float q = v[e] * (1.0f / (NS_M * NS_M));
      if (i >= m.m || j + e >= m.m) {
        o[e] = 0.0f;
      } else if (i == j + e) {
        db[i] = c.cb * di + c.cc * (di * di + q);
        o[e] = 0.0f;
      } else {
        const float x = ((float)h[e] + (float)l[e]) * (1.0f / NS_M);
        o[e] = (c.cb * x + c.cc * (q + (di + da[j + e]) * x)) * NS_M;
      }
    }
    write_symmetric(c, m, m.b, i, j, ti != tj, o);
  });
}

template <class S>
__global__ void __launch_bounds__(S::THREADS, 2) k_ns_apply(const NsCommon c, const int at, const NsLast last, const NsParts p) {
  extern __shared__ char lds_raw[];
  if (left_out(c)) return;
  NsMat m;
  uint32_t ti, tj;
  const uint32_t mat = my_part(c, p, xcd_order(blockIdx.x, gridDim.x), m, ti, tj);
  const uint32_t i0 = ti * S::BM, j0 = tj * S::BN;
  const uint64_t from = at ? m.y : m.x;
  const bool wide = m.rows <= m.cols;
  MmSums<S> sums;
  const int nseg = m.exact ? 3 : 1;
  if (wide)
    mm_tile<S, DT_F16, false, true, false>(
        sums, (TG_LDS char*)lds_raw,
        [&](int s, MmOperand& a, MmOperand& b, MmOperand&) {
          a = ns_operand(c, m, m.b, m.m, m.ldm, kPartsA, s);
          b = ns_operand(c, m, from, m.rows, m.ldx, kPartsB, s);
        },
        nseg, m.ldm, i0, j0, m.ldm, m.ldx);
  else
    mm_tile<S, DT_F16, false, false, false>(
        sums, (TG_LDS char*)lds_raw,
        [&](int s, MmOperand& a, MmOperand& b, MmOperand&) {
          a = ns_operand(c, m, from, m.rows, m.ldx, kPartsA, s);
          b = ns_operand(c, m, m.b, m.m, m.ldm, kPartsB, s);
        },
        nseg, m.ldx, i0, j0, m.ldx, m.ldm);
  const float* const db = (const float*)(c.ws + m.db);
  const _Float16* const xh = (const _Float16*)(c.ws + from);
  _Float16* const nh = (_Float16*)(c.ws + (at ? m.x : m.y));
  const uint64_t part = (uint64_t)m.rows * m.ldx;
  const float step = (float)(last.lr * m.scale), decay = (float)(1.0 - last.lr * m.wd);
  each_four(sums, i0, j0, [&](uint32_t i, uint32_t j, f32x4 v) {
    if (i >= m.rows || j >= m.ldx) return;
    const uint64_t o = (uint64_t)i * m.ldx + j;
    _Float16 h[4], l[4];
    *(uint2*)h = *(const uint2*)(xh + o);
    *(uint2*)l = *(const uint2*)(xh + part + o);
    float r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float d = c.ca + (wide ? db[i] : j + e < m.m ? db[j + e] : 0.0f);
      r[e] = d * ((float)h[e] + (float)l[e]) + v[e] * (1.0f / NS_M);   // under NS_X
    }
    if (!last.last) {
#pragma unroll
      for (int e = 0; e < 4; ++e) two_parts(j + e < m.cols ? r[e] : 0.0f, h[e], l[e]);
      *(uint2*)(nh + o) = *(const uint2*)h;
      *(uint2*)(nh + part + o) = *(const uint2*)l;
      return;
    }
    const uint64_t to = (last.w ? m.elem : (uint64_t)mat * m.rows * m.cols) + (uint64_t)i * m.cols + j;
    void* const out = last.w ? last.w[m.tensor] : last.out;
    with_type(m.wdt, [&](auto zero) {
      using T = decltype(zero);
      T* const o = (T*)out + to;
      T y[4] = {};
      if (j + 4 <= m.cols) {
        if (last.w) load_values<4>(o, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = r[e] * (1.0f / NS_X);
          y[e] = from_f32<T>(last.w ? to_f32(y[e]) * decay - step * v : v);
        }
        store_values<4>(o, y);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          if (j + e >= m.cols) continue;
          const float v = r[e] * (1.0f / NS_X);
          o[e] = from_f32<T>(last.w ? to_f32(o[e]) * decay - step * v : v);
        }
      }
    });
  });
}

template <class S, class K, class... A>
hipError_t launch_shape(K* k, uint32_t n, hipStream_t s, const A&... a) {
  if (n == 0) return hipSuccess;
  if (n > 0x7FFFFFFFu / S::THREADS) return hipErrorInvalidValue;
  const hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS_BYTES);
  if (e != hipSuccess) return e;
  k<<<n, S::THREADS, S::LDS_BYTES, s>>>(a...);
  return hipGetLastError();
}
using Big = MmBig;
using Mid = MmMid;
using Small = MmSmall;

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
  return tile == 0   ? launch_shape<Big>(k_ns_gram<Big>, n, s, c, at, p)
         : tile == 1 ? launch_shape<Mid>(k_ns_gram<Mid>, n, s, c, at, p)
                     : launch_shape<Small>(k_ns_gram<Small>, n, s, c, at, p);
}
hipError_t launch_ns_poly(const NsCommon& c, int tile, const NsParts& p, uint32_t n, hipStream_t s) {
  return tile == 0   ? launch_shape<Big>(k_ns_poly<Big>, n, s, c, p)
         : tile == 1 ? launch_shape<Mid>(k_ns_poly<Mid>, n, s, c, p)
                     : launch_shape<Small>(k_ns_poly<Small>, n, s, c, p);
}
hipError_t launch_ns_apply(const NsCommon& c, int at, int tile, const NsLast& l, const NsParts& p, uint32_t n,
                           hipStream_t s) {
  return tile == 0   ? launch_shape<Big>(k_ns_apply<Big>, n, s, c, at, l, p)
         : tile == 1 ? launch_shape<Mid>(k_ns_apply<Mid>, n, s, c, at, l, p)
                     : launch_shape<Small>(k_ns_apply<Small>, n, s, c, at, l, p);
}

}  // namespace tg
