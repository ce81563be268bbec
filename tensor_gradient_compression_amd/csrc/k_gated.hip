// Gated linear layer, y = act(x Wg^T + bg) * (x Wu^T + bu): the forward product, and the first
// product of the gradients.
//
// Both products are one: a tile's columns are 16 of the gate's and 16 of the other weight's by
// turns, so that a lane's sums hold g and u of the same places, and the activation and the
// product follow in registers. The backward pass keeps nothing of the forward's: the same tile
// forms g and u again (a third of its operations, and no 4 or 8 bytes a value in memory between
// the passes), then dg = dy u act'(g) and du = dy act(g), which leave rounded to x's type as
// the operands of the products for dx and the weights (k_gated_bwd.hip).
//
// fp32 values are multiplied in three bf16 parts, which add up to them exactly, by six of the
// nine products of parts; the three that are left out are 2^-24 of the whole and less. The
// matrix instructions do 16 times as much in bf16 as in fp32.
#include <type_traits>

#include "gated.h"

namespace tg {

namespace {

// Phi(-x) for x >= 0, the normal distribution's lower tail: t 2^(p(t) - x^2 log2(e) / 2) with
// t = 1 / (1 + x / sqrt(8)) and p a polynomial fitted to log2(erfcx(x / sqrt 2) / 2t) at
// Chebyshev points, 3.4e-7 of the value for every x. The rounding of the exponent's argument comes
// on top: 1.4e-6 of the value at x = 5, 3e-6 at 8, 8e-6 at 13.
__device__ __forceinline__ float normal_tail(float x) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.353553391f * x);
  float p = 0.253258819f;
  p = __builtin_fmaf(p, t, -1.21736752f);
  p = __builtin_fmaf(p, t, 2.20788314f);
  p = __builtin_fmaf(p, t, -1.70057641f);
  p = __builtin_fmaf(p, t, 0.440011764f);
  p = __builtin_fmaf(p, t, -0.281599746f);
  p = __builtin_fmaf(p, t, 0.141806747f);
  p = __builtin_fmaf(p, t, 0.53962246f);
  p = __builtin_fmaf(p, t, 1.4427072f);
  p = __builtin_fmaf(p, t, -2.82574634f);
  return t * __builtin_amdgcn_exp2f(__builtin_fmaf(x * -0.721347520f, x, p));
}
// The same for 16-bit results: a polynomial fitted to log2 Phi(-x) for x up to 6.5 (7.4e-6 of
// the value; Phi(-6.5) is 4e-11) that falls ever faster beyond.
__device__ __forceinline__ float short_normal_tail(float x) {
  float p = -1.76984737e-6f;
  p = __builtin_fmaf(p, x, 6.02403488e-5f);
  p = __builtin_fmaf(p, x, -9.19429847e-4f);
  p = __builtin_fmaf(p, x, 8.46320244e-3f);
  p = __builtin_fmaf(p, x, -5.38683020e-2f);
  p = __builtin_fmaf(p, x, -4.58553402e-1f);
  p = __builtin_fmaf(p, x, -1.15121899f);
  p = __builtin_fmaf(p, x, -0.999997157f);
  return __builtin_amdgcn_exp2f(p);
}

constexpr float kLog2e = 1.44269504f;

// act(g), and act'(g) for the gradients. SHORT: for 16-bit results, in fewer instructions: an
// epilogue of 67M GELUs is bound by them. A NaN stays one, and infinities give the limits. Neither
// value nor slope is a difference of larger ones where it falls off with the gate.
template <int ACT, bool SHORT, bool SLOPE>
__device__ __forceinline__ float activate(float g, float& slope) {
  const float x = __builtin_fabsf(g);
  if constexpr (ACT == GATED_RELU) {
    if (SLOPE) slope = g > 0.0f ? 1.0f : 0.0f;
    return g < 0.0f ? 0.0f : g;
  } else if constexpr (ACT == GATED_GELU && SHORT) {
    // g Phi(g) = max(g, 0) - |g| Phi(-|g|);  its slope q = Phi(-|g|) - |g| phi(g) below zero, 1 - q above
    const float tail = short_normal_tail(x), near = __builtin_fminf(x, 30.0f);
    if (SLOPE) {
      const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(g * -0.721347520f, g, -1.32574806f));
      const float q = __builtin_fmaf(-near, e, tail);
      slope = g < 0.0f ? q : 1.0f - q;
    }
    return __builtin_fmaxf(g, 0.0f) - near * tail;      // (not the mean of g and |g|, whose sum may overflow)
  } else if constexpr (ACT == GATED_GELU) {
    const float tail = normal_tail(x);
    const float cdf = g < 0.0f ? tail : 1.0f - tail;
    if (SLOPE) {
      const float e = 0.398942280f * __builtin_amdgcn_exp2f(g * -0.721347520f * g);
      slope = e == 0.0f ? cdf : __builtin_fmaf(g, e, cdf);
    }
    // -infinity times a tail of zero is the limit, zero
    return tail == 0.0f ? (g < 0.0f ? 0.0f : g) : g * cdf;
  } else if constexpr (SHORT) {
    const float e = __builtin_amdgcn_exp2f(-kLog2e * g), r = __builtin_amdgcn_rcpf(1.0f + e);
    if constexpr (ACT == GATED_SIGMOID) {
      // 1 - r keeps nothing of r's counterpart e r where that is small
      if (SLOPE) slope = g > 0.0f ? e * r * r : __builtin_fmaf(-r, r, r);
      return r;
    }
    const float low = __builtin_fmaxf(g, -200.0f);
    if (SLOPE) slope = __builtin_fmaf(__builtin_fminf(low, 200.0f) * r, 1.0f - r, r);
    return low * r;
  } else {
    // 1 / (1 + e^-|g|) and its counterpart e^-|g| / (1 + e^-|g|)
    const float e = __builtin_amdgcn_exp2f(-kLog2e * x);
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    const float p = g < 0.0f ? e * r : r, q = g < 0.0f ? r : e * r;
    if constexpr (ACT == GATED_SIGMOID) {
      if (SLOPE) slope = p * q;
      return p;
    }
    if (SLOPE) slope = q == 0.0f ? p : p == 0.0f ? 0.0f : p * __builtin_fmaf(g, q, 1.0f);
    return p == 0.0f ? 0.0f : g * p;
  }
}

// f with the activation as a constant
template <class F>
__device__ __forceinline__ void with_activation(int act, const F& f) {
  if (act == GATED_SILU) f(std::integral_constant<int, GATED_SILU>{});
  else if (act == GATED_GELU) f(std::integral_constant<int, GATED_GELU>{});
  else if (act == GATED_SIGMOID) f(std::integral_constant<int, GATED_SIGMOID>{});
  else f(std::integral_constant<int, GATED_RELU>{});
}

template <class S, int DT>
__device__ __forceinline__ void gate_and_up(MmSums<S>& sums, TG_LDS char* lds, const GatedArgs& a, int64_t row0, uint32_t f0) {
  using G = GatedType<DT>;
  mm_tile<S, G::MM, false, false, true>(
      sums, lds,
      [&](int s, MmOperand& x, MmOperand& g, MmOperand& u) {
        x = gated_operand<G::SEGS>(a.x, GATED_PART_A, s, 0, false);
        g = gated_operand<G::SEGS>(a.wg, GATED_PART_B, s, 0, false);
        u = gated_operand<G::SEGS>(a.wu, GATED_PART_B, s, 0, false);
      },
      G::SEGS, gated_sum(a.x, a.wg, f0, a.hidden), row0, f0, a.x.stride, a.wg.stride);
}

// The biases of eight columns of a lane, gate and up. (All loads of an epilogue go out before its first
// store, which the compiler would not let them pass.)
template <typename T>
__device__ __forceinline__ void load_biases(const GatedArgs& a, uint32_t f, float (&b)[2][8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const T* const p = (const T*)(h ? a.bu : a.bg);
#pragma unroll
    for (int e = 0; e < 8; ++e) b[h][e] = p && f + e < a.hidden ? to_f32(p[f + e]) : 0.0f;
  }
}

// Eight values of T on end through a window, `n` of them in the matrix; wide: by 16 bytes.
template <typename T>
__device__ __forceinline__ void window_store(const MmWindow& w, const T* v, int n, bool wide, uint32_t lane, uint32_t all) {
  constexpr int E = 16 / sizeof(T);
  if (wide) {
#pragma unroll
    for (int e = 0; e < 8; e += E) w.store16(*(const u32x4*)(v + e), e < n, lane + e * sizeof(T), all);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (sizeof(T) == 4) w.store4(__builtin_bit_cast(uint32_t, v[e]), e < n, lane + e * 4, all);
      else w.store2(__builtin_bit_cast(uint16_t, v[e]), e < n, lane + e * 2, all);
    }
  }
}
template <typename T>
__device__ __forceinline__ void window_load(const MmWindow& w, T* v, int n, bool wide, uint32_t lane, uint32_t all) {
  constexpr int E = 16 / sizeof(T);
  if (wide) {
#pragma unroll
    for (int e = 0; e < 8; e += E) *(u32x4*)(v + e) = w.load16(e < n, lane + e * sizeof(T), all);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (sizeof(T) == 4) v[e] = __builtin_bit_cast(T, w.load4(e < n, lane + e * 4, all));
      else v[e] = __builtin_bit_cast(T, w.load2(e < n, lane + e * 2, all));
    }
  }
}
// whether a row's pieces of 16 bytes are whole and aligned
template <typename T>
__device__ __forceinline__ bool wide_rows(const void* p, uint32_t cols, int64_t stride) {
  constexpr uint32_t E = 16 / sizeof(T);
  return cols % E == 0 && stride % E == 0 && ((uintptr_t)p & 15u) == 0;
}

// what a value's rounding left, nothing of one that is not finite
template <typename T>
__device__ __forceinline__ T rest(float v, T rounded) {
  const float r = v - to_f32(rounded);
  return from_f32<T>(__builtin_fabsf(r) <= __builtin_fabsf(v) ? r : 0.0f);
}

// A lane's eight columns of a row: g in two blocks, u in the two between them.
template <class S>
__device__ __forceinline__ void eight(const MmSums<S>& sums, int i, int j, float (&g)[8], float (&u)[8]) {
  static_assert(S::FN % 4 == 0, "pairs of blocks of both");
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    g[e] = sums.c[i][j + (e >> 2) * 2][e & 3];
    u[e] = sums.c[i][j + (e >> 2) * 2 + 1][e & 3];
  }
}

// y. Short sums are bound by the epilogue and by writing y (65536 x 256 x 1024 in bf16 with gelu:
// 119 us, the matrix unit 28% busy, 1.1 TB/s written), long ones by matrix instructions and LDS.
template <class S, int DT>
__global__ void __launch_bounds__(S::THREADS, 2) k_gated_forward(const GatedArgs a) {
  using T = typename GatedType<DT>::T;
  extern __shared__ char lds_raw[];
  TG_LDS char* const lds = (TG_LDS char*)lds_raw;
  const uint32_t nj = (a.hidden + S::BN / 2 - 1) / (S::BN / 2), ni = (uint32_t)((a.rows + S::BM - 1) / S::BM);
  uint32_t ti, tj;
  tile_at(xcd_order(blockIdx.x, gridDim.x), ni, nj, ti, tj);
  const int64_t row0 = (int64_t)ti * S::BM;
  const uint32_t f0 = tj * (S::BN / 2);
  MmSums<S> sums;
  gate_and_up<S, DT>(sums, lds, a, row0, f0);
  const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const bool wide = wide_rows<T>(a.y, a.hidden, a.hidden);
  const uint32_t r = wm * S::FM * 16 + (lane & 15), c = wn * S::FN * 8 + (lane >> 4) * 8;
  const MmWindow out((T*)a.y + row0 * a.hidden + f0);
  with_activation(a.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
#pragma unroll
    for (int j = 0; j < S::FN; j += 4) {
      const uint32_t f = f0 + c + j * 8;
      float bias[2][8];
      load_biases<T>(a, f, bias);
#pragma unroll
      for (int i = 0; i < S::FM; ++i) {
        float g[8], u[8];
        eight(sums, i, j, g, u);
        alignas(16) T y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float slope;
          const float p = activate<ACT, DT != DT_F32, false>(g[e] + bias[0][e], slope);
          y[e] = from_f32<T>(p * (u[e] + bias[1][e]));
        }
        const int n = row0 + r + i * 16 < a.rows ? (int)a.hidden - (int)f : 0;
        window_store<T>(out, y, n, wide, (r * a.hidden + c) * sizeof(T), (i * 16 * a.hidden + j * 8) * sizeof(T));
      }
    }
  });
}

// dg and du, and their sums over a wave's rows. As k_gated_forward, with dy read and two values
// written (65536 x 256 x 1024 in bf16: 242 us traced, 135 MB of dy read and 268 written; 8192 x 4096 x 8192:
// 942 us, 1167 TFLOP/s). By 256 x 256 it holds sums and a row of parts in more registers than there are: 100
// bytes a lane go to memory in 16 bits, 356 in fp32.
template <class S, int DT>
__global__ void __launch_bounds__(S::THREADS, 2) k_gated_grads(const GatedArgs a) {
  using T = typename GatedType<DT>::T;
  extern __shared__ char lds_raw[];
  TG_LDS char* const lds = (TG_LDS char*)lds_raw;
  const uint32_t pad = gated_pad(a.hidden);
  const uint32_t nj = (pad + S::BN / 2 - 1) / (S::BN / 2), ni = (uint32_t)((a.rows + S::BM - 1) / S::BM);
  if (a.counters && blockIdx.x == 0)
    for (uint32_t i = threadIdx.x; i < MM_MOST_SPLIT; i += S::THREADS) a.counters[i] = 0;
  uint32_t ti, tj;
  tile_at(xcd_order(blockIdx.x, gridDim.x), ni, nj, ti, tj);
  const int64_t row0 = (int64_t)ti * S::BM;
  const uint32_t f0 = tj * (S::BN / 2);
  MmSums<S> sums;
  gate_and_up<S, DT>(sums, lds, a, row0, f0);
  const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int64_t part = a.rows * 2 * (int64_t)pad;
  const bool wide = wide_rows<T>(a.dy, a.hidden, a.dy_stride);
  const uint32_t r0 = wm * S::FM * 16 + (lane & 15), c0 = wn * S::FN * 8 + (lane >> 4) * 8;
  const uint32_t dy_stride = (uint32_t)a.dy_stride;
  const MmWindow in((const T*)a.dy + row0 * a.dy_stride + f0);
  with_activation(a.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    // (what is alike for all activations would be computed before them, into more registers than are there)
    uint32_t r = r0, c = c0;
    __asm__ volatile("" : "+v"(r), "+v"(c));
#pragma unroll
    for (int j = 0; j < S::FN; j += 4) {
      const uint32_t f = f0 + c + j * 8;
      float bias[2][8];
      load_biases<T>(a, f, bias);
      float sg[8] = {}, su[8] = {};
      // dy of some rows' blocks, as many as there are registers for
      constexpr int ROWS = S::FM < 4 ? S::FM : 4;
      alignas(16) T dy[ROWS][8];
#pragma unroll
      for (int i = 0; i < S::FM; ++i) {
        if (i % ROWS == 0) {
#pragma unroll
          for (int k = 0; k < ROWS; ++k)
            window_load<T>(in, dy[k], row0 + r + (i + k) * 16 < a.rows ? (int)a.hidden - (int)f : 0, wide,
                           (r * dy_stride + c) * sizeof(T), ((i + k) * 16 * dy_stride + j * 8) * sizeof(T));
        }
        float g[8], u[8], dg[8], du[8];
        eight(sums, i, j, g, u);
        const bool row = row0 + r + i * 16 < a.rows;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float slope;
          const float d = to_f32(dy[i % ROWS][e]);
          const float p = activate<ACT, DT != DT_F32, true>(g[e] + bias[0][e], slope);
          const bool real = row && f + e < a.hidden;     // zeros behind (not zero times a bias)
          dg[e] = real ? d * (u[e] + bias[1][e]) * slope : 0.0f;
          du[e] = real ? d * p : 0.0f;
          sg[e] += dg[e];
          su[e] += du[e];
        }
        const int n = row && f < pad ? 8 : 0;
        const uint32_t to_lane = (r * 2 * pad + c) * 2, to_all = (i * 32 * pad + j * 8) * 2;
        if constexpr (DT == DT_F32) {
          alignas(16) bf16_t g[3][8], u[3][8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            bf16_t p[3];
            three_parts(dg[e], p);
            for (int q = 0; q < 3; ++q) g[q][e] = p[q];
            three_parts(du[e], p);
            for (int q = 0; q < 3; ++q) u[q][e] = p[q];
          }
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            const MmWindow to((bf16_t*)a.grads + q * part + row0 * 2 * (int64_t)pad + f0);
            window_store<bf16_t>(to, g[q], n, true, to_lane, to_all);
            window_store<bf16_t>(to, u[q], n, true, to_lane, to_all + pad * 2);
          }
        } else {
          alignas(16) T g[8], u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = from_f32<T>(dg[e]), u[e] = from_f32<T>(du[e]);
          const MmWindow to((T*)a.grads + row0 * 2 * (int64_t)pad + f0);
          window_store<T>(to, g, n, true, to_lane, to_all);
          window_store<T>(to, u, n, true, to_lane, to_all + pad * 2);
          if constexpr (S::BM <= 128) {           // few values: no larger tiles
            if (a.parts == 2) {
#pragma unroll
              for (int e = 0; e < 8; ++e) g[e] = rest(dg[e], g[e]), u[e] = rest(du[e], u[e]);
              const MmWindow more((T*)a.grads + part + row0 * 2 * (int64_t)pad + f0);
              window_store<T>(more, g, n, true, to_lane, to_all);
              window_store<T>(more, u, n, true, to_lane, to_all + pad * 2);
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);   // a row after the other: registers for few at a time
      }
      if (a.row_sums) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) {
            sg[e] += __shfl_xor(sg[e], o);
            su[e] += __shfl_xor(su[e], o);
          }
        if ((lane & 15) == 0 && f < pad) {
          float* const s = a.row_sums + ((int64_t)ti * S::WM + wm) * 2 * (int64_t)pad + f;
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            *(f32x4*)(s + e) = f32x4{sg[e], sg[e + 1], sg[e + 2], sg[e + 3]};
            *(f32x4*)(s + pad + e) = f32x4{su[e], su[e + 1], su[e + 2], su[e + 3]};
          }
        }
      }
    }
  });
}

// One workgroup's 256 pieces of 8 values of a row-padded copy. Rows that start anywhere are read by
// single values (9.6M in fp16 17 us, 2.3 TB/s).
struct PackArgs {
  GatedPack m[3];
  uint64_t first[4];    // workgroups before each
};
__global__ void __launch_bounds__(256) k_gated_pack(const PackArgs a) {
  const int w = blockIdx.x >= a.first[2] ? 2 : blockIdx.x >= a.first[1] ? 1 : 0;
  const GatedPack& m = a.m[w];
  const uint32_t pieces = gated_pad(m.cols) / 8;
  const uint64_t at = (blockIdx.x - a.first[w]) * 256 + threadIdx.x;
  const uint64_t row = at / pieces;
  if (row >= (uint64_t)m.rows) return;
  const uint32_t c = (uint32_t)(at % pieces) * 8;
  const int64_t part = m.rows * (int64_t)pieces * 8;
  const uint64_t from = row * (uint64_t)m.stride + c;
  if (m.dt == DT_F32) {
    bf16_t out[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      bf16_t p[3];
      three_parts(c + e < m.cols ? ((const float*)m.src)[from + e] : 0.0f, p);
      for (int q = 0; q < 3; ++q) out[q][e] = p[q];
    }
    for (int q = 0; q < 3; ++q) *(uint4*)((bf16_t*)m.dst + q * part + at * 8) = *(const uint4*)out[q];
  } else {
    uint16_t out[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = c + e < m.cols ? ((const uint16_t*)m.src)[from + e] : (uint16_t)0;
    *(uint4*)((uint16_t*)m.dst + at * 8) = *(const uint4*)out;
  }
}

template <class S, int DT>
hipError_t launch_tiles(bool grads, const GatedArgs& a, hipStream_t s) {
  const int64_t ni = (a.rows + S::BM - 1) / S::BM;
  const int64_t nj = ((grads ? gated_pad(a.hidden) : a.hidden) + S::BN / 2 - 1) / (S::BN / 2);
  if (ni * nj > kMostThreads / S::THREADS) return hipErrorInvalidValue;
  void (*k)(GatedArgs) = k_gated_forward<S, DT>;
  if constexpr (S::MODE != MM_EVEN || S::BN == 128)   // those of gated_tile()
    if (grads) k = k_gated_grads<S, DT>;
  const hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS_BYTES);
  if (e != hipSuccess) return e;
  k<<<(uint32_t)(ni * nj), S::THREADS, S::LDS_BYTES, s>>>(a);
  return hipGetLastError();
}
template <int DT>
hipError_t launch_type(bool grads, const GatedArgs& a, hipStream_t s) {
  switch (gated_tile(a.rows, a.hidden, a.in, grads)) {
    case 0: return launch_tiles<MmBig, DT>(grads, a, s);
    case 1: return launch_tiles<MmMid, DT>(grads, a, s);
    case 3: return launch_tiles<MmHalf, DT>(false, a, s);   // the forward pass alone
    case 4: return launch_tiles<MmNearRows, DT>(grads, a, s);
    default: return launch_tiles<MmSmall, DT>(grads, a, s);
  }
}
hipError_t launch_any(bool grads, const GatedArgs& a, hipStream_t s) {
  return a.dt == DT_F32 ? launch_type<DT_F32>(grads, a, s)
         : a.dt == DT_F16 ? launch_type<DT_F16>(grads, a, s) : launch_type<DT_BF16>(grads, a, s);
}

}  // namespace

int64_t gated_sum_rows(int64_t rows, uint32_t in, uint32_t hidden) {
  const int t = gated_tile(rows, hidden, in, true);
  auto sums = [&](auto shape) { return (rows + shape.BM - 1) / shape.BM * shape.WM; };
  return t == 0 ? sums(MmBig{}) : t == 1 ? sums(MmMid{}) : t == 2 ? sums(MmSmall{}) : sums(MmNearRows{});
}

hipError_t launch_gated_forward(const GatedArgs& a, hipStream_t s) { return launch_any(false, a, s); }
hipError_t launch_gated_grads(const GatedArgs& a, hipStream_t s) { return launch_any(true, a, s); }

hipError_t launch_gated_pack(const GatedPack* m, int n, hipStream_t s) {
  if (n < 1) return hipSuccess;
  PackArgs a{};
  uint64_t groups = 0;
  for (int i = 0; i < 3; ++i) {
    a.first[i] = groups;
    if (i >= n) continue;
    a.m[i] = m[i];
    groups += ((uint64_t)m[i].rows * (gated_pad(m[i].cols) / 8) + 255) / 256;
  }
  if (groups == 0) return hipSuccess;
  if (groups > kMostThreads / 256) return hipErrorInvalidValue;
  k_gated_pack<<<(uint32_t)groups, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace tg
