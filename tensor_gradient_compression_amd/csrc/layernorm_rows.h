// Layer norm: how rows are held by threads (gfx950 only). Shared by k_layernorm.hip and
// k_layernorm_bwd.hip.
//
// Both directions read and write every value once: a row stays in the registers of its
// threads, 8 or 16 values each, between the sums and the result. LANES lanes of a wave hold a
// row of up to 1024 columns (a wave then works on 64 / LANES rows at once); a workgroup of 4
// waves holds one of up to 4096 and one of 16 waves one of up to 16384, whose waves meet in LDS
// once for each sum. A workgroup walks over rows: the weight and the bias stay in registers,
// and the next row is loaded while the sums of this one are formed. Longer rows are read again
// from the cache for each sum.
//
// Every access is 16 bytes wide, at the element's alignment, which the hardware takes for
// global memory: rows start anywhere (odd column counts, strides). Where the columns do not
// divide into pieces of 16 bytes, the last piece of a row is moved back to end with it. It then
// holds some columns of the piece before as well, computes the same results for them and
// writes those twice; its sums leave them out.
#pragma once
#include "layernorm.h"

namespace tg {

// Raw values of one wide access.
template <typename T>
struct Piece {
  static constexpr int V = 16 / sizeof(T);
  T v[V];
};
template <typename T, int N>
struct __attribute__((packed, aligned(sizeof(T)))) Unaligned {
  T v[N];
};
template <typename T>
__device__ __forceinline__ void load_piece(const T* __restrict__ p, Piece<T>& x) {
  __builtin_memcpy(x.v, (const Unaligned<T, Piece<T>::V>*)p, 16);
}
template <typename T>
__device__ __forceinline__ void store_piece(T* __restrict__ p, const float* x) {
  constexpr int V = Piece<T>::V;
  T v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = from_f32<T>(x[j]);
  __builtin_memcpy((Unaligned<T, V>*)p, v, 16);
}

// How the columns of a row divide: into whole pieces; with a last piece moved back; or less
// than one piece, which is read and written value by value.
enum Columns { WHOLE = 0, RAGGED = 1, TINY = 2 };

// One piece of a row: its first column, and from which of its values on they are its own (V
// where the piece lies past the row's end: nothing is read or written).
template <typename T, int COLS>
struct Place {
  static constexpr int V = Piece<T>::V;
  uint32_t c;
  int own;
  __device__ __forceinline__ Place() {}
  __device__ __forceinline__ Place(uint32_t at, uint32_t cols) : c(at), own(at < cols ? 0 : V) {
    if (COLS == RAGGED && at < cols && at + V > cols) {
      c = cols - V;
      own = (int)(at + V - cols);
    }
  }
  // whether value j counts in sums
  __device__ __forceinline__ bool mine(int j, uint32_t cols) const {
    return COLS == TINY ? c + j < cols : j >= own;
  }
  __device__ __forceinline__ void load(const T* __restrict__ row, uint32_t cols, Piece<T>& x) const {
    if (COLS == TINY) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c + j < cols) x.v[j] = row[c + j];
    } else if (own < V) {
      load_piece(row + c, x);
    }
  }
  __device__ __forceinline__ void store(T* __restrict__ row, uint32_t cols, const float* x) const {
    if (COLS == TINY) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c + j < cols) row[c + j] = from_f32<T>(x[j]);
    } else if (own < V) {
      store_piece(row + c, x);
    }
  }
  // the weights of these columns, `none` without any
  __device__ __forceinline__ void weights(const void* w, int wdt, uint32_t cols, float none, float* x) const {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = none;
    if (!w || own >= V) return;
    if (COLS == TINY) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c + j < cols) x[j] = wdt == DT_F32 ? ((const float*)w)[c + j] : to_f32(((const T*)w)[c + j]);
    } else if (wdt == DT_F32) {
      __builtin_memcpy(x, (const Unaligned<float, V>*)((const float*)w + c), V * sizeof(float));
    } else {
      Piece<T> p;
      load_piece((const T*)w + c, p);
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = to_f32(p.v[j]);
    }
  }
};
template <typename T>
__device__ __forceinline__ void clear(Piece<T>& x) {
#pragma unroll
  for (int j = 0; j < Piece<T>::V; ++j) x.v[j] = zero_of<T>();
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
// The sum over each aligned group of LANES lanes, in all of them: neighbours, pairs, then
// mirrored halves of 8 and 16, rows and halves of the wave.
template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
  if (LANES > 1) x += dpp<0xB1>(x);
  if (LANES > 2) x += dpp<0x4E>(x);
  if (LANES > 4) x += dpp<0x141>(x);
  if (LANES > 8) x += dpp<0x140>(x);
  if (LANES > 16) {
    auto r = __builtin_amdgcn_permlane16_swap((unsigned)__float_as_int(x), (unsigned)__float_as_int(x), false, false);
    x = __int_as_float((int)r[0]) + __int_as_float((int)r[1]);
  }
  if (LANES > 32) {
    auto r = __builtin_amdgcn_permlane32_swap((unsigned)__float_as_int(x), (unsigned)__float_as_int(x), false, false);
    x = __int_as_float((int)r[0]) + __int_as_float((int)r[1]);
  }
  return x;
}

// The threads of a row: LANES lanes of a wave, or (LANES = 64) all WAVES waves of the
// workgroup.
template <int WAVES, int LANES>
struct RowThreads {
  static constexpr int kThreads = WAVES == 1 ? 256 : WAVES * 64;   // of a workgroup
  static constexpr int kCount = WAVES * LANES;
  static constexpr int kRows = kThreads / kCount;                   // of a workgroup at a time
  static constexpr int kLds = WAVES > 1 ? 4 * WAVES : 1;
  float* lds;
  int turn = 0;
  static __device__ __forceinline__ uint32_t index() { return threadIdx.x % kCount; }
  static __device__ __forceinline__ uint32_t row() { return threadIdx.x / kCount; }
  // s and t summed over the row's threads. The waves' sums alternate between two places, so
  // that one barrier a sum is enough: before a place is written again, every wave has passed
  // the barrier of the sum between.
  template <bool TWO>
  __device__ __forceinline__ void sum(float& s, float& t) {
    s = group_sum<LANES>(s);
    if (TWO) t = group_sum<LANES>(t);
    if (WAVES == 1) return;
    float* at = lds + turn * 2 * WAVES;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
      at[threadIdx.x >> 6] = s;
      if (TWO) at[WAVES + (threadIdx.x >> 6)] = t;
    }
    lds_barrier();
    s = group_sum<WAVES>(at[threadIdx.x & (WAVES - 1)]);
    if (TWO) t = group_sum<WAVES>(at[WAVES + (threadIdx.x & (WAVES - 1))]);
  }
};

constexpr uint32_t LN_MAX_COLS = 16384;   // of a row in registers

// Calls f.template operator()<WAVES, LANES, NV>() for the threads that hold rows of `cols`
// values, `v` to a piece: as few lanes as hold it with 8 or 16 values each.
template <typename F>
bool ln_dispatch(uint32_t cols, F f) {
  if (cols <= 8) f.template run<1, 1, 8>();
  else if (cols <= 32) f.template run<1, 4, 8>();
  else if (cols <= 128) f.template run<1, 16, 8>();
  else if (cols <= 256) f.template run<1, 16, 16>();
  else if (cols <= 512) f.template run<1, 64, 8>();
  else if (cols <= 1024) f.template run<1, 64, 16>();
  else if (cols <= 2048) f.template run<4, 64, 8>();
  else if (cols <= 4096) f.template run<4, 64, 16>();
  else if (cols <= 8192) f.template run<16, 64, 8>();
  else if (cols <= LN_MAX_COLS) f.template run<16, 64, 16>();
  else return false;
  return true;
}

// Workgroups of a walk over `rows`, `per` rows at a time: no more than `most`.
inline uint32_t ln_walk(int64_t rows, int per, uint32_t most) {
  const int64_t n = (rows + per - 1) / per;
  return (uint32_t)(n < (int64_t)most ? n : (int64_t)most);
}

constexpr int LN_LONG = 1024;   // threads of a row beyond the registers

}  // namespace tg
