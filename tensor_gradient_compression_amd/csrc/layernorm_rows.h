// Layer norm: how rows are held by threads (gfx950 only). Shared by k_layernorm.hip and
// k_layernorm_bwd.hip.
//
// Both directions read and write every value once: a row stays in the registers of its
// threads, 8 or 16 values each, between the sums and the result. LANES lanes of a wave hold a
// row of up to 1024 columns (a wave then works on 64 / LANES rows at once); longer rows of up
// to 16384 columns are held by as many waves as they need, which meet in LDS once for each
// sum. A workgroup walks over rows: the weight and the bias stay in registers, and the next row
// is loaded while the sums of this one are formed. Longer rows are read again from the cache for
// each sum, by one workgroup each (3000 x 32768 bf16: forward 114 us, 3.4 TB/s of what it needs;
// backward 319, 1.8 TB/s).
//
// Every access is 16 bytes wide, at the element's alignment, which the hardware takes for
// global memory: rows start anywhere (odd column counts, strides). Where the columns do not
// divide into pieces of 16 bytes, the last piece of a row is moved back to end with it. It then
// holds some columns of the piece before as well, computes the same results for them and
// writes those twice; its sums leave them out.
//
// Both directions are bound by memory where rows are many (rates at 67M values): forward 5.8 to
// 6.2 TB/s in bf16 and 6.2 to 6.7 in fp32, backward 5.2 to 5.9 and 5.5 to 6.4, for whole pieces
// of any width; bf16 rows of several waves that start at odd values (2001 to 12001 columns) 5.5 to
// 6.0 and 4.8 to 5.2. Held by their threads as the fewest lanes with 8 values each, since
// fewer lanes with 16 leave room for fewer waves (backward, 65536 x 256 bf16: 20 us, 18.4).
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
// The same, marked as not to be kept in the caches.
template <typename T>
__device__ __forceinline__ void load_piece_once(const T* __restrict__ p, Piece<T>& x) {
  typedef uint32_t Q __attribute__((ext_vector_type(4)));
  typedef Q QU __attribute__((aligned(2)));
  const Q q = __builtin_nontemporal_load((const QU*)p);
  __builtin_memcpy(x.v, &q, 16);
}
template <typename T>
__device__ __forceinline__ void store_piece(T* __restrict__ p, const float* x) {
  constexpr int V = Piece<T>::V;
  T v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = from_f32<T>(x[j]);
  __builtin_memcpy((Unaligned<T, V>*)p, v, 16);
}

// How the columns of a row divide: into whole pieces; with a last piece moved back; less than
// one piece, which is read and written value by value; or, of rows of 16-bit values that several
// waves hold and some of which start at odd ones, as RAGGED but read by whole words: loads off the
// words make 15 to 25% of a call (33M fp16 values: 4099 columns forward 30 -> 25 us, 2001
// backward 59 -> 50, 12001 76 -> 58; rows that a wave holds gain nothing, 255 columns 44 -> 48).
enum Columns { WHOLE = 0, RAGGED = 1, TINY = 2, ODD = 3 };
constexpr bool ln_moves(int columns) { return columns == RAGGED || columns == ODD; }

// A piece as it is loaded. ODD: as the four words that begin at its first value or one before
// (which is in the same word); the value that ends it then comes from the next lane, or by itself
// where that holds no neighbour.
template <typename T, int COLS>
struct Raw {
  Piece<T> x;
  uint32_t end;
};

// One piece of a row: its first column, and from which of its values on they are its own (V
// where the piece lies past the row's end: nothing is read or written).
template <typename T, int COLS>
struct Place {
  static constexpr int V = Piece<T>::V;
  uint32_t c;
  int own;
  bool alone;   // whether the next lane of the wave does not hold the next piece of the row
  __device__ __forceinline__ Place() {}
  __device__ __forceinline__ Place(uint32_t at, uint32_t cols, bool last_lane = true)
      : c(at), own(at < cols ? 0 : V), alone(last_lane || at + 2 * V > cols) {
    if (ln_moves(COLS) && at < cols && at + V > cols) {
      c = cols - V;
      own = (int)(at + V - cols);
    }
  }
  // whether value j counts in sums
  __device__ __forceinline__ bool mine(int j, uint32_t cols) const {
    return COLS == TINY ? c + j < cols : j >= own;
  }
  __device__ __forceinline__ void load(const T* __restrict__ row, uint32_t cols, bool once, Piece<T>& x) const {
    if (COLS == TINY) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c + j < cols) x.v[j] = row[c + j];
    } else if (own < V) {
      if (once) load_piece_once(row + c, x);
      else load_piece(row + c, x);
    }
  }
  // the same, of the walks: fetch() and, when it is used, piece() with the same row
  __device__ __forceinline__ void fetch(const T* __restrict__ row, uint32_t cols, bool once, Raw<T, COLS>& r) const {
    if constexpr (COLS != ODD) {
      load(row, cols, once, r.x);
    } else {
      if (own >= V) return;
      const T* p = row + c;
      const uint32_t odd = (uint32_t)(uintptr_t)p >> 1 & 1u;
      if (once) load_piece_once(p - odd, r.x);
      else load_piece(p - odd, r.x);
      // without a branch, whose end would wait for it: the others read the row's first value
      r.end = __builtin_bit_cast(uint16_t, *(alone && odd ? p + V - 1 : row));
    }
  }
  __device__ __forceinline__ Piece<T> piece(const T* row, const Raw<T, COLS>& r) const {
    if constexpr (COLS != ODD) return r.x;
    uint32_t q[5];
    __builtin_memcpy(q, r.x.v, 16);
    const uint32_t next = (uint32_t)__builtin_amdgcn_mov_dpp((int)q[0], 0x130, 0xF, 0xF, true);   // the next lane's
    q[4] = alone ? r.end : next;
    const uint32_t by = (uint32_t)(uintptr_t)(row + c) << 3 & 16u;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __builtin_amdgcn_alignbit(q[i + 1], q[i], by);
    Piece<T> x;
    __builtin_memcpy(x.v, q, 16);
    return x;
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
template <typename T, int COLS>
__device__ __forceinline__ void clear(Raw<T, COLS>& r) {
#pragma unroll
  for (int j = 0; j < Piece<T>::V; ++j) r.x.v[j] = zero_of<T>();
  r.end = 0;
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

// s / cols from the rounded reciprocal `inv`: the product, corrected by its exact residual, so
// that a quotient that fp32 holds comes out as it is (the product alone is off by a unit for
// some constant rows of 7, 13, 15 ... columns, and eps makes hundreds of that distance).
__device__ __forceinline__ float mean_of(float s, float cols, float inv) {
  const float m = s * inv;
  return fabsf(m) < INFINITY ? __builtin_fmaf(__builtin_fmaf(-m, cols, s), inv, m) : m;
}

// 1 / sqrt(a): the hardware's estimate and one Newton step, within 1.5 units of the last place;
// outside a range that keeps both away from overflow and subnormal numbers the slow exact way.
__device__ __forceinline__ float reciprocal_root(float a) {
  const float y = __builtin_amdgcn_rsqf(a);
  float r = __builtin_fmaf(0.5f * y, __builtin_fmaf(-a * y, y, 1.0f), y);
  if (__any(!(a >= 0x1p-100f && a <= 0x1p100f))) {
    __asm__ volatile("" : "+v"(a));   // a branch of its own, not computed beside the other
    r = 1.0f / sqrtf(a);
  }
  return r;
}

// The threads of a row: LANES lanes of a wave in a workgroup of 4 waves, or (LANES = 0) all
// threads of the workgroup, up to 16 waves.
template <int LANES>
struct RowThreads {
  static constexpr bool kWave = LANES > 0;
  static constexpr int kMost = kWave ? 256 : 1024;           // threads of a workgroup
  static constexpr int kRows = kWave ? 256 / (LANES + !LANES) : 1;   // of a workgroup at a time
  static constexpr int kLds = kWave ? 1 : 64;
  float* lds;
  int turn = 0;
  __device__ __forceinline__ explicit RowThreads(float* l) : lds(l) {
    // the places of waves that the workgroup does not have stay zero
    if (!kWave && threadIdx.x < 64) lds[threadIdx.x] = 0.0f;
    if (!kWave) lds_barrier();
  }
  static __device__ __forceinline__ uint32_t count() { return kWave ? LANES : blockDim.x; }
  static __device__ __forceinline__ uint32_t index() { return kWave ? threadIdx.x % (LANES + !LANES) : threadIdx.x; }
  // whether the next lane of the wave, if any, holds another row
  static __device__ __forceinline__ bool last_lane() { return (threadIdx.x + 1) % (kWave ? LANES : 64) == 0; }
  static __device__ __forceinline__ uint32_t row() { return kWave ? threadIdx.x / (LANES + !LANES) : 0; }
  // s and t summed over the row's threads. The waves' sums alternate between two places, so
  // that one barrier a sum is enough: before a place is written again, every wave has passed
  // the barrier of the sum between.
  template <bool TWO>
  __device__ __forceinline__ void sum(float& s, float& t) {
    s = group_sum<kWave ? LANES : 64>(s);
    if (TWO) t = group_sum<kWave ? LANES : 64>(t);
    if (kWave) return;
    float* at = lds + turn * 32;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
      at[threadIdx.x >> 6] = s;
      if (TWO) at[16 + (threadIdx.x >> 6)] = t;
    }
    lds_barrier();
    s = group_sum<16>(at[threadIdx.x & 15]);
    if (TWO) t = group_sum<16>(at[16 + (threadIdx.x & 15)]);
  }
};

// Waves of a kernel that a CU holds at once; the launch bounds keep the registers to that. A
// walk takes as many workgroups as then run at the same time: with some more the last ones
// start alone (1536 columns of bf16, forward: 5.8 TB/s, 5.2 with 7% too many).
constexpr uint32_t LN_CUS = 256;
constexpr uint32_t ln_forward_waves(int nv) { return nv == 8 ? 32 : 20; }
constexpr uint32_t ln_backward_waves(int lanes, int nv) { return nv == 8 ? 20 : lanes ? 12 : 16; }

constexpr uint32_t LN_MAX_COLS = 16384;   // of a row in registers

// Whether some row starts at an odd 16-bit value.
template <typename T>
bool ln_odd(const void* p, int64_t stride) {
  return sizeof(T) == 2 && (((uintptr_t)p >> 1 | (uintptr_t)stride) & 1);
}

// Calls f.run<LANES, NV>(threads) for the threads that hold rows of `cols` values: as few lanes
// of a wave as do with 8 values each, a wave with 16, or a workgroup of as many waves as do with
// 8 or 16.
template <typename F>
bool ln_dispatch(uint32_t cols, F f) {
  if (cols <= 8) f.template run<1, 8>(256);
  else if (cols <= 16) f.template run<2, 8>(256);
  else if (cols <= 32) f.template run<4, 8>(256);
  else if (cols <= 64) f.template run<8, 8>(256);
  else if (cols <= 128) f.template run<16, 8>(256);
  else if (cols <= 256) f.template run<32, 8>(256);
  else if (cols <= 512) f.template run<64, 8>(256);
  else if (cols <= 1024) f.template run<64, 16>(256);
  else if (cols <= 8192) f.template run<0, 8>((cols + 511) / 512 * 64);
  else if (cols <= LN_MAX_COLS) f.template run<0, 16>((cols + 1023) / 1024 * 64);
  else return false;
  return true;
}

// Whether a call that reads and writes this much asks the caches not to keep what it reads:
// more than they hold anyway (fp32, 67M values: forward 5.3 -> 6.5 TB/s, backward 5.2 -> 6.2;
// bf16 backward 5.2 -> 5.8). Below, part of it may be there still (bf16 forward, 268 MB: 5.9
// with and 5.6 TB/s without).
inline bool ln_once(int64_t bytes) { return bytes > 300000000; }

// Workgroups of a walk over `rows`, `per` rows at a time: no more than `most`.
inline uint32_t ln_walk(int64_t rows, int per, uint32_t most) {
  const int64_t n = (rows + per - 1) / per;
  return (uint32_t)(n < (int64_t)most ? n : (int64_t)most);
}

constexpr int LN_LONG = 1024;   // threads of a row beyond the registers
// Workgroups that walk over such rows: a launch whose threads along an axis pass 32 bits is cut
// to the rest without an error.
constexpr uint32_t LN_LONG_GROUPS = 1 << 16;

}  // namespace tg
