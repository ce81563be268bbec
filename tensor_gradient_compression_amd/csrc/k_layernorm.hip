// Layer norm over the last axis of (rows, cols), and its gradients.
//   mean = sum x / cols;  var = sum (x - mean)^2 / cols;  rstd = 1 / sqrt(var + eps)
//   n = (x - mean) rstd;  y = n w + b
//   h = dy w;  dx = rstd (h - mean(h) - n mean(h n));  dw = sum_rows dy n;  db = sum_rows dy
// Statistics and sums are fp32, results are rounded once. The variance is the mean of the
// squared distances from the mean: the mean of squares less the squared mean would cancel
// for rows far from zero.
//
// Both directions read and write every value once: a row stays in the registers of its
// threads, 8 or 16 values each, between the sums and the result. Rows of up to 512 columns are
// held by 1 to 64 lanes of a wave, so that a wave works on up to 64 rows at once; up to 1024 by
// a wave; up to 4096 by a workgroup of 4 waves and up to 16384 by one of 16, whose waves meet
// in LDS once for each sum. A workgroup walks over rows: the weight and the bias stay in
// registers, and the next row is loaded while the sums of this one are formed. Longer rows are
// read again from the cache for each sum.
// Backward, each thread sums dy n and dy over its rows for its own columns; a workgroup's sums
// become one row of `partial`, and a second kernel adds those rows up in a fixed order.
//
// Rows start anywhere (odd column counts, strides): vector accesses are made at the element's
// alignment, which the hardware takes for global memory.
#include "layernorm.h"

namespace tg {

namespace {

constexpr int kMaxCols = 16384;   // of a row in registers

// Raw values of one wide access, 16 bytes, at the element's alignment.
template <typename T>
struct Piece {
  static constexpr int V = 16 / sizeof(T);
  struct __attribute__((packed, aligned(sizeof(T)))) At {
    T v[V];
  };
  T v[V];
};
// Values c .. c + V - 1 of a row of `cols`; zeros past its end.
template <typename T>
__device__ __forceinline__ void load_piece(const T* __restrict__ row, uint32_t c, uint32_t cols, Piece<T>& p) {
  constexpr int V = Piece<T>::V;
  if (c + V <= cols) {
    __builtin_memcpy(p.v, (const typename Piece<T>::At*)(row + c), 16);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) p.v[j] = c + j < cols ? row[c + j] : zero_of<T>();
  }
}
template <typename T>
__device__ __forceinline__ void store_piece(T* __restrict__ row, uint32_t c, uint32_t cols, const float* x) {
  constexpr int V = Piece<T>::V;
  T v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = from_f32<T>(x[j]);
  if (c + V <= cols) {
    __builtin_memcpy((typename Piece<T>::At*)(row + c), v, 16);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c + j < cols) row[c + j] = v[j];
  }
}
// The weights of columns c .. c + n - 1 as fp32 (`none` where there are none or past the end).
template <typename WT>
__device__ __forceinline__ void load_weights(const WT* __restrict__ w, uint32_t c, int n, uint32_t cols, float none, float* x) {
#pragma unroll
  for (int j = 0; j < n; ++j) x[j] = w && c + j < cols ? to_f32(w[c + j]) : none;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
// The sum over each aligned group of `lanes` lanes (a power of two, the same in the whole
// wave), in all of them: neighbours, pairs, then mirrored halves, rows and halves of the wave.
__device__ __forceinline__ float group_sum(float x, int lanes) {
  if (lanes > 1) x += dpp<0xB1>(x);
  if (lanes > 2) x += dpp<0x4E>(x);
  if (lanes > 4) x += dpp<0x141>(x);
  if (lanes > 8) x += dpp<0x140>(x);
  if (lanes > 16) {
    auto r = __builtin_amdgcn_permlane16_swap((unsigned)__float_as_int(x), (unsigned)__float_as_int(x), false, false);
    x = __int_as_float((int)r[0]) + __int_as_float((int)r[1]);
  }
  if (lanes > 32) {
    auto r = __builtin_amdgcn_permlane32_swap((unsigned)__float_as_int(x), (unsigned)__float_as_int(x), false, false);
    x = __int_as_float((int)r[0]) + __int_as_float((int)r[1]);
  }
  return x;
}

// The threads of a row. WAVES = 1: `lanes` of a wave; else all WAVES waves of the workgroup.
template <int WAVES>
struct RowThreads {
  int lanes;
  float* lds;        // WAVES > 1: 2 x 2 x WAVES floats
  int turn = 0;
  __device__ __forceinline__ uint32_t count() const { return WAVES == 1 ? (uint32_t)lanes : WAVES * 64u; }
  __device__ __forceinline__ uint32_t index() const { return WAVES == 1 ? threadIdx.x & (uint32_t)(lanes - 1) : threadIdx.x; }
  // s and t summed over the row's threads. The waves' sums alternate between two places, so
  // that one barrier a sum is enough: before a place is written again, every wave has passed
  // the barrier of the sum between.
  template <bool TWO>
  __device__ __forceinline__ void sum(float& s, float& t) {
    s = group_sum(s, WAVES == 1 ? lanes : 64);
    if (TWO) t = group_sum(t, WAVES == 1 ? lanes : 64);
    if (WAVES == 1) return;
    float* at = lds + turn * 2 * WAVES;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
      at[threadIdx.x >> 6] = s;
      if (TWO) at[WAVES + (threadIdx.x >> 6)] = t;
    }
    lds_barrier();
    s = group_sum(at[threadIdx.x & (WAVES - 1)], WAVES);
    if (TWO) t = group_sum(at[WAVES + (threadIdx.x & (WAVES - 1))], WAVES);
  }
};

// Threads of a workgroup: 256 for rows in waves.
template <int WAVES>
constexpr int threads_of() { return WAVES == 1 ? 256 : WAVES * 64; }

template <typename T, typename WT, int WAVES, int NV>
__global__ void __launch_bounds__(threads_of<WAVES>()) k_ln_forward(LnForward a, int lanes) {
  constexpr int V = Piece<T>::V, K = NV / V;
  __shared__ float lds[WAVES > 1 ? 4 * WAVES : 1];
  RowThreads<WAVES> rt{lanes, lds};
  const uint32_t per = blockDim.x / rt.count(), t = rt.index(), step = rt.count() * V;
  const int64_t first = (int64_t)blockIdx.x * per + (WAVES == 1 ? threadIdx.x / (uint32_t)lanes : 0);
  const int64_t stride = (int64_t)gridDim.x * per;
  const float inv = 1.0f / (float)a.cols;
  float w[NV], b[NV];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    load_weights((const WT*)a.w, t * V + k * step, V, a.cols, 1.0f, w + k * V);
    load_weights((const WT*)a.b, t * V + k * step, V, a.cols, 0.0f, b + k * V);
  }
  Piece<T> next[K];
  if (first < a.rows)
#pragma unroll
    for (int k = 0; k < K; ++k) load_piece((const T*)a.x + first * a.x_stride, t * V + k * step, a.cols, next[k]);
  // Every thread of a workgroup makes the same number of turns, for the barriers in the sums.
  for (int64_t base = (int64_t)blockIdx.x * per; base < a.rows; base += stride) {
    const int64_t row = base + (first - (int64_t)blockIdx.x * per);
    float x[NV], s = 0.0f, unused;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[k * V + j] = to_f32(next[k].v[j]);
        s += x[k * V + j];
      }
    if (row + stride < a.rows)
#pragma unroll
      for (int k = 0; k < K; ++k)
        load_piece((const T*)a.x + (row + stride) * a.x_stride, t * V + k * step, a.cols, next[k]);
    rt.template sum<false>(s, unused);
    const float mean = s * inv;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = x[k * V + j] - mean;
        x[k * V + j] = d;
        s = __builtin_fmaf(d, t * V + k * step + j < a.cols ? d : 0.0f, s);
      }
    rt.template sum<false>(s, unused);
    const float rstd = 1.0f / sqrtf(s * inv + a.eps);
    if (row >= a.rows) continue;
    T* y = (T*)a.y + row * (int64_t)a.cols;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = __builtin_fmaf(x[k * V + j] * rstd, w[k * V + j], b[k * V + j]);
      store_piece(y, t * V + k * step, a.cols, o);
    }
    if (t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
  }
}

// partial: for every workgroup a row of sums of dy n and one of sums of dy
template <typename T, typename WT, int WAVES, int NV>
__global__ void __launch_bounds__(threads_of<WAVES>()) k_ln_backward(LnBackward a, int lanes) {
  constexpr int V = Piece<T>::V, K = NV / V;
  __shared__ float lds[WAVES > 1 ? 4 * WAVES : 4 * 2 * NV * 64];
  RowThreads<WAVES> rt{lanes, lds};
  const uint32_t per = blockDim.x / rt.count(), t = rt.index(), step = rt.count() * V;
  const int64_t first = (int64_t)blockIdx.x * per + (WAVES == 1 ? threadIdx.x / (uint32_t)lanes : 0);
  const int64_t stride = (int64_t)gridDim.x * per;
  const float inv = 1.0f / (float)a.cols;
  float w[NV], sw[NV], sb[NV];
#pragma unroll
  for (int k = 0; k < K; ++k) load_weights((const WT*)a.w, t * V + k * step, V, a.cols, 1.0f, w + k * V);
#pragma unroll
  for (int i = 0; i < NV; ++i) sw[i] = sb[i] = 0.0f;
  Piece<T> xn[K], dn[K];
  float mean_n = 0.0f, rstd_n = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (first < a.rows) {
      load_piece((const T*)a.x + first * a.x_stride, t * V + k * step, a.cols, xn[k]);
      load_piece((const T*)a.dy + first * a.dy_stride, t * V + k * step, a.cols, dn[k]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) xn[k].v[j] = dn[k].v[j] = zero_of<T>();
    }
  }
  if (first < a.rows) mean_n = a.mean[first], rstd_n = a.rstd[first];
  for (int64_t base = (int64_t)blockIdx.x * per; base < a.rows; base += stride) {
    const int64_t row = base + (first - (int64_t)blockIdx.x * per);
    const float mean = mean_n, rstd = rstd_n;
    float n[NV], h[NV], s = 0.0f, u = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = k * V + j;
        const float dy = to_f32(dn[k].v[j]);
        n[i] = (to_f32(xn[k].v[j]) - mean) * rstd;
        h[i] = dy * w[i];
        s += h[i];
        u = __builtin_fmaf(h[i], n[i], u);
        if (row < a.rows) {
          sw[i] = __builtin_fmaf(dy, n[i], sw[i]);
          sb[i] += dy;
        }
      }
    if (row + stride < a.rows) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        load_piece((const T*)a.x + (row + stride) * a.x_stride, t * V + k * step, a.cols, xn[k]);
        load_piece((const T*)a.dy + (row + stride) * a.dy_stride, t * V + k * step, a.cols, dn[k]);
      }
      mean_n = a.mean[row + stride];
      rstd_n = a.rstd[row + stride];
    }
    rt.template sum<true>(s, u);
    s *= inv;
    u *= inv;
    if (row >= a.rows) continue;
    T* dx = (T*)a.dx + row * (int64_t)a.cols;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = rstd * ((h[k * V + j] - s) - n[k * V + j] * u);
      store_piece(dx, t * V + k * step, a.cols, o);
    }
  }
  if (!a.partial) return;
  float* pw = a.partial + (uint64_t)blockIdx.x * 2 * a.cols;
  if (WAVES > 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t c = t * V + k * step + j;
        if (c < a.cols) {
          pw[c] = sw[k * V + j];
          pw[a.cols + c] = sb[k * V + j];
        }
      }
    return;
  }
  // the row groups of a wave, then the four waves, always in the same order
#pragma unroll
  for (int i = 0; i < NV; ++i)
    for (int o = lanes; o < 64; o <<= 1) {
      sw[i] += __shfl_xor(sw[i], o, 64);
      sb[i] += __shfl_xor(sb[i], o, 64);
    }
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    lds[(wave * 2 * NV + i) * 64 + lane] = sw[i];
    lds[(wave * 2 * NV + NV + i) * 64 + lane] = sb[i];
  }
  __syncthreads();
  // wave q sums half of the values of one kind
#pragma unroll
  for (int i = 0; i < NV / 2; ++i) {
    const uint32_t v = (wave & 1) * (NV / 2) + i, kind = wave >> 1;
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) s += lds[(q * 2 * NV + kind * NV + v) * 64 + lane];
    const uint32_t c = t * V + (v / V) * step + v % V;
    if (lane < (uint32_t)lanes && c < a.cols) pw[kind * a.cols + c] = s;
  }
}

// ---------------------------------------------------------------- rows beyond the registers
constexpr int kLong = 1024;

template <typename T, typename WT>
__global__ void __launch_bounds__(kLong) k_ln_forward_long(LnForward a) {
  constexpr int V = Piece<T>::V;
  __shared__ float lds[4 * (kLong / 64)];
  RowThreads<kLong / 64> rt{64, lds};
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.x_stride;
  T* y = (T*)a.y + row * (int64_t)a.cols;
  float s = 0.0f, unused;
  Piece<T> p;
  for (uint32_t c = threadIdx.x * V; c < a.cols; c += kLong * V) {
    load_piece(x, c, a.cols, p);
#pragma unroll
    for (int j = 0; j < V; ++j) s += to_f32(p.v[j]);
  }
  rt.template sum<false>(s, unused);
  const float mean = s / (float)a.cols;
  s = 0.0f;
  for (uint32_t c = threadIdx.x * V; c < a.cols; c += kLong * V) {
    load_piece(x, c, a.cols, p);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = to_f32(p.v[j]) - mean;
      s = __builtin_fmaf(d, c + j < a.cols ? d : 0.0f, s);
    }
  }
  rt.template sum<false>(s, unused);
  const float rstd = 1.0f / sqrtf(s / (float)a.cols + a.eps);
  for (uint32_t c = threadIdx.x * V; c < a.cols; c += kLong * V) {
    float w[V], b[V], o[V];
    load_piece(x, c, a.cols, p);
    load_weights((const WT*)a.w, c, V, a.cols, 1.0f, w);
    load_weights((const WT*)a.b, c, V, a.cols, 0.0f, b);
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = __builtin_fmaf((to_f32(p.v[j]) - mean) * rstd, w[j], b[j]);
    store_piece(y, c, a.cols, o);
  }
  if (threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
}

template <typename T, typename WT>
__global__ void __launch_bounds__(kLong) k_ln_dx_long(LnBackward a) {
  constexpr int V = Piece<T>::V;
  __shared__ float lds[4 * (kLong / 64)];
  RowThreads<kLong / 64> rt{64, lds};
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.x_stride;
  const T* dy = (const T*)a.dy + row * a.dy_stride;
  T* dx = (T*)a.dx + row * (int64_t)a.cols;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s = 0.0f, u = 0.0f, w[V];
  Piece<T> p, q;
  for (uint32_t c = threadIdx.x * V; c < a.cols; c += kLong * V) {
    load_piece(x, c, a.cols, p);
    load_piece(dy, c, a.cols, q);
    load_weights((const WT*)a.w, c, V, a.cols, 1.0f, w);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float h = to_f32(q.v[j]) * w[j];
      s += h;
      u = __builtin_fmaf(h, (to_f32(p.v[j]) - mean) * rstd, u);
    }
  }
  rt.template sum<true>(s, u);
  s /= (float)a.cols;
  u /= (float)a.cols;
  for (uint32_t c = threadIdx.x * V; c < a.cols; c += kLong * V) {
    float o[V];
    load_piece(x, c, a.cols, p);
    load_piece(dy, c, a.cols, q);
    load_weights((const WT*)a.w, c, V, a.cols, 1.0f, w);
#pragma unroll
    for (int j = 0; j < V; ++j)
      o[j] = rstd * ((to_f32(q.v[j]) * w[j] - s) - (to_f32(p.v[j]) - mean) * rstd * u);
    store_piece(dx, c, a.cols, o);
  }
}

// partial row r: the sums over rows r, r + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256) k_ln_columns(LnBackward a) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.cols) return;
  float s = 0.0f, t = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float dy = to_f32(((const T*)a.dy)[row * a.dy_stride + i]);
    s = __builtin_fmaf(dy, (to_f32(((const T*)a.x)[row * a.x_stride + i]) - a.mean[row]) * a.rstd[row], s);
    t += dy;
  }
  a.partial[(uint64_t)blockIdx.y * 2 * a.cols + i] = s;
  a.partial[((uint64_t)blockIdx.y * 2 + 1) * a.cols + i] = t;
}

// ---------------------------------------------------------------- the partial rows' sums
// blockIdx.y: dw or db; 32 columns a workgroup, 32 threads a column
template <typename WT>
__global__ void __launch_bounds__(1024) k_ln_reduce(const float* __restrict__ partial, uint32_t n, uint32_t cols,
                                                    WT* __restrict__ dw, WT* __restrict__ db) {
  __shared__ float lds[32][33];
  const uint32_t tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  WT* out = blockIdx.y ? db : dw;
  if (!out) return;
  float s = 0.0f;
  if (c < cols) {
    const float* p = partial + (uint64_t)blockIdx.y * cols + c;
#pragma unroll 8
    for (uint32_t r = ty; r < n; r += 32) s += p[(uint64_t)r * 2 * cols];
  }
  lds[ty][tx] = s;
  __syncthreads();
  s = group_sum(lds[tx][ty], 32);
  const uint32_t o = blockIdx.x * 32 + ty;
  if (tx == 0 && o < cols) out[o] = from_f32<WT>(s);
}

// ---------------------------------------------------------------- launches
// Workgroups of a walk over `rows`, `per` rows at a time: no more than `most`.
uint32_t walk(int64_t rows, uint32_t per, uint32_t most) {
  const int64_t n = (rows + per - 1) / per;
  return (uint32_t)(n < (int64_t)most ? n : (int64_t)most);
}
int lanes_of(uint32_t cols) {
  int lanes = 1;
  while (lanes < 64 && (uint32_t)lanes * 8 < cols) lanes *= 2;
  return lanes;
}

template <typename T, typename WT>
hipError_t forward(const LnForward& a, hipStream_t s) {
  const int lanes = lanes_of(a.cols);
  if (a.cols <= 512)
    k_ln_forward<T, WT, 1, 8><<<walk(a.rows, 256 / lanes, 2048), 256, 0, s>>>(a, lanes);
  else if (a.cols <= 1024)
    k_ln_forward<T, WT, 1, 16><<<walk(a.rows, 4, 2048), 256, 0, s>>>(a, 64);
  else if (a.cols <= 2048)
    k_ln_forward<T, WT, 4, 8><<<walk(a.rows, 1, 2048), 256, 0, s>>>(a, 64);
  else if (a.cols <= 4096)
    k_ln_forward<T, WT, 4, 16><<<walk(a.rows, 1, 2048), 256, 0, s>>>(a, 64);
  else if (a.cols <= 8192)
    k_ln_forward<T, WT, 16, 8><<<walk(a.rows, 1, 512), 1024, 0, s>>>(a, 64);
  else if (a.cols <= kMaxCols)
    k_ln_forward<T, WT, 16, 16><<<walk(a.rows, 1, 512), 1024, 0, s>>>(a, 64);
  else
    k_ln_forward_long<T, WT><<<(uint32_t)a.rows, kLong, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, typename WT>
hipError_t backward(LnBackward a, hipStream_t s) {
  const uint32_t n = ln_partial_rows(a.rows, a.cols);
  const bool params = a.dw || a.db;
  if (!params) a.partial = nullptr;
  const int lanes = lanes_of(a.cols);
  if (!a.rows) {
  } else if (a.cols <= 512) {
    k_ln_backward<T, WT, 1, 8><<<n, 256, 0, s>>>(a, lanes);
  } else if (a.cols <= 1024) {
    k_ln_backward<T, WT, 1, 16><<<n, 256, 0, s>>>(a, 64);
  } else if (a.cols <= 2048) {
    k_ln_backward<T, WT, 4, 8><<<n, 256, 0, s>>>(a, 64);
  } else if (a.cols <= 4096) {
    k_ln_backward<T, WT, 4, 16><<<n, 256, 0, s>>>(a, 64);
  } else if (a.cols <= 8192) {
    k_ln_backward<T, WT, 16, 8><<<n, 1024, 0, s>>>(a, 64);
  } else if (a.cols <= kMaxCols) {
    k_ln_backward<T, WT, 16, 16><<<n, 1024, 0, s>>>(a, 64);
  } else {
    k_ln_dx_long<T, WT><<<(uint32_t)a.rows, kLong, 0, s>>>(a);
    if (params) k_ln_columns<T><<<dim3((a.cols + 255) / 256, n), 256, 0, s>>>(a);
  }
  if (params)
    k_ln_reduce<WT><<<dim3((a.cols + 31) / 32, 2), 1024, 0, s>>>(a.partial, n, a.cols, (WT*)a.dw, (WT*)a.db);
  return hipGetLastError();
}

}  // namespace

// Workgroups of the backward walk, each of which leaves one row of sums: as many as keep the
// CUs busy, and no more than there are rows for.
uint32_t ln_partial_rows(int64_t rows, uint32_t cols) {
  if (cols <= 512) return walk(rows, 256 / lanes_of(cols), 1024);
  if (cols <= 1024) return walk(rows, 4, 1024);
  if (cols <= 4096) return walk(rows, 1, 1024);
  return walk(rows, 1, 512);
}

hipError_t launch_ln_forward(const LnForward& a, hipStream_t s) {
  if (!a.rows) return hipSuccess;
  if (a.dt == DT_F32) return forward<float, float>(a, s);
  if (a.dt == DT_F16 && a.wdt == DT_F32) return forward<_Float16, float>(a, s);
  if (a.dt == DT_F16) return forward<_Float16, _Float16>(a, s);
  if (a.wdt == DT_F32) return forward<bf16_t, float>(a, s);
  return forward<bf16_t, bf16_t>(a, s);
}

hipError_t launch_ln_backward(const LnBackward& a, hipStream_t s) {
  if (a.dt == DT_F32) return backward<float, float>(a, s);
  if (a.dt == DT_F16 && a.wdt == DT_F32) return backward<_Float16, float>(a, s);
  if (a.dt == DT_F16) return backward<_Float16, _Float16>(a, s);
  if (a.wdt == DT_F32) return backward<bf16_t, float>(a, s);
  return backward<bf16_t, bf16_t>(a, s);
}

}  // namespace tg
