// The gradients of layer norm over the last axis of (rows, cols), from its inputs and
// statistics:
//   n = (x - mean) rstd;  h = dy w;  dx = rstd (h - mean(h) - n mean(h n))
//   dw = sum_rows dy n;  db = sum_rows dy
// Sums are fp32, results are rounded once. Rows and threads: layernorm_rows.h. Each thread
// also sums dy n and dy over its rows for its own columns; a workgroup's sums become one row of
// `partial`, and a second kernel adds those rows up, always in the same order. A workgroup that
// is alone writes dw and db at once.
#include "layernorm_rows.h"

namespace tg {

namespace {

// Values of dw or db, from the place's `from`-th on.
template <typename WT, int V>
__device__ __forceinline__ void put(WT* out, int from, const float* x) {
  WT v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = from_f32<WT>(x[j]);
  if (from == 0) {
    __builtin_memcpy((Unaligned<WT, V>*)out, v, sizeof v);
    return;
  }
#pragma unroll
  for (int j = 1; j < V; ++j)
    if (j >= from) out[j] = v[j];
}
template <typename T, int V>
__device__ __forceinline__ void put(void* out, int wdt, uint32_t c, int from, const float* x) {
  if (!out) return;
  if (sizeof(T) == 4 || wdt == DT_F32) put<float, V>((float*)out + c, from, x);
  else put<T, V>((T*)out + c, from, x);
}

// Up to 16 values a thread their sums over rows, the weights and two rows fit the registers;
// with 16 waves and 16 values (128 registers a thread) the weights stay in LDS as fp32.
// ONCE: see ln_once; as an argument the choice between two loads makes every one wait at once.
template <typename T, int LANES, int NV, int COLS, bool ONCE>
__global__ void __launch_bounds__(RowThreads<LANES>::kMost, ln_backward_waves(LANES, NV) / 4)
    k_ln_backward(LnBackward a) {
  using RT = RowThreads<LANES>;
  constexpr int V = Piece<T>::V, K = NV / V;
  constexpr bool kKeep = !(LANES == 0 && NV == 16);
  __shared__ float lds[RT::kWave ? 4 * 2 * NV * LANES : RT::kLds];
  __shared__ float wl[kKeep ? 1 : LN_MAX_COLS];
  RT rt(lds);
  const int64_t stride = (int64_t)gridDim.x * RT::kRows;
  const float inv = 1.0f / (float)a.cols;
  int64_t row = (int64_t)blockIdx.x * RT::kRows + RT::row();
  Place<T, COLS> at[K];
  Raw<T, COLS> xn[K], dn[K];
  float mean_n = 0.0f, rstd_n = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    at[k] = Place<T, COLS>((RT::index() + k * RT::count()) * V, a.cols, RT::last_lane());
    clear(xn[k]);
    clear(dn[k]);
    if (row < a.rows) {
      at[k].fetch((const T*)a.x + row * a.x_stride, a.cols, ONCE, xn[k]);
      at[k].fetch((const T*)a.dy + row * a.dy_stride, a.cols, ONCE, dn[k]);
    }
  }
  if (row < a.rows) mean_n = a.mean[row], rstd_n = a.rstd[row];
  float w[kKeep ? NV : V], sw[NV], sb[NV];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    at[k].weights(a.w, a.wdt, a.cols, 1.0f, w + (kKeep ? k * V : 0));
    if (!kKeep) {   // read back by this thread alone
#pragma unroll
      for (int j = 0; j < V; ++j) wl[(k * V + j) * 1024 + threadIdx.x] = w[j];
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) sw[i] = sb[i] = 0.0f;
  for (int64_t base = (int64_t)blockIdx.x * RT::kRows; base < a.rows; base += stride, row += stride) {
    Piece<T> xp[K], dp[K];
    const float mean = mean_n, rstd = rstd_n;
    float s = 0.0f, u = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      xp[k] = at[k].piece((const T*)a.x + row * a.x_stride, xn[k]);
      dp[k] = at[k].piece((const T*)a.dy + row * a.dy_stride, dn[k]);
    }
    if (row + stride < a.rows) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        at[k].fetch((const T*)a.x + (row + stride) * a.x_stride, a.cols, ONCE, xn[k]);
        at[k].fetch((const T*)a.dy + (row + stride) * a.dy_stride, a.cols, ONCE, dn[k]);
      }
      mean_n = a.mean[row + stride];
      rstd_n = a.rstd[row + stride];
    } else {
      // a row past the end adds zeros
#pragma unroll
      for (int k = 0; k < K; ++k) clear(dn[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!kKeep) {
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = wl[(k * V + j) * 1024 + threadIdx.x];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = k * V + j;
        const float dy = to_f32(dp[k].v[j]), d = to_f32(xp[k].v[j]) - mean;
        const float h = ln_moves(COLS) && !at[k].mine(j, a.cols) ? 0.0f : dy * w[kKeep ? i : j];
        s += h;
        u = __builtin_fmaf(h, d, u);
        sw[i] = __builtin_fmaf(dy, d * rstd, sw[i]);
        sb[i] += dy;
      }
    }
    rt.template sum<true>(s, u);
    // dx = rstd (h - mean(h) + d du), with d = x - mean. mean(h) is taken off h itself, where
    // rstd h less rstd mean(h) would leave the rounding of one product: with a single column,
    // or the same h in all of them, nothing may be left
    const float mh = mean_of(s, (float)a.cols, inv), du = -rstd * (rstd * (u * inv));
    if (row >= a.rows) continue;
    T* dx = (T*)a.dx + row * (int64_t)a.cols;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float o[V];
      if (!kKeep) {
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = wl[(k * V + j) * 1024 + threadIdx.x];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = to_f32(xp[k].v[j]) - mean, h = to_f32(dp[k].v[j]) * w[kKeep ? k * V + j : j];
        o[j] = rstd * __builtin_fmaf(d, du, h - mh);
      }
      at[k].store(dx, a.cols, o);
    }
  }
  if (!a.partial) return;
  float* pw = a.partial + (uint64_t)blockIdx.x * 2 * a.cols;
  if (RT::kWave) {
    // the row groups of a wave, then the four waves, always in the same order
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int o = LANES + !LANES; o < 64; o <<= 1) {
        sw[i] += __shfl_xor(sw[i], o, 64);
        sb[i] += __shfl_xor(sb[i], o, 64);
      }
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane < LANES) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        lds[(wave * 2 * NV + i) * LANES + lane] = sw[i];
        lds[(wave * 2 * NV + NV + i) * LANES + lane] = sb[i];
      }
    }
    __syncthreads();
    if (wave > 0 || lane >= LANES) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int q = 1; q < 4; ++q) {
        sw[i] += lds[(q * 2 * NV + i) * LANES + lane];
        sb[i] += lds[(q * 2 * NV + NV + i) * LANES + lane];
      }
    }
  }
  void* const dw = gridDim.x == 1 ? a.dw : pw;
  void* const db = gridDim.x == 1 ? a.db : pw + a.cols;
  const int dt = gridDim.x == 1 ? a.wdt : DT_F32;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (at[k].own >= V) continue;
    if (COLS == TINY) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < (int)a.cols) {
          put<T, 1>(dw, dt, j, 0, sw + j);
          put<T, 1>(db, dt, j, 0, sb + j);
        }
    } else {
      put<T, V>(dw, dt, at[k].c, COLS == WHOLE ? 0 : at[k].own, sw + k * V);
      put<T, V>(db, dt, at[k].c, COLS == WHOLE ? 0 : at[k].own, sb + k * V);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(LN_LONG) k_ln_dx_long(LnBackward a) {
  using RT = RowThreads<0>;
  constexpr int V = Piece<T>::V;
  __shared__ float lds[RT::kLds];
  RT rt(lds);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.x_stride;
    const T* dy = (const T*)a.dy + row * a.dy_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s = 0.0f, u = 0.0f, w[V];
    Piece<T> p, q;
    for (uint32_t c = threadIdx.x * V; c < a.cols; c += LN_LONG * V) {
      const Place<T, RAGGED> at(c, a.cols);
      at.load(x, a.cols, false, p);
      at.load(dy, a.cols, false, q);
      at.weights(a.w, a.wdt, a.cols, 1.0f, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float h = at.mine(j, a.cols) ? to_f32(q.v[j]) * w[j] : 0.0f;
        s += h;
        u = __builtin_fmaf(h, (to_f32(p.v[j]) - mean) * rstd, u);
      }
    }
    rt.template sum<true>(s, u);
    s /= (float)a.cols;
    u /= (float)a.cols;
    for (uint32_t c = threadIdx.x * V; c < a.cols; c += LN_LONG * V) {
      const Place<T, RAGGED> at(c, a.cols);
      float o[V];
      at.load(x, a.cols, false, p);
      at.load(dy, a.cols, false, q);
      at.weights(a.w, a.wdt, a.cols, 1.0f, w);
#pragma unroll
      for (int j = 0; j < V; ++j)
        o[j] = rstd * ((to_f32(q.v[j]) * w[j] - s) - (to_f32(p.v[j]) - mean) * rstd * u);
      at.store((T*)a.dx + row * (int64_t)a.cols, a.cols, o);
    }
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

// The partial rows' sums. blockIdx.y: dw or db; 32 columns a workgroup at a time, 32 threads a
// column. Workgroups walk over the columns of the widest rows: a launch whose threads along an
// axis pass 32 bits is cut to the rest without an error.
constexpr uint32_t kReduceGroups = 1 << 16;
template <typename WT>
__global__ void __launch_bounds__(1024) k_ln_reduce(const float* __restrict__ partial, uint32_t n, uint32_t cols,
                                                    WT* __restrict__ dw, WT* __restrict__ db) {
  __shared__ float lds[32][33];
  const uint32_t tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  WT* out = blockIdx.y ? db : dw;
  if (!out) return;
  for (uint32_t first = blockIdx.x * 32; first < cols; first += kReduceGroups * 32) {
    const uint32_t c = first + tx;
    float s = 0.0f;
    if (c < cols) {
      const float* p = partial + (uint64_t)blockIdx.y * cols + c;
#pragma unroll 8
      for (uint32_t r = ty; r < n; r += 32) s += p[(uint64_t)r * 2 * cols];
    }
    lds[ty][tx] = s;
    __syncthreads();
    s = group_sum<32>(lds[tx][ty]);
    const uint32_t o = first + ty;
    if (tx == 0 && o < cols) out[o] = from_f32<WT>(s);
    __syncthreads();   // read before it is written again
  }
}

template <typename T>
struct Backward {
  const LnBackward& a;
  uint32_t n;
  bool once;
  hipStream_t s;
  template <int LANES, int NV>
  void run(uint32_t threads) const {
    constexpr uint32_t V = Piece<T>::V;
    if constexpr (LANES == 0 && sizeof(T) == 2) {
      if (ln_odd<T>(a.x, a.x_stride) || ln_odd<T>(a.dy, a.dy_stride)) {
        if (once) k_ln_backward<T, LANES, NV, ODD, true><<<n, threads, 0, s>>>(a);
        else k_ln_backward<T, LANES, NV, ODD, false><<<n, threads, 0, s>>>(a);
        return;
      }
    }
    if (LANES == 1 && a.cols < V) k_ln_backward<T, 1, 8, TINY, false><<<n, threads, 0, s>>>(a);
    else if (a.cols % V == 0 && once) k_ln_backward<T, LANES, NV, WHOLE, true><<<n, threads, 0, s>>>(a);
    else if (a.cols % V == 0) k_ln_backward<T, LANES, NV, WHOLE, false><<<n, threads, 0, s>>>(a);
    else if (once) k_ln_backward<T, LANES, NV, RAGGED, true><<<n, threads, 0, s>>>(a);
    else k_ln_backward<T, LANES, NV, RAGGED, false><<<n, threads, 0, s>>>(a);
  }
};
// Workgroups of the backward walk, each of which leaves one row of sums: as many as run at
// once, so that none waits for a place (8192 columns of bf16: 72 us with 256 workgroups of 16
// waves, 81 with 512), at most 768, and few enough that each has four turns: fewer rows of sums
// are sooner added up (4M values of bf16 in rows of 1024: 14 -> 11.4 us).
// One alone writes dw and db itself, which saves the second launch: up to eight turns of a wave
// with 8 values a thread (32 x 333 fp32: 8.0 -> 6.5 us a call, but 64 rows 7.9 -> 10.5), else
// four, of the longest rows two (2 x 16384 bf16 6.7, 8 rows in as many workgroups 9.6, four of
// them in one 10.1). Few long rows take fewer turns: a turn costs more than their sums do, up to
// 32 rows two turns more than one and up to 256 rows four more than two (16384 bf16, four turns,
// two and one: 16 rows 14.8, 11.5 and 10.3 us; 64 rows 15.4, 13.2 and 14.1; four and two: 192
// rows 19.4 and 17.6, 256 20.1 and 19.1, 384 20.1 and 22.0; 8192 bf16 11.7 and 11.4, 12.4 and
// 12.7, 13.9 and 14.4).
// Without dw and db there is nothing to add up, and every row that finds a place has its own
// (512 x 8192 bf16: 8.4 -> 6.6 us; 4 rows 6.6 -> 4.5).
struct BackwardGroups {
  int64_t rows;
  bool params;
  uint32_t& n;
  template <int LANES, int NV>
  void run(uint32_t threads) const {
    constexpr int kRows = RowThreads<LANES>::kRows;
    const uint32_t held = LN_CUS * (ln_backward_waves(LANES, NV) / (threads / 64)), most = held < 768 ? held : 768;
    if (!params) n = ln_walk(rows, kRows, most);
    else if (rows <= kRows * (LANES && NV == 8 ? 8 : LANES || NV == 8 ? 4 : 2)) n = rows > 0;
    else n = ln_walk(rows, kRows * (LANES || rows > 256 ? 4 : rows > 32 ? 2 : 1), most);
  }
};

uint32_t ln_groups(int64_t rows, uint32_t cols, bool params) {
  uint32_t n = 0;
  if (!ln_dispatch(cols, BackwardGroups{rows, params, n})) n = ln_walk(rows, 1, 512);
  return n;
}

template <typename T>
hipError_t backward(LnBackward a, hipStream_t s) {
  const bool once = ln_once(a.rows * a.cols * 3 * (int64_t)sizeof(T));
  const bool params = a.dw || a.db;
  const uint32_t n = ln_groups(a.rows, a.cols, params);
  bool alone = n == 1;   // that workgroup has written dw and db
  if (!params) a.partial = nullptr;
  if (a.rows && !ln_dispatch(a.cols, Backward<T>{a, n, once, s})) {
    alone = false;
    k_ln_dx_long<T><<<ln_walk(a.rows, 1, LN_LONG_GROUPS), LN_LONG, 0, s>>>(a);
    if (params) k_ln_columns<T><<<dim3((a.cols + 255) / 256, n), 256, 0, s>>>(a);
  }
  if (params && !alone) {
    const uint32_t groups = (a.cols + 31) / 32;
    const dim3 grid(groups < kReduceGroups ? groups : kReduceGroups, 2);
    if (a.wdt == DT_F32) k_ln_reduce<float><<<grid, 1024, 0, s>>>(a.partial, n, a.cols, (float*)a.dw, (float*)a.db);
    else k_ln_reduce<T><<<grid, 1024, 0, s>>>(a.partial, n, a.cols, (T*)a.dw, (T*)a.db);
  }
  return hipGetLastError();
}

}  // namespace

uint32_t ln_partial_rows(int64_t rows, uint32_t cols) { return ln_groups(rows, cols, true); }

hipError_t launch_ln_backward(const LnBackward& a, hipStream_t s) {
  if (a.dt == DT_F32) return backward<float>(a, s);
  if (a.dt == DT_F16) return backward<_Float16>(a, s);
  return backward<bf16_t>(a, s);
}

}  // namespace tg
