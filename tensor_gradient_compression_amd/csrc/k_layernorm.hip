// Layer norm over the last axis of (rows, cols).
//   mean = sum x / cols;  var = sum (x - mean)^2 / cols;  rstd = 1 / sqrt(var + eps)
//   n = (x - mean) rstd;  y = n w + b
// Statistics and sums are fp32, results are rounded once. The variance is the mean of the
// squared distances from the mean: the mean of squares less the squared mean would cancel
// for rows far from zero. Rows and threads: layernorm_rows.h.
#include "layernorm_rows.h"

namespace tg {

namespace {

template <typename T, int LANES, int NV, int COLS>
__global__ void __launch_bounds__(RowThreads<LANES>::kMost, ln_forward_waves(NV) / 4) k_ln_forward(LnForward a, bool once) {
  using RT = RowThreads<LANES>;
  constexpr int V = Piece<T>::V, K = NV / V;
  __shared__ float lds[RT::kLds];
  RT rt(lds);
  const int64_t stride = (int64_t)gridDim.x * RT::kRows;
  const float inv = 1.0f / (float)a.cols;
  Place<T, COLS> at[K];
  Raw<T, COLS> next[K];
  int64_t row = (int64_t)blockIdx.x * RT::kRows + RT::row();
  // pointers to the row whose values are used next, and to the one that is written next
  const T* xr = (const T*)a.x + row * a.x_stride;
  T* yr = (T*)a.y + row * (int64_t)a.cols;
  const int64_t x_step = stride * a.x_stride, y_step = stride * (int64_t)a.cols;
  bool moved = false;   // whether a thread of this wave holds a piece that was moved back
#pragma unroll
  for (int k = 0; k < K; ++k) {
    at[k] = Place<T, COLS>((RT::index() + k * RT::count()) * V, a.cols, RT::last_lane());
    moved = moved || (COLS != WHOLE && at[k].own > 0);
    clear(next[k]);
    if (row < a.rows) at[k].fetch(xr, a.cols, once, next[k]);
  }
  moved = COLS == TINY || __any(moved);
  float w[NV], b[NV];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    at[k].weights(a.w, a.wdt, a.cols, 1.0f, w + k * V);
    at[k].weights(a.b, a.wdt, a.cols, 0.0f, b + k * V);
  }
  // Every thread of a workgroup makes the same number of turns, for the barriers in the sums.
  for (int64_t base = (int64_t)blockIdx.x * RT::kRows; base < a.rows; base += stride, row += stride) {
    float x[NV], s = 0.0f, unused;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Piece<T> p = at[k].piece(xr, next[k]);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float v = to_f32(p.v[j]);
        x[k * V + j] = v;
        s += v;
      }
    }
    if (ln_moves(COLS) && moved) {
      s = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) s += at[k].mine(j, a.cols) ? x[k * V + j] : 0.0f;
    }
    xr += x_step;
    if (row + stride < a.rows)
#pragma unroll
      for (int k = 0; k < K; ++k) at[k].fetch(xr, a.cols, once, next[k]);
    rt.template sum<false>(s, unused);
    const float mean = mean_of(s, (float)a.cols, inv);
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float sk = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = x[k * V + j] - mean;
        x[k * V + j] = d;
        sk = __builtin_fmaf(d, d, sk);
      }
      s += at[k].own < V ? sk : 0.0f;
    }
    if (COLS != WHOLE && moved) {
      s = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = at[k].mine(j, a.cols) ? x[k * V + j] : 0.0f;
          s = __builtin_fmaf(d, d, s);
        }
    }
    rt.template sum<false>(s, unused);
    const float rstd = reciprocal_root(s * inv + a.eps);
    T* y = yr;
    yr += y_step;
    if (row >= a.rows) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = __builtin_fmaf(x[k * V + j] * rstd, w[k * V + j], b[k * V + j]);
      at[k].store(y, a.cols, o);
    }
    if (RT::index() == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(LN_LONG) k_ln_forward_long(LnForward a) {
  using RT = RowThreads<0>;
  constexpr int V = Piece<T>::V;
  __shared__ float lds[RT::kLds];
  RT rt(lds);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.x_stride;
    float s = 0.0f, unused;
    Piece<T> p;
    for (uint32_t c = threadIdx.x * V; c < a.cols; c += LN_LONG * V) {
      const Place<T, RAGGED> at(c, a.cols);
      at.load(x, a.cols, false, p);
#pragma unroll
      for (int j = 0; j < V; ++j) s += at.mine(j, a.cols) ? to_f32(p.v[j]) : 0.0f;
    }
    rt.template sum<false>(s, unused);
    const float mean = s / (float)a.cols;
    s = 0.0f;
    for (uint32_t c = threadIdx.x * V; c < a.cols; c += LN_LONG * V) {
      const Place<T, RAGGED> at(c, a.cols);
      at.load(x, a.cols, false, p);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = to_f32(p.v[j]) - mean;
        s = __builtin_fmaf(d, at.mine(j, a.cols) ? d : 0.0f, s);
      }
    }
    rt.template sum<false>(s, unused);
    const float rstd = 1.0f / sqrtf(s / (float)a.cols + a.eps);
    for (uint32_t c = threadIdx.x * V; c < a.cols; c += LN_LONG * V) {
      const Place<T, RAGGED> at(c, a.cols);
      float w[V], b[V], o[V];
      at.load(x, a.cols, false, p);
      at.weights(a.w, a.wdt, a.cols, 1.0f, w);
      at.weights(a.b, a.wdt, a.cols, 0.0f, b);
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = __builtin_fmaf((to_f32(p.v[j]) - mean) * rstd, w[j], b[j]);
      at.store((T*)a.y + row * (int64_t)a.cols, a.cols, o);
    }
    if (threadIdx.x == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
  }
}

template <typename T>
struct Forward {
  const LnForward& a;
  hipStream_t s;
  template <int LANES, int NV>
  void run(uint32_t threads) const {
    constexpr uint32_t V = Piece<T>::V;
    const uint32_t n = ln_walk(a.rows, RowThreads<LANES>::kRows, LN_CUS * (ln_forward_waves(NV) / (threads / 64)));
    const bool once = ln_once(a.rows * a.cols * 2 * (int64_t)sizeof(T));
    if constexpr (LANES == 0 && sizeof(T) == 2) {
      if (ln_odd<T>(a.x, a.x_stride)) {
        k_ln_forward<T, LANES, NV, ODD><<<n, threads, 0, s>>>(a, once);
        return;
      }
    }
    if (LANES == 1 && a.cols < V) k_ln_forward<T, 1, 8, TINY><<<n, threads, 0, s>>>(a, once);
    else if (a.cols % V == 0) k_ln_forward<T, LANES, NV, WHOLE><<<n, threads, 0, s>>>(a, once);
    else k_ln_forward<T, LANES, NV, RAGGED><<<n, threads, 0, s>>>(a, once);
  }
};

template <typename T>
hipError_t forward(const LnForward& a, hipStream_t s) {
  if (!ln_dispatch(a.cols, Forward<T>{a, s})) k_ln_forward_long<T><<<ln_walk(a.rows, 1, LN_LONG_GROUPS), LN_LONG, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ln_forward(const LnForward& a, hipStream_t s) {
  if (!a.rows) return hipSuccess;
  if (a.dt == DT_F32) return forward<float>(a, s);
  if (a.dt == DT_F16) return forward<_Float16>(a, s);
  return forward<bf16_t>(a, s);
}

}  // namespace tg
