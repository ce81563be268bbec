// Layer norm over the last axis of (rows, cols), and its gradients.
//   mean = sum x / cols;  var = sum (x - mean)^2 / cols;  rstd = 1 / sqrt(var + eps)
//   n = (x - mean) rstd;  y = n w + b
//   h = dy w;  dx = rstd (h - mean(h) - n mean(h n));  dw = sum_rows dy n;  db = sum_rows dy
// Statistics and sums are fp32, results are rounded once. The variance is the mean of the
// squared distances from the mean: the mean of squares less the squared mean would cancel
// for rows far from zero.
#include "layernorm.h"

namespace tg {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float s, float* lds) {
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

template <typename T, typename WT>
__global__ void __launch_bounds__(kThreads) k_ln_forward(LnForward a) {
  __shared__ float lds[4];
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.x_stride;
  T* y = (T*)a.y + row * (int64_t)a.cols;
  const WT *w = (const WT*)a.w, *b = (const WT*)a.b;
  float s = 0.0f;
  for (uint32_t i = threadIdx.x; i < a.cols; i += kThreads) s += to_f32(x[i]);
  const float mean = block_sum(s, lds) / (float)a.cols;
  s = 0.0f;
  for (uint32_t i = threadIdx.x; i < a.cols; i += kThreads) {
    const float d = to_f32(x[i]) - mean;
    s += d * d;
  }
  const float rstd = 1.0f / sqrtf(block_sum(s, lds) / (float)a.cols + a.eps);
  for (uint32_t i = threadIdx.x; i < a.cols; i += kThreads) {
    float n = (to_f32(x[i]) - mean) * rstd;
    if (w) n *= to_f32(w[i]);
    if (b) n += to_f32(b[i]);
    y[i] = from_f32<T>(n);
  }
  if (threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
}

template <typename T, typename WT>
__global__ void __launch_bounds__(kThreads) k_ln_dx(LnBackward a) {
  __shared__ float lds[4];
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.x_stride;
  const T* dy = (const T*)a.dy + row * a.dy_stride;
  T* dx = (T*)a.dx + row * (int64_t)a.cols;
  const WT* w = (const WT*)a.w;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s = 0.0f, t = 0.0f;
  for (uint32_t i = threadIdx.x; i < a.cols; i += kThreads) {
    const float h = to_f32(dy[i]) * (w ? to_f32(w[i]) : 1.0f);
    s += h;
    t += h * ((to_f32(x[i]) - mean) * rstd);
  }
  s = block_sum(s, lds) / (float)a.cols;
  t = block_sum(t, lds) / (float)a.cols;
  for (uint32_t i = threadIdx.x; i < a.cols; i += kThreads) {
    const float h = to_f32(dy[i]) * (w ? to_f32(w[i]) : 1.0f);
    const float n = (to_f32(x[i]) - mean) * rstd;
    dx[i] = from_f32<T>(rstd * (h - s - n * t));
  }
}

// partial row r: the sums over rows r, r + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(kThreads) k_ln_columns(LnBackward a) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.cols) return;
  float s = 0.0f, t = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float dy = to_f32(((const T*)a.dy)[row * a.dy_stride + i]);
    s += dy * ((to_f32(((const T*)a.x)[row * a.x_stride + i]) - a.mean[row]) * a.rstd[row]);
    t += dy;
  }
  a.partial[(uint64_t)blockIdx.y * 2 * a.cols + i] = s;
  a.partial[((uint64_t)blockIdx.y * 2 + 1) * a.cols + i] = t;
}

template <typename WT>
__global__ void __launch_bounds__(kThreads) k_ln_reduce(const float* __restrict__ partial, uint32_t n,
                                                        uint32_t cols, WT* __restrict__ dw,
                                                        WT* __restrict__ db) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= cols) return;
  float s = 0.0f, t = 0.0f;
  for (uint32_t r = 0; r < n; ++r) {
    s += partial[(uint64_t)r * 2 * cols + i];
    t += partial[((uint64_t)r * 2 + 1) * cols + i];
  }
  if (dw) dw[i] = from_f32<WT>(s);
  if (db) db[i] = from_f32<WT>(t);
}

template <typename T, typename WT>
hipError_t forward(const LnForward& a, hipStream_t s) {
  k_ln_forward<T, WT><<<(uint32_t)a.rows, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, typename WT>
hipError_t backward(const LnBackward& a, hipStream_t s) {
  const uint32_t n = ln_partial_rows(a.rows, a.cols), blocks = (a.cols + kThreads - 1) / kThreads;
  if (a.rows) k_ln_dx<T, WT><<<(uint32_t)a.rows, kThreads, 0, s>>>(a);
  if (a.dw || a.db) {
    if (a.rows) k_ln_columns<T><<<dim3(blocks, n), kThreads, 0, s>>>(a);
    k_ln_reduce<WT><<<blocks, kThreads, 0, s>>>(a.partial, n, a.cols, (WT*)a.dw, (WT*)a.db);
  }
  return hipGetLastError();
}

}  // namespace

uint32_t ln_partial_rows(int64_t rows, uint32_t) { return (uint32_t)(rows < 256 ? rows : 256); }

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
