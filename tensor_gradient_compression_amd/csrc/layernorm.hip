// Host side of layer norm: argument checks and the launches of k_layernorm.hip.
#include <cmath>

#include "layernorm.h"
#include "tgrad.h"

using namespace tg;

namespace {

uintptr_t low_bits(int dtype) { return dtype == TGRAD_F32 ? 3 : 1; }

// sizes, types and strides that the kernels' indexes hold
bool shape_ok(int64_t rows, int64_t cols, int dtype, int weight_dtype) {
  if (rows < 0 || rows > 0x7FFFFFFF || cols < 1 || cols > 0x7FFFFFFF - 65536) return false;
  if (dtype < TGRAD_F32 || dtype > TGRAD_BF16) return false;
  return weight_dtype == dtype || weight_dtype == TGRAD_F32;
}
bool stride_ok(int64_t stride, int64_t rows, int64_t cols) {
  return rows <= 1 || (stride >= cols && stride <= (int64_t(1) << 40));
}
bool bad(const void* p, int dtype) { return ((uintptr_t)p & low_bits(dtype)) != 0; }

}  // namespace

extern "C" {

int tgrad_layer_norm_forward(const void* x, int64_t x_stride, const void* weight, const void* bias,
                             void* y, float* mean, float* rstd, int64_t rows, int64_t cols,
                             int dtype, int weight_dtype, double eps, void* stream) {
  if (!shape_ok(rows, cols, dtype, weight_dtype) || !stride_ok(x_stride, rows, cols))
    return TGRAD_EINVAL;
  if (!(eps >= 0.0 && std::isfinite(eps))) return TGRAD_EINVAL;
  if (bad(weight, weight_dtype) || bad(bias, weight_dtype)) return TGRAD_EINVAL;
  if (rows == 0) return TGRAD_OK;
  if (!x || !y || !mean || !rstd || bad(x, dtype) || bad(y, dtype) || bad(mean, TGRAD_F32) ||
      bad(rstd, TGRAD_F32))
    return TGRAD_EINVAL;
  LnForward a;
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.x_stride = x_stride;
  a.cols = (uint32_t)cols;
  a.dt = dtype;
  a.wdt = weight_dtype;
  a.eps = (float)eps;
  return launch_ln_forward(a, (hipStream_t)stream) == hipSuccess ? TGRAD_OK : TGRAD_EHIP;
}

int64_t tgrad_layer_norm_workspace(int64_t rows, int64_t cols) {
  if (!shape_ok(rows, cols, TGRAD_F32, TGRAD_F32)) return -1;
  return (int64_t)ln_partial_rows(rows, (uint32_t)cols) * 2 * cols * (int64_t)sizeof(float);
}

int tgrad_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                              const void* weight, const float* mean, const float* rstd, void* dx,
                              void* dweight, void* dbias, int64_t rows, int64_t cols, int dtype,
                              int weight_dtype, void* workspace, void* stream) {
  if (!shape_ok(rows, cols, dtype, weight_dtype) || !stride_ok(x_stride, rows, cols) ||
      !stride_ok(dy_stride, rows, cols))
    return TGRAD_EINVAL;
  if (bad(weight, weight_dtype) || bad(dweight, weight_dtype) || bad(dbias, weight_dtype))
    return TGRAD_EINVAL;
  if (rows > 0) {
    if (!dy || !x || !mean || !rstd || !dx || bad(dy, dtype) || bad(x, dtype) || bad(dx, dtype) ||
        bad(mean, TGRAD_F32) || bad(rstd, TGRAD_F32))
      return TGRAD_EINVAL;
    if ((dweight || dbias) && (!workspace || ((uintptr_t)workspace & 15u))) return TGRAD_EINVAL;
  }
  LnBackward a;
  a.dy = dy;
  a.x = x;
  a.w = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  a.dw = dweight;
  a.db = dbias;
  a.rows = rows;
  a.dy_stride = dy_stride;
  a.x_stride = x_stride;
  a.cols = (uint32_t)cols;
  a.dt = dtype;
  a.wdt = weight_dtype;
  a.partial = (float*)workspace;
  return launch_ln_backward(a, (hipStream_t)stream) == hipSuccess ? TGRAD_OK : TGRAD_EHIP;
}

}  // extern "C"
