// Layer norm: what the host side (layernorm.hip) and the kernels (k_layernorm.hip) share.
#pragma once
#include "tg_common.h"

namespace tg {

struct LnForward {
  const void* x;
  const void* w;   // may be NULL: 1
  const void* b;   // may be NULL: 0
  void* y;
  float* mean;
  float* rstd;
  int64_t rows, x_stride;
  uint32_t cols;
  int dt, wdt;
  float eps;
};
hipError_t launch_ln_forward(const LnForward& a, hipStream_t s);

struct LnBackward {
  const void* dy;
  const void* x;
  const void* w;      // may be NULL: 1
  const float* mean;
  const float* rstd;
  void* dx;
  void* dw;           // may be NULL
  void* db;           // may be NULL
  int64_t rows, dy_stride, x_stride;
  uint32_t cols;
  int dt, wdt;
  float* partial;     // ln_partial_rows() x 2 x cols: sums over rows of dy xhat, and of dy
};
uint32_t ln_partial_rows(int64_t rows, uint32_t cols);
hipError_t launch_ln_backward(const LnBackward& a, hipStream_t s);

}  // namespace tg
