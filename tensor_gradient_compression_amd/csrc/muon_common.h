// Newton-Schulz orthogonalisation: what the kernels of k_muon.hip and k_muon_small.hip share.
#pragma once
#include "muon.h"

namespace tg {

__device__ __forceinline__ bool left_out(const NsCommon& c) {
  return c.clip && !(__builtin_fabsf(c.clip[0]) <= 3.40282347e38f);
}

// this workgroup's matrix (its offsets those of its own) and part
__device__ __forceinline__ uint32_t my_part(const NsCommon& c, const NsParts& p, uint32_t b, NsMat& m, uint32_t& i,
                                            uint32_t& j) {
  if (p.list) {
    const NsPart q = p.list[b];
    m = c.mats[q.mat];
    i = q.i;
    j = q.j;
    return q.mat;
  }
  const uint32_t each = p.lower ? p.ni * (p.ni + 1) / 2 : p.ni * p.nj, mat = b / each, t = b - mat * each;
  if (p.lower) {
    i = (uint32_t)((__builtin_sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    j = t - i * (i + 1) / 2;
  } else {
    tile_at(t, p.ni, p.nj, i, j);
  }
  m = c.one;
  const uint64_t o = mat * c.pitch;
  m.x += o;
  m.y += o;
  m.a += o;
  m.b += o;
  m.da += o;
  m.db += o;
  m.sums += o;
  return mat;
}

__device__ __forceinline__ float load_as(const void* p, uint32_t dt, uint64_t i) {
  return dt == DT_F32 ? ((const float*)p)[i] : dt == DT_F16 ? to_f32(((const _Float16*)p)[i]) : to_f32(((const bf16_t*)p)[i]);
}

// f with a zero of the type
template <class F>
__device__ __forceinline__ void with_type(uint32_t dt, const F& f) {
  if (dt == DT_F32) f(0.0f);
  else if (dt == DT_F16) f((_Float16)0.0f);
  else f(bf16_t{0});
}

// v as two fp16 parts
__device__ __forceinline__ void two_parts(float v, _Float16& hi, _Float16& lo) {
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

__device__ __forceinline__ void store_as(void* p, uint32_t dt, uint64_t i, float y) {
  if (dt == DT_F32) ((float*)p)[i] = y;
  else if (dt == DT_F16) ((_Float16*)p)[i] = from_f32<_Float16>(y);
  else ((bf16_t*)p)[i] = from_f32<bf16_t>(y);
}

__device__ __forceinline__ float updated(float g, float m, const MuonFirst& f) { return f.nesterov ? f.nu * g + f.mu * m : m; }

}  // namespace tg
