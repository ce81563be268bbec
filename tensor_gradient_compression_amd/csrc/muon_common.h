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

// f with a zero of the type
template <class F>
__device__ __forceinline__ void with_type(uint32_t dt, const F& f) {
  if (dt == DT_F32) f(0.0f);
  else if (dt == DT_F16) f((_Float16)0.0f);
  else f(bf16_t{0});
}

// N values at p, which is aligned to one of them (16 bytes at a time all the same)
template <int N, typename T>
__device__ __forceinline__ void load_values(const T* p, T* v) { __builtin_memcpy(v, p, N * sizeof(T)); }
template <int N, typename T>
__device__ __forceinline__ void store_values(T* p, const T* v) { __builtin_memcpy(p, v, N * sizeof(T)); }

// 2^12 / (|U| + eps) from the sum of U's squares, in two factors: a norm below 1.2e-35 has a reciprocal
// that fp32 does not hold, so such values are lifted by a power of two before.
struct NsScale {
  float lift, rest;
  __device__ __forceinline__ NsScale(double squares, double eps) {
    const double s = (double)NS_X / (__builtin_sqrt(squares) + eps);
    lift = 1.0f;
    rest = (float)s;
    if (__builtin_expect(rest > 0x1p126f, 0)) {
      lift = 0x1p100f;
      rest = (float)(s * 0x1p-100);
    }
  }
  __device__ __forceinline__ float operator()(float v) const { return v * lift * rest; }
};

// v as two fp16 parts. (Without the empty statement the compiler rounds a product that v is twice,
// once from its exact value and once from its fp32 one, and where these differ the lower part
// belongs to another upper part than the one that is stored.)
__device__ __forceinline__ void two_parts(float v, _Float16& hi, _Float16& lo) {
  __asm__("" : "+v"(v));
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

__device__ __forceinline__ float updated(float g, float m, const MuonFirst& f) { return f.nesterov ? f.nu * g + f.mu * m : m; }

}  // namespace tg
