// AdamW over many tensors in one launch (up to ADAMW_LAUNCH_TENSORS a launch), with fp32
// moments or with moments in 8 bits, and the norm of all their gradients.
//
// A step, each operation rounded to fp32:
//   g' = g * coefficient (of the norm; without one g' = g)
//   m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) (g' g');  q = sqrt(v)
//   w <- round(w * decay - (lr / (1 - b1^t) m) / (q / sqrt(1 - b2^t) + eps))
// with decay = fp32(1 - lr * weight_decay) formed in fp64.
//
// 8-bit state: groups of 128 values of a tensor share a scale for m and one for q = sqrt(v)
// (the root has half v's exponents, so 16 binades hold what 32 of v would). The scale byte is
// the exponent field f of the group's largest magnitude as fp32. A code is a small float: m a
// sign, 4 bits of exponent and 3 of mantissa; q 4 and 4 bits. Its value is the fp32 number
// with the bits code << 20 (q: << 19) times 2^(f - 14), gradual underflow included, so that
// encoding is a scaling by a power of two (exact), an integer addition of random low bits and
// a shift. The random bits make the rounding unbiased: with b2 = 0.999 a step changes v by
// less than half a code, and rounding to nearest would never move it. They are a hash of the
// seed, the step and the value's place, so a run can be repeated bit for bit. A q above zero
// keeps at least the least code: an element whose v vanished beside its group's largest would
// otherwise divide by eps alone. A group with a value that is not finite gets f = 255, which
// stands for NaN in all of it.
//
// Every workgroup keeps the step number and its powers for itself (AdamwClock) and writes
// those of the next step back at its end: nothing is passed from the host, so that a step
// captured in a graph counts on when it is replayed, and a step that the norm cancels leaves
// them alone, with no workgroup waiting for another.
#include "adamw.h"

namespace tg {

namespace {

constexpr int kThreads = 256;

struct StepK {
  float b1, c1, b2, c2, eps, step, is2, decay, coef;
};

__device__ __forceinline__ float moments(float g, float& m, float& v, const StepK& k) {
  const float gc = g * k.coef;
  m = k.b1 * m + k.c1 * gc;
  v = k.b2 * v + k.c2 * (gc * gc);
  return sqrtf(v);
}
__device__ __forceinline__ float updated(float w, float m, float q, const StepK& k) {
  return w * k.decay - (k.step * m) / (q * k.is2 + k.eps);
}

// SplitMix64's output for the state seed + t * 0x9E3779B97F4A7C15, its low half: the step's
// key. A value's 32 bits mix its place in the state with the key (two multiplications by the
// high halves of the same function's constants).
__device__ __forceinline__ uint32_t step_key(uint64_t seed, uint64_t t) {
  uint64_t z = seed + t * 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return (uint32_t)(z ^ (z >> 31));
}
__device__ __forceinline__ uint32_t random_bits(uint32_t place, uint32_t key) {
  uint32_t h = (place ^ key) * 0xBF58476Du;
  h ^= h >> 16;
  h *= 0x94D049BBu;
  return h ^ (h >> 13);
}

// largest over the 16 lanes of a row, in all of them (rotations within the row)
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x128, 0xF, 0xF, true));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x124, 0xF, 0xF, true));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x122, 0xF, 0xF, true));
  return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x121, 0xF, 0xF, true));
}

__device__ __forceinline__ uint32_t nan_bits(uint32_t field) {
  return field == 255u ? 0x7FC00000u : 0u;
}

// N values from p on, of which `have` exist (the others read as zero and are not written);
// ALIGNED: p is aligned to N values and N * sizeof(T) is 8, 16 or 32 bytes.
template <int N, bool ALIGNED, typename T>
__device__ __forceinline__ void load(const T* __restrict__ p, int have, float* x) {
  if (ALIGNED && have >= N) {
    T v[N];
    __builtin_memcpy(v, __builtin_assume_aligned(p, N * sizeof(T) < 16 ? N * sizeof(T) : 16), sizeof v);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = to_f32(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = j < have ? to_f32(p[j]) : 0.0f;
  }
}
template <int N, bool ALIGNED, typename T>
__device__ __forceinline__ void store(T* __restrict__ p, int have, const float* x) {
  if (ALIGNED && have >= N) {
    T v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = from_f32<T>(x[j]);
    __builtin_memcpy(__builtin_assume_aligned(p, N * sizeof(T) < 16 ? N * sizeof(T) : 16), v, sizeof v);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < have) p[j] = from_f32<T>(x[j]);
  }
}

// fp32 moments: four values a thread and two such pieces a pass, so that a wave's accesses to
// the moments are whole 1 KiB runs and both pieces' loads are in flight together.
template <typename WT, typename GT, bool ALIGNED>
__device__ __forceinline__ void chunk32(WT* __restrict__ w, const GT* __restrict__ g,
                                        float* __restrict__ m, float* __restrict__ v, uint32_t n,
                                        const StepK& k, bool skip) {
  for (uint32_t base = threadIdx.x * 4; base < n; base += kThreads * 8) {
    float wx[2][4], gx[2][4], mx[2][4], vx[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t i = base + u * kThreads * 4;
      if (i >= n) break;
      load<4, ALIGNED>(w + i, (int)(n - i), wx[u]);
      load<4, ALIGNED>(g + i, (int)(n - i), gx[u]);
      load<4, true>(m + i, 4, mx[u]);
      load<4, true>(v + i, 4, vx[u]);
    }
    if (skip) continue;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t i = base + u * kThreads * 4;
      if (i >= n) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float q = moments(gx[u][j], mx[u][j], vx[u][j], k);
        wx[u][j] = updated(wx[u][j], mx[u][j], q, k);
      }
      store<4, ALIGNED>(w + i, (int)(n - i), wx[u]);
      store<4, true>(m + i, 4, mx[u]);
      store<4, true>(v + i, 4, vx[u]);
    }
  }
}

// 8-bit moments: 16 lanes hold a group, 8 values each
template <typename WT, typename GT, bool ALIGNED, bool VALUES>
__device__ __forceinline__ void chunk8(WT* __restrict__ w, const GT* __restrict__ g,
                                       uint8_t* __restrict__ mc, uint8_t* __restrict__ qc,
                                       uint8_t* __restrict__ ms, uint8_t* __restrict__ qs,
                                       uint16_t* __restrict__ mo, uint16_t* __restrict__ qo,
                                       uint32_t n, uint32_t place, uint32_t key, const StepK& k,
                                       bool skip) {
  const uint32_t end = (n + ADAMW_GROUP - 1) / ADAMW_GROUP * ADAMW_GROUP;
  for (uint32_t i = threadIdx.x * 8; i < end; i += kThreads * 8) {
    const uint32_t grp = i / ADAMW_GROUP;
    const int have = (int)n - (int)i;
    float wx[8], gx[8], m[8], q[8];
    load<8, ALIGNED>(w + i, have, wx);
    load<8, ALIGNED>(g + i, have, gx);
    uint2 cm = *(const uint2*)(mc + i), cq = *(const uint2*)(qc + i);
    const int fm = ms[grp], fq = qs[grp];
    if (skip) continue;
    const uint32_t nan_m = nan_bits(fm), nan_q = nan_bits(fq);
    uint32_t tm = 0, tq = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = (j < 4 ? cm.x : cm.y) >> (8 * (j & 3)), b = (j < 4 ? cq.x : cq.y) >> (8 * (j & 3));
      m[j] = ldexpf(__uint_as_float(((a & 127u) << 20) | ((a & 128u) << 24) | nan_m), fm - 14);
      const float old = ldexpf(__uint_as_float(((b & 255u) << 19) | nan_q), fq - 14);
      float v = old * old;
      q[j] = moments(gx[j], m[j], v, k);
      wx[j] = updated(wx[j], m[j], q[j], k);
      tm = max(tm, __float_as_uint(m[j]) & 0x7FFFFFFFu);
      tq = max(tq, __float_as_uint(q[j]) & 0x7FFFFFFFu);
    }
    store<8, ALIGNED>(w + i, have, wx);
    const int nm = (int)(row_max(tm) >> 23), nq = (int)(row_max(tq) >> 23);
    uint32_t ym[8], yq[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = random_bits(place + i + j, key);
      // the sign stays in bit 31: a code's magnitude ends below bit 27, and so does the sum
      ym[j] = __float_as_uint(ldexpf(m[j], 14 - nm)) + (h >> 12);
      yq[j] = __float_as_uint(ldexpf(q[j], 14 - nq)) + (h & 0x7FFFFu);
      // a q above zero is above 2^-75, so its bits are more than the least code's
      yq[j] = max(yq[j], min(__float_as_uint(q[j]), 1u << 19));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = ((ym[j] >> 20) & 127u) | ((ym[j] >> 24) & 128u), b = (yq[j] >> 19) & 255u;
      uint32_t &x = j < 4 ? cm.x : cm.y, &y = j < 4 ? cq.x : cq.y;
      x = (j & 3) ? x | a << (8 * (j & 3)) : a;
      y = (j & 3) ? y | b << (8 * (j & 3)) : b;
    }
    *(uint2*)(mc + i) = cm;
    *(uint2*)(qc + i) = cq;
    if ((threadIdx.x & 15) == 0) {
      ms[grp] = (uint8_t)nm;
      qs[grp] = (uint8_t)nq;
    }
    if (VALUES) {
      // at most five significant bits: the upper half of the fp32 value is the bf16 one
      uint32_t om[8], oq[8];
      const uint32_t new_nan_m = nan_bits(nm), new_nan_q = nan_bits(nq);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        om[j] = __float_as_uint(ldexpf(__uint_as_float((ym[j] & 0x87F00000u) | new_nan_m), nm - 14));
        oq[j] = __float_as_uint(ldexpf(__uint_as_float((yq[j] & 0x07F80000u) | new_nan_q), nq - 14));
      }
      uint4 a, b;
      a.x = __builtin_amdgcn_perm(om[1], om[0], 0x07060302u);
      a.y = __builtin_amdgcn_perm(om[3], om[2], 0x07060302u);
      a.z = __builtin_amdgcn_perm(om[5], om[4], 0x07060302u);
      a.w = __builtin_amdgcn_perm(om[7], om[6], 0x07060302u);
      b.x = __builtin_amdgcn_perm(oq[1], oq[0], 0x07060302u);
      b.y = __builtin_amdgcn_perm(oq[3], oq[2], 0x07060302u);
      b.z = __builtin_amdgcn_perm(oq[5], oq[4], 0x07060302u);
      b.w = __builtin_amdgcn_perm(oq[7], oq[6], 0x07060302u);
      *(uint4*)(mo + i) = a;
      *(uint4*)(qo + i) = b;
    }
  }
}

template <int BITS, bool VALUES, typename WT, typename GT, bool ALIGNED>
__device__ __forceinline__ void chunk_as(const AdamwArgs& a, const AdamwChunk& c, WT* w, const GT* g,
                                         uint32_t key, const StepK& k, bool skip) {
  if (BITS == 32)
    chunk32<WT, GT, ALIGNED>(w, g, (float*)a.m + c.state, (float*)a.v + c.state, c.n, k, skip);
  else
    chunk8<WT, GT, ALIGNED, VALUES>(w, g, (uint8_t*)a.m + c.state, (uint8_t*)a.v + c.state,
                                    a.ms + c.state / ADAMW_GROUP, a.vs + c.state / ADAMW_GROUP,
                                    a.m_out + c.state, a.v_out + c.state, c.n, (uint32_t)c.state, key, k,
                                    skip);
}

// Wide accesses where both addresses allow them: chunks start at multiples of 128 values, so
// the tensors' own addresses decide.
template <int BITS, bool VALUES, typename WT, typename GT>
__device__ __forceinline__ void chunk(const AdamwArgs& a, const AdamwChunk& c, void* w, const void* g,
                                      uint32_t key, const StepK& k, bool skip) {
  if ((((uintptr_t)w | (uintptr_t)g) & 15u) == 0)
    chunk_as<BITS, VALUES, WT, GT, true>(a, c, (WT*)w + c.start, (const GT*)g + c.start, key, k, skip);
  else
    chunk_as<BITS, VALUES, WT, GT, false>(a, c, (WT*)w + c.start, (const GT*)g + c.start, key, k, skip);
}

template <int BITS, bool VALUES>
__global__ void __launch_bounds__(kThreads) k_adamw(AdamwArgs a, AdamwTable tab) {
  const AdamwChunk c = a.chunks[blockIdx.x];
  const AdamwClock now = a.clocks[blockIdx.x];
  StepK k;
  k.coef = 1.0f;
  // a norm that is not finite: some gradient is not, and the step is left out. The chunks'
  // loads do not wait for that.
  bool skip = false;
  if (a.clip) {
    skip = !(fabsf(a.clip[0]) < INFINITY);
    k.coef = a.clip[1];
  }
  k.b1 = a.b1;
  k.c1 = a.c1;
  k.b2 = a.b2;
  k.c2 = a.c2;
  k.eps = a.eps;
  k.step = (float)a.lr * now.ic1;
  k.is2 = now.is2;
  k.decay = (float)(1.0 - a.lr * c.wd);
  void* w = tab.w[c.tensor - a.first_tensor];
  const void* g = tab.g[c.tensor - a.first_tensor];
  const uint32_t key = BITS == 8 ? step_key(a.seed, (uint64_t)now.t) : 0;
  if (c.wdt == DT_F32) chunk<BITS, VALUES, float, float>(a, c, w, g, key, k, skip);
  else if (c.wdt == DT_F16 && c.gdt == DT_F16) chunk<BITS, VALUES, _Float16, _Float16>(a, c, w, g, key, k, skip);
  else if (c.wdt == DT_F16) chunk<BITS, VALUES, _Float16, float>(a, c, w, g, key, k, skip);
  else if (c.gdt == DT_BF16) chunk<BITS, VALUES, bf16_t, bf16_t>(a, c, w, g, key, k, skip);
  else chunk<BITS, VALUES, bf16_t, float>(a, c, w, g, key, k, skip);
  __syncthreads();   // every wave has read its clock
  if (threadIdx.x == 0 && !skip) {
    AdamwClock next;
    next.t = now.t + 1;
    next.p1 = now.p1 * a.b1d;
    next.p2 = now.p2 * a.b2d;
    next.ic1 = (float)(1.0 / (1.0 - next.p1));
    next.is2 = (float)(1.0 / sqrt(1.0 - next.p2));
    a.clocks[blockIdx.x] = next;
  }
}

template <typename GT>
__device__ double squares(const GT* __restrict__ g, uint32_t n) {
  constexpr int N = 16 / sizeof(GT);
  double s = 0.0;
  if (((uintptr_t)g & 15u) != 0) {
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
      const double x = (double)to_f32(g[i]);
      s += x * x;
    }
    return s;
  }
  for (uint32_t base = threadIdx.x * N; base < n; base += kThreads * N * 4) {
    float x[4][N];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t i = base + u * kThreads * N;
      load<N, true>(g + i, (int)n - (int)i, x[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < N; ++j) s = fma((double)x[u][j], (double)x[u][j], s);
  }
  return s;
}

__device__ __forceinline__ double block_sum(double s, double* lds) {
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__global__ void __launch_bounds__(kThreads) k_adamw_squares(const AdamwChunk* __restrict__ chunks,
                                                            uint32_t first, AdamwTable tab,
                                                            double* __restrict__ partial) {
  __shared__ double lds[4];
  const AdamwChunk c = chunks[blockIdx.x];
  const void* g = tab.g[c.tensor - first];
  double s;
  if (c.gdt == DT_F32) s = squares((const float*)g + c.start, c.n);
  else if (c.gdt == DT_F16) s = squares((const _Float16*)g + c.start, c.n);
  else s = squares((const bf16_t*)g + c.start, c.n);
  s = block_sum(s, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) k_adamw_norm(const double* __restrict__ partial, uint32_t n,
                                                         double max_norm, double scale,
                                                         float* __restrict__ out) {
  __shared__ double lds[4];
  double s = 0.0;
  for (uint32_t i = threadIdx.x; i < n; i += kThreads) s += partial[i];
  s = block_sum(s, lds);
  if (threadIdx.x == 0) {
    const double norm = sqrt(s) * scale;
    out[0] = (float)norm;
    out[1] = (float)(norm > max_norm ? scale * (max_norm / norm) : scale);
  }
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, const AdamwTable& tab, hipStream_t s) {
  if (a.bits == 32) k_adamw<32, false><<<a.nchunks, kThreads, 0, s>>>(a, tab);
  else if (!a.m_out) k_adamw<8, false><<<a.nchunks, kThreads, 0, s>>>(a, tab);
  else k_adamw<8, true><<<a.nchunks, kThreads, 0, s>>>(a, tab);
  return hipGetLastError();
}

hipError_t launch_adamw_squares(const AdamwChunk* chunks, uint32_t first_tensor, uint32_t nchunks,
                                const AdamwTable& tab, double* partial, hipStream_t s) {
  k_adamw_squares<<<nchunks, kThreads, 0, s>>>(chunks, first_tensor, tab, partial);
  return hipGetLastError();
}

hipError_t launch_adamw_norm(const double* partial, uint32_t n, double max_norm, double scale,
                             float* out, hipStream_t s) {
  k_adamw_norm<<<1, kThreads, 0, s>>>(partial, n, max_norm, scale, out);
  return hipGetLastError();
}

}  // namespace tg
