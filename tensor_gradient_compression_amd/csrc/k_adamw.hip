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

// largest over the 16 lanes of a row, in all of them
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, (uint32_t)__shfl_xor((int)x, 8, 64));
  x = max(x, (uint32_t)__shfl_xor((int)x, 4, 64));
  x = max(x, (uint32_t)__shfl_xor((int)x, 2, 64));
  return max(x, (uint32_t)__shfl_xor((int)x, 1, 64));
}

__device__ __forceinline__ uint32_t nan_bits(uint32_t field) {
  return field == 255u ? 0x7FC00000u : 0u;
}

template <typename WT, typename GT>
__device__ void chunk32(WT* __restrict__ w, const GT* __restrict__ g, float* __restrict__ m,
                        float* __restrict__ v, uint32_t n, const StepK& k) {
  for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
    float mi = m[i], vi = v[i];
    const float q = moments(to_f32(g[i]), mi, vi, k);
    w[i] = from_f32<WT>(updated(to_f32(w[i]), mi, q, k));
    m[i] = mi;
    v[i] = vi;
  }
}

// 16 lanes hold a group, 8 values each
template <typename WT, typename GT>
__device__ void chunk8(WT* __restrict__ w, const GT* __restrict__ g, uint8_t* __restrict__ mc,
                       uint8_t* __restrict__ qc, uint8_t* __restrict__ ms, uint8_t* __restrict__ qs,
                       bf16_t* __restrict__ mo, bf16_t* __restrict__ qo, uint32_t n, uint32_t place,
                       uint32_t key, const StepK& k) {
  const uint32_t end = (n + ADAMW_GROUP - 1) / ADAMW_GROUP * ADAMW_GROUP;
  for (uint32_t i = threadIdx.x * 8; i < end; i += kThreads * 8) {
    const uint32_t grp = i / ADAMW_GROUP;
    const int fm = ms[grp], fq = qs[grp];
    float m[8], q[8];
    uint32_t tm = 0, tq = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t cm = mc[i + j], cq = qc[i + j];
      const bool in = i + j < n;
      m[j] = ldexpf(__uint_as_float(((cm & 127u) << 20) | ((cm & 128u) << 24) | nan_bits(fm)), fm - 14);
      const float qold = ldexpf(__uint_as_float((cq << 19) | nan_bits(fq)), fq - 14);
      float v = qold * qold;
      q[j] = moments(in ? to_f32(g[i + j]) : 0.0f, m[j], v, k);
      if (in) w[i + j] = from_f32<WT>(updated(to_f32(w[i + j]), m[j], q[j], k));
      tm = max(tm, __float_as_uint(m[j]) & 0x7FFFFFFFu);
      tq = max(tq, __float_as_uint(q[j]) & 0x7FFFFFFFu);
    }
    const int nm = (int)(row_max(tm) >> 23), nq = (int)(row_max(tq) >> 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = random_bits(place + i + j, key);
      const uint32_t ym = __float_as_uint(ldexpf(m[j], 14 - nm));
      const uint32_t yq = __float_as_uint(ldexpf(q[j], 14 - nq));
      const uint32_t cm = ((((ym & 0x7FFFFFFFu) + (h >> 12)) >> 20) & 127u) | ((ym >> 24) & 128u);
      const uint32_t cq = max(((yq + (h & 0x7FFFFu)) >> 19) & 255u, q[j] > 0.0f ? 1u : 0u);
      mc[i + j] = (uint8_t)cm;
      qc[i + j] = (uint8_t)cq;
      if (mo) {
        mo[i + j] = from_f32<bf16_t>(ldexpf(
            __uint_as_float(((cm & 127u) << 20) | ((cm & 128u) << 24) | nan_bits(nm)), nm - 14));
        qo[i + j] = from_f32<bf16_t>(ldexpf(__uint_as_float((cq << 19) | nan_bits(nq)), nq - 14));
      }
    }
    if ((threadIdx.x & 15) == 0) {
      ms[grp] = (uint8_t)nm;
      qs[grp] = (uint8_t)nq;
    }
  }
}

template <typename WT, typename GT>
__device__ void chunk(const AdamwArgs& a, const AdamwChunk& c, void* w, const void* g, uint32_t key,
                      const StepK& k) {
  WT* wp = (WT*)w + c.start;
  const GT* gp = (const GT*)g + c.start;
  if (a.bits == 32)
    chunk32(wp, gp, (float*)a.m + c.state, (float*)a.v + c.state, c.n, k);
  else
    chunk8(wp, gp, (uint8_t*)a.m + c.state, (uint8_t*)a.v + c.state, a.ms + c.state / ADAMW_GROUP,
           a.vs + c.state / ADAMW_GROUP, a.m_out ? (bf16_t*)a.m_out + c.state : nullptr,
           a.m_out ? (bf16_t*)a.v_out + c.state : nullptr, c.n, (uint32_t)c.state, key, k);
}

__global__ void __launch_bounds__(kThreads) k_adamw(AdamwArgs a, AdamwTable tab) {
  const AdamwChunk c = a.chunks[blockIdx.x];
  const AdamwClock now = a.clocks[blockIdx.x];
  StepK k;
  k.coef = 1.0f;
  if (a.clip) {
    // a norm that is not finite: some gradient is not, and the step is left out
    if (!(fabsf(a.clip[0]) < INFINITY)) return;
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
  const uint32_t key = step_key(a.seed, (uint64_t)now.t);
  if (c.wdt == DT_F32) chunk<float, float>(a, c, w, g, key, k);
  else if (c.wdt == DT_F16 && c.gdt == DT_F16) chunk<_Float16, _Float16>(a, c, w, g, key, k);
  else if (c.wdt == DT_F16) chunk<_Float16, float>(a, c, w, g, key, k);
  else if (c.gdt == DT_BF16) chunk<bf16_t, bf16_t>(a, c, w, g, key, k);
  else chunk<bf16_t, float>(a, c, w, g, key, k);
  __syncthreads();   // every wave has read its clock
  if (threadIdx.x == 0) {
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
  double s = 0.0;
  for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
    const double x = (double)to_f32(g[i]);
    s += x * x;
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
  k_adamw<<<a.nchunks, kThreads, 0, s>>>(a, tab);
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
