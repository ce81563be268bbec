// AdamW over many tensors in one launch (up to ADAMW_LAUNCH_TENSORS a launch), with fp32
// moments or with moments in 8 bits, and the norm of all their gradients.
//
// A step, each operation rounded to fp32:
//   g' = g * coefficient (of the norm; without one g' = g)
//   m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) (g' g');  q = sqrt(v)
//   w <- round(w * decay - (lr / (1 - b1^t) m) / (q / sqrt(1 - b2^t) + eps))
// with decay = fp32(1 - lr * weight_decay) formed in fp64, and the division as a product with
// the hardware's reciprocal (within one unit of the last place: the weights' own rounding or a
// step of lr hides it, and the stored state does not depend on it).
//
// What bounds it. A step moves 2 weights, a gradient and 16 bytes of state a value (fp32
// moments) or 4.06 (8 bits, 4 more where the values are asked back) and is bound by memory:
// bf16 weights, fp32 moments, 236M values 842 us (6.2 TB/s; a large copy with the same mix of
// reads and writes reaches 5.9), 150 tensors of 18.7M values 63 us (5.9 TB/s); 8 bits, fp16,
// 67M values with values back 167 us (5.6 TB/s), 30M bf16 values without 51 us (6.0 TB/s). The
// 8-bit step was bound by its instructions at first (92 issue slots a value): the pairwise
// conversion of m's codes, one multiplication of the hash shared by 8 values, the short root
// and bytes packed by permutes brought them to about 70. Small models are bound by latency and
// by the host's launches: 12 tensors 3.6 us of a kernel's time.
// One workgroup steps 2048 values in a straight line, all its loads in flight at once: with
// 32768 values a workgroup (fewer, longer walks) the same tensors took 1040 and 85 us, since the
// open pieces of a walk are spread over all of memory.
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
static_assert(kThreads * 8 == ADAMW_CHUNK, "a workgroup steps its chunk in one pass");

struct StepK {
  float b1, c1, b2, c2, eps, step, is2, decay, coef;
};

__device__ __forceinline__ void moments(float g, float& m, float& v, const StepK& k) {
  const float gc = g * k.coef;
  m = k.b1 * m + k.c1 * gc;
  v = k.b2 * v + k.c2 * (gc * gc);
}
__device__ __forceinline__ float updated(float w, float m, float q, const StepK& k) {
  return w * k.decay - (k.step * m) * __builtin_amdgcn_rcpf(q * k.is2 + k.eps);
}

// A value's 32 random bits: its place in the state mixed with the step's key (two
// multiplications by the high halves of SplitMix64's constants).
// `head` is (place ^ key) * 0xBF58476D.
__device__ __forceinline__ uint32_t random_bits(uint32_t head) {
  uint32_t h = head ^ (head >> 16);
  h *= 0x94D049BBu;
  return h ^ (h >> 13);
}

// sqrt(v), correctly rounded for 2^-96 <= v <= 2^126 and for 0: v times its reciprocal root
// and one correction by the exact residual. Compared with sqrtf for every mantissa of both
// exponent parities at both ends of that range and between; sqrtf's own care for the rest
// costs twice the instructions. kRootLow and kRootHigh bound the results of that range.
__device__ __forceinline__ float root(float v) {
  const float y = __builtin_amdgcn_rsqf(fmaxf(v, 0x1p-96f));
  const float s = v * y, h = 0.5f * y;
  return __builtin_fmaf(__builtin_fmaf(-s, s, v), h, s);
}
constexpr uint32_t kRootLow = (127 - 48) << 23, kRootHigh = (127 + 63) << 23;

// Whole accesses of 8 or 16 bytes, marked as not to be kept: a step touches every byte once,
// and what the caches keep of it is gone before the next one. At the element's alignment, which
// the hardware takes for global memory: tensors may be views that start anywhere.
template <typename T, int N>
struct Wide {
  static constexpr int kBytes = N * sizeof(T) < 16 ? N * sizeof(T) : 16;
  typedef uint32_t V __attribute__((ext_vector_type(kBytes / 4)));
  typedef V At __attribute__((aligned(2)));
  static constexpr int kPieces = N * sizeof(T) / kBytes;
};
template <typename T, int N>
__device__ __forceinline__ void load_wide(const T* __restrict__ p, T (&v)[N]) {
  using W = Wide<T, N>;
  typename W::V t[W::kPieces];
#pragma unroll
  for (int i = 0; i < W::kPieces; ++i) t[i] = __builtin_nontemporal_load((const typename W::At*)p + i);
  __builtin_memcpy(v, t, sizeof v);
}
template <typename T, int N>
__device__ __forceinline__ void store_wide(T* __restrict__ p, const T (&v)[N]) {
  using W = Wide<T, N>;
  typename W::V t[W::kPieces];
  __builtin_memcpy(t, v, sizeof v);
#pragma unroll
  for (int i = 0; i < W::kPieces; ++i) __builtin_nontemporal_store(t[i], (typename W::At*)p + i);
}

// The largest over the 16 lanes of a row, in all of them (rotations within the row)
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x128, 0xF, 0xF, true));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x124, 0xF, 0xF, true));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x122, 0xF, 0xF, true));
  return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x121, 0xF, 0xF, true));
}

__device__ __forceinline__ uint32_t nan_bits(uint32_t field) {
  return field == 255u ? 0x7FC00000u : 0u;
}

// The upper bytes of four words, the first lowest.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0703u), hi = __builtin_amdgcn_perm(d, c, 0x0C0C0703u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}
// The upper halves of two words.
__device__ __forceinline__ uint32_t top_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// The weights and gradients of a chunk. They are converted apart from their loads, so that
// every load of the chunk is in flight before the first is waited for. In a chunk that ends
// early (WHOLE false) one lane's piece may end inside: it is read and written value by value.
template <typename WT, typename GT, bool WHOLE>
struct Chunk {
  static constexpr bool kWhole = WHOLE;
  WT* w;
  const GT* g;
  uint32_t n;
  template <int N>
  struct Raw {
    WT w[N];
    GT g[N];
  };
  template <int N>
  __device__ __forceinline__ void load(uint32_t i, Raw<N>& r) const {
    if (WHOLE || i + N <= n) {
      load_wide(w + i, r.w);
      load_wide(g + i, r.g);
      return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const bool in = i + j < n;
      r.w[j] = in ? w[i + j] : zero_of<WT>();
      r.g[j] = in ? g[i + j] : zero_of<GT>();
    }
  }
  template <int N>
  __device__ __forceinline__ void values(const Raw<N>& r, float* wx, float* gx) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      wx[j] = to_f32(r.w[j]);
      gx[j] = to_f32(r.g[j]);
    }
  }
  template <int N>
  __device__ __forceinline__ void store(uint32_t i, const float* wx) const {
    WT v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = from_f32<WT>(wx[j]);
    if (WHOLE || i + N <= n) {
      store_wide(w + i, v);
      return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (i + j < n) w[i + j] = v[j];
  }
};

// fp32 moments: two pieces of four values a thread, so that a wave's accesses to the moments
// are whole 1 KiB runs and all loads of both pieces are in flight together.
template <typename IO>
__device__ __forceinline__ void chunk32(const AdamwArgs& a, const AdamwChunk& c, const IO& io,
                                        const StepK& k, bool skip) {
  float* m = (float*)a.m + c.state;
  float* v = (float*)a.v + c.state;
  typename IO::template Raw<4> raw[2];
  float mx[2][4], vx[2][4];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t i = (u * kThreads + threadIdx.x) * 4;
    if (!IO::kWhole && i >= c.n) break;
    load_wide(m + i, mx[u]);
    load_wide(v + i, vx[u]);
    io.load(i, raw[u]);
  }
  if (skip) return;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t i = (u * kThreads + threadIdx.x) * 4;
    if (!IO::kWhole && i >= c.n) break;
    float wx[4], gx[4];
    io.values(raw[u], wx, gx);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      moments(gx[j], mx[u][j], vx[u][j], k);
      wx[j] = updated(wx[j], mx[u][j], sqrtf(vx[u][j]), k);
    }
    io.template store<4>(i, wx);
    store_wide(m + i, mx[u]);
    store_wide(v + i, vx[u]);
  }
}

// 8-bit moments: 16 lanes hold a group, 8 values each
template <bool VALUES, typename IO>
__device__ __forceinline__ void chunk8(const AdamwArgs& a, const AdamwChunk& c, const IO& io,
                                       uint32_t key, const StepK& k, bool skip) {
  const uint32_t i = threadIdx.x * 8;
  if (!IO::kWhole && i >= (c.n + ADAMW_GROUP - 1) / ADAMW_GROUP * ADAMW_GROUP) return;
  const uint64_t at = c.state + i;
  uint2* mc = (uint2*)((uint8_t*)a.m + at);
  uint2* qc = (uint2*)((uint8_t*)a.v + at);
  uint8_t *ms = a.ms + at / ADAMW_GROUP, *qs = a.vs + at / ADAMW_GROUP;
  const uint2 cm = *mc, cq = *qc;
  const int fm = *ms, fq = *qs;
  typename IO::template Raw<8> raw;
  io.load(i, raw);
  if (skip) return;
  float wx[8], gx[8], m[8], q[8];
  io.values(raw, wx, gx);
  // m's codes are the fp8 numbers (4 bits of exponent, 3 of mantissa) that the hardware
  // converts in pairs: those stand for 2^120 times the number with the bits code << 20. A
  // group that stands for NaN makes its products with b1 and b2 that.
  typedef float Pair __attribute__((ext_vector_type(2)));
  const float sm = ldexpf(1.0f, fm - 134);
  StepK kg = k;
  if (fm == 255) kg.b1 = kg.b2 = __uint_as_float(0x7FC00000u);
  if (fq == 255) kg.b2 = __uint_as_float(0x7FC00000u);
  const Pair p0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)cm.x, false), p1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)cm.x, true);
  const Pair p2 = __builtin_amdgcn_cvt_pk_f32_fp8((int)cm.y, false), p3 = __builtin_amdgcn_cvt_pk_f32_fp8((int)cm.y, true);
  m[0] = p0.x, m[1] = p0.y, m[2] = p1.x, m[3] = p1.y, m[4] = p2.x, m[5] = p2.y, m[6] = p3.x, m[7] = p3.y;
  float v[8], tm = 0.0f;
  uint32_t tq = 0, lq = 0xFFFFFFFFu;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t y = ((j < 4 ? cq.x : cq.y) >> (8 * (j & 3))) & 255u;
    const float old = ldexpf(__uint_as_float(y << 19), fq - 14);
    m[j] *= sm;
    v[j] = old * old;
    moments(gx[j], m[j], v[j], kg);
    q[j] = root(v[j]);
    tm = fmaxf(tm, fabsf(m[j]));
    tq = max(tq, __float_as_uint(q[j]) & 0x7FFFFFFFu);
    lq = min(lq, __float_as_uint(q[j]));
  }
  if (__any(tq >= kRootHigh || lq < kRootLow)) {   // zeros among them
    tq = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      __asm__ volatile("" : "+v"(v[j]));   // a branch of its own, not computed beside the other
      q[j] = sqrtf(v[j]);
      tq = max(tq, __float_as_uint(q[j]) & 0x7FFFFFFFu);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) wx[j] = updated(wx[j], m[j], q[j], k);
  io.template store<8>(i, wx);
  // where m is not finite v is not either: both groups then stand for NaN
  const int nq = (int)(row_max(tq) >> 23);
  const int nm = nq == 255 ? 255 : (int)(row_max(__float_as_uint(tm)) >> 23);
  const uint32_t ks = (uint32_t)__builtin_amdgcn_readfirstlane((int)key), low = ks & 7u;
  const uint32_t head = ((uint32_t)at ^ (ks & ~7u)) * 0xBF58476Du;
  uint32_t ym[8], yq[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // (at + j) ^ key: at is a multiple of 8, so its product and that of the low bits add up
    const uint32_t h = random_bits(head + (j ^ low) * 0xBF58476Du);
    // the sign stays in bit 31: a code's magnitude ends below bit 27, and so does the sum
    ym[j] = __float_as_uint(ldexpf(m[j], 14 - nm)) + (h >> 12);
    yq[j] = __float_as_uint(ldexpf(q[j], 14 - nq)) + (h & 0x7FFFFu);
    // a q above zero is above 2^-75, so its bits are more than the least code's
    yq[j] = max(yq[j], min(__float_as_uint(q[j]), 1u << 19));
  }
  uint32_t bm[8], bq[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    bm[j] = (ym[j] & 0x80000000u) | ((ym[j] << 4) & 0x7F000000u);
    bq[j] = yq[j] << 5;
  }
  *mc = make_uint2(top_bytes(bm[0], bm[1], bm[2], bm[3]), top_bytes(bm[4], bm[5], bm[6], bm[7]));
  *qc = make_uint2(top_bytes(bq[0], bq[1], bq[2], bq[3]), top_bytes(bq[4], bq[5], bq[6], bq[7]));
  if ((threadIdx.x & 15) == 0) {
    *ms = (uint8_t)nm;
    *qs = (uint8_t)nq;
  }
  if (VALUES) {
    // at most five significant bits: the upper half of the fp32 value is the bf16 one
    uint32_t om[8], oq[8];
    const uint32_t nan_m = nan_bits(nm), nan_q = nan_bits(nq);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      om[j] = __float_as_uint(ldexpf(__uint_as_float((ym[j] & 0x87F00000u) | nan_m), nm - 14));
      oq[j] = __float_as_uint(ldexpf(__uint_as_float((yq[j] & 0x07F80000u) | nan_q), nq - 14));
    }
    *(uint4*)(a.m_out + at) = make_uint4(top_halves(om[0], om[1]), top_halves(om[2], om[3]),
                                         top_halves(om[4], om[5]), top_halves(om[6], om[7]));
    *(uint4*)(a.v_out + at) = make_uint4(top_halves(oq[0], oq[1]), top_halves(oq[2], oq[3]),
                                         top_halves(oq[4], oq[5]), top_halves(oq[6], oq[7]));
  }
}

template <int BITS, bool VALUES, typename IO>
__device__ __forceinline__ void chunk(const AdamwArgs& a, const AdamwChunk& c, const IO& io,
                                      uint32_t key, const StepK& k, bool skip) {
  if (BITS == 32) chunk32(a, c, io, k, skip);
  else chunk8<VALUES>(a, c, io, key, k, skip);
}
template <int BITS, bool VALUES, typename WT, typename GT>
__device__ __forceinline__ void chunk_of(const AdamwArgs& a, const AdamwChunk& c, void* w, const void* g,
                                         uint32_t key, const StepK& k, bool skip) {
  WT* wp = (WT*)w + c.start;
  const GT* gp = (const GT*)g + c.start;
  if (c.n == ADAMW_CHUNK) chunk<BITS, VALUES>(a, c, Chunk<WT, GT, true>{wp, gp, c.n}, key, k, skip);
  else chunk<BITS, VALUES>(a, c, Chunk<WT, GT, false>{wp, gp, c.n}, key, k, skip);
}

template <int BITS, bool VALUES, typename Table>
__global__ void __launch_bounds__(kThreads) k_adamw(AdamwArgs a, Table tab) {
  const AdamwChunk c = a.chunks[blockIdx.x];
  const AdamwClock now = a.clocks[blockIdx.x];
  StepK k;
  k.coef = 1.0f;
  // a norm that is not finite: some gradient is not, and the step is left out. The chunk's
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
  if (c.wdt == DT_F32) chunk_of<BITS, VALUES, float, float>(a, c, w, g, now.key, k, skip);
  else if (c.wdt == DT_F16 && c.gdt == DT_F16) chunk_of<BITS, VALUES, _Float16, _Float16>(a, c, w, g, now.key, k, skip);
  else if (c.wdt == DT_F16) chunk_of<BITS, VALUES, _Float16, float>(a, c, w, g, now.key, k, skip);
  else if (c.gdt == DT_BF16) chunk_of<BITS, VALUES, bf16_t, bf16_t>(a, c, w, g, now.key, k, skip);
  else chunk_of<BITS, VALUES, bf16_t, float>(a, c, w, g, now.key, k, skip);
  __syncthreads();   // every wave has read its clock
  if (threadIdx.x == 0 && !skip) {
    // the hardware's estimates (2^-26 and better) with one Newton step each are exact far
    // below fp32's rounding, and shorter than a division and a root
    AdamwClock next;
    next.t = now.t + 1;
    next.p1 = now.p1 * a.b1d;
    next.p2 = now.p2 * a.b2d;
    const double d1 = 1.0 - next.p1, d2 = 1.0 - next.p2;
    const double r = __builtin_amdgcn_rcp(d1), q = __builtin_amdgcn_rsq(d2);
    next.ic1 = (float)__builtin_fma(__builtin_fma(-d1, r, 1.0), r, r);
    next.is2 = (float)__builtin_fma(__builtin_fma(-d2 * q, q, 1.0), 0.5 * q, q);
    next.key = adamw_step_key(a.seed, (uint64_t)next.t);
    a.clocks[blockIdx.x] = next;
  }
}

// Over n values from g on, by THREADS threads of which this is number `t`: four pieces of 16
// bytes a thread in flight, the last ones by themselves.
template <int THREADS, typename GT>
__device__ __forceinline__ double squares(const GT* __restrict__ g, uint32_t n, uint32_t t) {
  constexpr uint32_t N = 16 / sizeof(GT), kPass = THREADS * N;
  double s = 0.0;
  auto add = [&](const GT (&x)[N]) {
#pragma unroll
    for (uint32_t j = 0; j < N; ++j) {
      const double v = (double)to_f32(x[j]);
      s = fma(v, v, s);
    }
  };
  uint32_t i = t * N, left = n;
  for (; left >= 4 * kPass; left -= 4 * kPass, i += 4 * kPass) {
    GT x[4][N];
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u) load_wide(g + i + u * kPass, x[u]);
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u) add(x[u]);
  }
  if (!left) return s;
  GT x[4][N];
#pragma unroll
  for (uint32_t u = 0; u < 4; ++u) {
    const uint32_t k = i + u * kPass;
#pragma unroll
    for (uint32_t j = 0; j < N; ++j) x[u][j] = zero_of<GT>();
    if (k + N <= n) load_wide(g + k, x[u]);
  }
  // the end of the last piece
  if (n % N && (n / N) % THREADS == t)
    for (uint32_t k = n / N * N; k < n; ++k) {
      const double v = (double)to_f32(g[k]);
      s = fma(v, v, s);
    }
#pragma unroll
  for (uint32_t u = 0; u < 4; ++u) add(x[u]);
  return s;
}

template <int THREADS>
__device__ __forceinline__ double span_squares(const AdamwSpan& c, const void* g, uint32_t t) {
  if (c.gdt == DT_F32) return squares<THREADS>((const float*)g + c.start, c.n, t);
  if (c.gdt == DT_F16) return squares<THREADS>((const _Float16*)g + c.start, c.n, t);
  return squares<THREADS>((const bf16_t*)g + c.start, c.n, t);
}

__device__ __forceinline__ double block_sum(double s, double* lds) {
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__device__ __forceinline__ void write_norm(const AdamwNorm& a, double squares) {
  const double norm = sqrt(squares) * a.scale;
  a.out[0] = (float)norm;
  a.out[1] = (float)(norm > a.max_norm ? a.scale * (a.max_norm / norm) : a.scale);
}

// Adds one to a count and returns whether it is the last of `n`, which also clears it. The
// count is made where every workgroup sees it.
__device__ __forceinline__ bool last_of(uint32_t* count, uint32_t one, uint32_t n) {
  const uint32_t before = __hip_atomic_fetch_add(count, one, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (before != n - 1) return false;
  __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return true;
}

// The sums of squares of one launch's spans (67M fp16 values 27 us, 5.0 TB/s). JOIN (a call's last launch): the workgroup that
// finishes last also adds all the sums up, in their order, and writes the result; a kernel of
// its own for that would take 5 us with the gap before it. The sums go through atomic
// exchanges, whose answers the count waits for, and atomic loads: both act where every
// workgroup sees them, so no cache has to be written back in between (with fences that did,
// 32 ns a workgroup). Counting at one place takes 11 ns a workgroup; so 16 groups of them count
// apart, and their last ones together.
template <bool JOIN, typename Table>
__global__ void __launch_bounds__(kThreads) k_adamw_squares(AdamwNorm a, Table tab) {
  __shared__ double lds[4];
  __shared__ bool last;
  const AdamwSpan c = a.spans[blockIdx.x];
  double s = span_squares<kThreads>(c, tab.g[c.tensor - a.first_tensor], threadIdx.x);
  s = block_sum(s, lds);
  if (!JOIN) {
    if (threadIdx.x == 0) a.partial[blockIdx.x] = s;
    return;
  }
  if (threadIdx.x == 0) {
    unsigned long long old = __hip_atomic_exchange((unsigned long long*)a.partial + blockIdx.x,
                                                   __double_as_longlong(s), __ATOMIC_RELAXED,
                                                   __HIP_MEMORY_SCOPE_AGENT);
    uint32_t one = 1;
    __asm__ volatile("" : "+v"(one), "+v"(old));   // the count waits for the exchange
    const uint32_t groups = gridDim.x < ADAMW_COUNTS ? gridDim.x : ADAMW_COUNTS, mine = blockIdx.x % ADAMW_COUNTS;
    const uint32_t members = (gridDim.x - mine + ADAMW_COUNTS - 1) / ADAMW_COUNTS;
    last = last_of(a.counts + mine * ADAMW_COUNT_PITCH, one, members) &&
           last_of(a.counts + ADAMW_COUNTS * ADAMW_COUNT_PITCH, one, groups);
  }
  __syncthreads();
  if (!last) return;
  s = 0.0;
  for (uint32_t i = threadIdx.x; i < a.total_spans; i += kThreads)
    s += __longlong_as_double(__hip_atomic_load((unsigned long long*)a.all_partial + i, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT));
  s = block_sum(s, lds);
  if (threadIdx.x == 0) write_norm(a, s);
}

// The norm of up to 16 spans (of one launch, or none at all): one workgroup, a wave for each.
__global__ void __launch_bounds__(1024) k_adamw_norm(AdamwNorm a, AdamwTableOf<ADAMW_FEW_TENSORS> tab) {
  __shared__ double lds[16];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double s = 0.0;
  if (wave < a.total_spans) {
    const AdamwSpan c = a.spans[wave];
    s = span_squares<64>(c, tab.g[c.tensor - a.first_tensor], threadIdx.x & 63);
#pragma unroll
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o, 64);
  }
  if ((threadIdx.x & 63) == 0) lds[wave] = s;
  __syncthreads();
  if (threadIdx.x) return;
  s = 0.0;
  for (uint32_t i = 0; i < a.total_spans; ++i) s += lds[i];
  write_norm(a, s);
}

}  // namespace

namespace {

using FewTable = AdamwTableOf<ADAMW_FEW_TENSORS>;

FewTable few_of(int tensors, const AdamwTable& tab) {
  FewTable t;
  for (int i = 0; i < tensors; ++i) {
    t.w[i] = tab.w[i];
    t.g[i] = tab.g[i];
  }
  return t;
}

template <typename Table>
hipError_t step(const AdamwArgs& a, const Table& tab, hipStream_t s) {
  if (a.bits == 32) k_adamw<32, false><<<a.nchunks, kThreads, a.lds, s>>>(a, tab);
  else if (!a.m_out) k_adamw<8, false><<<a.nchunks, kThreads, 0, s>>>(a, tab);
  else k_adamw<8, true><<<a.nchunks, kThreads, 0, s>>>(a, tab);
  return hipGetLastError();
}
template <typename Table>
hipError_t sums(const AdamwNorm& a, uint32_t nspans, bool join, const Table& tab, hipStream_t s) {
  if (join) k_adamw_squares<true><<<nspans, kThreads, 0, s>>>(a, tab);
  else k_adamw_squares<false><<<nspans, kThreads, 0, s>>>(a, tab);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, int tensors, const AdamwTable& tab, hipStream_t s) {
  return tensors <= ADAMW_FEW_TENSORS ? step(a, few_of(tensors, tab), s) : step(a, tab, s);
}

hipError_t launch_adamw_squares(const AdamwNorm& a, uint32_t nspans, bool join, int tensors,
                                const AdamwTable& tab, hipStream_t s) {
  return tensors <= ADAMW_FEW_TENSORS ? sums(a, nspans, join, few_of(tensors, tab), s)
                                      : sums(a, nspans, join, tab, s);
}

hipError_t launch_adamw_norm(const AdamwNorm& a, int tensors, const AdamwTable& tab, hipStream_t s) {
  k_adamw_norm<<<1, 1024, 0, s>>>(a, few_of(tensors, tab));
  return hipGetLastError();
}

}  // namespace tg
