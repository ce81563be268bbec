// Newton-Schulz orthogonalisation and the Muon step (see k_muon.hip for the iteration and its
// formats) of matrices that a workgroup holds: one workgroup a matrix, one launch for all of it.
//
// Eight waves. A wave owns parts of 16 x 32 values of X, whose values it keeps in registers as
// fp32 from the first pass over the gradient to the last over the weights; LDS holds what the
// products read, the fp16 parts of X and of A, which B replaces. A launch of its own for each
// product of a 64 x 64 matrix takes 5 us, nearly all of it latency; here a step's three products
// are four barriers apart.
#include <type_traits>

#include "muon_common.h"

namespace tg {

namespace {

constexpr int kWaves = 8, kThreads = kWaves * 64;

// The places of a matrix in LDS, in 16-bit values: lines are padded to whole k of a matrix
// instruction and 8 more, so that eight lines' 16-byte pieces lie in eight different banks.
struct Places {
  uint32_t ldx, lds;         // lines of X, of A and B
  uint32_t xpart, spart;     // values of a part
  uint32_t s, diag, bytes;   // where A begins, the diagonals, all of it
};
__host__ __device__ inline Places places_of(uint32_t rows, uint32_t cols, bool exact) {
  Places p;
  const uint32_t m = rows < cols ? rows : cols, pm = (m + 31) & ~31u;
  p.ldx = ((cols + 31) & ~31u) + 8;
  p.lds = pm + 8;
  p.xpart = ((rows + 31) & ~31u) * p.ldx;
  p.spart = pm * p.lds;
  p.s = p.xpart * (exact ? 2 : 1);
  p.diag = p.s + p.spart * (exact ? 2 : 1);
  p.bytes = p.diag * 2 + 2 * pm * 4;
  return p;
}
typedef TG_LDS _Float16 lds_f16;
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// the fragment of 16 lines from `line` on, 32 values of k from k on (straight), or of 16 columns
// from `line` on (crossed)
template <bool CROSSED>
__device__ __forceinline__ s16x8 fragment(const lds_f16* p, uint32_t ld, uint32_t line, uint32_t k, uint32_t lane) {
  const uint32_t r = lane & 15, kg = lane >> 4;
  if constexpr (!CROSSED) {
    return *(const TG_LDS s16x8*)(p + (line + r) * ld + k + kg * 8);
  } else {
    const lds_f16* const a = p + (k + kg * 8 + (r >> 2)) * ld + line + (r & 3) * 4;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TG_LDS s16x4*)a);
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TG_LDS s16x4*)(a + 4 * ld));
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  }
}

// 16 x 32 sums over kk values of k of the products of the parts of a and b
template <bool EXACT, bool CA, bool CB>
__device__ __forceinline__ void product(f32x4 (&c)[2], const lds_f16* a, uint32_t lda, uint32_t pa, uint32_t i,
                                        const lds_f16* b, uint32_t ldb, uint32_t pb, uint32_t j, uint32_t kk, uint32_t lane) {
  c[0] = c[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (uint32_t k = 0; k < kk; k += 32) {
    const s16x8 ah = fragment<CA>(a, lda, i, k, lane);
    s16x8 al = {};
    if (EXACT) al = fragment<CA>(a + pa, lda, i, k, lane);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const s16x8 bh = fragment<CB>(b, ldb, j + 16 * h, k, lane);
      if (EXACT) {
        const s16x8 bl = fragment<CB>(b + pb, ldb, j + 16 * h, k, lane);
        c[h] = mm_mfma<DT_F16>(bh, al, c[h]);
        c[h] = mm_mfma<DT_F16>(bl, ah, c[h]);
      }
      c[h] = mm_mfma<DT_F16>(bh, ah, c[h]);
    }
  }
}

// four values to the parts of a matrix
template <bool EXACT>
__device__ __forceinline__ void put4(lds_f16* p, uint32_t part, const float* v) {
  _Float16 h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) two_parts(v[e], h[e], l[e]);
  *(TG_LDS f16x4*)p = f16x4{h[0], h[1], h[2], h[3]};
  if (EXACT) *(TG_LDS f16x4*)(p + part) = f16x4{l[0], l[1], l[2], l[3]};
}

struct NoTable {};

// SLOTS: parts of X that a wave owns at most. Table: MuonTable for a step, else matrices given as
// they are.
template <int SLOTS, bool EXACT, class Table>
__global__ void __launch_bounds__(kThreads, 2)
    k_ns_small(const NsCommon c, const NsSmall k, const MuonFirst f, const Table table, const NsSource src, const NsParts p) {
  constexpr bool MUON = std::is_same<Table, MuonTable>::value;
  extern __shared__ char lds_raw[];
  __shared__ double sums[kWaves];
  if (left_out(c)) return;
  NsMat m;
  uint32_t none0, none1;
  const uint32_t mat = my_part(c, p, blockIdx.x, m, none0, none1);
  const Places at = places_of(m.rows, m.cols, EXACT);
  lds_f16* x16 = (lds_f16*)lds_raw;
  uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, c4 = (lane >> 4) * 4;
  const uint32_t across = (m.cols + 31) / 32, sacross = (m.m + 31) / 32;
  // the first row and column of this wave's parts of X, and of A
  uint32_t xi[SLOTS], xj[SLOTS], si[4], sj[4];
  auto places = [&](uint32_t wide, uint32_t* i, uint32_t* j, int n) {
    uint32_t a = wave / wide, b = wave % wide;
#pragma unroll
    for (int s = 0; s < n; ++s) {
      i[s] = uniform(a * 16);
      j[s] = uniform(b * 32);
      for (b += kWaves; b >= wide; b -= wide) ++a;
    }
  };
  places(across, xi, xj, SLOTS);
  places(sacross, si, sj, 4);
  for (uint32_t i = threadIdx.x; i < (at.bytes + 15) / 16; i += kThreads) ((TG_LDS u32x4*)x16)[i] = u32x4{0, 0, 0, 0};

  // this wave's values: the gradient and momentum, or the matrix
  const float coef = c.clip ? c.clip[1] : 1.0f;
  const void* from = src.x;
  if constexpr (MUON) from = table.g[m.tensor - f.first_tensor];
  float x[SLOTS][2][4];
  double square = 0.0;
  with_type(m.gdt, [&](auto zero) {
    using T = decltype(zero);
    const T* const g = (const T*)from + (MUON ? m.elem : mat * src.matrix_stride);
    const int64_t pitch = MUON ? (int64_t)m.cols : src.row_stride;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const uint32_t i = xi[s] + r;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t j = xj[s] + h * 16 + c4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float u = 0.0f;
          if (i < m.rows && j + e < m.cols) {
            u = to_f32(g[i * pitch + j + e]);
            if (MUON) {
              float* const mom = f.momentum + m.state + (uint64_t)i * m.cols + j + e;
              const float v = u * coef, w = f.mu * *mom + f.nu * v;
              *mom = w;
              u = updated(v, w, f);
            }
          }
          x[s][h][e] = u;
          square += (double)u * u;
        }
      }
    }
  });
#pragma unroll
  for (int o = 32; o; o >>= 1) square += __shfl_xor(square, o);
  if (lane == 0) sums[wave] = square;
  __syncthreads();
  double total = 0.0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) total += sums[i];
  const float scale = (float)((double)NS_X / (__builtin_sqrt(total) + k.eps));
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[s][h][e] *= scale;

  const bool wide = m.rows <= m.cols;
#pragma unroll 1
  for (int t = 0; t < k.steps; ++t) {
    // (taken as another lane each time: the compiler would keep the addresses of all parts in
    // registers over the steps, and spill)
    __asm__ volatile("" : "+v"(lane));
    r = lane & 15;
    c4 = (lane >> 4) * 4;
    lds_f16* const s16 = x16 + at.s;
    TG_LDS float* const da = (TG_LDS float*)(x16 + at.diag);
    TG_LDS float* const db = da + (at.lds - 8);
    // X's parts (the last reads of X and of B ended at a barrier)
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (xi[s] >= m.rows) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) put4<EXACT>(x16 + (xi[s] + r) * at.ldx + xj[s] + h * 16 + c4, at.xpart, x[s][h]);
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s) {                                  // A
      const uint32_t i = si[s], j = sj[s];
      if (i >= m.m) continue;
      f32x4 q[2];
      if (wide) product<EXACT, false, false>(q, x16, at.ldx, at.xpart, i, x16, at.ldx, at.xpart, j, m.cols, lane);
      else product<EXACT, true, true>(q, x16, at.ldx, at.xpart, i, x16, at.ldx, at.xpart, j, m.rows, lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t on = i + r - (j + h * 16 + c4);     // which of the four lies on the diagonal
        float o[4], d = 0.0f;
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          const float v = q[h][e] * (1.0f / (NS_X * NS_X));
          d = on == e ? v : d;
          o[e] = on == e ? 0.0f : v * NS_M;
        }
        if (on < 4) da[i + r] = d;
        put4<EXACT>(s16 + (i + r) * at.lds + j + h * 16 + c4, at.spart, o);
      }
    }
    __syncthreads();
    float b[4][2][4], d[4] = {};                                    // B
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t i = si[s], j = sj[s];
      if (i >= m.m) continue;
      f32x4 q[2];
      product<EXACT, false, false>(q, s16, at.lds, at.spart, i, s16, at.lds, at.spart, j, m.m, lane);
      const float di = da[i + r];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t o = (i + r) * at.lds + j + h * 16 + c4;
        const f16x4 oh = *(const TG_LDS f16x4*)(s16 + o);
        f16x4 ol = {};
        if (EXACT) ol = *(const TG_LDS f16x4*)(s16 + at.spart + o);
        const f32x4 dj = *(const TG_LDS f32x4*)(da + j + h * 16 + c4);
        const uint32_t on = i + r - (j + h * 16 + c4);
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          const float q2 = q[h][e] * (1.0f / (NS_M * NS_M));
          const float v = ((float)oh[e] + (float)ol[e]) * (1.0f / NS_M);
          const float w = c.cb * v + c.cc * (q2 + (di + dj[e]) * v);
          d[s] = on == e ? c.cb * di + c.cc * (di * di + q2) : d[s];
          b[s][h][e] = on == e ? 0.0f : w * NS_M;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t i = si[s], j = sj[s];
      if (i >= m.m) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        put4<EXACT>(s16 + (i + r) * at.lds + j + h * 16 + c4, at.spart, b[s][h]);
        const uint32_t first = j + h * 16 + c4;
        if (i + r >= first && i + r < first + 4) db[i + r] = d[s];
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {                              // X
      const uint32_t i = xi[s], j = xj[s];
      if (i >= m.rows) continue;
      f32x4 q[2];
      if (wide) product<EXACT, false, true>(q, s16, at.lds, at.spart, i, x16, at.ldx, at.xpart, j, m.rows, lane);
      else product<EXACT, false, false>(q, x16, at.ldx, at.xpart, i, s16, at.lds, at.spart, j, m.cols, lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 dj = *(const TG_LDS f32x4*)(wide ? db + (i + r) / 4 * 4 : db + j + h * 16 + c4);
        const float di = db[wide ? i + r : 0];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[s][h][e] = (c.ca + (wide ? di : dj[e])) * x[s][h][e] + q[h][e] * (1.0f / NS_M);
      }
    }
    __syncthreads();
  }

  const float step = (float)(k.lr * m.scale), decay = (float)(1.0 - k.lr * m.wd);
  void* to = k.out;
  if constexpr (MUON) to = table.w[m.tensor - f.first_tensor];
  with_type(m.wdt, [&](auto zero) {
    using T = decltype(zero);
    T* const out = (T*)to + (MUON ? m.elem : (uint64_t)mat * m.rows * m.cols);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const uint32_t i = xi[s] + r;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t j = xj[s] + h * 16 + c4 + e;
          if (i >= m.rows || j >= m.cols) continue;
          T* const o = out + (uint64_t)i * m.cols + j;
          const float y = x[s][h][e] * (1.0f / NS_X);
          *o = from_f32<T>(MUON ? to_f32(*o) * decay - step * y : y);
        }
    }
  });
}

template <int SLOTS, bool EXACT, class Table>
hipError_t launch(const NsCommon& c, const NsSmall& k, const MuonFirst& f, const Table& t, const NsSource& src,
                  const NsParts& p, uint32_t n, hipStream_t s) {
  auto* const kernel = k_ns_small<SLOTS, EXACT, Table>;
  const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, NS_SMALL_LDS);
  if (e != hipSuccess) return e;
  kernel<<<n, kThreads, k.lds, s>>>(c, k, f, t, src, p);
  return hipGetLastError();
}
template <class Table>
hipError_t launch_any(const NsCommon& c, const NsSmall& k, const MuonFirst& f, const Table& t, const NsSource& src,
                      const NsParts& p, uint32_t n, hipStream_t s) {
  if (k.exact)
    return k.slots <= 2   ? launch<2, true>(c, k, f, t, src, p, n, s)
           : k.slots <= 6 ? launch<6, true>(c, k, f, t, src, p, n, s) : launch<12, true>(c, k, f, t, src, p, n, s);
  return k.slots <= 2   ? launch<2, false>(c, k, f, t, src, p, n, s)
         : k.slots <= 6 ? launch<6, false>(c, k, f, t, src, p, n, s) : launch<12, false>(c, k, f, t, src, p, n, s);
}
static_assert(sizeof(NsCommon) + sizeof(NsSmall) + sizeof(MuonFirst) + sizeof(MuonTable) + sizeof(NsSource) + sizeof(NsParts) <=
                  4096, "kernel arguments");

}  // namespace

int ns_small_slots(uint32_t rows, uint32_t cols, bool exact) {
  if ((rows < cols ? rows : cols) > 128 || rows > 65536 || cols > 65536) return 0;
  const uint32_t parts = ((rows + 15) / 16) * ((cols + 31) / 32);
  if (parts > 12 * kWaves || ns_small_lds(rows, cols, exact) > NS_SMALL_LDS) return 0;
  return (int)((parts + kWaves - 1) / kWaves);
}
uint32_t ns_small_lds(uint32_t rows, uint32_t cols, bool exact) { return (places_of(rows, cols, exact).bytes + 15) & ~15u; }

hipError_t launch_ns_small(const NsCommon& c, const NsSmall& k, const MuonFirst& f, const MuonTable* t, const NsSource& src,
                           const NsParts& p, uint32_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  if (n > 0x7FFFFFFFu / kThreads) return hipErrorInvalidValue;
  return t ? launch_any(c, k, f, *t, src, p, n, s) : launch_any(c, k, f, NoTable{}, src, p, n, s);
}

}  // namespace tg
