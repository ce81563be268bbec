// Newton-Schulz orthogonalisation and the Muon step (see k_muon.hip for the iteration and its
// formats) of matrices that a workgroup holds: one workgroup a matrix, one launch for all of it.
//
// Eight or 16 waves. A wave owns parts of 16 or 32 x 32 values of X, which it keeps in registers as
// fp32 from the first pass over the gradient to the last over the weights; LDS holds what the
// products read, the fp16 parts of X and of A, which B replaces. A launch of its own for each
// product of a 64 x 64 matrix takes 5 us, nearly all of it latency; here a step's three products
// are four barriers apart.
#include <algorithm>
#include <type_traits>

#include "muon_common.h"

namespace tg {

namespace {

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
    return *(const TG_LDS s16x8*)(p + __umul24(line + r, ld) + k + kg * 8);
  } else {
    const lds_f16* const a = p + __umul24(k + kg * 8 + (r >> 2), ld) + line + (r & 3) * 4;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TG_LDS s16x4*)a);
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TG_LDS s16x4*)(a + 4 * ld));
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  }
}

// 16 RB x 32 sums over kk values of k of the products of the parts of a and b
template <int RB, bool EXACT, bool CA, bool CB>
__device__ __forceinline__ void product(f32x4 (&c)[RB][2], const lds_f16* a, uint32_t lda, uint32_t pa, uint32_t i,
                                        const lds_f16* b, uint32_t ldb, uint32_t pb, uint32_t j, uint32_t kk, uint32_t lane) {
#pragma unroll
  for (int g = 0; g < RB; ++g) c[g][0] = c[g][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (uint32_t k = 0; k < kk; k += 32) {
    s16x8 ah[RB], al[RB], bh[2], bl[2];
#pragma unroll
    for (int g = 0; g < RB; ++g) {
      ah[g] = fragment<CA>(a, lda, i + 16 * g, k, lane);
      if (EXACT) al[g] = fragment<CA>(a + pa, lda, i + 16 * g, k, lane);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bh[h] = fragment<CB>(b, ldb, j + 16 * h, k, lane);
      if (EXACT) bl[h] = fragment<CB>(b + pb, ldb, j + 16 * h, k, lane);
    }
#pragma unroll
    for (int g = 0; g < RB; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (EXACT) {
          c[g][h] = mm_mfma<DT_F16>(bh[h], al[g], c[g][h]);
          c[g][h] = mm_mfma<DT_F16>(bl[h], ah[g], c[g][h]);
        }
        c[g][h] = mm_mfma<DT_F16>(bh[h], ah[g], c[g][h]);
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

// Four values of a line from column j on, without a branch where the line has four at all.
template <typename T>
struct Four {
  typedef uint32_t V __attribute__((ext_vector_type(sizeof(T))));   // four values' bits
  V v;
  __device__ __forceinline__ void load(const T* line, uint32_t j, uint32_t cols) {
    if (cols >= 4) {
      __builtin_memcpy(&v, line + (j + 4 <= cols ? j : cols - 4), sizeof(V));
    } else {
      T t[4];
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) t[e] = line[e < cols ? e : 0];
      __builtin_memcpy(&v, t, sizeof(V));
    }
  }
  __device__ __forceinline__ float one(int e) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(v[e]);
    } else {
      const uint16_t b = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
      T t;
      __builtin_memcpy(&t, &b, 2);
      return to_f32(t);
    }
  }
  // value j + e, anything past the line
  __device__ __forceinline__ float value(int e, uint32_t j, uint32_t cols) const {
    const uint32_t turn = cols >= 4 && j + 4 > cols ? j + 4 - cols : 0;
    float x = one(e);
    if (e < 3) x = turn == 1 ? one(e < 3 ? e + 1 : 3) : x;
    if (e < 2) x = turn == 2 ? one(e < 2 ? e + 2 : 3) : x;
    if (e < 1) x = turn == 3 ? one(3) : x;
    return x;
  }
};
template <typename T>
__device__ __forceinline__ void store_four(T* line, uint32_t j, uint32_t cols, const T* v) {
  if (j + 4 <= cols) {
    store_values<4>(line + j, v);
  } else {
#pragma unroll
    for (uint32_t e = 0; e < 3; ++e)
      if (j + e < cols) line[j + e] = v[e];
  }
}

struct NoTable {};

// SLOTS: parts of 16 RB x 32 values of X that a wave owns at most (of A: one). Table: MuonTable for a step, else matrices given as
// they are.
template <int WAVES, int RB, int SLOTS, bool EXACT, class Table>
__global__ void __launch_bounds__(WAVES * 64, WAVES / 4)
    k_ns_small(const NsCommon c, const NsSmall k, const MuonFirst f, const Table table, const NsSource src, const NsParts p) {
  constexpr uint32_t kWaves = WAVES, kThreads = WAVES * 64;
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
  uint32_t xi[SLOTS], xj[SLOTS], si[1], sj[1];
  auto places = [&](uint32_t wide, uint32_t* i, uint32_t* j, int n) {
    uint32_t a = wave / wide, b = wave % wide;
#pragma unroll
    for (int s = 0; s < n; ++s) {
      i[s] = uniform(a * 16 * RB);
      j[s] = uniform(b * 32);
      for (b += kWaves; b >= wide; b -= wide) ++a;
    }
  };
  places(across, xi, xj, SLOTS);
  places(sacross, si, sj, 1);
  for (uint32_t i = threadIdx.x; i < (at.bytes + 15) / 16; i += kThreads) ((TG_LDS u32x4*)x16)[i] = u32x4{0, 0, 0, 0};

  // this wave's values: the gradient and momentum, or the matrix
  const float coef = c.clip ? c.clip[1] : 1.0f;
  const void* from = src.x;
  if constexpr (MUON) from = table.g[m.tensor - f.first_tensor];
  float x[SLOTS][RB][2][4];
  double square = 0.0;
  with_type(m.gdt, [&](auto zero) {
    using T = decltype(zero);
    const T* const g = (const T*)from + (MUON ? m.elem : mat * src.matrix_stride);
    const int64_t pitch = MUON ? (int64_t)m.cols : src.row_stride;
    float* const mom = MUON ? f.momentum + m.state : nullptr;
    // all of a part's loads at once, four values each: those that would pass a line's end begin
    // four before it and are turned, those outside the matrix take its first line
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      Four<T> raw[2 * RB];
      Four<float> old[2 * RB];
#pragma unroll
      for (int gh = 0; gh < 2 * RB; ++gh) {
        const uint32_t i = xi[s] + (gh >> 1) * 16 + r, j = xj[s] + (gh & 1) * 16 + c4, row = i < m.rows ? i : 0;
        raw[gh].load(g + row * pitch, j, m.cols);
        if (MUON) old[gh].load(mom + (uint64_t)row * m.cols, j, m.cols);
      }
#pragma unroll
      for (int gh = 0; gh < 2 * RB; ++gh) {
        const uint32_t i = xi[s] + (gh >> 1) * 16 + r, j = xj[s] + (gh & 1) * 16 + c4;
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float u = raw[gh].value(e, j, m.cols);
          if (MUON) {
            const float v = u * coef;
            w[e] = f.mu * old[gh].value(e, j, m.cols) + f.nu * v;
            u = updated(v, w[e], f);
          }
          u = i < m.rows && j + e < m.cols ? u : 0.0f;
          x[s][gh >> 1][gh & 1][e] = u;
          square += (double)u * u;
        }
        if (MUON && i < m.rows) store_four(mom + (uint64_t)i * m.cols, j, m.cols, w);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  });
#pragma unroll
  for (int o = 32; o; o >>= 1) square += __shfl_xor(square, o);
  if (lane == 0) sums[wave] = square;
  __syncthreads();
  double total = 0.0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) total += sums[i];
  const NsScale scale(total, k.eps);
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
#pragma unroll
    for (int gh = 0; gh < 2 * RB; ++gh)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[s][gh >> 1][gh & 1][e] = scale(x[s][gh >> 1][gh & 1][e]);

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
      for (int gh = 0; gh < 2 * RB; ++gh)
        put4<EXACT>(x16 + __umul24(xi[s] + (gh >> 1) * 16 + r, at.ldx) + xj[s] + (gh & 1) * 16 + c4, at.xpart,
                    x[s][gh >> 1][gh & 1]);
    }
    __syncthreads();
    const uint32_t i0 = si[0], j0 = sj[0];
    const bool mine = i0 < m.m;
    f32x4 q[RB][2];
    if (mine) {                                                    // A
      if (wide) product<RB, EXACT, false, false>(q, x16, at.ldx, at.xpart, i0, x16, at.ldx, at.xpart, j0, m.cols, lane);
      else product<RB, EXACT, true, true>(q, x16, at.ldx, at.xpart, i0, x16, at.ldx, at.xpart, j0, m.rows, lane);
#pragma unroll
      for (int gh = 0; gh < 2 * RB; ++gh) {
        const uint32_t i = i0 + (gh >> 1) * 16 + r, j = j0 + (gh & 1) * 16 + c4, on = i - j;   // on: which lies on the diagonal
        float o[4], d = 0.0f;
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          const float v = q[gh >> 1][gh & 1][e] * (1.0f / (NS_X * NS_X));
          d = on == e ? v : d;
          o[e] = on == e ? 0.0f : v * NS_M;
        }
        if (on < 4) da[i] = d;
        put4<EXACT>(s16 + __umul24(i, at.lds) + j, at.spart, o);
      }
    }
    __syncthreads();
    float b[2 * RB][4], db0[RB] = {};                              // B
    if (mine) {
      product<RB, EXACT, false, false>(q, s16, at.lds, at.spart, i0, s16, at.lds, at.spart, j0, m.m, lane);
#pragma unroll
      for (int gh = 0; gh < 2 * RB; ++gh) {
        const uint32_t i = i0 + (gh >> 1) * 16 + r, j = j0 + (gh & 1) * 16 + c4, on = i - j, o = __umul24(i, at.lds) + j;
        const f16x4 oh = *(const TG_LDS f16x4*)(s16 + o);
        f16x4 ol = {};
        if (EXACT) ol = *(const TG_LDS f16x4*)(s16 + at.spart + o);
        const f32x4 dj = *(const TG_LDS f32x4*)(da + j);
        const float di = da[i];
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          const float q2 = q[gh >> 1][gh & 1][e] * (1.0f / (NS_M * NS_M));
          const float v = ((float)oh[e] + (float)ol[e]) * (1.0f / NS_M);
          const float w = c.cb * v + c.cc * (q2 + (di + dj[e]) * v);
          db0[gh >> 1] = on == e ? c.cb * di + c.cc * (di * di + q2) : db0[gh >> 1];
          b[gh][e] = on == e ? 0.0f : w * NS_M;
        }
      }
    }
    __syncthreads();
    if (mine) {
#pragma unroll
      for (int gh = 0; gh < 2 * RB; ++gh) {
        const uint32_t i = i0 + (gh >> 1) * 16 + r, j = j0 + (gh & 1) * 16 + c4;
        put4<EXACT>(s16 + __umul24(i, at.lds) + j, at.spart, b[gh]);
        if (i - j < 4) db[i] = db0[gh >> 1];
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {                              // X
      if (xi[s] >= m.rows) continue;
      f32x4 v[RB][2];
      if (wide) product<RB, EXACT, false, true>(v, s16, at.lds, at.spart, xi[s], x16, at.ldx, at.xpart, xj[s], m.rows, lane);
      else product<RB, EXACT, false, false>(v, x16, at.ldx, at.xpart, xi[s], s16, at.lds, at.spart, xj[s], m.cols, lane);
#pragma unroll
      for (int gh = 0; gh < 2 * RB; ++gh) {
        const uint32_t i = xi[s] + (gh >> 1) * 16 + r, j = xj[s] + (gh & 1) * 16 + c4;
        const f32x4 dj = *(const TG_LDS f32x4*)(wide ? db + i / 4 * 4 : db + j);
        const float di = db[wide ? i : 0];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[s][gh >> 1][gh & 1][e] =
              (c.ca + (wide ? di : dj[e])) * x[s][gh >> 1][gh & 1][e] + v[gh >> 1][gh & 1][e] * (1.0f / NS_M);
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
      Four<T> old[2 * RB];
      if (MUON)
#pragma unroll
        for (int gh = 0; gh < 2 * RB; ++gh) {
          const uint32_t i = xi[s] + (gh >> 1) * 16 + r;
          old[gh].load(out + (uint64_t)(i < m.rows ? i : 0) * m.cols, xj[s] + (gh & 1) * 16 + c4, m.cols);
        }
#pragma unroll
      for (int gh = 0; gh < 2 * RB; ++gh) {
        const uint32_t i = xi[s] + (gh >> 1) * 16 + r, j = xj[s] + (gh & 1) * 16 + c4;
        T y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = x[s][gh >> 1][gh & 1][e] * (1.0f / NS_X);
          y[e] = from_f32<T>(MUON ? old[gh].value(e, j, m.cols) * decay - step * v : v);
        }
        if (i < m.rows) store_four(out + (uint64_t)i * m.cols, j, m.cols, y);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  });
}

template <int WAVES, int RB, int SLOTS, bool EXACT, class Table>
hipError_t launch(const NsCommon& c, const NsSmall& k, const MuonFirst& f, const Table& t, const NsSource& src,
                  const NsParts& p, uint32_t n, hipStream_t s) {
  if (n > 0xFFFFFFFFu / (WAVES * 64)) return hipErrorInvalidValue;   // threads of a launch in 32 bits
  auto* const kernel = k_ns_small<WAVES, RB, SLOTS, EXACT, Table>;
  const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, NS_SMALL_LDS);
  if (e != hipSuccess) return e;
  kernel<<<n, WAVES * 64, k.lds, s>>>(c, k, f, t, src, p);
  return hipGetLastError();
}
// Matrices of up to eight parts of 16 x 32 have a wave for each; others parts of 32 x 32, which
// take two thirds of the reads of LDS that set their pace (113 x 156 fp32: 105 us in parts of
// 16 x 32, 70 in these). Four to a wave need more registers than there are: 68 to 112 bytes a lane go to
// memory, in bf16 without a step none.
template <bool EXACT, class Table>
hipError_t launch_any(const NsCommon& c, const NsSmall& k, const MuonFirst& f, const Table& t, const NsSource& src,
                      const NsParts& p, uint32_t n, hipStream_t s) {
  return k.parts == 1   ? launch<8, 1, 1, EXACT>(c, k, f, t, src, p, n, s)
         : k.parts <= 32 ? launch<16, 2, 2, EXACT>(c, k, f, t, src, p, n, s) : launch<16, 2, 4, EXACT>(c, k, f, t, src, p, n, s);
}
static_assert(sizeof(NsCommon) + sizeof(NsSmall) + sizeof(MuonFirst) + sizeof(MuonTable) + sizeof(NsSource) + sizeof(NsParts) <=
                  4096, "kernel arguments");

}  // namespace

uint32_t ns_small_parts(uint32_t rows, uint32_t cols, bool exact) {
  const uint32_t m = rows < cols ? rows : cols;
  if (m > 128 || rows > 65536 || cols > 65536) return 0;
  if (ns_small_lds(rows, cols, exact) > NS_SMALL_LDS) return 0;
  const uint32_t wide = (cols + 31) / 32;
  if (((rows + 15) / 16) * wide <= 8 && ((m + 15) / 16) * ((m + 31) / 32) <= 8) return 1;
  const uint32_t parts = ((rows + 31) / 32) * wide;
  return parts <= 64 ? std::max(parts, 2u) : 0;
}
uint32_t ns_small_lds(uint32_t rows, uint32_t cols, bool exact) { return (places_of(rows, cols, exact).bytes + 15) & ~15u; }

hipError_t launch_ns_small(const NsCommon& c, const NsSmall& k, const MuonFirst& f, const MuonTable* t, const NsSource& src,
                           const NsParts& p, uint32_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  if (t) return k.exact ? launch_any<true>(c, k, f, *t, src, p, n, s) : launch_any<false>(c, k, f, *t, src, p, n, s);
  return k.exact ? launch_any<true>(c, k, f, NoTable{}, src, p, n, s) : launch_any<false>(c, k, f, NoTable{}, src, p, n, s);
}

}  // namespace tg
