// A workgroup's tile of a product of 16-bit matrices, C = A B^T with fp32 sums, for gfx950's
// matrix instructions. Shared by the Newton-Schulz products (k_muon.hip) and the gated linear
// layer (k_gated.hip), which differ in what they do with the sums.
//
// C[i][j] = sum over k of A(i, k) B(j, k). Each operand lies in memory either by its own rows
// ("straight": the k of one row are contiguous) or by k ("crossed": the rows of one k are
// contiguous). Both go to LDS as they lie, 16 bytes a lane through buffer resources that end
// with the operand (what lies beyond reads as zero, so no size has to fit the tile), and are
// read back as fragments of v_mfma_f32_16x16x32: straight ones 8 values a lane at once, crossed
// ones by the transposing reads (ds_read_b64_tr_b16: 16 lanes name 4 rows of 16 values, each
// lane receives its column of them). A transfer fills LDS in lane order, so bank conflicts are
// avoided by permuting what each lane fetches: a straight row's eight 16-byte pieces by the
// row's low bits, a crossed row's 32-byte pairs by those bits of k in which the 32 lanes of a
// read differ.
//
// k may run over several segments, each with operands of its own: a value held in two or three
// 16-bit parts is multiplied by naming its parts' products one after another (the smallest
// first), and [dg du] [Wg; Wu] without laying the weights together.
#pragma once
#include "tg_common.h"

namespace tg {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#define TG_LDS __attribute__((address_space(3)))

// A matrix of 16-bit values as it lies: `lines` lines of `len` contiguous values, `stride`
// values apart. `p` and the lines are 16-byte aligned and len is a multiple of 8 (rows are
// padded to that, with zeros where k runs along them).
struct MmOperand {
  const void* p;
  int64_t lines;
  uint32_t len, stride;
};

// at most 2^21 values between lines: a tile's offsets stay under 2^31
constexpr int64_t MM_MOST_STRIDE = 1 << 21;

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// One operand's way into LDS: ROWS rows (or columns of C) by 64 values of k, PER transfers of
// 1 KB for each of WAVES waves.
template <int ROWS, int WAVES, bool CROSSED>
struct MmLoader {
  static constexpr int PER = ROWS / 8 / WAVES;
  static constexpr int BYTES = ROWS * 128;
  static_assert(PER * 8 * WAVES == ROWS, "the waves share the transfers evenly");
  uint32_t v[PER];       // lane's byte offsets from the stage's first byte
  uint32_t k_of_lane;    // straight: the k of the lane's piece within the stage
  uint64_t at;           // the stage's first byte
  int64_t left;          // bytes from there to the operand's end

  // The row of the tile that transfer i of a wave begins at (straight).
  __device__ static int row0(int wave, int i) { return (wave * PER + i) * 8; }

  __device__ __forceinline__ void init(int wave, int lane, uint32_t stride) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int q = wave * PER + i;
      if constexpr (!CROSSED) {
        const int r = lane >> 3;
        k_of_lane = (uint32_t)(((lane & 7) ^ r) * 8);
        v[i] = (uint32_t)(q * 8 + r) * (stride * 2) + k_of_lane * 2;
      } else {
        constexpr int LANES = ROWS / 8;   // of one k
        const int k = q * (64 / LANES) + lane / LANES, c = lane % LANES;
        v[i] = (uint32_t)k * (stride * 2) + (uint32_t)(c ^ (turn(k) << 1)) * 16;
        k_of_lane = 0;
      }
    }
  }
  // crossed: how a k's pairs are permuted
  __device__ static constexpr int turn(int k) { return ((k & 3) | (((k >> 3) & 1) << 2)) & (ROWS / 16 - 1); }

  // from row `row` and k = 0 on
  __device__ __forceinline__ void start(const MmOperand& o, int64_t row) {
    const uint64_t skip = CROSSED ? (uint64_t)row * 2 : (uint64_t)row * o.stride * 2;
    at = (uint64_t)o.p + skip;
    left = ((o.lines - 1) * (int64_t)o.stride + o.len) * 2 - (int64_t)skip;
  }
  // past 64 values of k
  __device__ __forceinline__ void next(uint32_t stride) {
    const uint32_t step = CROSSED ? stride * 128 : 128;
    at += step;
    left -= step;
  }
  // `rem`: values of k from the stage's first one on; `i0`, `n`: which transfers
  template <int I0 = 0, int N = PER>
  __device__ __forceinline__ void issue(TG_LDS char* lds, int wave, uint32_t rem) const {
    const int64_t l = left < 0 ? 0 : left;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)at, 0, (int)(l > 0xFFFFFFF0ll ? 0xFFFFFFF0u : (uint32_t)l), 0x00020000);
#pragma unroll
    for (int i = I0; i < I0 + N; ++i) {
      const uint32_t o = CROSSED || k_of_lane < rem ? v[i] : 0xFFFFFFF0u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (TG_LDS void*)(lds + (wave * PER + i) * 1024), 16, (int)o, 0, 0, 0);
    }
  }
};

// One operand's fragments: a wave's N blocks of 16 rows from `row` (a multiple of 16 N) on.
template <int ROWS, int N, bool CROSSED>
struct MmReader {
  uint32_t at[CROSSED ? N : 2];

  __device__ __forceinline__ void init(int row, int lane) {
    const int r = lane & 15, kg = lane >> 4;
    if constexpr (!CROSSED) {
      at[0] = (uint32_t)((row + r) * 128 + ((kg ^ (r & 7)) * 16));
      at[1] = at[0] ^ 64;
    } else {
      const int k = kg * 8 + (r >> 2);
#pragma unroll
      for (int i = 0; i < N; ++i)
        at[i] = (uint32_t)(k * (ROWS * 2) + (((row >> 4) + i) ^ MmLoader<ROWS, 1, true>::turn(k)) * 32 + (r & 3) * 8);
    }
  }
  // block i, the 32 values of k from 32 half on
  __device__ __forceinline__ s16x8 get(const TG_LDS char* lds, int i, int half) const {
    if constexpr (!CROSSED) {
      return *(const TG_LDS s16x8*)(lds + at[half] + i * 2048);
    } else {
      const TG_LDS char* const a = lds + at[i] + half * (ROWS * 64);
      const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TG_LDS s16x4*)a);
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TG_LDS s16x4*)(a + ROWS * 8));
      return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

template <int DT>
__device__ __forceinline__ f32x4 mm_mfma(s16x8 a, s16x8 b, f32x4 c) {
  if constexpr (DT == DT_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A tile of BM x BN by WM x WN waves.
template <int BM_, int BN_, int WM_, int WN_>
struct MmShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int STAGE = (BM + BN) * 128, LDS_BYTES = 2 * STAGE;
};

// The sums of a wave: c[i][j] holds, in lane l, row 16 i + (l & 15) and columns
// 16 j + 4 (l >> 4) + 0..3 of the wave's part.
template <class S>
struct MmSums {
  f32x4 c[S::FM][S::FN];
};

// `source(s, a, b)` names the operands of segment s; all straight (crossed) As have the stride
// sa, all Bs sb. k values in each of nseg segments. B's rows may come from two matrices, one
// for every other 16 (DUAL: source(s, a, b, b2), tile row 32 q + r < 16 from b, 16 more from b2, both
// at row 16 q + r of them; bj counts in rows of either).
template <class S, int DT, bool CA, bool CB, bool DUAL, class Source>
__device__ __forceinline__ void mm_tile(MmSums<S>& sums, TG_LDS char* lds, const Source& source, int nseg, int64_t k,
                                        int64_t ai, int64_t bj, uint32_t sa, uint32_t sb) {
  static_assert(!DUAL || !CB, "two matrices by turns: straight ones");
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6);
  using LA = MmLoader<S::BM, S::WAVES, CA>;
  using LB = MmLoader<S::BN, S::WAVES, CB>;
  LA la;
  LB lb, lb2;
  la.init(wave, lane, sa);
  lb.init(wave, lane, sb);
  if constexpr (DUAL) {
    // tile row 8 q + lane / 8 of transfer q: matrix (q >> 1) & 1, its row 16 (q >> 2) + 8 (q & 1) + lane / 8
#pragma unroll
    for (int i = 0; i < LB::PER; ++i) {
      const int q = wave * LB::PER + i;
      lb.v[i] -= (uint32_t)(q * 8 - (16 * (q >> 2) + 8 * (q & 1))) * (sb * 2);
    }
  }
  MmReader<S::BM, S::FM, CA> ra;
  MmReader<S::BN, S::FN, CB> rb;
  const int wm = wave / S::WN, wn = wave % S::WN;
  ra.init(wm * S::FM * 16, lane);
  rb.init(wn * S::FN * 16, lane);
#pragma unroll
  for (int i = 0; i < S::FM; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j) sums.c[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int64_t per_seg = (k + 63) >> 6, total = per_seg * nseg;
  if (total <= 0) return;
  int seg = 0;
  int64_t rem = 0;
  auto begin = [&](int s) {
    MmOperand a, b, b2;
    source(s, a, b, b2);
    la.start(a, ai);
    if constexpr (DUAL && LB::PER == 2) lb.start(wave & 1 ? b2 : b, bj);
    else lb.start(b, bj);
    if constexpr (DUAL && LB::PER == 4) lb2.start(b2, bj);
    rem = k;
  };
  constexpr int LOADS = LA::PER + LB::PER;
  auto issue = [&](int buf) {
    TG_LDS char* const l = lds + buf * S::STAGE;
    const uint32_t r = (uint32_t)(rem < 64 ? rem : 64);
    la.issue(l, wave, r);
    if constexpr (!DUAL || LB::PER == 2) {
      lb.issue(l + LA::BYTES, wave, r);
    } else {
      // a wave's four transfers: two from either matrix (of two, every other wave's from one)
      static_assert(LB::PER == 4, "a wave's transfers end where the matrices change");
#pragma unroll
      for (int i = 0; i < 4; ++i) lb2.v[i] = lb.v[i];
      lb2.k_of_lane = lb.k_of_lane;
      lb.template issue<0, 2>(l + LA::BYTES, wave, r);
      lb2.template issue<2, 2>(l + LA::BYTES, wave, r);
    }
    rem -= 64;
    if (rem > 0) {
      la.next(sa);
      lb.next(sb);
      if constexpr (DUAL && LB::PER == 4) lb2.next(sb);
    } else if (++seg < nseg) {
      begin(seg);
    }
  };
  begin(0);
  issue(0);
  if (total > 1) issue(1);
  for (int64_t t = 0; t < total; ++t) {
    if (t + 1 < total) wait_vm<LOADS>();
    else wait_vm<0>();
    lds_barrier();
    const TG_LDS char* const l = lds + (t & 1) * S::STAGE;
    s16x8 fa[S::FM], fb[S::FN];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < S::FN; ++j) fb[j] = rb.get(l + LA::BYTES, j, h);
#pragma unroll
      for (int i = 0; i < S::FM; ++i) fa[i] = ra.get(l, i, h);
#pragma unroll
      for (int i = 0; i < S::FM; ++i)
#pragma unroll
        for (int j = 0; j < S::FN; ++j) sums.c[i][j] = mm_mfma<DT>(fb[j], fa[i], sums.c[i][j]);
    }
    lds_barrier();
    if (t + 2 < total) issue((int)(t & 1));
  }
}

// Workgroup b of n to a place in the order of tiles, so that each of the eight XCDs (workgroups
// go to them by turns) walks a run of neighbours, which share operands in its L2.
__device__ __forceinline__ uint32_t xcd_order(uint32_t b, uint32_t n) {
  const uint32_t x = b & 7u, y = b >> 3, q = n >> 3, r = n & 7u;
  return x * q + (x < r ? x : r) + y;
}
// Place t of a grid of ni x nj tiles, eight rows of tiles at a time.
__device__ __forceinline__ void tile_at(uint32_t t, uint32_t ni, uint32_t nj, uint32_t& i, uint32_t& j) {
  const uint32_t band = t / (8 * nj), first = band * 8, rows = ni - first < 8 ? ni - first : 8;
  const uint32_t in = t - first * nj;
  i = first + in % rows;
  j = in / rows;
}

}  // namespace tg
