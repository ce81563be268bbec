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
// avoided by permuting what each lane fetches: a straight row's 16-byte pieces by the row's
// low bits, a crossed row's 32-byte pairs by those bits of k in which the 32 lanes of a
// read differ.
//
// k may run over several segments, each with operands of its own: a value held in two or three
// 16-bit parts is multiplied by naming its parts' products one after another (the smallest
// first), and [dg du] [Wg; Wu] without laying the weights together.
#pragma once
#include <type_traits>

#include "tg_common.h"

namespace tg {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#define TG_LDS __attribute__((address_space(3)))
// what a host program computes too, to check what a tile reads against its operands
#define TG_BOTH __host__ __device__ __forceinline__

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

TG_BOTH uint32_t uniform(uint32_t x) {
#if __HIP_DEVICE_COMPILE__
  x = __builtin_amdgcn_readfirstlane(x);
#endif
  return x;
}

// Waits until at most N of this wave's transfers are under way. The compiler knows nothing of
// them: no read of LDS may move across.
template <int N>
__device__ __forceinline__ void wait_vm() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
  __asm__ volatile("" ::: "memory");
}

// Waits for this wave's reads and writes of LDS.
__device__ __forceinline__ void wait_lds() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __asm__ volatile("" ::: "memory");
}

// One operand's way into LDS: ROWS rows (or columns of C) by K values of k, PER transfers of
// 1 KB for each of WAVES waves.
template <int ROWS, int K, int WAVES, bool CROSSED>
struct MmLoader {
  static constexpr int BYTES = ROWS * K * 2;
  static constexpr int PER = BYTES / 1024 / WAVES;
  static constexpr int PIECES = K / 8;   // of a straight row
  static_assert(PER * 1024 * WAVES == BYTES, "the waves share the transfers evenly");
  uint32_t v[PER];       // lane's byte offsets from the stage's first byte
  uint32_t k_of_lane;    // of the lane's piece within the stage (crossed: of the first transfer)
  u32x4 rs;              // buffer resource from the segment's first byte (or a later one) to the operand's end
  uint32_t at;           // the stage's first byte there

  // BY_TURNS: the operand holds every other 16 of the tile's rows; of 32 of its rows 0..3, 8..11, ..
  // are in the first 16 that it holds of 64, the others in the second: a lane's sums of the
  // two blocks are those of eight rows on end
  template <bool BY_TURNS = false>
  TG_BOTH void init(int wave, int lane, uint32_t stride) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int q = wave * PER + i;
      if constexpr (!CROSSED) {
        constexpr int LINES = 64 / PIECES;   // of a transfer
        const int r = lane / PIECES;
        k_of_lane = (uint32_t)(((lane % PIECES) ^ turn_row(r)) * 8);
        const int row = q * LINES + r;
        const int of = (row >> 6) * 32 + ((row >> 2) & 3) * 8 + ((row >> 5) & 1) * 4 + (row & 3);
        v[i] = (uint32_t)(BY_TURNS ? of : row) * (stride * 2) + k_of_lane * 2;
      } else {
        constexpr int LANES = ROWS / 8;   // of one k
        const int k = q * (64 / LANES) + lane / LANES, c = lane % LANES;
        v[i] = (uint32_t)k * (stride * 2) + (uint32_t)(c ^ (turn(k) << 1)) * 16;
        if (i == 0) k_of_lane = (uint32_t)k;
      }
    }
  }
  // straight: how a row's pieces are permuted; crossed: how a k's pairs are
  __host__ __device__ static constexpr int turn_row(int r) { return K == 64 ? r & 7 : (r >> 1) & 3; }
  __host__ __device__ static constexpr int turn(int k) { return ((k & 3) | (((k >> 3) & 1) << 2)) & (ROWS / 16 - 1); }

  // from row `row` and value `k` of k on, both inside the operand
  TG_BOTH void start(const MmOperand& o, int64_t row, int64_t k) {
    const int64_t skip = (CROSSED ? row + k * o.stride : row * o.stride + k) * 2;
    resource((uint64_t)o.p + (uint64_t)skip, ((o.lines - 1) * (int64_t)o.stride + o.len) * 2 - skip);
  }
  // (What lies behind the operand is none of it. The check takes the stage's offset off the size, so
  // that may not pass it: k ends where the operand's lines do.)
  TG_BOTH void resource(uint64_t from, int64_t left) {
    rs[0] = uniform((uint32_t)from);
    rs[1] = uniform((uint32_t)(from >> 32)) & 0xFFFFu;
    rs[2] = uniform(left <= 0 ? 0u : left >> 32 ? 0xFFFFFFF0u : (uint32_t)left);
    rs[3] = 0x00020000u;
    at = 0;
  }
  TG_BOTH void next(const MmOperand& o, uint32_t stride) {
    at += (CROSSED ? uniform(stride) : 1) * (K * 2);
    if (CROSSED && at >= 0x40000000u) {   // 32 bits do not reach through a long operand
      const uint64_t from = (((uint64_t)rs[1] << 32) | rs[0]) + at;
      resource(from, (int64_t)((uint64_t)o.p + (uint64_t)(((o.lines - 1) * (int64_t)o.stride + o.len) * 2) - from));
    }
  }
  // the lane's offset in transfer i of a stage of which only `rem` values of k are there
  TG_BOTH uint32_t offset(int i, int rem) const {
    return (int)k_of_lane + (CROSSED ? i * (512 / ROWS) : 0) < rem ? v[i] : 0xFFFFFFF0u;
  }
  // Whether transfer i is of the second matrix of two that alternate.
  __device__ static constexpr bool second(int i) { return ((i * (64 / PIECES)) >> 4) & 1; }

  // The transfers (BY_TURNS: those of one matrix) of a stage; PART: only `rem` values of k of it are
  // there. Written as instructions: the compiler would wait for all transfers before any read of LDS.
  template <bool PART, bool BY_TURNS = false, bool SECOND = false>
  __device__ __forceinline__ void issue(uint32_t lds, int wave, int rem) const {
    bool first = true;
    lds += (uint32_t)(wave * PER) * 1024u;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (BY_TURNS && second(i) != SECOND) continue;
      const uint32_t o = PART ? offset(i, rem) : v[i];
      // a scalar register that the vector unit wrote takes five states to reach a transfer
      if (first)
        __asm__ volatile("s_add_u32 m0, %0, %4\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                         ::"s"(lds), "v"(o), "s"(rs), "s"(at), "i"(i * 1024)
                         : "memory", "scc");
      else
        __asm__ volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                         ::"s"(lds), "v"(o), "s"(rs), "s"(at), "i"(i * 1024)
                         : "memory", "scc");
      first = false;
    }
  }
};

// One operand's fragments: a wave's N blocks of 16 rows from `row` (a multiple of 16 N) on.
template <int ROWS, int K, int N, bool CROSSED>
struct MmReader {
  uint32_t at[CROSSED ? N : K / 32];

  __device__ __forceinline__ void init(int row, int lane) {
    using L = MmLoader<ROWS, K, 1, CROSSED>;
    const int r = lane & 15, kg = lane >> 4;
    if constexpr (!CROSSED) {
      at[0] = (uint32_t)((row + r) * (K * 2) + ((kg ^ L::turn_row(r)) * 16));
      if constexpr (K == 64) at[1] = at[0] ^ 64;
    } else {
      const int k = kg * 8 + (r >> 2);
#pragma unroll
      for (int i = 0; i < N; ++i)
        at[i] = (uint32_t)(k * (ROWS * 2) + (((row >> 4) + i) ^ L::turn(k)) * 32 + (r & 3) * 8);
    }
  }
  // block i, the 32 values of k from 32 part on
  __device__ __forceinline__ s16x8 get(const TG_LDS char* lds, int i, int part) const {
    if constexpr (!CROSSED) {
      return *(const TG_LDS s16x8*)(lds + at[part] + i * (K * 32));
    } else {
      const TG_LDS char* const a = lds + at[i] + part * (ROWS * 64);
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

// How the waves of a workgroup share a tile.
//   MM_TURNS  eight waves, each a part of the tile over all of k, in two groups that read
//             fragments and multiply by turns: one wave of either group is on each SIMD, so the
//             matrix instructions of one run while the other waits for LDS.
//   MM_EVEN   four waves, each a part of the tile over all of k; two workgroups fit a CU and
//             overlap by themselves.
//   MM_ALONE  four waves, each the whole tile over a quarter of k, from stages of its own and
//             without a barrier; their sums are added at the end. For few tiles and long sums.
//   MM_AHEAD  each wave a part of the tile over all of k; it reads the fragments of one half of a
//             stage while it multiplies the other's, the next stage's among them. For tiles whose
//             workgroups have a CU to themselves or share it with one (2048 x 2048 x 2048 by 128 x 128:
//             27.6 us MM_EVEN, 25.9 so; by 64 x 64: 47.9 MM_ALONE, 34.4 so).
enum MmMode { MM_TURNS, MM_EVEN, MM_ALONE, MM_AHEAD };

// A tile of BM x BN by WM x WN waves, in stages of K values of k of which STAGES fit. FM x FN: a
// wave's blocks of 16 x 16, as it ends with them.
// Four stages of 32 keep a transfer in flight for two stages' products; two of 64 fetch straight
// rows by whole cache lines and have half the barriers (MM_TURNS, 8192 x 8192 x 8192: 1014 us with
// four of 32, 1032 with two of 64; MM_EVEN, 18 Grams of 1024 x 4096: 148 and 136).
template <int BM_, int BN_, int WM_, int WN_, MmMode MODE_, int K_, int STAGES_>
struct MmShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr MmMode MODE = MODE_;
  static constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int K = K_, STAGES = STAGES_;
  static constexpr int STAGE = (BM + BN) * K * 2;
  static constexpr int LDS_BYTES = STAGES * STAGE * (MODE == MM_ALONE ? WAVES : 1);
};
using MmBig = MmShape<256, 256, 2, 4, MM_TURNS, 32, 4>;
using MmHalf = MmShape<128, 256, 1, 4, MM_EVEN, 32, 3>;
using MmMid = MmShape<128, 128, 2, 2, MM_EVEN, 64, 2>;
using MmDeep = MmShape<128, 128, 2, 4, MM_AHEAD, 64, 4>;
using MmNear = MmShape<64, 64, 2, 2, MM_AHEAD, 64, 4>;
using MmNearRows = MmShape<64, 64, 4, 1, MM_AHEAD, 64, 4>;   // whole rows of the tile in a wave
using MmSmall = MmShape<64, 64, 4, 1, MM_ALONE, 32, 4>;

// The sums of a wave: c[i][j] holds, in lane l, row 16 i + (l & 15) and columns
// 16 j + 4 (l >> 4) + 0..3 of the wave's part.
template <class S>
struct MmSums {
  f32x4 c[S::FM][S::FN];
};

// `source(s, a, b, b2)` names the operands of segment s; all straight (crossed) As have the
// stride sa, all Bs sb. k values in each of nseg segments. B's rows may come from two matrices
// (DUAL): 16 by turns, as MmLoader's init has them; bj counts in rows of either. Of `splits` parts of every segment's k only part `split` is summed.
template <class S, int DT, bool CA, bool CB, bool DUAL, class Source>
__device__ __forceinline__ void mm_tile(MmSums<S>& sums, TG_LDS char* lds, const Source& source, int nseg, int64_t k,
                                        int64_t ai, int64_t bj, uint32_t sa, uint32_t sb, uint32_t split = 0,
                                        uint32_t splits = 1) {
  static_assert(!DUAL || !CB, "two matrices by turns: straight ones");
  constexpr bool ALONE = S::MODE == MM_ALONE;
  constexpr int LOADERS = ALONE ? 1 : S::WAVES;
  constexpr int FM = ALONE ? S::BM / 16 : S::FM, FN = ALONE ? S::BN / 16 : S::FN;   // while summing
  constexpr int STAGES = S::STAGES, K = S::K;
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6);
  const int loader = ALONE ? 0 : wave;
  using LA = MmLoader<S::BM, K, LOADERS, CA>;
  using LB = MmLoader<S::BN, K, LOADERS, CB>;
  constexpr int LOADS = LA::PER + LB::PER;
  // of two matrices by turns a wave's transfers are whole pairs of blocks, or one block
  constexpr bool ONE = DUAL && LB::PER * (64 / LB::PIECES) == 16;
  static_assert(!DUAL || ONE || LB::PER * (64 / LB::PIECES) % 32 == 0, "whole blocks");
  LA la;
  LB lb, lb2;
  la.init(loader, lane, sa);
  lb.template init<DUAL>(loader, lane, sb);
  if constexpr (DUAL && !ONE) lb2 = lb;
  MmReader<S::BM, K, FM, CA> ra;
  MmReader<S::BN, K, FN, CB> rb;
  const int wm = ALONE ? 0 : wave / S::WN, wn = ALONE ? 0 : wave % S::WN;
  ra.init(wm * FM * 16, lane);
  rb.init(wn * FN * 16, lane);
  f32x4 c[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) c[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // this wave's k of every segment
  const uint32_t pieces = splits * (ALONE ? S::WAVES : 1);
  const int64_t piece = (k + K * pieces - 1) / (K * pieces) * K;
  const int64_t from = (ALONE ? split * S::WAVES + wave : split) * piece;
  const int64_t many = k - from < piece ? k - from : piece;
  if constexpr (ALONE) lds += wave * (STAGES * S::STAGE);
  const int total = many > 0 ? (int)((many + K - 1) / K) * nseg : 0;
  const uint32_t lds0 = uniform((uint32_t)(uintptr_t)lds);
  int seg = 0, issued = 0, rem = 0;
  uint32_t into = 0;       // where the next stage goes
  MmOperand oa, ob, ob2;
  auto begin = [&](int s) {
    source(s, oa, ob, ob2);
    la.start(oa, ai, from);
    lb.start(ONE && (loader & 1) ? ob2 : ob, bj, from);
    if constexpr (DUAL && !ONE) lb2.start(ob2, bj, from);
    rem = (int)many;
  };
  auto after = [&](uint32_t at) { return at == (STAGES - 1) * S::STAGE ? 0u : at + S::STAGE; };
  auto transfers = [&](auto part, uint32_t l) {
    constexpr bool PART = decltype(part)::value;
    la.template issue<PART>(l, loader, rem);
    if constexpr (!DUAL || ONE) {
      lb.template issue<PART>(l + LA::BYTES, loader, rem);
    } else {
      lb.template issue<PART, true, false>(l + LA::BYTES, loader, rem);
      lb2.template issue<PART, true, true>(l + LA::BYTES, loader, rem);
    }
  };
  auto issue = [&]() {
    const uint32_t l = lds0 + into;
    into = after(into);
    ++issued;
    if (rem >= K) transfers(std::false_type{}, l);
    else transfers(std::true_type{}, l);
    rem -= K;
    if (rem > 0) {
      la.next(oa, sa);
      lb.next(ONE && (loader & 1) ? ob2 : ob, sb);
      if constexpr (DUAL && !ONE) lb2.next(ob2, sb);
    } else if (++seg < nseg) {
      begin(seg);
    }
  };
  auto fragments = [&](uint32_t at, int part, s16x8 (&fa)[FM], s16x8 (&fb)[FN]) {
    const TG_LDS char* const l = lds + at;
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = rb.get(l + LA::BYTES, j, part);
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = ra.get(l, i, part);
  };
  auto multiply = [&](const s16x8 (&fa)[FM], const s16x8 (&fb)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) c[i][j] = mm_mfma<DT>(fb[j], fa[i], c[i][j]);
  };
  // waits until stage t has arrived
  auto arrived = [&](int t) {
    const int behind = issued - 1 - t;
    if (behind >= 3) wait_vm<3 * LOADS>();
    else if (behind == 2) wait_vm<2 * LOADS>();
    else if (behind == 1) wait_vm<LOADS>();
    else wait_vm<0>();
  };
  if (total > 0) begin(0);
  int t = 0;
  uint32_t at = 0;
  if constexpr (S::MODE == MM_TURNS) {
    // Phases between barriers:  group 0: read t    multiply  read t + 1  multiply
    //                           group 1:           read t    multiply    read t + 1  multiply
    // Stage t + 3 goes where t - 1 was, whose reads by both groups ended at a barrier before either
    // reads t; what a group reads in its next phase both have awaited before the barrier there.
    const int group = wave >> 2;
    for (int i = 0; i < 3; ++i)
      if (i < total) issue();
    arrived(0);
    lds_barrier();
    if (group) lds_barrier();
    auto product = [&](const s16x8 (&fa)[FM], const s16x8 (&fb)[FN]) {
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
      multiply(fa, fb);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      lds_barrier();
    };
    for (; t + 3 < total; ++t, at = after(at)) {
      // (crossed reads take longer than straight ones: transfers that wait for them come late;
      // 8192 x 8192 x 8192 with both operands crossed 1048 -> 990 us, straight 975 -> 993)
      s16x8 fa[FM], fb[FN];
      if (CA) issue();
      fragments(at, 0, fa, fb);
      if (!CA) issue();
      wait_vm<2 * LOADS>();
      product(fa, fb);
    }
    for (; t < total; ++t, at = after(at)) {
      s16x8 fa[FM], fb[FN];
      fragments(at, 0, fa, fb);
      arrived(t + 1);
      product(fa, fb);
    }
    if (!group) lds_barrier();
  } else if constexpr (S::MODE == MM_EVEN) {
    for (int i = 0; i < STAGES - 1; ++i)
      if (i < total) issue();
    for (; t < total; ++t, at = after(at)) {
      arrived(t);
      lds_barrier();       // every wave's part of this stage is there, and the one before is read
      if (issued < total) issue();
#pragma unroll
      for (int part = 0; part < K / 32; ++part) {
        s16x8 fa[FM], fb[FN];
        fragments(at, part, fa, fb);
        multiply(fa, fb);
      }
    }
  } else if constexpr (S::MODE == MM_AHEAD) {
    // Between the two halves of a stage a barrier: all waves have read it, and what each has awaited
    // of the next is there for all.
    static_assert(S::MODE != MM_AHEAD || K == 64, "two halves of a stage");
    for (int i = 0; i < STAGES; ++i)
      if (i < total) issue();
    s16x8 fa[2][FM], fb[2][FN];
    if (total > 0) {
      arrived(0);
      lds_barrier();
      fragments(at, 0, fa[0], fb[0]);
    }
    for (; t < total; ++t) {
      fragments(at, 1, fa[1], fb[1]);
      multiply(fa[0], fb[0]);
      if (t + 1 < total) arrived(t + 1);
      lds_barrier();
      if (issued < total) issue();
      at = after(at);
      fragments(at, 0, fa[0], fb[0]);      // behind the last: not used
      multiply(fa[1], fb[1]);
    }
  } else {
    // a stage's fragments are read while the one before is multiplied, and its place filled again
    // once they are there
    static_assert(!ALONE || (STAGES == 4 && K == 32), "at most three stages behind the one that is awaited");
    for (int i = 0; i < STAGES; ++i)
      if (i < total) issue();
    s16x8 fa[2][FM], fb[2][FN];
    if (total > 0) {
      arrived(0);
      fragments(at, 0, fa[0], fb[0]);
    }
    for (; t + STAGES + 1 < total; t += 2) {
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        wait_lds();
        issue();
        at = after(at);
        wait_vm<3 * LOADS>();
        fragments(at, 0, fa[o ^ 1], fb[o ^ 1]);
        multiply(fa[o], fb[o]);
      }
    }
    for (; t < total; ++t) {
      wait_lds();
      if (issued < total) issue();
      at = after(at);
      if (t + 1 < total) arrived(t + 1);
      fragments(at, 0, fa[1], fb[1]);      // behind the last: not used
      multiply(fa[0], fb[0]);
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[0][i] = fa[1][i];
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[0][j] = fb[1][j];
    }
  }
  if constexpr (!ALONE) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) sums.c[i][j] = c[i][j];
  } else {
    // every wave's sums to LDS; wave w then adds those of its row of blocks, in the waves' order
    lds -= wave * (STAGES * S::STAGE);
    lds_barrier();
    TG_LDS f32x4* const all = (TG_LDS f32x4*)lds;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) all[((wave * FM + i) * FN + j) * 64 + lane] = c[i][j];
    lds_barrier();
    static_assert(S::FM * S::WAVES == FM && S::FN == FN, "a row of blocks for each wave");
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      f32x4 s = all[(wave * FN + j) * 64 + lane];
#pragma unroll
      for (int w = 1; w < S::WAVES; ++w) s += all[((w * FM + wave) * FN + j) * 64 + lane];
      sums.c[0][j] = s;
    }
  }
}

// At most so many workgroups share sums in a launch, at most so many those of a tile.
constexpr uint32_t MM_MOST_SPLIT = 512, MM_MOST_SPLITS = 8;
// Bytes of the counters and the sums.
inline uint64_t mm_split_bytes(uint64_t tiles, uint64_t splits, uint64_t side) {
  return splits > 1 ? MM_MOST_SPLIT * 4 + tiles * splits * side * side * 4 : 0;
}

// Leaves this workgroup's sums to the last of its tile, which adds all in their order: true for that
// one, and its sums are the whole. Behind MM_MOST_SPLIT counters (zero, and so again when it ends) lie the
// tiles' sums, a tile's one after another. The sums pass the L2s,
// which the XCDs do not share, by accesses of agent scope; every wave waits until its own are
// there before the workgroup is counted. (A release and an acquire around plain accesses write back
// and empty an XCD's L2 for all its workgroups: 777 x 2051 in fp16 took 1057 us with them.)
template <class S>
__device__ __forceinline__ bool whole_sums(MmSums<S>& sums, uint32_t* counters, uint32_t tile, uint32_t split, uint32_t splits,
                                           TG_LDS char* lds) {
  if (splits == 1) return true;
  TG_LDS uint32_t* const before = (TG_LDS uint32_t*)lds;   // what was there has been read
  constexpr uint32_t EACH = S::FM * S::FN * S::THREADS * 2;
  uint64_t* const all = (uint64_t*)(counters + MM_MOST_SPLIT) + (uint64_t)tile * splits * EACH + threadIdx.x;
#pragma unroll
  for (int i = 0; i < S::FM; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x2 v = {sums.c[i][j][2 * h], sums.c[i][j][2 * h + 1]};
        __hip_atomic_store(all + split * EACH + ((i * S::FN + j) * 2 + h) * S::THREADS, __builtin_bit_cast(uint64_t, v),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
  wait_vm<0>();
  __syncthreads();
  if (threadIdx.x == 0) *before = __hip_atomic_fetch_add(counters + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (*before != splits - 1) return false;
  if (threadIdx.x == 0) __hip_atomic_store(counters + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int i = 0; i < S::FM; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j) sums.c[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (uint32_t q = 0; q < splits; ++q)
#pragma unroll
    for (int i = 0; i < S::FM; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x2 v = __builtin_bit_cast(f32x2, __hip_atomic_load(all + q * EACH + ((i * S::FN + j) * 2 + h) * S::THREADS,
                                                                      __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
          sums.c[i][j][2 * h] += v[0];
          sums.c[i][j][2 * h + 1] += v[1];
        }
  return true;
}

// A matrix around a tile, for what follows a product. Loads and stores at byte offsets from `first`
// (of one lane, and of all together) happen where `in` holds; loads give zeros elsewhere. Through a
// buffer resource that takes no branch, and the loads of many blocks go out together.
struct MmWindow {
  __amdgpu_buffer_rsrc_t rs;
  __device__ __forceinline__ explicit MmWindow(const void* first)
      : rs(__builtin_amdgcn_make_buffer_rsrc(
            (void*)((uint64_t)uniform((uint32_t)((uint64_t)first >> 32)) << 32 | uniform((uint32_t)(uint64_t)first)), 0,
            0x80000000u, 0x20000)) {}
  __device__ static __forceinline__ uint32_t at(bool in, uint32_t lane) { return in ? lane : 0xFFFFFFF0u; }
  __device__ __forceinline__ uint16_t load2(bool in, uint32_t lane, uint32_t all) const {
    return __builtin_amdgcn_raw_buffer_load_b16(rs, at(in, lane), all, 0);
  }
  __device__ __forceinline__ uint32_t load4(bool in, uint32_t lane, uint32_t all) const {
    return __builtin_amdgcn_raw_buffer_load_b32(rs, at(in, lane), all, 0);
  }
  __device__ __forceinline__ u32x2 load8(bool in, uint32_t lane, uint32_t all) const {
    return __builtin_amdgcn_raw_buffer_load_b64(rs, at(in, lane), all, 0);
  }
  __device__ __forceinline__ u32x4 load16(bool in, uint32_t lane, uint32_t all) const {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, at(in, lane), all, 0);
  }
  __device__ __forceinline__ void store2(uint16_t v, bool in, uint32_t lane, uint32_t all) const {
    __builtin_amdgcn_raw_buffer_store_b16(v, rs, at(in, lane), all, 0);
  }
  __device__ __forceinline__ void store4(uint32_t v, bool in, uint32_t lane, uint32_t all) const {
    __builtin_amdgcn_raw_buffer_store_b32(v, rs, at(in, lane), all, 0);
  }
  __device__ __forceinline__ void store8(u32x2 v, bool in, uint32_t lane, uint32_t all) const {
    __builtin_amdgcn_raw_buffer_store_b64(v, rs, at(in, lane), all, 0);
  }
  // (The offset is one register: with a scalar one beside it the compiler lets the next instruction
  // write the stored registers, and the store then takes some of the new values.)
  __device__ __forceinline__ void store16(u32x4 v, bool in, uint32_t lane, uint32_t all) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, rs, at(in, lane + all), 0, 0);
  }
};

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
