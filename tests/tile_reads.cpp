// What the tiles of mm_tile.h read, lane by lane, on the host: the loaders' own offsets and resources
// against the operands, for the products of the gated linear layer and of Newton-Schulz. A buffer
// access is taken to happen where its offset is below the resource's size less the scalar offset, as
// 32 bits without a sign: one that is larger than the size lets every lane pass.
#include <stdio.h>

#include "gated.h"

using namespace tg;

static long failures = 0;
static const char* what = "";
static int64_t sizes[3];

// One loader over `many` values of k from (row, from) on.
template <class L, int K, bool BY_TURNS>
static void walk(const MmOperand& o, int64_t row, int64_t from, int64_t many, int waves) {
  const uint64_t begin = (uint64_t)o.p, end = begin + (uint64_t)((o.lines - 1) * (int64_t)o.stride + o.len) * 2;
  for (int wave = 0; wave < waves; ++wave)
    for (int lane = 0; lane < 64; ++lane) {
      L l;
      l.template init<BY_TURNS>(wave, lane, o.stride);
      l.start(o, row, from);
      for (int64_t rem = many; rem > 0;) {
        for (int i = 0; i < L::PER; ++i) {
          const uint32_t off = rem < K ? l.offset(i, (int)rem) : l.v[i];
          if (off >= l.rs[2] - l.at) continue;
          const uint64_t at = ((uint64_t)l.rs[1] << 32 | l.rs[0]) + l.at + off;
          if (at >= begin && at + 16 <= end) continue;
          if (failures++ < 5)
            printf("%s %lld %lld %lld: row %lld, k %lld of %lld: %lld bytes behind the operand\n", what,
                   (long long)sizes[0], (long long)sizes[1], (long long)sizes[2], (long long)row,
                   (long long)(from + many - rem), (long long)many, (long long)(at + 16 - end));
        }
        rem -= K;
        if (rem > 0) l.next(o, o.stride);
      }
    }
}

// Both operands of a tile at (ai, bj), as mm_tile() divides k.
template <class S, bool CA, bool CB, bool DUAL>
static void tile(const MmOperand& a, const MmOperand& b, int64_t k, int64_t ai, int64_t bj, int splits) {
  constexpr bool ALONE = S::MODE == MM_ALONE;
  constexpr int LOADERS = ALONE ? 1 : S::WAVES, K = S::K;
  const int pieces = splits * (ALONE ? S::WAVES : 1);
  const int64_t piece = (k + K * pieces - 1) / (K * pieces) * K;
  for (int p = 0; p < pieces; ++p) {
    const int64_t from = p * piece, many = k - from < piece ? k - from : piece;
    if (many <= 0) continue;
    walk<MmLoader<S::BM, K, LOADERS, CA>, K, false>(a, ai, from, many, LOADERS);
    walk<MmLoader<S::BN, K, LOADERS, CB>, K, DUAL>(b, bj, from, many, LOADERS);
  }
}
template <class S, bool CA, bool CB>
static void tiles(const MmOperand& a, const MmOperand& b, int64_t k, int64_t ni, int64_t nj, int splits) {
  for (int64_t i = 0; i < ni; i += S::BM)
    for (int64_t j = 0; j < nj; j += S::BN) tile<S, CA, CB, false>(a, b, k, i, j, splits);
}

static char* const kAt = (char*)0x7f0000001000;
static GatedParts parts(int64_t lines, uint32_t cols, bool lies, uint32_t gap) {
  const uint32_t pad = gated_pad(cols);
  return lies ? GatedParts{kAt, lines, 0, cols, lines <= 1 ? cols : cols + gap} : GatedParts{kAt, lines, lines * pad, pad, pad};
}
static MmOperand whole(const GatedParts& m) { return {m.p, m.lines, m.len, m.stride}; }

template <class S>
static void gate_and_up(const GatedParts& x, const GatedParts& w, int64_t rows, uint32_t hidden, bool grads) {
  const uint32_t n = grads ? gated_pad(hidden) : hidden;
  for (uint32_t f0 = 0; f0 < n; f0 += S::BN / 2)
    if (const uint32_t k = gated_sum(x, w, f0, hidden))
      for (int64_t i = 0; i < rows; i += S::BM) tile<S, false, false, true>(whole(x), whole(w), k, i, f0, 1);
}
template <class S>
static void gated_behind(const GatedParts& x, const GatedParts& w, int64_t rows, uint32_t in, uint32_t hidden) {
  const uint32_t pad = gated_pad(hidden);
  for (int splits = 1; splits < (S::MODE == MM_AHEAD ? 4 : 2); ++splits) {
    const MmOperand g{kAt, rows, pad, 2 * pad}, both{kAt, rows, 2 * pad, 2 * pad};
    what = "dx";
    tiles<S, false, true>(g, whole(w), hidden, rows, in, splits);
    what = "dw";
    tiles<S, true, true>(both, whole(x), rows, 2 * pad, in, splits);
  }
}

static void gated(int64_t rows, uint32_t in, uint32_t hidden) {
  sizes[0] = rows, sizes[1] = in, sizes[2] = hidden;
  const bool may = in % 8 == 0;
  for (int lies = 0; lies < (may ? 4 : 1); ++lies) {
    const GatedParts x = parts(rows, in, lies & 1, 8), w = parts(hidden, in, lies & 2, 0);
    what = "gradients of gate and up";
    gate_and_up<MmBig>(x, w, rows, hidden, true);
    gate_and_up<MmMid>(x, w, rows, hidden, true);
    gate_and_up<MmSmall>(x, w, rows, hidden, true);
    gate_and_up<MmNearRows>(x, w, rows, hidden, true);
    what = "gate and up";
    gate_and_up<MmHalf>(x, w, rows, hidden, false);
    gate_and_up<MmSmall>(x, w, rows, hidden, false);
    gated_behind<MmBig>(x, w, rows, in, hidden);
    gated_behind<MmMid>(x, w, rows, in, hidden);
    gated_behind<MmSmall>(x, w, rows, in, hidden);
    gated_behind<MmNear>(x, w, rows, in, hidden);
  }
}

static uint32_t line(uint32_t n) { return n >= 256 ? (n + 63u) & ~63u : (n + 7u) & ~7u; }
template <class S>
static void newton_schulz(uint32_t rows, uint32_t cols) {
  const uint32_t m = rows < cols ? rows : cols, ldx = line(cols), ldm = line(m);
  const MmOperand x{kAt, rows, ldx, ldx}, a{kAt, m, ldm, ldm};
  const int most = S::MODE == MM_TURNS ? 1 : 3;
  for (int splits = 1; splits <= most; ++splits) {
    what = "A";
    if (rows <= cols) tiles<S, false, false>(x, x, (cols + 7) & ~7u, m, m, splits);
    else tiles<S, true, true>(x, x, rows, m, m, splits);
    what = "B";
    tiles<S, false, false>(a, a, (m + 7) & ~7u, m, m, splits);
    what = "X";
    if (rows <= cols) tiles<S, false, true>(a, x, m, rows, cols, splits);
    else tiles<S, false, false>(x, a, (cols + 7) & ~7u, rows, cols, splits);
  }
}

// dg and du in two parts never meet the kernel of 256 x 256 tiles, which writes one.
static void two_parts_in_small_tiles() {
  what = "two parts in the largest tiles";
  for (int64_t rows = 1; rows <= 1 << 19; rows += rows < 600 ? 1 : rows / 7)
    for (int64_t hidden = 1; hidden <= 1 << 19; hidden += hidden < 300 ? 1 : hidden / 7)
      for (int64_t in : {1, 8, 512, 1024, 1025, 1 << 19})
        if (gated_grad_parts(rows, in, hidden, DT_BF16) == 2 && gated_tile(rows, hidden, in, true) == 0 && failures++ < 5)
          printf("%s: %lld %lld %lld\n", what, (long long)rows, (long long)in, (long long)hidden);
}

int main() {
  two_parts_in_small_tiles();
  for (int64_t rows : {1, 70, 300})
    for (uint32_t in : {1u, 8u, 65u, 136u, 264u, 320u, 333u, 520u})
      for (uint32_t hidden : {1u, 33u, 64u, 129u, 257u, 264u, 288u, 289u, 330u}) gated(rows, in, hidden);
  for (uint32_t rows : {1u, 129u, 260u, 333u})
    for (uint32_t cols : {7u, 130u, 257u, 520u}) {
      sizes[0] = rows, sizes[1] = cols, sizes[2] = 0;
      newton_schulz<MmBig>(rows, cols);
      newton_schulz<MmMid>(rows, cols);
      newton_schulz<MmDeep>(rows, cols);
      newton_schulz<MmNear>(rows, cols);
    }
  printf("%ld failures\n", failures);
  return failures != 0;
}
