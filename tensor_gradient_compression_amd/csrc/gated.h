// Gated linear layer: what the host side (gated.hip) and the kernels (k_gated.hip,
// k_gated_bwd.hip) share. gfx950 only.
#pragma once
#include "mm_tile.h"

namespace tg {

constexpr int64_t kMostThreads = 0xFFFFFFFF;   // of a launch

enum GatedAct { GATED_SILU = 0, GATED_GELU, GATED_SIGMOID, GATED_RELU, GATED_ACTS };

// A matrix in the parts that the products take: one of its own 16-bit values, or three of bf16
// that add up to an fp32 value, `part` values apart.
struct GatedParts {
  const void* p;
  int64_t lines, part;
  uint32_t len, stride;
};
// Products of parts, the smallest first: A's and B's part of segment s (of 6; the last alone
// for 16-bit values).
constexpr uint32_t GATED_PART_A = 0x001102, GATED_PART_B = 0x010120;

// (long lines are whole cache lines, which the tiles' transfers take in halves)
__host__ __device__ inline uint32_t gated_pad(uint32_t n) { return n >= 256 ? (n + 63u) & ~63u : (n + 7u) & ~7u; }

// Copies of rows whose lines are not 16-byte aligned (16 bits), or their parts (fp32).
struct GatedPack {
  const void* src;
  int64_t rows, stride;
  uint32_t cols;
  int dt;
  void* dst;          // rows of gated_pad(cols) values, zeros behind; fp32: three times
};
hipError_t launch_gated_pack(const GatedPack* a, int n, hipStream_t s);

// Values of k that the tile of g and u from column f0 of the weights on sums over: those that the lines of
// both x and the weights have (a copy's padding may pass the end of a line that goes as it lies), and none
// behind the weights, where the gradients have tiles for their padding alone.
__host__ __device__ inline uint32_t gated_sum(const GatedParts& x, const GatedParts& w, uint32_t f0, uint32_t hidden) {
  return f0 >= hidden ? 0 : x.len < w.len ? x.len : w.len;
}

struct GatedArgs {
  GatedParts x, wg, wu;
  const void* bg;      // may be NULL: 0
  const void* bu;
  int64_t rows;
  uint32_t in, hidden;
  int dt, act;
  // forward
  void* y;
  // backward: dg and du side by side, rows of 2 gated_pad(hidden) values, `parts` times
  const void* dy;
  int64_t dy_stride;
  void* grads;
  int parts;
  uint32_t* counters;  // or NULL: cleared for the products behind
  float* row_sums;     // or NULL: sums of dg and du over a tile's rows, as rows of 2 gated_pad(hidden)
};
hipError_t launch_gated_forward(const GatedArgs& a, hipStream_t s);
hipError_t launch_gated_grads(const GatedArgs& a, hipStream_t s);
// rows of row_sums
int64_t gated_sum_rows(int64_t rows, uint32_t in, uint32_t hidden);

// How a product behind is divided: a tile, and splits of its sum with what they need of memory:
// counters and sums that the last workgroup of a tile adds (counted), or a result for every split.
struct GatedWay {
  int tile, splits;
  bool counted;
  size_t bytes;
};
GatedWay gated_dx_way(int64_t rows, uint32_t in, uint32_t hidden, int parts);
GatedWay gated_dw_way(int64_t rows, uint32_t in, uint32_t hidden, int parts);

// The parts of dg and du that the products take. 16-bit ones are rounded once where they are many: the
// gradients are then sqrt(2) times as far off as their own rounding, since as many independent
// roundings as there are dg enter them. Few do not average (33 values: 1.55 times), nor do few results: up to
// 2^14 values, or 2^19 of which some result has up to 2^10, go in two parts, whose products are bound by
// their launches anyway. (None of them is of 256 x 256 tiles, whose kernel writes one part: 2^14 values are
// 129 such tiles at most, and where some result has 2^10 values `in` is not above 1024.)
inline int gated_grad_parts(int64_t rows, int64_t in, int64_t hidden, int dt) {
  if (dt == DT_F32) return 3;
  const int64_t n = rows * hidden, results = (rows < hidden ? rows : hidden) * in;
  return n <= 1 << 14 || (n <= 1 << 19 && results <= 1 << 10) ? 2 : 1;
}
// and the segments of a product with them
inline int gated_grad_segs(int parts) { return parts == 3 ? 6 : parts; }

// dx = dg Wg + du Wu
struct GatedDx {
  GatedParts grads, wg, wu;
  void* dx;
  int64_t rows;
  uint32_t in, hidden;
  int dt;
  int parts;           // of dg and du
  GatedWay way;
  void* sums;          // of way.bytes, if any
};
hipError_t launch_gated_dx(const GatedDx& a, hipStream_t s);

// dWg = dg^T x, dWu = du^T x, and the biases' gradients
struct GatedDw {
  GatedParts grads, x;
  void* dwg;
  void* dwu;
  void* dbg;           // may be NULL, together
  void* dbu;
  const float* row_sums;
  int64_t sum_rows;
  int64_t rows;
  uint32_t in, hidden;
  int dt;
  int parts;           // of dg and du
  GatedWay way;
  void* sums;          // of way.bytes, if any
};
hipError_t launch_gated_dw(const GatedDw& a, hipStream_t s);

// The tile of the products of g and u: 0: 256 x 256, 1: 128 x 128, 2 and 4: 64 x 64, 3: 128 x 256.
// 256 x 256 where its tiles fill the chip, smaller ones for short sums, whose epilogue is most of the
// time: two workgroups of a CU overlap theirs. 8192 rows to 8192 in bf16 with silu, forward and gradients in
// us, by 256 x 256 and by smaller tiles:  in = 256: 100, 211 and 91, 186;  512: 155, 257 and 152, 257;
// 1024: 250, 355 and 269, 371;  2048: 445, 544 and 496, 609;  4096: 865, 924 and 1007, 1095. The smaller one
// is of 128 x 256 forward (65536 x 256 x 1024: 170 us, 128 x 128 183) and of 128 x 128 for the gradients, which
// need more registers (128 x 256 283 us, 128 x 128 221).
// 64 x 64 for few tiles: by one workgroup a CU that splits the sum, or two that do not (768 x 2048 over
// 768, 384 tiles: 11.8 us and 9.2; 768 x 768 over 2048, 144 tiles: 10.6 and 13.0).
inline int gated_tile(int64_t rows, int64_t hidden, int64_t in, bool grads) {
  auto tiles = [&](int64_t t) { return ((rows + t - 1) / t) * ((2 * hidden + t - 1) / t); };
  if (tiles(256) >= 200) return in > 1024 ? 0 : grads ? 1 : 3;
  return tiles(128) >= 200 ? 1 : tiles(64) > 256 ? 4 : 2;
}

template <int DT> struct GatedType;
template <> struct GatedType<DT_F32> { using T = float; static constexpr int MM = DT_BF16, SEGS = 6; };
template <> struct GatedType<DT_F16> { using T = _Float16; static constexpr int MM = DT_F16, SEGS = 1; };
template <> struct GatedType<DT_BF16> { using T = bf16_t; static constexpr int MM = DT_BF16, SEGS = 1; };

// Segment s of SEGS: a part of a matrix from k0 on.
template <int SEGS>
__device__ __forceinline__ MmOperand gated_operand(const GatedParts& m, uint32_t parts, int s, int64_t k0, bool crossed) {
  const uint32_t part = (parts >> (4 * (SEGS == 1 ? 5 : s))) & 3u;
  MmOperand o;
  o.p = (const char*)m.p + (int64_t)part * m.part * 2 + (crossed ? k0 * m.stride : k0) * 2;
  o.lines = crossed ? m.lines - k0 : m.lines;
  o.len = crossed ? m.len : m.len - (uint32_t)k0;
  o.stride = m.stride;
  return o;
}

// The same of dg and du, of which 16-bit ones are in one part or two.
template <int SEGS>
__device__ __forceinline__ MmOperand gated_grad_operand(const GatedParts& m, int parts, int s, int64_t k0, bool crossed) {
  if constexpr (SEGS != 1) {
    return gated_operand<SEGS>(m, GATED_PART_A, s, k0, crossed);
  } else {
    GatedParts p = m;
    p.p = (const char*)p.p + (parts == 2 && s == 0 ? m.part * 2 : 0);   // the lower part first
    return gated_operand<1>(p, GATED_PART_A, 0, k0, crossed);
  }
}

// A value as three of bf16 that add up to it: each the nearest to what is left, so that the
// second is 2^-8 and the third 2^-16 of the value at most. The first of one that is not finite
// holds it; one that would round to infinity is cut instead.
__device__ __forceinline__ void three_parts(float x, bf16_t* p) {
  p[0] = from_f32<bf16_t>(x);
  if ((p[0].b & 0x7F80u) == 0x7F80u) {
    const uint32_t b = __float_as_uint(x);
    if ((b & 0x7F800000u) == 0x7F800000u) {
      p[1].b = p[2].b = 0;
      return;
    }
    p[0].b = (uint16_t)(b >> 16);
  }
  const float r = x - to_f32(p[0]);   // exact, as the next
  p[1] = from_f32<bf16_t>(r);
  p[2] = from_f32<bf16_t>(r - to_f32(p[1]));
}

}  // namespace tg
