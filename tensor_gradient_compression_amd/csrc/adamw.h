// AdamW over many tensors: what the host side (adamw.hip) and the kernels (k_adamw.hip)
// share. gfx950 only.
#pragma once
#include "tg_common.h"

namespace tg {

// Values that share one scale of the 8-bit state; every tensor's state starts at a multiple.
constexpr uint32_t ADAMW_GROUP = 128;
// Tensors whose addresses one launch carries in its arguments (16 bytes each, under 4 KiB).
constexpr int ADAMW_LAUNCH_TENSORS = 240;
// Launches of up to this many tensors carry a table of their own: 0.4 us less on the host.
constexpr int ADAMW_FEW_TENSORS = 24;

// Values that one workgroup steps.
constexpr uint32_t ADAMW_CHUNK = 2048;

// A workgroup's share of one tensor: `n` values from `start` on, all of them multiples of
// ADAMW_CHUNK except the tensor's end. `state` is the place of the first in the flat state.
struct AdamwChunk {
  uint64_t start, state;
  double wd;
  uint32_t tensor, n;
  uint32_t wdt, gdt;   // Dt of the weight and the gradient, DT_F32 for complex (its parts)
};

// A workgroup's share of the sum of squares.
struct AdamwSpan {
  uint64_t start;
  uint32_t tensor, n, gdt;
};

// What a workgroup knows of the step it makes next: its number t (the first is 1), the
// powers b1^t and b2^t, the corrections 1 / (1 - b1^t) and 1 / sqrt(1 - b2^t), and the key of
// its random bits.
struct AdamwClock {
  int64_t t;
  double p1, p2;
  float ic1, is2;
  uint32_t key;
};
// SplitMix64's output for the state seed + t * 0x9E3779B97F4A7C15, its low half
__host__ __device__ inline uint32_t adamw_step_key(uint64_t seed, uint64_t t) {
  uint64_t z = seed + t * 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return (uint32_t)(z ^ (z >> 31));
}

template <int N>
struct AdamwTableOf {
  void* w[N];
  const void* g[N];
};
using AdamwTable = AdamwTableOf<ADAMW_LAUNCH_TENSORS>;

struct AdamwArgs {
  const AdamwChunk* chunks;   // of this launch
  AdamwClock* clocks;         // of this launch
  uint32_t first_tensor;
  uint32_t nchunks;
  int bits;                   // 32 or 8
  uint32_t lds;               // 32 bits: LDS that a workgroup reserves, unused
  void* m;                    // fp32, or codes
  void* v;                    // fp32, or codes of sqrt(v)
  uint8_t* ms;                // 8 bits: the groups' exponent fields
  uint8_t* vs;
  uint16_t* m_out;            // 8 bits, or NULL: the new values as bf16
  uint16_t* v_out;
  const float* clip;          // NULL, or {norm, coefficient}
  double lr, b1d, b2d;
  uint64_t seed;
  float b1, c1, b2, c2, eps;
};

// `tensors` of the table are set.
hipError_t launch_adamw(const AdamwArgs& a, int tensors, const AdamwTable& tab, hipStream_t s);

// Counts of workgroups that have finished, by their number's remainder, and one of the groups,
// each in a cache line of its own.
constexpr uint32_t ADAMW_COUNTS = 16, ADAMW_COUNT_PITCH = 64;

// Spans that one workgroup sums up alone.
constexpr uint32_t ADAMW_NORM_SPANS = 16;

// norm = scale * sqrt(sum of squares), coefficient = scale * min(1, max_norm / norm)
struct AdamwNorm {
  const AdamwSpan* spans;     // of this launch
  double* partial;            // a sum of squares for each of them
  double* all_partial;        // those of all launches
  uint32_t* counts;           // join: workgroups that have finished; 0 between calls
  uint32_t first_tensor;      // of this launch
  uint32_t total_spans;
  float* out;                 // {norm, coefficient}
  double max_norm, scale;
};
// The sums of squares of a launch's spans, with join also the result.
hipError_t launch_adamw_squares(const AdamwNorm& a, uint32_t nspans, bool join, int tensors,
                                const AdamwTable& tab, hipStream_t s);
// The result alone, of at most ADAMW_NORM_SPANS spans of one launch.
hipError_t launch_adamw_norm(const AdamwNorm& a, int tensors, const AdamwTable& tab, hipStream_t s);

}  // namespace tg
