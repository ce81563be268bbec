// Newton-Schulz orthogonalisation and the Muon step: what the host side (muon.hip) and the
// kernels (k_muon.hip) share. gfx950 only.
#pragma once
#include "mm_tile.h"

namespace tg {

// Tensors whose addresses the first launch of a step carries in its arguments.
constexpr int MUON_LAUNCH_TENSORS = 220;
// Values that one workgroup takes in the passes over values.
constexpr uint32_t MUON_CHUNK = 8192;

// The powers of two that X, and A and B, are held under.
constexpr float NS_X = 4096.0f, NS_M = 256.0f;

// One matrix. Offsets are bytes from the workspace's first.
struct NsMat {
  uint64_t x, y;       // X and the next X: rows lines of ldx, the upper parts, then the lower ones
  uint64_t a, b;       // A and B off their diagonals: m lines of ldm; with `exact` the lower parts behind
  uint64_t da, db;     // their diagonals, m floats each
  uint64_t sums;       // `chunks` doubles: sums of squares
  uint64_t elem;       // the first value in its tensor
  uint64_t state;      // and in the momentum
  double scale, wd;
  uint32_t rows, cols, ldx, ldm, m, chunks, tensor;
  uint32_t wdt, gdt, exact;
};
// A workgroup's part of a matrix: a tile of a product, or a chunk of values.
struct NsPart {
  uint32_t mat, i, j;
};
// Either a list of parts (and matrices), or `count` matrices alike with ni x nj parts each.
struct NsParts {
  const NsPart* list;
  uint32_t ni, nj;
  bool lower;          // alike: only those with j <= i, ni = nj
  uint32_t splits;     // products: workgroups to a tile, each over a part of the sum
};

struct NsCommon {
  const NsMat* mats;   // or NULL: all like `one`, `pitch` bytes of the workspace apart
  NsMat one;
  uint64_t pitch;
  char* ws;
  uint32_t* counters;  // of whole_sums(), or NULL if no product is split
  const float* clip;   // NULL, or {norm, coefficient}: nothing happens where the norm is not finite
  float ca, cb, cc;
};

struct MuonTable {
  void* w[MUON_LAUNCH_TENSORS];
  const void* g[MUON_LAUNCH_TENSORS];
};
// A step's first pass: new momentum and sums of squares of the update.
struct MuonFirst {
  void** w;            // device: every tensor's addresses, for the launches after
  const void** g;
  uint32_t first_tensor, tensors;
  float* momentum;
  float mu, nu;        // momentum and 1 - momentum
  bool nesterov;
};
hipError_t launch_muon_first(const NsCommon& c, const MuonFirst& f, const MuonTable& t, const NsParts& p, uint32_t n,
                             hipStream_t s);
// X from the update and its norm
hipError_t launch_muon_start(const NsCommon& c, const MuonFirst& f, double eps, const NsParts& p, uint32_t n,
                             hipStream_t s);
// The same two from matrices given as they are.
struct NsSource {
  const void* x;
  int64_t row_stride, matrix_stride;
};
hipError_t launch_ns_norm(const NsCommon& c, const NsSource& f, const NsParts& p, uint32_t n, hipStream_t s);
hipError_t launch_ns_start(const NsCommon& c, const NsSource& f, double eps, const NsParts& p, uint32_t n, hipStream_t s);

// The products. `tile`: 0: 256 x 256, 1: 128 x 128, 2: 64 x 64, 3: 128 x 128 of a
// workgroup alone on its compute unit; n: tiles; `at`: which X is read.
hipError_t launch_ns_gram(const NsCommon& c, int at, int tile, const NsParts& p, uint32_t n, hipStream_t s);
hipError_t launch_ns_poly(const NsCommon& c, int tile, const NsParts& p, uint32_t n, hipStream_t s);
// X to the other X, or at the end to the weights or a result
struct NsLast {
  bool last;
  void* const* w;      // weights: device addresses, or NULL
  double lr;
  void* out;           // else contiguous matrices
};
hipError_t launch_ns_apply(const NsCommon& c, int at, int tile, const NsLast& l, const NsParts& p, uint32_t n,
                           hipStream_t s);

// All of a step or an orthogonalisation, a workgroup a matrix: for those with ns_small_parts()
// above zero (1: eight parts of 16 x 32 at most; others: parts of 32 x 32). parts, lds: the largest of the launch's ns_small_parts() and ns_small_lds(); exact:
// theirs. With t a step, whose addresses it has, else of src.
constexpr uint32_t NS_SMALL_LDS = 160 * 1024 - 512;
uint32_t ns_small_parts(uint32_t rows, uint32_t cols, bool exact);
uint32_t ns_small_lds(uint32_t rows, uint32_t cols, bool exact);
struct NsSmall {
  int steps;
  bool exact;
  uint32_t parts, lds;
  double eps, lr;
  void* out;           // without t: contiguous matrices
};
hipError_t launch_ns_small(const NsCommon& c, const NsSmall& k, const MuonFirst& f, const MuonTable* t, const NsSource& src,
                           const NsParts& p, uint32_t n, hipStream_t s);

constexpr uint32_t ns_tile_size(int tile) { return tile == 0 ? 256 : tile == 2 ? 64 : 128; }

}  // namespace tg
