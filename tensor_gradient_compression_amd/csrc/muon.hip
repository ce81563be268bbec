// Host side of Newton-Schulz orthogonalisation and of the Muon step: the handle, the division
// of the matrices into tiles and chunks, and the launches. Kernels and arithmetic: k_muon.hip.
#include <algorithm>
#include <cmath>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "muon.h"
#include "tgrad.h"

using namespace tg;

struct tgrad_muon {
  struct Tensor {
    int64_t values;
    int dtype, grad_dtype;
  };
  struct Small {             // a launch over matrices that a workgroup holds
    uint32_t first = 0, n = 0, parts = 0, lds = 0;
  };
  struct First {             // launches over some tensors, whose addresses their arguments carry
    uint32_t first_tensor, tensors, first_chunk, chunks;
    Small small[2];          // bf16, and those whose products take both parts
  };
  struct List {              // a launch of a product over all matrices
    uint32_t first = 0, n = 0, splits = 1;
    int tile = 2;
  };
  int device = 0, steps = 5;
  double lr = 0, momentum = 0, eps = 0, coef[3] = {};
  bool nesterov = true;
  std::vector<Tensor> tensors;
  std::vector<First> firsts;
  List chunks, starts, gram, poly, apply;
  void* block = nullptr;     // device: matrices, parts, addresses, then the workspace
  NsMat* mats = nullptr;
  NsPart* parts = nullptr;
  void** w = nullptr;
  const void** g = nullptr;
  char* ws = nullptr;
  uint32_t* counters = nullptr;
  float* state = nullptr;    // the caller's
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;   // of a step's weights
  std::string err;
};

namespace {

constexpr uint64_t kGroup = 128;           // every tensor's momentum starts at a multiple
constexpr int64_t kMostSide = 1 << 19;     // tiles' offsets stay under 2^31 bytes
constexpr uint64_t kMostParts = 1 << 21;   // of one launch
constexpr int kMostSteps = 100;
// So few values do not average what the products of upper parts are off (2 x 2 in bf16: 1.8 times a
// rounding), and take those of both in a launch that waits for its barriers anyway.
constexpr int64_t kFewValues = 1024;

struct OnDevice {
  int prev = -1;
  explicit OnDevice(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) prev = -1;
    if (prev != dev) (void)hipSetDevice(dev);
    else prev = -1;
  }
  ~OnDevice() {
    if (prev >= 0) (void)hipSetDevice(prev);
  }
};

int fail(tgrad_muon_t* h, hipError_t e, const char* what) {
  try {
    h->err = std::string(what) + ": " + hipGetErrorString(e);
  } catch (...) {
  }
  return TGRAD_EHIP;
}

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

bool side_ok(int64_t rows, int64_t cols) { return rows >= 1 && rows <= kMostSide && cols >= 1 && cols <= kMostSide; }
bool type_ok(int dtype) { return dtype >= TGRAD_F32 && dtype <= TGRAD_BF16; }
bool numbers_ok(int steps, const double* c, double eps) {
  return steps >= 1 && steps <= kMostSteps && c && std::isfinite(c[0]) && std::isfinite(c[1]) && std::isfinite(c[2]) &&
         eps >= 0.0 && std::isfinite(eps);
}

// A line's values with its padding: long ones are whole cache lines, which the tiles' transfers
// take in halves (2048 x 2048 x 2048 in lines of 2056: 60 us, of 2048: 48).
uint32_t line(uint64_t n) { return (uint32_t)up(n, n >= 256 ? 64 : 8); }

// Sizes of a matrix and its place in a workspace, from `at` on; returns the end.
uint64_t lay_out(NsMat& m, int64_t rows, int64_t cols, int dtype, uint64_t at) {
  m.rows = (uint32_t)rows;
  m.cols = (uint32_t)cols;
  m.ldx = line(cols);
  m.m = (uint32_t)(rows < cols ? rows : cols);
  m.ldm = line(m.m);
  m.exact = dtype != TGRAD_BF16 || rows * cols <= kFewValues;
  m.wdt = (uint32_t)dtype;
  m.chunks = (uint32_t)(((uint64_t)rows * (m.ldx / 8) + MUON_CHUNK / 8 - 1) / (MUON_CHUNK / 8));
  auto take = [&](uint64_t bytes) {
    const uint64_t o = at;
    at += up(bytes, 256);
    return o;
  };
  const uint64_t x = (uint64_t)rows * m.ldx * 4, s = (uint64_t)m.m * m.ldm * (m.exact ? 4 : 2);
  m.x = take(x);
  m.y = take(x);
  m.a = take(s);
  m.b = take(s);
  m.da = take(m.m * 4ull);
  m.db = take(m.m * 4ull);
  m.sums = take(m.chunks * 8ull);
  return at;
}
uint64_t across(uint64_t n, int tile) { return (n + ns_tile_size(tile) - 1) / ns_tile_size(tile); }
uint64_t lower_tiles(uint64_t m, int tile) { return across(m, tile) * (across(m, tile) + 1) / 2; }

// A tile, and how many workgroups share each.
struct Way {
  int tile = 2;
  uint32_t splits = 1;
  uint64_t tiles = 0;
  uint64_t sums() const { return mm_split_bytes(tiles, splits, ns_tile_size(tile)); }
};
// The one after which the compute unit with most to do ends first, in ns, by what was measured:
// 256 x 256 tiles bring 36 bytes a ns of their operands to LDS (matrix instructions bind them),
// 128 x 128 ones 50, smaller ones 68 where two workgroups share a unit and 52 where one is alone;
// what follows the product takes 0.5 ns a place, and the sums of a split pass memory at 4 TB/s after
// 2 us of waiting. (1536 x 1536 in fp16: Gram of 128 x 128 tiles in three splits 34 us, in six 42;
// 18 of 1024 x 4096 in bf16: 256 x 256 tiles 123, 128 x 128 141; 777 x 2051 in fp16, B X: 128 x 128
// in four splits 41, in two 32, 64 x 64 unsplit 25.)
template <class Each>
Way choose(const Each& each) {
  Way best;
  double least = 0;
  for (int tile = 0; tile < 3; ++tile) {
    const double side = ns_tile_size(tile);
    uint64_t tiles = 0, longest = 0;
    double total = 0;
    each(tile, [&](uint64_t n, uint64_t k) {   // n tiles with sums over k
      tiles += n;
      longest = std::max(longest, k);
      total += (double)n * k;
    });
    if (!tiles) return best;
    for (uint32_t splits = 1; splits <= (tile ? MM_MOST_SPLITS : 1); ++splits) {
      if (splits > 1 && (tiles * splits > MM_MOST_SPLIT || longest < splits * 256)) break;
      const double one = (double)longest / splits, loads = std::ceil(total / 256 / one - 1e-6);
      const double rate = tile == 0 ? 36 : tile == 1 ? 50 : loads > 1 ? 68 : 52;
      const double cost = loads * (one * side * 4 / rate + side * side / 2) +
                          (splits > 1 ? 2000 + tiles * splits * side * side * 8 / 4000 : 0);
      if (!(tile == 0 && splits == 1) && cost >= least) continue;
      least = cost;
      best = {tile, splits, tiles};
    }
  }
  if (best.tile == 1 && best.tiles * best.splits <= 256) best.tile = 3;
  return best;
}

// Those of `count` matrices alike.
struct Ways {
  Way gram, poly, apply;
  Ways(const NsMat& m, uint64_t count) {
    const uint64_t parts = m.exact ? 3 : 1;
    gram = choose([&](int t, auto&& add) { add(count * lower_tiles(m.m, t), parts * std::max(m.rows, m.cols)); });
    poly = choose([&](int t, auto&& add) { add(count * lower_tiles(m.m, t), parts * m.m); });
    apply = choose([&](int t, auto&& add) { add(count * across(m.rows, t) * across(m.cols, t), parts * m.m); });
  }
  uint64_t sums() const { return std::max({gram.sums(), poly.sums(), apply.sums()}); }
};

// `products` steps of the iteration, X in place
struct Launches {
  NsParts gram, poly, apply;
  uint32_t ngram, npoly, napply;
  int tgram, tpoly, tapply;
};
hipError_t iterate(const NsCommon& c, const Launches& l, int steps, NsLast last, hipStream_t s) {
  hipError_t e = hipSuccess;
  for (int i = 0; i < steps && e == hipSuccess; ++i) {
    const int at = i & 1;
    e = launch_ns_gram(c, at, l.tgram, l.gram, l.ngram, s);
    if (e == hipSuccess) e = launch_ns_poly(c, l.tpoly, l.poly, l.npoly, s);
    last.last = i == steps - 1;
    if (e == hipSuccess) e = launch_ns_apply(c, at, l.tapply, last, l.apply, l.napply, s);
  }
  return e;
}

// Values of the flat momentum, or -1.
int64_t state_values(int n, const int64_t* count, const int64_t* rows, const int64_t* cols) {
  if (n < 1 || !count || !rows || !cols) return -1;
  uint64_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (count[i] < 0 || count[i] > (int64_t(1) << 40) || !side_ok(rows[i], cols[i])) return -1;
    const uint64_t each = (uint64_t)rows[i] * cols[i];
    if ((uint64_t)count[i] > (1ull << 40) / each) return -1;
    total += up(count[i] * each, kGroup);
    if (total > (1ull << 40)) return -1;
  }
  return (int64_t)total;
}

}  // namespace

extern "C" {

int64_t tgrad_muon_state_values(int n, const int64_t* count, const int64_t* rows, const int64_t* cols) {
  return state_values(n, count, rows, cols);
}

int tgrad_muon_init(tgrad_muon_t** out, int n, const int64_t* count, const int64_t* rows, const int64_t* cols,
                    const int* dtype, const int* grad_dtype, const double* weight_decay, const double* scale, double lr,
                    double momentum, int nesterov, int steps, const double* coefficients, double eps, float* state) {
  if (!out) return TGRAD_EINVAL;
  *out = nullptr;
  const int64_t total = state_values(n, count, rows, cols);
  if (total < 0 || !dtype || !grad_dtype || !weight_decay || !scale || !numbers_ok(steps, coefficients, eps))
    return TGRAD_EINVAL;
  if (!(lr >= 0.0 && std::isfinite(lr)) || !(momentum >= 0.0 && momentum < 1.0)) return TGRAD_EINVAL;
  if ((total > 0 && !state) || ((uintptr_t)state & 15u) != 0) return TGRAD_EINVAL;
  uint64_t matrices = 0;
  for (int i = 0; i < n; ++i) {
    if (!type_ok(dtype[i]) || (grad_dtype[i] != dtype[i] && grad_dtype[i] != TGRAD_F32)) return TGRAD_EINVAL;
    if (!(weight_decay[i] >= 0.0 && std::isfinite(weight_decay[i])) || !(scale[i] >= 0.0 && std::isfinite(scale[i])))
      return TGRAD_EINVAL;
    matrices += (uint64_t)count[i];
    if (matrices > kMostParts) return TGRAD_EINVAL;
  }
  tgrad_muon_t* h = nullptr;
  try {
    h = new tgrad_muon_t();
    if (hipGetDevice(&h->device) != hipSuccess) {
      delete h;
      return TGRAD_EHIP;
    }
    h->lr = lr;
    h->momentum = momentum;
    h->nesterov = nesterov != 0;
    h->steps = steps;
    h->eps = eps;
    h->state = state;
    h->spans.reserve(n);
    for (int i = 0; i < 3; ++i) h->coef[i] = coefficients[i];
    std::vector<NsMat> mats;
    std::vector<NsPart> parts;
    uint64_t ws = 0, at = 0, over = 0;
    for (int i = 0; i < n; ++i) {
      const uint64_t each = (uint64_t)rows[i] * cols[i];
      h->tensors.push_back({(int64_t)(count[i] * each), dtype[i], grad_dtype[i]});
      for (int64_t k = 0; k < count[i]; ++k) {
        NsMat m{};
        const uint64_t end = lay_out(m, rows[i], cols[i], dtype[i], ws);
        if (!ns_small_parts(m.rows, m.cols, m.exact != 0)) ws = end;   // others need none of it
        m.gdt = (uint32_t)grad_dtype[i];
        m.elem = k * each;
        m.state = at + k * each;
        m.scale = scale[i];
        m.wd = weight_decay[i];
        m.tensor = (uint32_t)i;
        mats.push_back(m);
        over += 2 * m.chunks + 1;
        if (over > 2 * kMostParts) {
          delete h;
          return TGRAD_EINVAL;
        }
      }
      at += up(count[i] * each, kGroup);
    }
    auto small = [](const NsMat& m) { return ns_small_parts(m.rows, m.cols, m.exact != 0); };
    // matrices that a workgroup holds, and chunks of the others' values, in launches of the
    // tensors whose addresses fit one
    size_t mat = 0;
    for (int i = 0; i < n || h->firsts.empty(); i += MUON_LAUNCH_TENSORS) {
      const int t = n - i < MUON_LAUNCH_TENSORS ? n - i : MUON_LAUNCH_TENSORS;
      tgrad_muon::First f{(uint32_t)i, (uint32_t)t, 0, 0, {}};
      size_t end = mat;
      while (end < mats.size() && mats[end].tensor < (uint32_t)(i + t)) ++end;
      for (int exact = 0; exact < 2; ++exact) {
        auto& l = f.small[exact];
        l.first = (uint32_t)parts.size();
        for (size_t k = mat; k < end; ++k) {
          const uint32_t n = small(mats[k]);
          if (!n || mats[k].exact != (uint32_t)exact) continue;
          parts.push_back({(uint32_t)k, 0, 0});
          l.parts = std::max(l.parts, n);
          l.lds = std::max(l.lds, ns_small_lds(mats[k].rows, mats[k].cols, exact != 0));
        }
        l.n = (uint32_t)parts.size() - l.first;
      }
      f.first_chunk = (uint32_t)parts.size();
      for (; mat < end; ++mat)
        for (uint32_t c = 0; !small(mats[mat]) && c < mats[mat].chunks; ++c) parts.push_back({(uint32_t)mat, c, 0});
      f.chunks = (uint32_t)parts.size() - f.first_chunk;
      h->firsts.push_back(f);
    }
    auto list = [&](tgrad_muon::List& l, Way way, auto&& add) {
      l.tile = way.tile;
      l.splits = way.splits;
      l.first = (uint32_t)parts.size();
      for (size_t k = 0; k < mats.size(); ++k)
        if (!small(mats[k])) add((uint32_t)k, mats[k]);
      l.n = (uint32_t)(parts.size() - l.first);
    };
    uint64_t sums = 0;
    auto way = [&](auto&& tiles, auto&& length) {
      const Way w = choose([&](int tile, auto&& add) {
        for (const NsMat& m : mats)
          if (!small(m)) add(tiles(m, tile), (uint64_t)length(m) * (m.exact ? 3 : 1));
      });
      sums = std::max(sums, w.sums());
      return w;
    };
    list(h->starts, Way{}, [&](uint32_t k, const NsMat& m) {
      for (uint32_t c = 0; c < m.chunks; ++c) parts.push_back({k, c, 0});
    });
    auto lower = [](const NsMat& m, int tile) { return lower_tiles(m.m, tile); };
    const Way ways[2] = {way(lower, [](const NsMat& m) { return std::max(m.rows, m.cols); }),
                         way(lower, [](const NsMat& m) { return m.m; })};
    for (int o = 0; o < 2; ++o)
      list(o ? h->poly : h->gram, ways[o], [&](uint32_t k, const NsMat& m) {
        for (uint32_t i = 0; i < across(m.m, ways[o].tile); ++i)
          for (uint32_t j = 0; j <= i; ++j) parts.push_back({k, i, j});
      });
    const Way whole = way([](const NsMat& m, int t) { return across(m.rows, t) * across(m.cols, t); },
                          [](const NsMat& m) { return m.m; });
    list(h->apply, whole, [&](uint32_t k, const NsMat& m) {
      const uint32_t ni = (uint32_t)across(m.rows, whole.tile), nj = (uint32_t)across(m.cols, whole.tile);
      for (uint32_t b = 0; b < ni; b += 8)
        for (uint32_t j = 0; j < nj; ++j)
          for (uint32_t i = b; i < ni && i < b + 8; ++i) parts.push_back({k, i, j});
    });
    if (parts.size() > 4 * kMostParts) {
      delete h;
      return TGRAD_EINVAL;
    }
    const uint64_t bm = up(mats.size() * sizeof(NsMat), 256), bp = up(parts.size() * sizeof(NsPart), 256);
    const uint64_t bt = up((uint64_t)n * 8, 256);
    if (hipMalloc(&h->block, bm + bp + 2 * bt + ws + sums) != hipSuccess) {
      (void)hipGetLastError();
      delete h;
      return TGRAD_ENOMEM;
    }
    char* b = (char*)h->block;
    h->mats = (NsMat*)b;
    h->parts = (NsPart*)(b += bm);
    h->w = (void**)(b += bp);
    h->g = (const void**)(b += bt);
    h->ws = b + bt;
    if (sums) h->counters = (uint32_t*)(h->ws + ws);
    hipError_t e = hipSuccess;
    if (!mats.empty()) e = hipMemcpy(h->mats, mats.data(), mats.size() * sizeof(NsMat), hipMemcpyHostToDevice);
    if (e == hipSuccess && !parts.empty())
      e = hipMemcpy(h->parts, parts.data(), parts.size() * sizeof(NsPart), hipMemcpyHostToDevice);
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) {
      (void)hipFree(h->block);
      delete h;
      return TGRAD_EHIP;
    }
  } catch (const std::bad_alloc&) {
    if (h && h->block) (void)hipFree(h->block);
    delete h;
    return TGRAD_ENOMEM;
  }
  *out = h;
  return TGRAD_OK;
}

int tgrad_muon_destroy(tgrad_muon_t* h) {
  if (!h) return TGRAD_OK;
  {
    OnDevice g(h->device);
    (void)hipFree(h->block);
  }
  delete h;
  return TGRAD_OK;
}

const char* tgrad_muon_last_error(const tgrad_muon_t* h) { return h ? h->err.c_str() : ""; }

int tgrad_muon_set_lr(tgrad_muon_t* h, double lr) {
  if (!h || !(lr >= 0.0 && std::isfinite(lr))) return TGRAD_EINVAL;
  h->lr = lr;
  return TGRAD_OK;
}

int tgrad_muon_step(tgrad_muon_t* h, void* const* weights, const void* const* grads, const float* clip, void* stream) {
  if (!h || !weights || !grads || ((uintptr_t)clip & 3u)) return TGRAD_EINVAL;
  for (size_t i = 0; i < h->tensors.size(); ++i) {
    const auto& t = h->tensors[i];
    if (!t.values) continue;
    const uintptr_t wa = t.dtype == TGRAD_F32 ? 3 : 1, ga = t.grad_dtype == TGRAD_F32 ? 3 : 1;
    if (!weights[i] || !grads[i] || ((uintptr_t)weights[i] & wa) || ((uintptr_t)grads[i] & ga)) return TGRAD_EINVAL;
  }
  h->spans.clear();          // within what was reserved
  for (size_t i = 0; i < h->tensors.size(); ++i) {
    const auto& t = h->tensors[i];
    const uintptr_t at = (uintptr_t)weights[i];
    if (t.values) h->spans.emplace_back(at, at + (uintptr_t)t.values * (t.dtype == TGRAD_F32 ? 4 : 2));
  }
  std::sort(h->spans.begin(), h->spans.end());
  for (size_t i = 1; i < h->spans.size(); ++i)
    if (h->spans[i].first < h->spans[i - 1].second) return TGRAD_EINVAL;   // two workgroups' at once
  OnDevice dev(h->device);
  const hipStream_t s = (hipStream_t)stream;
  NsCommon c{};
  c.mats = h->mats;
  c.ws = h->ws;
  c.counters = h->counters;
  c.clip = clip;
  c.ca = (float)h->coef[0];
  c.cb = (float)h->coef[1];
  c.cc = (float)h->coef[2];
  MuonFirst f{};
  f.w = h->w;
  f.g = h->g;
  f.momentum = h->state;
  f.mu = (float)h->momentum;
  f.nu = (float)(1.0 - h->momentum);
  f.nesterov = h->nesterov;
  hipError_t e = hipSuccess;
  for (const auto& l : h->firsts) {
    MuonTable t;
    for (uint32_t i = 0; i < l.tensors; ++i) {
      t.w[i] = weights[l.first_tensor + i];
      t.g[i] = grads[l.first_tensor + i];
    }
    f.first_tensor = l.first_tensor;
    f.tensors = l.tensors;
    for (int exact = 0; exact < 2; ++exact) {
      const auto& q = l.small[exact];
      const NsSmall k{h->steps, exact != 0, q.parts, q.lds, h->eps, h->lr, nullptr};
      if (e == hipSuccess) e = launch_ns_small(c, k, f, &t, NsSource{}, {h->parts + q.first, 0, 0, false, 1}, q.n, s);
    }
    if (e == hipSuccess) e = launch_muon_first(c, f, t, {h->parts + l.first_chunk, 0, 0, false, 1}, l.chunks, s);
  }
  auto parts = [&](const tgrad_muon::List& l) { return NsParts{h->parts + l.first, 0, 0, false, l.splits}; };
  if (!h->starts.n) return e == hipSuccess ? TGRAD_OK : fail(h, e, "Muon step");
  if (e == hipSuccess) e = launch_muon_start(c, f, h->eps, parts(h->starts), h->starts.n, s);
  const Launches l{parts(h->gram), parts(h->poly), parts(h->apply), h->gram.n, h->poly.n, h->apply.n,
                   h->gram.tile,   h->poly.tile,   h->apply.tile};
  NsLast last{};
  last.w = h->w;
  last.lr = h->lr;
  if (e == hipSuccess) e = iterate(c, l, h->steps, last, s);
  return e == hipSuccess ? TGRAD_OK : fail(h, e, "Muon step");
}

int64_t tgrad_orthogonalize_workspace(int64_t count, int64_t rows, int64_t cols, int dtype) {
  if (count < 0 || count > (int64_t)kMostParts || !side_ok(rows, cols) || !type_ok(dtype)) return -1;
  NsMat m{};
  const uint64_t each = lay_out(m, rows, cols, dtype, 0);
  if (ns_small_parts(m.rows, m.cols, m.exact != 0)) return 0;
  if ((uint64_t)count > (1ull << 46) / each) return -1;
  return (int64_t)(each * count + (count ? Ways(m, count).sums() : 0));
}

int tgrad_orthogonalize(const void* x, int64_t matrix_stride, int64_t row_stride, void* out, int64_t count,
                        int64_t rows, int64_t cols, int dtype, int steps, const double* coefficients, double eps,
                        void* workspace, void* stream) {
  const int64_t bytes = tgrad_orthogonalize_workspace(count, rows, cols, dtype);
  if (bytes < 0 || !numbers_ok(steps, coefficients, eps)) return TGRAD_EINVAL;
  if ((rows > 1 && row_stride < cols) || row_stride > (int64_t(1) << 40)) return TGRAD_EINVAL;
  if (count > 1 && (matrix_stride < (rows - 1) * (rows > 1 ? row_stride : 0) + cols || matrix_stride > (int64_t(1) << 42)))
    return TGRAD_EINVAL;
  if (count == 0) return TGRAD_OK;
  const uintptr_t low = dtype == TGRAD_F32 ? 3 : 1;
  if (!x || !out || (bytes && !workspace) || ((uintptr_t)x & low) || ((uintptr_t)out & low) || ((uintptr_t)workspace & 15u))
    return TGRAD_EINVAL;
  const hipStream_t s = (hipStream_t)stream;
  NsCommon c{};
  c.pitch = lay_out(c.one, rows, cols, dtype, 0);
  c.one.gdt = (uint32_t)dtype;
  c.ws = (char*)workspace;
  c.ca = (float)coefficients[0];
  c.cb = (float)coefficients[1];
  c.cc = (float)coefficients[2];
  const NsSource f{x, row_stride, matrix_stride};
  if (const uint32_t most = ns_small_parts(c.one.rows, c.one.cols, c.one.exact != 0)) {
    c.pitch = 0;
    const NsSmall k{steps, c.one.exact != 0, most, ns_small_lds(c.one.rows, c.one.cols, c.one.exact != 0), eps, 0.0, out};
    const hipError_t e = launch_ns_small(c, k, MuonFirst{}, nullptr, f, {nullptr, 1, 1, false, 1}, (uint32_t)count, s);
    return e == hipSuccess ? TGRAD_OK : TGRAD_EHIP;
  }
  const uint64_t n = (uint64_t)count, m = c.one.m;
  const Ways w(c.one, n);
  const uint64_t chunks = n * c.one.chunks;
  for (uint64_t k : {chunks, w.gram.tiles, w.poly.tiles, w.apply.tiles})
    if (k > kMostParts) return TGRAD_EINVAL;
  if (w.sums()) c.counters = (uint32_t*)(c.ws + c.pitch * n);
  auto parts = [&](const Way& y, uint64_t r, uint64_t k, bool lower) {
    return NsParts{nullptr, (uint32_t)across(r, y.tile), (uint32_t)across(k, y.tile), lower, y.splits};
  };
  const Launches l{parts(w.gram, m, m, true), parts(w.poly, m, m, true), parts(w.apply, rows, cols, false),
                   (uint32_t)w.gram.tiles,    (uint32_t)w.poly.tiles,    (uint32_t)w.apply.tiles,
                   w.gram.tile,               w.poly.tile,               w.apply.tile};
  hipError_t e = launch_ns_norm(c, f, {nullptr, c.one.chunks, 1, false, 1}, (uint32_t)chunks, s);
  if (e == hipSuccess) e = launch_ns_start(c, f, eps, {nullptr, c.one.chunks, 1, false, 1}, (uint32_t)chunks, s);
  NsLast last{};
  last.out = out;
  if (e == hipSuccess) e = iterate(c, l, steps, last, s);
  return e == hipSuccess ? TGRAD_OK : TGRAD_EHIP;
}

}  // extern "C"
