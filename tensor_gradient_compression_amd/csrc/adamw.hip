// Host side of AdamW over many tensors: the handle, its division of the tensors into
// workgroups' chunks, and the launches. Kernels and arithmetic: k_adamw.hip.
#include <cfloat>
#include <cmath>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "adamw.h"
#include "tgrad.h"

using namespace tg;

struct tgrad_adamw {
  struct Tensor {
    int64_t numel;
    uint64_t values, state;   // real values, place of the first in the flat state
    int dtype, grad_dtype;
    double wd;
  };
  struct Launch {
    int first_tensor, tensors;
    uint32_t first_chunk, chunks, first_span, spans;
  };
  int device = 0;
  int bits = 32;
  double lr = 0, b1 = 0, b2 = 0, eps = 0;
  uint64_t seed = 0, total = 0;   // total: values of the flat state
  uint32_t lds = 0;               // see kStreamBytes
  std::vector<Tensor> tensors;
  std::vector<Launch> launches;
  uint32_t nchunks = 0, nspans = 0;
  AdamwChunk* chunks = nullptr;   // device, one block of memory with those below
  AdamwClock* clocks = nullptr;
  AdamwSpan* spans = nullptr;
  double* partial = nullptr;
  uint32_t* counts = nullptr;
  void* block = nullptr;
  void* state = nullptr;          // the caller's
  std::string err;
};

namespace {

// A step with fp32 moments that reads and writes this much runs two workgroups a CU instead of
// eight: each reserves half of the LDS. Fewer of its seven streams' pieces are then open at a
// time (bf16, 236M values, 5.2 GB: 945 us with eight, 850 with two; three models of 100M values
// in turn 1171 and 1066). Below, more loads in flight win: 60M values 198 and 214 us, 18.7M in
// 150 tensors 64 and 69.
constexpr uint64_t kStreamBytes = 1500000000;
constexpr uint32_t kStreamLds = 80 * 1024;

// Chunks of one launch: a launch whose threads along an axis pass 32 bits, which 2^24 workgroups'
// do, is cut to the rest without an error.
constexpr uint32_t kLaunchChunks = 1 << 21;

// Chunks of a handle, for each of which the host makes a record of 80 bytes: more values than any
// card holds a state of.
constexpr uint64_t kMostChunks = 1 << 27;

constexpr size_t kCountBytes = (ADAMW_COUNTS + 1) * ADAMW_COUNT_PITCH * sizeof(uint32_t);

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

int fail(tgrad_adamw_t* h, hipError_t e, const char* what) {
  try {
    h->err = std::string(what) + ": " + hipGetErrorString(e);
  } catch (...) {
  }
  return TGRAD_EHIP;
}

// -1 where the sizes do not form a state: values of the flat state otherwise
int64_t state_values(int n, const int64_t* numel, const int* dtype) {
  if (n < 1 || !numel || !dtype) return -1;
  uint64_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (numel[i] < 0 || numel[i] > (int64_t(1) << 40) || dtype[i] < TGRAD_F32 || dtype[i] > TGRAD_C64)
      return -1;
    const uint64_t v = (uint64_t)numel[i] * (dtype[i] == TGRAD_C64 ? 2 : 1);
    total += (v + ADAMW_GROUP - 1) / ADAMW_GROUP * ADAMW_GROUP;
    if (total > (1ull << 42)) return -1;
  }
  return (int64_t)total;
}

// The clock of the step after `t` steps.
AdamwClock clock_after(const tgrad_adamw_t* h, int64_t t) {
  AdamwClock c;
  c.t = t + 1;
  c.p1 = std::pow(h->b1, (double)c.t);
  c.p2 = std::pow(h->b2, (double)c.t);
  c.ic1 = (float)(1.0 / (1.0 - c.p1));
  c.is2 = (float)(1.0 / std::sqrt(1.0 - c.p2));
  c.key = adamw_step_key(h->seed, (uint64_t)c.t);
  return c;
}

hipError_t set_clocks(tgrad_adamw_t* h, const std::vector<AdamwClock>& host) {
  hipError_t e = hipDeviceSynchronize();
  if (e == hipSuccess)
    e = hipMemcpy(h->clocks, host.data(), host.size() * sizeof(AdamwClock), hipMemcpyHostToDevice);
  return e;
}

}  // namespace

extern "C" {

int64_t tgrad_adamw_state_values(int n, const int64_t* numel, const int* dtype) {
  return state_values(n, numel, dtype);
}

int64_t tgrad_adamw_state_bytes(int n, const int64_t* numel, const int* dtype, int state_bits) {
  const int64_t v = state_values(n, numel, dtype);
  if (v < 0 || (state_bits != 32 && state_bits != 8)) return -1;
  return state_bits == 32 ? 8 * v : 2 * v + 2 * (v / ADAMW_GROUP);
}

int tgrad_adamw_init(tgrad_adamw_t** out, int n, const int64_t* numel, const int* dtype,
                     const int* grad_dtype, const double* weight_decay, int state_bits, double lr,
                     double beta1, double beta2, double eps, uint64_t seed, void* state) {
  if (!out) return TGRAD_EINVAL;
  *out = nullptr;
  const int64_t total = state_values(n, numel, dtype);
  if (total < 0 || !grad_dtype || !weight_decay || (state_bits != 32 && state_bits != 8))
    return TGRAD_EINVAL;
  if (!(lr >= 0.0 && std::isfinite(lr)) || !(beta1 >= 0.0 && beta1 < 1.0) ||
      !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0 && std::isfinite(eps)))
    return TGRAD_EINVAL;
  if ((total > 0 && !state) || ((uintptr_t)state & 15u) != 0) return TGRAD_EINVAL;
  uint64_t pieces = 0;
  for (int i = 0; i < n; ++i) {
    const uint64_t values = (uint64_t)numel[i] * (dtype[i] == TGRAD_C64 ? 2 : 1);
    pieces += (values + ADAMW_CHUNK - 1) / ADAMW_CHUNK;
    if (pieces > kMostChunks) return TGRAD_EINVAL;
    const bool half = dtype[i] == TGRAD_F16 || dtype[i] == TGRAD_BF16;
    if (grad_dtype[i] != dtype[i] && !(half && grad_dtype[i] == TGRAD_F32)) return TGRAD_EINVAL;
    if (!(weight_decay[i] >= 0.0 && std::isfinite(weight_decay[i]))) return TGRAD_EINVAL;
  }
  tgrad_adamw_t* h = nullptr;
  try {
    h = new tgrad_adamw_t();
    if (hipGetDevice(&h->device) != hipSuccess) {
      delete h;
      return TGRAD_EHIP;
    }
    int cu = 0;
    if (hipDeviceGetAttribute(&cu, hipDeviceAttributeMultiprocessorCount, h->device) != hipSuccess ||
        cu < 1)
      cu = 256;
    h->bits = state_bits;
    h->lr = lr;
    h->b1 = beta1;
    h->b2 = beta2;
    h->eps = eps;
    h->seed = seed;
    h->total = (uint64_t)total;
    h->state = state;
    // Spans of the sum of squares: five workgroups a CU are enough to fill the memory's queues,
    // and few sums are sooner joined (bf16, 18.7M values in 150 tensors: 30 us with spans of
    // 2048, 12.6 with 8192, 10.6 with 16384, 15.8 with 98304; one of 236M: 107, 91 and 79 with
    // 8192, 16384 and 98304). A workgroup takes 4096 or 8192 values (of 4 or 2 bytes) at a time.
    const uint64_t even = (uint64_t)total / ((uint64_t)cu * 5);
    uint64_t size = even <= 2 * ADAMW_CHUNK ? 2 * ADAMW_CHUNK : (even + 4 * ADAMW_CHUNK - 1) / (4 * ADAMW_CHUNK) * (4 * ADAMW_CHUNK);
    if (size > 48 * ADAMW_CHUNK) size = 48 * ADAMW_CHUNK;
    std::vector<AdamwChunk> chunks;
    std::vector<AdamwSpan> spans;
    uint64_t at = 0, bytes = 0;
    for (int i = 0; i < n; ++i) {
      tgrad_adamw::Tensor t;
      t.numel = numel[i];
      t.values = (uint64_t)numel[i] * (dtype[i] == TGRAD_C64 ? 2 : 1);
      t.state = at;
      t.dtype = dtype[i];
      t.grad_dtype = grad_dtype[i];
      t.wd = weight_decay[i];
      auto new_launch = [&] {
        h->launches.push_back({i, 0, (uint32_t)chunks.size(), 0, (uint32_t)spans.size(), 0});
      };
      // closes a launch for now, with this tensor in it
      auto up_to_here = [&](tgrad_adamw::Launch& l) {
        l.tensors = i - l.first_tensor + 1;
        l.chunks = (uint32_t)chunks.size() - l.first_chunk;
        l.spans = (uint32_t)spans.size() - l.first_span;
      };
      if (i % ADAMW_LAUNCH_TENSORS == 0) new_launch();
      AdamwChunk c{};
      c.wd = t.wd;
      c.tensor = (uint32_t)i;
      c.wdt = dtype[i] == TGRAD_C64 ? DT_F32 : (uint32_t)dtype[i];
      c.gdt = grad_dtype[i] == TGRAD_C64 ? DT_F32 : (uint32_t)grad_dtype[i];
      for (uint64_t s = 0; s < t.values; s += ADAMW_CHUNK) {
        if (chunks.size() - h->launches.back().first_chunk == kLaunchChunks) {
          up_to_here(h->launches.back());
          new_launch();
        }
        c.start = s;
        c.state = at + s;
        c.n = (uint32_t)(t.values - s < ADAMW_CHUNK ? t.values - s : ADAMW_CHUNK);
        chunks.push_back(c);
      }
      for (uint64_t s = 0; s < t.values; s += size)
        spans.push_back({s, (uint32_t)i, (uint32_t)(t.values - s < size ? t.values - s : size), c.gdt});
      if (i == 0 && chunks.empty()) chunks.push_back(c);   // the step count needs a keeper
      up_to_here(h->launches.back());
      h->tensors.push_back(t);
      bytes += t.values * (16 + (c.wdt == DT_F32 ? 8 : 4) + (c.gdt == DT_F32 ? 4 : 2));
      at += (t.values + ADAMW_GROUP - 1) / ADAMW_GROUP * ADAMW_GROUP;
    }
    if (state_bits == 32 && bytes >= kStreamBytes) h->lds = kStreamLds;
    h->nchunks = (uint32_t)chunks.size();
    h->nspans = (uint32_t)spans.size();
    const size_t bc = chunks.size() * sizeof(AdamwChunk), bk = chunks.size() * sizeof(AdamwClock);
    const size_t bs = spans.size() * sizeof(AdamwSpan), bp = spans.size() * sizeof(double);
    // one block, filled by one copy: counts of zero, chunks, clocks, spans, room for the sums
    std::vector<char> host(kCountBytes + bc + bk + bs, 0);
    const std::vector<AdamwClock> clocks(chunks.size(), clock_after(h, 0));
    std::memcpy(host.data() + kCountBytes, chunks.data(), bc);
    std::memcpy(host.data() + kCountBytes + bc, clocks.data(), bk);
    if (bs) std::memcpy(host.data() + kCountBytes + bc + bk, spans.data(), bs);
    if (hipMalloc(&h->block, host.size() + bp) != hipSuccess) {
      delete h;
      return TGRAD_ENOMEM;
    }
    char* at_block = (char*)h->block;
    h->counts = (uint32_t*)at_block;
    h->chunks = (AdamwChunk*)(at_block += kCountBytes);
    h->clocks = (AdamwClock*)(at_block += bc);
    h->spans = (AdamwSpan*)(at_block += bk);
    h->partial = (double*)(at_block += bs);
    hipError_t e = hipMemcpy(h->block, host.data(), host.size(), hipMemcpyHostToDevice);
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

int tgrad_adamw_destroy(tgrad_adamw_t* h) {
  if (!h) return TGRAD_OK;
  {
    OnDevice g(h->device);
    (void)hipFree(h->block);
  }
  delete h;
  return TGRAD_OK;
}

const char* tgrad_adamw_last_error(const tgrad_adamw_t* h) { return h ? h->err.c_str() : ""; }

int tgrad_adamw_set_lr(tgrad_adamw_t* h, double lr) {
  if (!h || !(lr >= 0.0 && std::isfinite(lr))) return TGRAD_EINVAL;
  h->lr = lr;
  return TGRAD_OK;
}

int tgrad_adamw_get_steps(tgrad_adamw_t* h, int64_t* steps) {
  if (!h || !steps) return TGRAD_EINVAL;
  OnDevice g(h->device);
  AdamwClock c;
  hipError_t e = hipDeviceSynchronize();
  if (e == hipSuccess) e = hipMemcpy(&c, h->clocks, sizeof c, hipMemcpyDeviceToHost);
  if (e != hipSuccess) return fail(h, e, "reading the step count");
  *steps = c.t - 1;
  return TGRAD_OK;
}

int tgrad_adamw_set_steps(tgrad_adamw_t* h, int64_t steps) {
  if (!h || steps < 0) return TGRAD_EINVAL;
  OnDevice g(h->device);
  try {
    const hipError_t e = set_clocks(h, std::vector<AdamwClock>(h->nchunks, clock_after(h, steps)));
    return e == hipSuccess ? TGRAD_OK : fail(h, e, "writing the step count");
  } catch (const std::bad_alloc&) {
    return TGRAD_ENOMEM;
  }
}

int tgrad_adamw_step(tgrad_adamw_t* h, void* const* weights, const void* const* grads,
                     const float* clip, void* m_out, void* v_out, void* stream) {
  if (!h || !weights || !grads || !m_out != !v_out) return TGRAD_EINVAL;
  if (m_out && (h->bits != 8 || (((uintptr_t)m_out | (uintptr_t)v_out) & 15u))) return TGRAD_EINVAL;
  if ((uintptr_t)clip & 3u) return TGRAD_EINVAL;
  for (size_t i = 0; i < h->tensors.size(); ++i) {
    const auto& t = h->tensors[i];
    if (!t.numel) continue;
    const uintptr_t wa = t.dtype == TGRAD_F32 || t.dtype == TGRAD_C64 ? 3 : 1;
    const uintptr_t ga = t.grad_dtype == TGRAD_F32 || t.grad_dtype == TGRAD_C64 ? 3 : 1;
    if (!weights[i] || !grads[i] || ((uintptr_t)weights[i] & wa) || ((uintptr_t)grads[i] & ga))
      return TGRAD_EINVAL;
  }
  OnDevice g(h->device);
  AdamwArgs a{};
  a.bits = h->bits;
  a.lds = h->lds;
  a.m = h->state;
  if (h->bits == 32) {
    a.v = (float*)h->state + h->total;
  } else {
    a.v = (uint8_t*)h->state + h->total;
    a.ms = (uint8_t*)h->state + 2 * h->total;
    a.vs = a.ms + h->total / ADAMW_GROUP;
  }
  a.m_out = (uint16_t*)m_out;
  a.v_out = (uint16_t*)v_out;
  a.clip = clip;
  a.lr = h->lr;
  a.b1d = h->b1;
  a.b2d = h->b2;
  a.seed = h->seed;
  a.b1 = (float)h->b1;
  a.c1 = (float)(1.0 - h->b1);
  a.b2 = (float)h->b2;
  a.c2 = (float)(1.0 - h->b2);
  // The reciprocal of a subnormal eps, or of one that rounds to 0, is infinite, and a value
  // without a gradient so far would become 0 * infinity. Beside any root of v above zero (2^-75
  // and more) the least normal number is as little as those.
  a.eps = h->eps > 0.0 && h->eps < FLT_MIN ? FLT_MIN : (float)h->eps;
  for (const auto& l : h->launches) {
    if (!l.chunks) continue;
    AdamwTable tab;
    for (int i = 0; i < l.tensors; ++i) {
      tab.w[i] = weights[l.first_tensor + i];
      tab.g[i] = grads[l.first_tensor + i];
    }
    a.chunks = h->chunks + l.first_chunk;
    a.clocks = h->clocks + l.first_chunk;
    a.first_tensor = (uint32_t)l.first_tensor;
    a.nchunks = l.chunks;
    const hipError_t e = launch_adamw(a, l.tensors, tab, (hipStream_t)stream);
    if (e != hipSuccess) return fail(h, e, "AdamW step");
  }
  return TGRAD_OK;
}

int tgrad_adamw_grad_norm(tgrad_adamw_t* h, const void* const* grads, double max_norm,
                          double grad_scale, float* out, void* stream) {
  if (!h || !grads || !out || ((uintptr_t)out & 3u)) return TGRAD_EINVAL;
  if (!(max_norm > 0.0) || !(grad_scale > 0.0 && std::isfinite(grad_scale))) return TGRAD_EINVAL;
  for (size_t i = 0; i < h->tensors.size(); ++i) {
    const auto& t = h->tensors[i];
    const uintptr_t ga = t.grad_dtype == TGRAD_F32 || t.grad_dtype == TGRAD_C64 ? 3 : 1;
    if (t.numel && (!grads[i] || ((uintptr_t)grads[i] & ga))) return TGRAD_EINVAL;
  }
  OnDevice g(h->device);
  AdamwNorm a{};
  a.counts = h->counts;
  a.all_partial = h->partial;
  a.total_spans = h->nspans;
  a.out = out;
  a.max_norm = max_norm;
  a.scale = grad_scale;
  AdamwTable tab;
  auto fill = [&](const tgrad_adamw::Launch& l) {
    for (int i = 0; i < l.tensors; ++i) {
      tab.w[i] = nullptr;
      tab.g[i] = grads[l.first_tensor + i];
    }
    a.spans = h->spans + l.first_span;
    a.partial = h->partial + l.first_span;
    a.first_tensor = (uint32_t)l.first_tensor;
  };
  hipError_t e = hipSuccess;
  if (!h->nspans) {
    e = launch_adamw_norm(a, 0, tab, (hipStream_t)stream);
  } else if (h->nspans <= ADAMW_NORM_SPANS && h->launches.size() == 1 &&
             h->launches[0].tensors <= ADAMW_FEW_TENSORS) {
    // a workgroup alone, without counting (14 spans 3.0 us against 5.2)
    fill(h->launches[0]);
    e = launch_adamw_norm(a, h->launches[0].tensors, tab, (hipStream_t)stream);
  } else {
    for (const auto& l : h->launches) {
      if (!l.spans || e != hipSuccess) continue;
      fill(l);
      const bool join = l.first_span + l.spans == h->nspans;
      e = launch_adamw_squares(a, l.spans, join, l.tensors, tab, (hipStream_t)stream);
    }
  }
  return e == hipSuccess ? TGRAD_OK : fail(h, e, "gradient norm");
}

}  // extern "C"
