// Host side of the gated linear layer: argument checks, the workspace's division and the
// launches of k_gated.hip and k_gated_bwd.hip.
#include "gated.h"
#include "tgrad.h"

using namespace tg;

namespace {

// sizes that the kernels' indexes and tiles' offsets hold
constexpr int64_t kMostSide = 1 << 19;
constexpr int64_t kMostDyStride = 1 << 20;   // 256 rows of a tile stay under 2^31 bytes

bool shape_ok(int64_t rows, int64_t in, int64_t hidden, int dtype, int act) {
  return rows >= 0 && rows <= 0x7FFFFFFF - 65536 && in >= 1 && in <= kMostSide && hidden >= 1 && hidden <= kMostSide &&
         dtype >= TGRAD_F32 && dtype <= TGRAD_BF16 && act >= 0 && act < GATED_ACTS;
}
bool stride_ok(int64_t stride, int64_t rows, int64_t cols) {
  return rows <= 1 || (stride >= cols && stride <= (int64_t(1) << 40));
}
bool bad(const void* p, int dtype) { return ((uintptr_t)p & (dtype == TGRAD_F32 ? 3 : 1)) != 0; }

// whether a matrix's lines go to the products as they lie
bool as_it_lies(const void* p, int64_t stride, int64_t rows, int64_t cols, int dtype) {
  if (dtype == TGRAD_F32 || (cols & 7) != 0 || ((uintptr_t)p & 15u) != 0) return false;
  return rows <= 1 || ((stride & 7) == 0 && stride <= MM_MOST_STRIDE);
}

size_t up16(size_t n) { return (n + 255) & ~(size_t)255; }

// A call's workspace, and what of it is copies.
struct Plan {
  GatedParts x, wg, wu;
  GatedPack pack[3];
  int packs = 0;
  size_t bytes = 0;
};
void place(Plan& p, GatedParts& m, const void* src, int64_t stride, int64_t rows, int64_t cols, int dtype, bool lies,
           char* ws) {
  if (lies) {
    m = {src, rows, 0, (uint32_t)cols, (uint32_t)(rows <= 1 ? cols : stride)};
    return;
  }
  const uint32_t pad = gated_pad((uint32_t)cols);
  m = {ws + p.bytes, rows, rows * (int64_t)pad, pad, pad};
  p.pack[p.packs++] = {src, rows, rows <= 1 ? cols : stride, (uint32_t)cols, dtype, ws + p.bytes};
  p.bytes += up16((size_t)rows * pad * 2 * (dtype == TGRAD_F32 ? 3 : 1));
}
Plan plan_of(const void* x, int64_t x_stride, const void* w_gate, const void* w_up, int64_t rows, int64_t in,
             int64_t hidden, int dtype, char* ws) {
  Plan p;
  place(p, p.x, x, x_stride, rows, in, dtype, as_it_lies(x, x_stride, rows, in, dtype), ws);
  // both weights alike: their strides are one
  const bool both = as_it_lies(w_gate, in, hidden, in, dtype) && as_it_lies(w_up, in, hidden, in, dtype);
  place(p, p.wg, w_gate, in, hidden, in, dtype, both, ws);
  place(p, p.wu, w_up, in, hidden, in, dtype, both, ws);
  return p;
}

struct Backward {
  size_t grads, sums, split, bytes;    // where each begins, behind the copies
  int parts;
  GatedWay dx, dw;
};
Backward backward_of(size_t at, int64_t rows, int64_t in, int64_t hidden, int dtype) {
  Backward b;
  const int64_t pad = gated_pad((uint32_t)hidden);
  b.grads = at;
  b.parts = gated_grad_parts(rows, in, hidden, dtype);
  at += up16((size_t)rows * 2 * pad * 2 * b.parts);
  b.sums = at;
  at += up16((size_t)gated_sum_rows(rows, (uint32_t)in, (uint32_t)hidden) * 2 * pad * 4);
  b.split = at;       // dx's, then dw's
  b.dx = gated_dx_way(rows, (uint32_t)in, (uint32_t)hidden, b.parts);
  b.dw = gated_dw_way(rows, (uint32_t)in, (uint32_t)hidden, b.parts);
  // what is counted has its counters first, cleared once for both; results of splits go behind them
  const size_t most = b.dx.bytes > b.dw.bytes ? b.dx.bytes : b.dw.bytes;
  b.bytes = at + (most ? MM_MOST_SPLIT * 4 + up16(most) : 0);
  return b;
}

int status(hipError_t e) { return e == hipSuccess ? TGRAD_OK : TGRAD_EHIP; }

}  // namespace

extern "C" {

int64_t tgrad_gated_linear_workspace(const void* x, int64_t x_stride, const void* w_gate, const void* w_up,
                                     int64_t rows, int64_t in, int64_t hidden, int dtype, int backward) {
  if (!shape_ok(rows, in, hidden, dtype, 0) || !stride_ok(x_stride, rows, in)) return -1;
  const Plan p = plan_of(x, x_stride, w_gate, w_up, rows, in, hidden, dtype, nullptr);
  return (int64_t)(backward ? backward_of(p.bytes, rows, in, hidden, dtype).bytes : p.bytes);
}

int tgrad_gated_linear_forward(const void* x, int64_t x_stride, const void* w_gate, const void* w_up,
                               const void* b_gate, const void* b_up, void* y, int64_t rows, int64_t in,
                               int64_t hidden, int dtype, int activation, void* workspace, void* stream) {
  if (!shape_ok(rows, in, hidden, dtype, activation) || !stride_ok(x_stride, rows, in)) return TGRAD_EINVAL;
  if (bad(x, dtype) || bad(w_gate, dtype) || bad(w_up, dtype) || bad(b_gate, dtype) || bad(b_up, dtype) ||
      bad(y, dtype) || ((uintptr_t)workspace & 15u))
    return TGRAD_EINVAL;
  if (!w_gate || !w_up) return TGRAD_EINVAL;
  if (rows == 0) return TGRAD_OK;
  if (!x || !y) return TGRAD_EINVAL;
  const Plan p = plan_of(x, x_stride, w_gate, w_up, rows, in, hidden, dtype, (char*)workspace);
  if (p.bytes && !workspace) return TGRAD_EINVAL;
  const hipStream_t s = (hipStream_t)stream;
  hipError_t e = launch_gated_pack(p.pack, p.packs, s);
  if (e != hipSuccess) return TGRAD_EHIP;
  GatedArgs a{};
  a.x = p.x;
  a.wg = p.wg;
  a.wu = p.wu;
  a.bg = b_gate;
  a.bu = b_up;
  a.rows = rows;
  a.in = (uint32_t)in;
  a.hidden = (uint32_t)hidden;
  a.dt = dtype;
  a.act = activation;
  a.y = y;
  return status(launch_gated_forward(a, s));
}

int tgrad_gated_linear_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                const void* w_gate, const void* w_up, const void* b_gate, const void* b_up, void* dx,
                                void* dw_gate, void* dw_up, void* db_gate, void* db_up, int64_t rows, int64_t in,
                                int64_t hidden, int dtype, int activation, void* workspace, void* stream) {
  if (!shape_ok(rows, in, hidden, dtype, activation) || !stride_ok(x_stride, rows, in) ||
      !stride_ok(dy_stride, rows, hidden) || (rows > 1 && dy_stride > kMostDyStride))
    return TGRAD_EINVAL;
  for (const void* q : {dy, x, w_gate, w_up, b_gate, b_up, (const void*)dx, (const void*)dw_gate, (const void*)dw_up,
                        (const void*)db_gate, (const void*)db_up})
    if (bad(q, dtype)) return TGRAD_EINVAL;
  if (!w_gate || !w_up || !dw_gate != !dw_up || !db_gate != !db_up) return TGRAD_EINVAL;
  if (((uintptr_t)workspace & 15u) || (rows > 0 && (!dy || !x))) return TGRAD_EINVAL;
  const hipStream_t s = (hipStream_t)stream;
  char* const ws = (char*)workspace;
  const Plan p = plan_of(x, x_stride, w_gate, w_up, rows, in, hidden, dtype, ws);
  const Backward b = backward_of(p.bytes, rows, in, hidden, dtype);
  if (b.bytes && !workspace) return TGRAD_EINVAL;
  const uint32_t pad = gated_pad((uint32_t)hidden);
  const GatedParts grads{ws + b.grads, rows, rows * 2 * (int64_t)pad, 2 * pad, 2 * pad};
  hipError_t e = hipSuccess;
  if (rows > 0) {
    e = launch_gated_pack(p.pack, p.packs, s);
    if (e != hipSuccess) return TGRAD_EHIP;
    GatedArgs a{};
    a.x = p.x;
    a.wg = p.wg;
    a.wu = p.wu;
    a.bg = b_gate;
    a.bu = b_up;
    a.rows = rows;
    a.in = (uint32_t)in;
    a.hidden = (uint32_t)hidden;
    a.dt = dtype;
    a.act = activation;
    a.dy = dy;
    a.dy_stride = rows > 1 ? dy_stride : hidden;
    a.grads = ws + b.grads;
    a.parts = b.parts;
    a.counters = b.dx.counted || b.dw.counted ? (uint32_t*)(ws + b.split) : nullptr;
    a.row_sums = db_gate ? (float*)(ws + b.sums) : nullptr;
    e = launch_gated_grads(a, s);
    if (e == hipSuccess && dx) {
      GatedDx d{};
      d.grads = grads;
      d.wg = p.wg;
      d.wu = p.wu;
      d.dx = dx;
      d.rows = rows;
      d.in = (uint32_t)in;
      d.hidden = (uint32_t)hidden;
      d.dt = dtype;
      d.parts = b.parts;
      d.way = b.dx;
      d.sums = ws + b.split + (d.way.counted ? 0 : MM_MOST_SPLIT * 4);
      e = launch_gated_dx(d, s);
    }
    if (e != hipSuccess) return TGRAD_EHIP;
  }
  if (!dw_gate && !db_gate) return TGRAD_OK;
  GatedDw d{};
  d.grads = grads;
  d.x = p.x;
  d.dwg = dw_gate;
  d.dwu = dw_up;
  d.dbg = db_gate;
  d.dbu = db_up;
  d.row_sums = (const float*)(ws + b.sums);
  d.sum_rows = gated_sum_rows(rows, (uint32_t)in, (uint32_t)hidden);
  d.rows = rows;
  d.in = (uint32_t)in;
  d.hidden = (uint32_t)hidden;
  d.dt = dtype;
  d.parts = b.parts;
  d.way = b.dw;
  d.sums = ws + b.split + (d.way.counted ? 0 : MM_MOST_SPLIT * 4);
  return status(launch_gated_dw(d, s));
}

}  // extern "C"
