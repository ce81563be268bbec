// Python side of the operators on lists of tensors and of layer norm: unpacks torch tensors,
// checks them against what the library will read and write, and calls the C functions of
// tgrad.h on the current stream. A step over some hundred small tensors takes the GPU less
// time than interpreted checks of each of them would take the host, so they are made here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>
#include <vector>

#include "tgrad.h"

namespace {

PyObject* g_error = nullptr;   // the package's TGradError

// A Python error that is already set, or one to be set as a ValueError.
struct Raised {};
struct Invalid {
  std::string what;
};

c10::ScalarType scalar_type(int code) {
  switch (code) {
    case TGRAD_F32: return c10::ScalarType::Float;
    case TGRAD_F16: return c10::ScalarType::Half;
    case TGRAD_BF16: return c10::ScalarType::BFloat16;
    case TGRAD_C64: return c10::ScalarType::ComplexFloat;
  }
  throw Invalid{"unknown dtype code"};
}

struct Plan {
  tgrad_adamw_t* h = nullptr;
  int device = 0, bits = 32;
  int64_t total = 0;
  std::vector<int64_t> numel;
  std::vector<c10::ScalarType> wt, gt;
  std::vector<void*> w;
  std::vector<const void*> g;
};

const char* kPlan = "tgrad.adamw_plan";

void free_plan(PyObject* cap) { delete (Plan*)PyCapsule_GetPointer(cap, kPlan); }

Plan* plan_of(PyObject* cap) {
  Plan* p = (Plan*)PyCapsule_GetPointer(cap, kPlan);
  if (!p) throw Raised{};
  return p;
}

std::string named(const char* what, long i) {
  return i < 0 ? std::string(what) : std::string(what) + "[" + std::to_string(i) + "]";
}

const at::Tensor& tensor(PyObject* o, const char* what, long i = -1) {
  if (!THPVariable_Check(o))
    throw Invalid{named(what, i) + ": expected a torch.Tensor, got " + Py_TYPE(o)->tp_name};
  return THPVariable_Unpack(o);
}

// a dense tensor of the type on the GPU `device` (any GPU if that is negative)
void on_gpu(const at::Tensor& t, c10::ScalarType type, int device, const char* what, long i = -1) {
  if (!t.is_cuda()) throw Invalid{named(what, i) + ": must be a GPU tensor"};
  if (t.layout() != c10::Layout::Strided) throw Invalid{named(what, i) + ": must be a dense tensor"};
  if (device >= 0 && t.get_device() != device)
    throw Invalid{named(what, i) + ": on cuda:" + std::to_string(t.get_device()) + ", expected cuda:" +
                  std::to_string(device)};
  if (t.scalar_type() != type)
    throw Invalid{named(what, i) + ": dtype " + c10::toString(t.scalar_type()) + ", expected " +
                  c10::toString(type)};
  if (t.is_conj() || t.is_neg())
    throw Invalid{named(what, i) + ": a lazily conjugated or negated view; call resolve_conj() or resolve_neg()"};
}

// Uninitialised memory from torch's allocator, ordered with the current stream, without the way
// through torch's dispatcher (layer norm forward 5.8 -> 5.4 us, backward 9.5 -> 8.7).
at::Tensor empty(at::IntArrayRef sizes, c10::ScalarType type, int device) {
  return at::Tensor(at::detail::empty_cuda(sizes, type, c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)device),
                                           std::nullopt));
}

void* data_of(const at::Tensor& t) { return const_cast<void*>(t.const_data_ptr()); }

// As torch's own in-place operations: what autograd saved of the tensor is out of date.
void changed(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

struct Sequence {
  PyObject* fast;
  Sequence(PyObject* o, const char* what) : fast(PySequence_Fast(o, what)) {
    if (!fast) throw Raised{};
  }
  ~Sequence() { Py_XDECREF(fast); }
  long size() const { return (long)PySequence_Fast_GET_SIZE(fast); }
  PyObject* operator[](long i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

void* pointer(PyObject* o, int device) {
  if (o == Py_None) return (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised{};
  return p;
}

void check_rc(int rc, const char* what, const char* detail) {
  if (rc == TGRAD_OK) return;
  std::string m = std::string(what) + ": " + tgrad_status_string(rc);
  if (detail && *detail) m += std::string(" ") + detail;
  PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, m.c_str());
  throw Raised{};
}

// Every entry: C++ exceptions end here as Python errors.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const Invalid& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

void want(Py_ssize_t n, Py_ssize_t m, const char* what) {
  if (n == m) return;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", what, m);
  throw Raised{};
}

std::vector<int64_t> ints(PyObject* o, const char* what) {
  Sequence s(o, what);
  std::vector<int64_t> v;
  for (long i = 0; i < s.size(); ++i) {
    const long long x = PyLong_AsLongLong(s[i]);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    v.push_back(x);
  }
  return v;
}

// set_error(class)
PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

// adamw_plan(handle, device, bits, total, numels, dtype codes, gradient dtype codes)
PyObject* adamw_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 7, "adamw_plan");
    std::vector<int64_t> wt = ints(a[5], "dtypes"), gt = ints(a[6], "grad dtypes");
    Plan* p = new Plan();
    try {
      p->h = (tgrad_adamw_t*)PyLong_AsVoidPtr(a[0]);
      p->device = (int)PyLong_AsLong(a[1]);
      p->bits = (int)PyLong_AsLong(a[2]);
      p->total = PyLong_AsLongLong(a[3]);
      if (PyErr_Occurred()) throw Raised{};
      p->numel = ints(a[4], "numels");
      for (int64_t c : wt) p->wt.push_back(scalar_type((int)c));
      for (int64_t c : gt) p->gt.push_back(scalar_type((int)c));
      p->w.resize(p->numel.size());
      p->g.resize(p->numel.size());
    } catch (...) {
      delete p;
      throw;
    }
    PyObject* cap = PyCapsule_New(p, kPlan, free_plan);
    if (!cap) delete p;
    return cap;
  });
}

void gradients(Plan* p, PyObject* list) {
  Sequence s(list, "grads: expected a list of tensors");
  if (s.size() != (long)p->numel.size())
    throw Invalid{"grads: " + std::to_string(s.size()) + " tensors, the handle has " +
                  std::to_string(p->numel.size())};
  for (long i = 0; i < s.size(); ++i) {
    const at::Tensor& t = tensor(s[i], "grads", i);
    on_gpu(t, p->gt[i], p->device, "grads", i);
    if (t.numel() != p->numel[i])
      throw Invalid{named("grads", i) + ": " + std::to_string(t.numel()) + " elements, expected " +
                    std::to_string(p->numel[i])};
    if (!t.is_contiguous()) throw Invalid{named("grads", i) + ": must be contiguous"};
    p->g[i] = data_of(t);
  }
}

float* pair_of_floats(Plan* p, PyObject* o, const char* what) {
  const at::Tensor& t = tensor(o, what);
  on_gpu(t, c10::ScalarType::Float, p->device, what);
  if (t.numel() != 2 || !t.is_contiguous())
    throw Invalid{std::string(what) + ": needs two contiguous float32 values, the norm and the coefficient"};
  return (float*)data_of(t);
}

// adamw_step(plan, weights, grads, clip or None, moments or None, stream or None)
PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 6, "adamw_step");
    Plan* p = plan_of(a[0]);
    Sequence ws(a[1], "weights: expected a list of tensors");
    if (ws.size() != (long)p->numel.size())
      throw Invalid{"weights: " + std::to_string(ws.size()) + " tensors, the handle has " +
                    std::to_string(p->numel.size())};
    for (long i = 0; i < ws.size(); ++i) {
      const at::Tensor& t = tensor(ws[i], "weights", i);
      on_gpu(t, p->wt[i], p->device, "weights", i);
      if (t.numel() != p->numel[i])
        throw Invalid{named("weights", i) + ": " + std::to_string(t.numel()) + " elements, expected " +
                      std::to_string(p->numel[i])};
      if (!t.is_contiguous()) throw Invalid{named("weights", i) + ": must be contiguous"};
      p->w[i] = data_of(t);
    }
    gradients(p, a[2]);
    const float* clip = a[3] == Py_None ? nullptr : pair_of_floats(p, a[3], "clip");
    void* out[2] = {nullptr, nullptr};
    std::vector<at::Tensor> moments;
    if (a[4] != Py_None) {
      if (p->bits != 8) throw Invalid{"moments: only for 8-bit states (32-bit ones are in `state`)"};
      Sequence ms(a[4], "moments: expected two tensors");
      if (ms.size() != 2) throw Invalid{"moments: expected two tensors"};
      for (long i = 0; i < 2; ++i) {
        const at::Tensor& t = tensor(ms[i], "moments", i);
        on_gpu(t, c10::ScalarType::BFloat16, p->device, "moments", i);
        if (t.numel() != p->total || !t.is_contiguous())
          throw Invalid{named("moments", i) + ": needs " + std::to_string(p->total) + " contiguous bfloat16 values"};
        out[i] = data_of(t);
        moments.push_back(t);
      }
      if (p->total && out[0] == out[1]) throw Invalid{"moments: the two tensors are the same"};
    }
    check_rc(tgrad_adamw_step(p->h, p->w.data(), p->g.data(), clip, out[0], out[1], pointer(a[5], p->device)),
             "tgrad_adamw_step", tgrad_adamw_last_error(p->h));
    for (long i = 0; i < ws.size(); ++i) changed(THPVariable_Unpack(ws[i]));
    for (const at::Tensor& t : moments) changed(t);
    Py_RETURN_NONE;
  });
}

// adamw_grad_norm(plan, grads, max_norm, grad_scale, out or None, stream or None) -> out
PyObject* adamw_grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 6, "adamw_grad_norm");
    Plan* p = plan_of(a[0]);
    gradients(p, a[1]);
    const double max_norm = PyFloat_AsDouble(a[2]), scale = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) throw Raised{};
    at::Tensor out;
    if (a[4] == Py_None) {
      // memory that torch hands out on the current stream is ordered with that stream alone
      if (a[5] != Py_None) throw Invalid{"out: give the result's tensor along with a stream"};
      out = empty({2}, at::kFloat, p->device);
    } else {
      pair_of_floats(p, a[4], "out");
      out = THPVariable_Unpack(a[4]);
    }
    check_rc(tgrad_adamw_grad_norm(p->h, p->g.data(), max_norm, scale, (float*)data_of(out),
                                   pointer(a[5], p->device)),
             "tgrad_adamw_grad_norm", tgrad_adamw_last_error(p->h));
    if (a[4] != Py_None) changed(out);
    return THPVariable_Wrap(out);
  });
}

int code_of(const at::Tensor& t, const char* what) {
  switch (t.scalar_type()) {
    case c10::ScalarType::Float: return TGRAD_F32;
    case c10::ScalarType::Half: return TGRAD_F16;
    case c10::ScalarType::BFloat16: return TGRAD_BF16;
    default: throw Invalid{std::string(what) + ": dtype must be float32, float16 or bfloat16"};
  }
}

// Rows of the last axis, `stride` elements apart: the leading axes have to lie as one.
struct Rows {
  int64_t rows = 1, cols = 0, stride = 0;
};
Rows rows_of(const at::Tensor& t, const char* what) {
  const int64_t d = t.dim();
  Rows r;
  if (d < 1) throw Invalid{std::string(what) + ": needs at least one axis"};
  r.cols = t.size(d - 1);
  if (r.cols < 1) throw Invalid{std::string(what) + ": the last axis is empty"};
  for (int64_t i = 0; i < d - 1; ++i) r.rows *= t.size(i);
  if (r.rows == 0) return r;
  if (t.stride(d - 1) != 1 && r.cols > 1) throw Invalid{std::string(what) + ": the last axis must be contiguous"};
  // of the axes from the last leading one outwards; none yet (an expanded axis has stride and span 0)
  int64_t span = -1;
  for (int64_t i = d - 2; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (span < 0) r.stride = t.stride(i);
    else if (t.stride(i) != span)
      throw Invalid{std::string(what) + ": the leading axes' strides do not form one; call contiguous()"};
    span = t.stride(i) * t.size(i);
  }
  if (r.rows > 1 && r.stride < r.cols)
    throw Invalid{std::string(what) + ": the rows overlap; call contiguous()"};
  if (span < 0) r.stride = r.cols;
  return r;
}

// a vector of the columns, or NULL for None
const at::Tensor* vector_of(PyObject* o, int64_t cols, int device, const char* what) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, what);
  code_of(t, what);
  on_gpu(t, t.scalar_type(), device, what);
  if (t.dim() != 1 || t.numel() != cols || !t.is_contiguous())
    throw Invalid{std::string(what) + ": needs " + std::to_string(cols) + " contiguous values on one axis"};
  return &t;
}

void weight_type(int dt, int wdt, const char* what) {
  if (wdt != dt && wdt != TGRAD_F32)
    throw Invalid{std::string(what) + ": dtype must be float32 or that of x"};
}

// layer_norm_forward(x, weight or None, bias or None, eps) -> (y, mean, rstd)
PyObject* layer_norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 4, "layer_norm_forward");
    const at::Tensor& x = tensor(a[0], "x");
    const int dt = code_of(x, "x");
    on_gpu(x, x.scalar_type(), -1, "x");
    const int dev = (int)x.get_device();
    const Rows r = rows_of(x, "x");
    const at::Tensor* w = vector_of(a[1], r.cols, dev, "weight");
    const at::Tensor* b = vector_of(a[2], r.cols, dev, "bias");
    const int wdt = w ? code_of(*w, "weight") : b ? code_of(*b, "bias") : dt;
    if (w) weight_type(dt, wdt, "weight");
    if (b && code_of(*b, "bias") != wdt) throw Invalid{"bias: dtype differs from the weight's"};
    if (b) weight_type(dt, wdt, "bias");
    const double eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) throw Raised{};
    const c10::DeviceGuard guard(x.device());
    at::Tensor y = empty(x.sizes(), x.scalar_type(), dev);
    const auto lead = x.sizes().slice(0, x.dim() - 1);
    at::Tensor mean = empty(lead, at::kFloat, dev), rstd = empty(lead, at::kFloat, dev);
    check_rc(tgrad_layer_norm_forward(data_of(x), r.stride, w ? data_of(*w) : nullptr, b ? data_of(*b) : nullptr,
                                      data_of(y), (float*)data_of(mean), (float*)data_of(rstd), r.rows, r.cols, dt,
                                      wdt, eps, pointer(Py_None, dev)),
             "tgrad_layer_norm_forward", "");
    return Py_BuildValue("(NNN)", THPVariable_Wrap(y), THPVariable_Wrap(mean), THPVariable_Wrap(rstd));
  });
}

// layer_norm_backward(dy, x, weight or None, mean, rstd, need_params) -> (dx, dweight or None, dbias or None)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 6, "layer_norm_backward");
    const at::Tensor& x = tensor(a[1], "x");
    const int dt = code_of(x, "x");
    on_gpu(x, x.scalar_type(), -1, "x");
    const int dev = (int)x.get_device();
    const at::Tensor& dy = tensor(a[0], "dy");
    on_gpu(dy, x.scalar_type(), dev, "dy");
    if (dy.sizes() != x.sizes()) throw Invalid{"dy: its shape is not x's"};
    const Rows r = rows_of(x, "x"), rd = rows_of(dy, "dy");
    const at::Tensor* w = vector_of(a[2], r.cols, dev, "weight");
    const int wdt = w ? code_of(*w, "weight") : dt;
    weight_type(dt, wdt, "weight");
    const at::Tensor* st[2];
    for (int i = 0; i < 2; ++i) {
      const char* what = i ? "rstd" : "mean";
      const at::Tensor& t = tensor(a[3 + i], what);
      on_gpu(t, c10::ScalarType::Float, dev, what);
      if (t.numel() != r.rows || !t.is_contiguous())
        throw Invalid{std::string(what) + ": needs " + std::to_string(r.rows) + " contiguous float32 values"};
      st[i] = &t;
    }
    const int params = PyObject_IsTrue(a[5]);
    if (params < 0) throw Raised{};
    const c10::DeviceGuard guard(x.device());
    at::Tensor dx = empty(x.sizes(), x.scalar_type(), dev), dw, db, ws;
    if (params) {
      dw = empty({r.cols}, scalar_type(wdt), dev);
      db = empty({r.cols}, scalar_type(wdt), dev);
      const int64_t bytes = tgrad_layer_norm_workspace(r.rows, r.cols);
      if (bytes < 0) throw Invalid{"x: too many rows or columns"};
      ws = empty({bytes}, at::kByte, dev);
    }
    check_rc(tgrad_layer_norm_backward(data_of(dy), rd.stride, data_of(x), r.stride, w ? data_of(*w) : nullptr,
                                       (const float*)data_of(*st[0]), (const float*)data_of(*st[1]), data_of(dx),
                                       params ? data_of(dw) : nullptr, params ? data_of(db) : nullptr, r.rows, r.cols,
                                       dt, wdt, params ? data_of(ws) : nullptr, pointer(Py_None, dev)),
             "tgrad_layer_norm_backward", "");
    if (!params) {
      Py_INCREF(Py_None);
      Py_INCREF(Py_None);
      return Py_BuildValue("(NNN)", THPVariable_Wrap(dx), Py_None, Py_None);
    }
    return Py_BuildValue("(NNN)", THPVariable_Wrap(dx), THPVariable_Wrap(dw), THPVariable_Wrap(db));
  });
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {{"set_error", set_error, METH_O, nullptr},
                          FAST(adamw_plan),
                          FAST(adamw_step),
                          FAST(adamw_grad_norm),
                          FAST(layer_norm_forward),
                          FAST(layer_norm_backward),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_tgrad_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tgrad_torch(void) { return PyModule_Create(&kModule); }
