// Python binding of libtide_step.so: checks of torch tensors, outputs and workspaces from torch's
// allocator, one call of the C ABI on torch's current stream.
//
// It is compiled because the smallest calls are bound by the host: the same checks and allocations
// written in Python took 9 to 22 us a call, where the kernels take 3.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/impl/VirtualGuardImpl.h>

#include <sstream>
#include <string>
#include <vector>

#include "../../include/tide_step.h"

#ifndef TIDE_BUILD_ID
#define TIDE_BUILD_ID "unknown"
#endif
// Found in the file by its mark, so that asking for it does not load torch.
extern "C" __attribute__((visibility("default"), used)) const char tide_step_binding_id[] =
    "tide_step_binding build id " TIDE_BUILD_ID;

namespace {

PyObject* g_error = nullptr;       // TideError
PyObject* g_raw_stream = nullptr;  // device index -> handle of torch's current stream

struct Refused {};  // a Python error is set

template <typename... Parts>
[[noreturn]] void refuse(PyObject* kind, const Parts&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  PyErr_SetString(kind, s.str().c_str());
  throw Refused();
}
// The message's parts are made only where they are needed: some cost more than the rest of a check.
#define NEED(ok, ...)                                                      \
  do {                                                                     \
    if (__builtin_expect(!(ok), 0)) refuse(PyExc_ValueError, __VA_ARGS__); \
  } while (0)

void check(tide_status status, const char* where) {
  if (status == TIDE_OK) return;
  const int hip = status == TIDE_ERR_HIP ? tide_step_last_hip_error() : 0;
  if (PyObject* e = PyObject_CallFunction(g_error, "isi", int(status), where, hip)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused();
}

// ---------------------------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------------------------

using Opt = const at::Tensor*;  // NULL where the caller passed None

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
Opt optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

int code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return TIDE_BF16;
    case at::kFloat: return TIDE_FP32;
    case at::kInt: return TIDE_INT32;
    case at::kLong: return TIDE_INT64;
    default: return -1;
  }
}
inline bool is_float(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }
inline bool is_id(at::ScalarType t) { return t == at::kInt || t == at::kLong; }
constexpr const char* kFloats = "torch.bfloat16 or torch.float32";

struct Device {
  int index;
  Device() : index(c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index()) {}
  void* stream() const {
    PyObject* i = PyLong_FromLong(index);
    PyObject* h = i != nullptr ? PyObject_CallOneArg(g_raw_stream, i) : nullptr;
    Py_XDECREF(i);
    if (h == nullptr) throw Refused();
    void* s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (s == nullptr && PyErr_Occurred()) throw Refused();
    return s;
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return at::empty(shape, at::TensorOptions().dtype(t).device(at::Device(c10::DeviceType::CUDA, c10::DeviceIndex(index))));
  }
};
void on_gpu(const at::Tensor& t, const char* name) {
  NEED(t.is_cuda(), name, " must be on the current device, got ", t.device().str());
}
void on(const Device& d, const at::Tensor& t, const char* name) {
  NEED(t.is_cuda() && t.get_device() == d.index, name, " must be on the current device (cuda:", d.index, "), got ",
       t.device().str());
  NEED(!t.is_neg(), name, " must not be a negated view: its memory holds the values of the other sign");
}
void like(const Device& d, const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  on(d, t, name);
  NEED(t.scalar_type() == type, name, " must be of ", c10::toString(type), ", got ", c10::toString(t.scalar_type()));
  NEED(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
}
void dense(const at::Tensor& t, const char* name) { NEED(t.is_contiguous(), name, " must be contiguous"); }
inline void* at_of(Opt t) { return t == nullptr ? nullptr : t->data_ptr(); }

// The caller's workspace if it is large enough, else a new one, kept alive until the call is enqueued.
struct Workspace {
  at::Tensor own;
  void* p;
  int64_t bytes;
  Workspace(const Device& d, Opt given, int64_t needed, const char* where) {
    if (needed < 0) check(TIDE_ERR_INVALID, where);
    if (given != nullptr) {
      on(d, *given, "workspace");
      NEED(given->scalar_type() == at::kByte, "workspace must be of torch.uint8");
      dense(*given, "workspace");
      NEED(given->numel() >= needed, "workspace must hold ", needed, " bytes, got ", given->numel());
    } else {
      own = d.empty({needed}, at::kByte);
      given = &own;
    }
    p = given->data_ptr();
    bytes = given->numel();
  }
};

// Tells autograd that a caller's tensor was written in place: what saved it for a backward pass refuses to
// use it.  Tensors of inference mode are not counted.
void changed(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
// What the caller passed, or what was made in its place.
struct Output {
  PyObject* given;
  at::Tensor made;
  const at::Tensor* t;
  template <typename Make>
  Output(PyObject* o, const char* name, Make&& make) : given(o), t(optional(o, name)) {
    if (t == nullptr) {
      made = make();
      t = &made;
    }
  }
  PyObject* result() const {  // of a call that has been enqueued
    if (given == Py_None) return wrap(made);
    changed(*t);
    Py_INCREF(given);
    return given;
  }
};
PyObject* triple(const Output& a, const Output& b, const Output& c) {
  PyObject* r = PyTuple_New(3);
  if (r == nullptr) return nullptr;
  const Output* o[] = {&a, &b, &c};
  for (int i = 0; i < 3; ++i) {
    PyObject* x = o[i]->result();
    if (x == nullptr) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, x);
  }
  return r;
}

// ---------------------------------------------------------------------------------------------
// Gradient norm and clipping
// ---------------------------------------------------------------------------------------------

// A reference to a Python object, which may be NULL.
struct Held {
  PyObject* o;
  explicit Held(PyObject* owned) : o(owned) {}
  Held(const Held& h) : o(h.o) { Py_XINCREF(o); }
  Held& operator=(const Held&) = delete;
  ~Held() { Py_XDECREF(o); }
};

// The tensors of a sequence or iterator.  They live as long as this does: what a generator makes would
// otherwise be freed before the call is enqueued, and its memory given to the call's own workspace.
struct List {
  Held held;
  std::vector<void*> p;
  std::vector<int64_t> n;
  at::ScalarType type = at::kFloat;
  int32_t count() const { return int32_t(p.size()); }
  void all_changed() const {
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(held.o); ++i)
      changed(THPVariable_Unpack(PySequence_Fast_GET_ITEM(held.o, i)));
  }

  List(const Device& d, PyObject* o, const char* name) : held(PySequence_Fast(o, "a sequence of tensors is wanted")) {
    PyObject* seq = held.o;
    if (seq == nullptr) throw Refused();
    const Py_ssize_t size = PySequence_Fast_GET_SIZE(seq);
    NEED(size <= INT32_MAX, "too many ", name);
    p.reserve(size_t(size));
    n.reserve(size_t(size));
    for (Py_ssize_t i = 0; i < size; ++i) {
      const at::Tensor& t = tensor(PySequence_Fast_GET_ITEM(seq, i), name);
      on(d, t, name);
      if (i == 0) type = t.scalar_type();
      NEED(is_float(t.scalar_type()), name, " must be of ", kFloats, ", got ", c10::toString(t.scalar_type()));
      NEED(t.scalar_type() == type, "all ", name, " must have one dtype");
      NEED(t.is_contiguous(), "all ", name, " must be contiguous");
      p.push_back(t.data_ptr());
      n.push_back(t.numel());
    }
  }
};

// outs: like the gradients, or None for the gradients themselves.
List outputs(const Device& d, PyObject* o, const List& g) {
  if (o == Py_None) return g;
  List outs(d, o, "outs");
  NEED(outs.n == g.n, "outs must have the gradients' sizes");
  NEED(g.p.empty() || outs.type == g.type, "outs must have the gradients' dtype");
  return outs;
}
void one_value(const Device& d, Opt t, const char* name, at::ScalarType type) {
  if (t == nullptr) return;
  on(d, *t, name);
  NEED(t->scalar_type() == type, name, " must be of ", c10::toString(type), ", got ", c10::toString(t->scalar_type()));
  NEED(t->numel() == 1, name, " must hold one value");
}
// The first of a list, or a matrix of which each row is one, tells a tensor of the host apart before the
// device is asked for.
void first_on_gpu(PyObject* list, const char* name) {
  if (THPVariable_Check(list)) return on_gpu(THPVariable_Unpack(list), name);
  if (PySequence_Check(list) && PySequence_Size(list) > 0)
    if (PyObject* o = PySequence_GetItem(list, 0)) {
      const bool host = THPVariable_Check(o) && !THPVariable_Unpack(o).is_cuda();
      Py_DECREF(o);
      NEED(!host, name, " must be on the current device");
    }
  if (PyErr_Occurred()) throw Refused();
}

using Args = PyObject* const*;
void arity(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "takes ", want, " arguments, got ", n);
}

// grads, norm, sumsq, workspace
PyObject* grad_norm(Args a, Py_ssize_t n) {
  arity(n, 4);
  first_on_gpu(a[0], "grads");
  const Device d;
  const List g(d, a[0], "grads");
  const Output norm(a[1], "norm", [&] { return d.empty({}, at::kFloat); });
  const Opt sumsq = optional(a[2], "sumsq");
  one_value(d, norm.t, "norm", at::kFloat);
  one_value(d, sumsq, "sumsq", at::kDouble);
  const int type = code(g.type);
  const Workspace ws(d, optional(a[3], "workspace"), tide_grad_norm_workspace(g.count(), g.n.data(), type),
                     "tide_grad_norm");
  check(tide_grad_norm(g.count(), g.p.data(), g.n.data(), type, static_cast<double*>(at_of(sumsq)),
                       static_cast<float*>(at_of(norm.t)), ws.p, ws.bytes, d.stream()),
        "tide_grad_norm");
  if (sumsq != nullptr) changed(*sumsq);
  return norm.result();
}

// grads, sumsq, max_norm, outs, norm
PyObject* grad_clip(Args a, Py_ssize_t n) {
  arity(n, 5);
  const at::Tensor& sumsq = tensor(a[1], "sumsq");
  on_gpu(sumsq, "sumsq");
  const double max_norm = number(a[2]);  // before addresses are taken: it may run Python code
  const Device d;
  const List g(d, a[0], "grads");
  const List outs = outputs(d, a[3], g);
  const Output norm(a[4], "norm", [&] { return d.empty({}, at::kFloat); });
  one_value(d, norm.t, "norm", at::kFloat);
  one_value(d, &sumsq, "sumsq", at::kDouble);
  check(tide_grad_clip(g.count(), g.p.data(), outs.p.data(), g.n.data(), code(g.type),
                       static_cast<double*>(sumsq.data_ptr()), max_norm, static_cast<float*>(at_of(norm.t)),
                       d.stream()),
        "tide_grad_clip");
  outs.all_changed();
  return norm.result();
}

// grads, max_norm, outs, norm, sumsq, workspace
PyObject* clip_grad_norm(Args a, Py_ssize_t n) {
  arity(n, 6);
  first_on_gpu(a[0], "grads");
  const double max_norm = number(a[1]);  // as in grad_clip
  const Device d;
  const List g(d, a[0], "grads");
  const List outs = outputs(d, a[2], g);
  const Output norm(a[3], "norm", [&] { return d.empty({}, at::kFloat); });
  const Opt sumsq = optional(a[4], "sumsq");
  one_value(d, norm.t, "norm", at::kFloat);
  one_value(d, sumsq, "sumsq", at::kDouble);
  const int type = code(g.type);
  const Workspace ws(d, optional(a[5], "workspace"), tide_grad_norm_workspace(g.count(), g.n.data(), type),
                     "tide_clip_grad_norm");
  check(tide_clip_grad_norm(g.count(), g.p.data(), outs.p.data(), g.n.data(), type, max_norm,
                            static_cast<double*>(at_of(sumsq)), static_cast<float*>(at_of(norm.t)), ws.p, ws.bytes,
                            d.stream()),
        "tide_clip_grad_norm");
  outs.all_changed();
  if (sumsq != nullptr) changed(*sumsq);
  return norm.result();
}

// ---------------------------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------------------------

// A tensor as rows of its last dimension.
struct Matrix {
  int64_t rows, cols, stride;
  Matrix(const at::Tensor& t, const char* name) {
    NEED(t.dim() >= 1, name, " must have at least one dimension");
    cols = t.size(-1);
    NEED(cols >= 1, name, " must have a last dimension of at least one");
    rows = t.numel() / cols;
    stride = cols;
    if (t.is_contiguous()) return;
    NEED(t.dim() == 2 && (t.stride(1) == 1 || cols == 1) && t.stride(0) >= cols, name,
         " must be contiguous, or a matrix whose rows are");
    stride = t.stride(0);
  }
};
void float_on(const Device& d, const at::Tensor& t, const char* name) {
  on(d, t, name);
  NEED(is_float(t.scalar_type()), name, " must be of ", kFloats, ", got ", c10::toString(t.scalar_type()));
}
// The parameters' one dtype: that of the first given, x's if there is none.
struct Params {
  at::ScalarType type;
  bool any = false;
  explicit Params(at::ScalarType x) : type(x) {}
  void add(const Device& d, Opt t, const char* name, int64_t cols) {
    if (t == nullptr) return;
    float_on(d, *t, name);
    NEED(t->dim() == 1 && t->size(0) == cols, name, " must have shape [", cols, "], got ", t->sizes());
    dense(*t, name);
    NEED(!any || t->scalar_type() == type, "weight, bias and their gradients must have one dtype");
    type = t->scalar_type();
    any = true;
  }
};

// x, weight, bias, eps, out, mean, rstd
PyObject* layer_norm(Args a, Py_ssize_t n) {
  arity(n, 7);
  const at::Tensor& x = tensor(a[0], "x");
  on_gpu(x, "x");
  const Device d;
  float_on(d, x, "x");
  const Matrix m(x, "x");
  const Opt weight = optional(a[1], "weight"), bias = optional(a[2], "bias");
  Params params(x.scalar_type());
  params.add(d, weight, "weight", m.cols);
  params.add(d, bias, "bias", m.cols);
  const auto per_row = x.sizes().slice(0, size_t(x.dim()) - 1);
  const Output y(a[4], "out", [&] { return d.empty(x.sizes(), x.scalar_type()); });
  const Output mean(a[5], "mean", [&] { return d.empty(per_row, at::kFloat); });
  const Output rstd(a[6], "rstd", [&] { return d.empty(per_row, at::kFloat); });
  like(d, *y.t, "out", x.scalar_type(), x.sizes());
  like(d, *mean.t, "mean", at::kFloat, per_row);
  like(d, *rstd.t, "rstd", at::kFloat, per_row);
  dense(*mean.t, "mean");
  dense(*rstd.t, "rstd");
  check(tide_layer_norm(m.rows, m.cols, x.data_ptr(), m.stride, code(x.scalar_type()), at_of(weight), at_of(bias),
                        code(params.type), float(number(a[3])), y.t->data_ptr(), Matrix(*y.t, "out").stride,
                        static_cast<float*>(mean.t->data_ptr()), static_cast<float*>(rstd.t->data_ptr()), d.stream()),
        "tide_layer_norm");
  return triple(y, mean, rstd);
}

// dy, x, weight, mean, rstd, dx, dweight, dbias, workspace
PyObject* layer_norm_bwd(Args a, Py_ssize_t n) {
  arity(n, 9);
  const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x");
  const at::Tensor &mean = tensor(a[3], "mean"), &rstd = tensor(a[4], "rstd");
  on_gpu(x, "x");
  const Device d;
  float_on(d, x, "x");
  const Matrix m(x, "x");
  like(d, dy, "dy", x.scalar_type(), x.sizes());
  const auto per_row = x.sizes().slice(0, size_t(x.dim()) - 1);
  like(d, mean, "mean", at::kFloat, per_row);
  like(d, rstd, "rstd", at::kFloat, per_row);
  dense(mean, "mean");
  dense(rstd, "rstd");
  const Opt weight = optional(a[2], "weight");
  Params params(x.scalar_type());
  params.add(d, weight, "weight", m.cols);
  params.add(d, optional(a[6], "dweight"), "dweight", m.cols);
  params.add(d, optional(a[7], "dbias"), "dbias", m.cols);
  const Output dx(a[5], "dx", [&] { return d.empty(x.sizes(), x.scalar_type()); });
  const Output dw(a[6], "dweight", [&] { return d.empty({m.cols}, params.type); });
  const Output db(a[7], "dbias", [&] { return d.empty({m.cols}, params.type); });
  like(d, *dx.t, "dx", x.scalar_type(), x.sizes());
  const int type = code(x.scalar_type());
  const Workspace ws(d, optional(a[8], "workspace"), tide_layer_norm_bwd_workspace(m.rows, m.cols, type),
                     "tide_layer_norm_bwd");
  check(tide_layer_norm_bwd(m.rows, m.cols, dy.data_ptr(), Matrix(dy, "dy").stride, x.data_ptr(), m.stride, type,
                            at_of(weight), code(params.type), static_cast<float*>(mean.data_ptr()),
                            static_cast<float*>(rstd.data_ptr()), dx.t->data_ptr(), Matrix(*dx.t, "dx").stride,
                            dw.t->data_ptr(), db.t->data_ptr(), ws.p, ws.bytes, d.stream()),
        "tide_layer_norm_bwd");
  return triple(dx, dw, db);
}

// ---------------------------------------------------------------------------------------------
// Embedding
// ---------------------------------------------------------------------------------------------

void ids_on(const Device& d, const at::Tensor& ids) {
  on(d, ids, "ids");
  NEED(is_id(ids.scalar_type()), "ids must be of torch.int32 or torch.int64, got ", c10::toString(ids.scalar_type()));
  dense(ids, "ids");
}

// ids, table, scale, out
PyObject* embedding(Args a, Py_ssize_t n) {
  arity(n, 4);
  const at::Tensor &ids = tensor(a[0], "ids"), &table = tensor(a[1], "table");
  on_gpu(ids, "ids");
  const Device d;
  ids_on(d, ids);
  float_on(d, table, "table");
  dense(table, "table");
  NEED(table.dim() == 2 && table.size(1) >= 1, "table must be [vocab, dim] with dim at least one");
  c10::SmallVector<int64_t, 6> shape(ids.sizes().begin(), ids.sizes().end());
  shape.push_back(table.size(1));
  const Output out(a[3], "out", [&] { return d.empty(shape, table.scalar_type()); });
  like(d, *out.t, "out", table.scalar_type(), shape);
  dense(*out.t, "out");
  check(tide_embedding(ids.numel(), ids.data_ptr(), code(ids.scalar_type()), table.size(0), table.size(1),
                       table.data_ptr(), code(table.scalar_type()), float(number(a[2])), out.t->data_ptr(), d.stream()),
        "tide_embedding");
  return out.result();
}

// ids, dy, vocab, scale, out, accumulate, workspace
PyObject* embedding_bwd(Args a, Py_ssize_t n) {
  arity(n, 7);
  const at::Tensor &ids = tensor(a[0], "ids"), &dy = tensor(a[1], "dy");
  on_gpu(ids, "ids");
  const Device d;
  ids_on(d, ids);
  float_on(d, dy, "dy");
  dense(dy, "dy");
  NEED(dy.dim() == ids.dim() + 1 && dy.sizes().slice(0, size_t(ids.dim())) == ids.sizes(),
       "dy must have shape ids.shape + (dim,)");
  const int64_t vocab = whole(a[2]), dim = dy.size(-1);
  NEED(dim >= 1, "dy must have a last dimension of at least one");
  NEED(vocab >= 0, "vocab must not be negative");
  const int accumulate = PyObject_IsTrue(a[5]);
  if (accumulate < 0) throw Refused();
  NEED(a[4] != Py_None || accumulate == 0, "accumulate needs the gradient to add to as `out`");
  const Output out(a[4], "out", [&] { return d.empty({vocab, dim}, dy.scalar_type()); });
  like(d, *out.t, "out", dy.scalar_type(), {vocab, dim});
  dense(*out.t, "out");
  const Workspace ws(d, optional(a[6], "workspace"), tide_embedding_bwd_workspace(ids.numel(), vocab, dim),
                     "tide_embedding_bwd");
  check(tide_embedding_bwd(ids.numel(), ids.data_ptr(), code(ids.scalar_type()), vocab, dim, dy.data_ptr(),
                           code(dy.scalar_type()), float(number(a[3])), accumulate, out.t->data_ptr(), ws.p, ws.bytes,
                           d.stream()),
        "tide_embedding_bwd");
  return out.result();
}

// TideError, raw stream of a device
PyObject* configure(Args a, Py_ssize_t n) {
  arity(n, 2);
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XDECREF(g_error);
  Py_XDECREF(g_raw_stream);
  g_error = a[0];
  g_raw_stream = a[1];
  Py_RETURN_NONE;
}

// No C++ exception passes into Python: torch's errors are translated, the others are already set.
template <PyObject* (*kFn)(Args, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return kFn(args, n);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*kFn)(Args, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kFn>)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {method<configure>("configure"),
                          method<grad_norm>("grad_norm"),
                          method<grad_clip>("grad_clip"),
                          method<clip_grad_norm>("clip_grad_norm"),
                          method<layer_norm>("layer_norm"),
                          method<layer_norm_bwd>("layer_norm_bwd"),
                          method<embedding>("embedding"),
                          method<embedding_bwd>("embedding_bwd"),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_step", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__step(void) { return PyModule_Create(&kModule); }
