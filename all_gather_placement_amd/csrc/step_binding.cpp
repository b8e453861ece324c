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
    } else if (needed > 0) {
      own = d.empty({needed}, at::kByte);
      given = &own;
    }
    p = at_of(given);
    bytes = given != nullptr ? given->numel() : 0;
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
template <typename... Outputs>
PyObject* together(const Outputs&... outputs) {
  const Output* o[] = {&outputs...};
  constexpr int kCount = int(sizeof...(Outputs));
  PyObject* r = PyTuple_New(kCount);
  if (r == nullptr) return nullptr;
  for (int i = 0; i < kCount; ++i) {
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
  return together(y, mean, rstd);
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
  return together(dx, dw, db);
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

// ---------------------------------------------------------------------------------------------
// Experts
// ---------------------------------------------------------------------------------------------

// experts, num_experts, align, place, source, offsets, workspace
PyObject* expert_sort(Args a, Py_ssize_t n) {
  arity(n, 7);
  const at::Tensor& ids = tensor(a[0], "experts");
  on_gpu(ids, "experts");
  const int64_t experts = whole(a[1]), align = whole(a[2]);
  NEED(experts >= 1 && experts <= TIDE_MAX_EXPERTS, "num_experts must be from 1 to ", TIDE_MAX_EXPERTS, ", got ", experts);
  NEED(align >= 1 && align <= INT32_MAX, "align must be at least one, got ", align);
  const Device d;
  on(d, ids, "experts");
  NEED(is_id(ids.scalar_type()), "experts must be of torch.int32 or torch.int64, got ", c10::toString(ids.scalar_type()));
  dense(ids, "experts");
  NEED(ids.dim() >= 1 && ids.size(-1) >= 1 && ids.size(-1) <= TIDE_MAX_CHOICES,
       "experts must be [..., choices] with 1 to ", TIDE_MAX_CHOICES, " choices, got ", ids.sizes());
  const int32_t choices = int32_t(ids.size(-1));
  const int64_t tokens = ids.numel() / choices;
  const int64_t rows = tide_expert_rows(tokens, choices, int32_t(experts), int32_t(align));
  NEED(rows >= 0, "there must be fewer than 2^31 pairs and rows");
  const Output place(a[3], "place", [&] { return d.empty(ids.sizes(), at::kInt); });
  const Output source(a[4], "source", [&] { return d.empty({rows}, at::kInt); });
  const Output offsets(a[5], "offsets", [&] { return d.empty({experts + 1}, at::kInt); });
  like(d, *place.t, "place", at::kInt, ids.sizes());
  like(d, *source.t, "source", at::kInt, {source.t->numel()});
  NEED(source.t->numel() >= rows, "source must hold ", rows, " rows at least, got ", source.t->numel());
  like(d, *offsets.t, "offsets", at::kInt, {experts + 1});
  dense(*place.t, "place");
  dense(*source.t, "source");
  dense(*offsets.t, "offsets");
  const Workspace ws(d, optional(a[6], "workspace"), tide_expert_sort_workspace(tokens, choices, int32_t(experts)),
                     "tide_expert_sort");
  check(tide_expert_sort(tokens, choices, ids.data_ptr(), code(ids.scalar_type()), int32_t(experts), int32_t(align),
                         static_cast<int32_t*>(place.t->data_ptr()), static_cast<int32_t*>(source.t->data_ptr()),
                         source.t->numel(), static_cast<int32_t*>(offsets.t->data_ptr()), ws.p, ws.bytes, d.stream()),
        "tide_expert_sort");
  return together(place, source, offsets);
}

// place and source, the first two of what expert_sort gives.
struct Sorted {
  const at::Tensor *place, *source;
  int64_t tokens, rows;
  int32_t choices;
  Sorted(const Device& d, PyObject* o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3)
      refuse(PyExc_TypeError, "sort must be the (place, source, offsets) of expert_sort");
    place = &tensor(PyTuple_GET_ITEM(o, 0), "place");
    source = &tensor(PyTuple_GET_ITEM(o, 1), "source");
    for (const auto& [t, name] : {std::pair(place, "place"), std::pair(source, "source")}) {
      on(d, *t, name);
      NEED(t->scalar_type() == at::kInt, name, " must be of Int, got ", c10::toString(t->scalar_type()));
      dense(*t, name);
    }
    NEED(place->dim() >= 1 && place->size(-1) >= 1 && place->size(-1) <= TIDE_MAX_CHOICES,
         "place must be [..., choices] with 1 to ", TIDE_MAX_CHOICES, " choices, got ", place->sizes());
    NEED(source->dim() == 1, "source must be [rows], got ", source->sizes());
    choices = int32_t(place->size(-1));
    tokens = place->numel() / choices;
    rows = source->numel();
  }
  const int32_t* at() const { return static_cast<const int32_t*>(place->data_ptr()); }
  const int32_t* from() const { return static_cast<const int32_t*>(source->data_ptr()); }
  // A tensor with a vector for each token.
  Matrix by_token(const at::Tensor& t, const char* name) const {
    const Matrix m(t, name);
    NEED(t.dim() == place->dim() && t.sizes().slice(0, size_t(t.dim()) - 1) == place->sizes().slice(0, size_t(t.dim()) - 1),
         name, " must have shape place.shape[:-1] + (dim,), got ", t.sizes(), " with place ", place->sizes());
    return m;
  }
  Matrix by_row(const at::Tensor& t, const char* name) const {
    const Matrix m(t, name);
    NEED(t.dim() == 2 && t.size(0) == rows, name, " must have shape [", rows, ", dim], got ", t.sizes());
    return m;
  }
  c10::SmallVector<int64_t, 6> token_shape(int64_t dim) const {
    c10::SmallVector<int64_t, 6> shape(place->sizes().begin(), place->sizes().end());
    shape.back() = dim;
    return shape;
  }
  void weights(const Device& d, const at::Tensor& t, const char* name) const {
    float_on(d, t, name);
    NEED(t.sizes() == place->sizes(), name, " must have shape ", place->sizes(), ", got ", t.sizes());
    dense(t, name);
  }
};

// x, sort, out
PyObject* expert_dispatch(Args a, Py_ssize_t n) {
  arity(n, 3);
  const at::Tensor& x = tensor(a[0], "x");
  on_gpu(x, "x");
  const Device d;
  float_on(d, x, "x");
  const Sorted s(d, a[1]);
  const Matrix m = s.by_token(x, "x");
  const Output out(a[2], "out", [&] { return d.empty({s.rows, m.cols}, x.scalar_type()); });
  like(d, *out.t, "out", x.scalar_type(), {s.rows, m.cols});
  check(tide_expert_dispatch(s.tokens, s.choices, m.cols, x.data_ptr(), m.stride, code(x.scalar_type()), s.at(), s.from(),
                             s.rows, out.t->data_ptr(), Matrix(*out.t, "out").stride, d.stream()),
        "tide_expert_dispatch");
  return out.result();
}

// rows, weights, sort, out
PyObject* expert_combine(Args a, Py_ssize_t n) {
  arity(n, 4);
  const at::Tensor& rows = tensor(a[0], "rows");
  on_gpu(rows, "rows");
  const Device d;
  float_on(d, rows, "rows");
  const Sorted s(d, a[2]);
  const Matrix m = s.by_row(rows, "rows");
  const Opt weights = optional(a[1], "weights");
  if (weights != nullptr) s.weights(d, *weights, "weights");
  const auto shape = s.token_shape(m.cols);
  const Output out(a[3], "out", [&] { return d.empty(shape, rows.scalar_type()); });
  like(d, *out.t, "out", rows.scalar_type(), shape);
  check(tide_expert_combine(s.tokens, s.choices, m.cols, rows.data_ptr(), m.stride, s.rows, code(rows.scalar_type()),
                            at_of(weights), weights != nullptr ? code(weights->scalar_type()) : TIDE_FP32, s.at(),
                            out.t->data_ptr(), Matrix(*out.t, "out").stride, d.stream()),
        "tide_expert_combine");
  return out.result();
}

// dy, rows, weights, sort, drows, dweights
PyObject* expert_combine_bwd(Args a, Py_ssize_t n) {
  arity(n, 6);
  const at::Tensor &dy = tensor(a[0], "dy"), &rows = tensor(a[1], "rows"), &weights = tensor(a[2], "weights");
  on_gpu(dy, "dy");
  const Device d;
  float_on(d, rows, "rows");
  const Sorted s(d, a[3]);
  const Matrix m = s.by_row(rows, "rows");
  like(d, dy, "dy", rows.scalar_type(), s.token_shape(m.cols));
  s.weights(d, weights, "weights");
  const Output drows(a[4], "drows", [&] { return d.empty(rows.sizes(), rows.scalar_type()); });
  const Output dweights(a[5], "dweights", [&] { return d.empty(weights.sizes(), weights.scalar_type()); });
  like(d, *drows.t, "drows", rows.scalar_type(), rows.sizes());
  like(d, *dweights.t, "dweights", weights.scalar_type(), weights.sizes());
  dense(*dweights.t, "dweights");
  check(tide_expert_combine_bwd(s.tokens, s.choices, m.cols, dy.data_ptr(), Matrix(dy, "dy").stride, rows.data_ptr(),
                                m.stride, s.rows, code(rows.scalar_type()), weights.data_ptr(),
                                code(weights.scalar_type()), s.at(), s.from(), drows.t->data_ptr(),
                                Matrix(*drows.t, "drows").stride, dweights.t->data_ptr(), d.stream()),
        "tide_expert_combine_bwd");
  return together(drows, dweights);
}

// ---------------------------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------------------------

// A tensor as vectors by token and head: [..., heads, dim] contiguous, or [tokens, heads, dim] of any strides
// but the last.
struct HeadVectors {
  int64_t tokens, heads, dim, token, head;
  HeadVectors(const at::Tensor& t, const char* name) {
    NEED(t.dim() >= 2, name, " must have shape [..., heads, dim], got ", t.sizes());
    heads = t.size(-2);
    dim = t.size(-1);
    tokens = 1;
    for (int64_t i = 0; i < t.dim() - 2; ++i) tokens *= t.size(i);
    token = heads * dim;
    head = dim;
    if (t.is_contiguous()) return;
    NEED(t.dim() == 3 && (t.stride(2) == 1 || dim <= 1), name,
         " must be contiguous, or [tokens, heads, dim] with contiguous vectors");
    token = t.stride(0);
    head = t.stride(1);
  }
};

// x, positions, freqs, sections, pairing, inverse, out
PyObject* rotary(Args a, Py_ssize_t n) {
  arity(n, 7);
  const at::Tensor &x = tensor(a[0], "x"), &positions = tensor(a[1], "positions"), &freqs = tensor(a[2], "freqs");
  on_gpu(x, "x");
  int32_t sections[TIDE_ROTARY_MAX_AXES];
  int64_t pairs = 0;
  int32_t axes = 0;
  {  // before addresses are taken: whole() may run Python code
    const Held seq(PySequence_Tuple(a[3]));
    if (seq.o == nullptr) throw Refused();
    const Py_ssize_t count = PyTuple_GET_SIZE(seq.o);
    NEED(count >= 1 && count <= TIDE_ROTARY_MAX_AXES, "there must be 1 to ", TIDE_ROTARY_MAX_AXES, " sections, got ", count);
    for (; axes < count; ++axes) {
      const int64_t v = whole(PyTuple_GET_ITEM(seq.o, axes));
      NEED(v >= 1 && v <= TIDE_ROTARY_MAX_DIM, "each section must have 1 to ", TIDE_ROTARY_MAX_DIM, " pairs, got ", v);
      sections[axes] = int32_t(v);
      pairs += v;
    }
  }
  const bool halves = PyUnicode_Check(a[4]) && PyUnicode_CompareWithASCIIString(a[4], "halves") == 0;
  NEED(halves || (PyUnicode_Check(a[4]) && PyUnicode_CompareWithASCIIString(a[4], "neighbours") == 0),
       "pairing must be 'halves' or 'neighbours'");
  const Device d;
  float_on(d, x, "x");
  const HeadVectors v(x, "x");
  NEED(v.dim >= 1 && v.dim <= TIDE_ROTARY_MAX_DIM && 2 * pairs <= v.dim, "sections of ", pairs, " pairs need vectors of ",
       2 * pairs, " to ", TIDE_ROTARY_MAX_DIM, " elements, got ", v.dim);
  NEED(v.heads <= TIDE_ROTARY_MAX_HEADS, "x must have at most ", TIDE_ROTARY_MAX_HEADS, " heads, got ", v.heads);
  on(d, positions, "positions");
  NEED(is_id(positions.scalar_type()) || positions.scalar_type() == at::kFloat,
       "positions must be of torch.int32, torch.int64 or torch.float32, got ", c10::toString(positions.scalar_type()));
  NEED(positions.dim() == x.dim() - 1 && positions.size(0) == axes &&
           positions.sizes().slice(1) == x.sizes().slice(0, size_t(x.dim()) - 2),
       "positions must have shape (", axes, ",) + x.shape[:-2], got ", positions.sizes());
  dense(positions, "positions");
  like(d, freqs, "freqs", at::kDouble, {pairs});
  dense(freqs, "freqs");
  const Output out(a[6], "out", [&] { return d.empty(x.sizes(), x.scalar_type()); });
  like(d, *out.t, "out", x.scalar_type(), x.sizes());
  const HeadVectors to(*out.t, "out");
  check(tide_rotary(v.tokens, v.heads, v.dim, x.data_ptr(), v.token, v.head, code(x.scalar_type()), positions.data_ptr(),
                    code(positions.scalar_type()), axes, sections, static_cast<const double*>(freqs.data_ptr()),
                    halves ? TIDE_ROTARY_HALVES : TIDE_ROTARY_NEIGHBOURS, a[5] == Py_True, out.t->data_ptr(), to.token,
                    to.head, d.stream()),
        "tide_rotary");
  return out.result();
}

// ---------------------------------------------------------------------------------------------
// Dropout
// ---------------------------------------------------------------------------------------------

// Any 64 bits, as a number with or without a sign.
uint64_t bits64(PyObject* o) {
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (over > 0) {
    const unsigned long long u = PyLong_AsUnsignedLongLong(o);
    if (u != ~0ull || !PyErr_Occurred()) return u;
    PyErr_Clear();
  }
  NEED(over == 0, "seed must fit 64 bits");
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return uint64_t(v);
}

// x, p, seed, offset, residual, out
PyObject* dropout(Args a, Py_ssize_t n) {
  arity(n, 6);
  const at::Tensor& x = tensor(a[0], "x");
  on_gpu(x, "x");
  const double p = number(a[1]);  // before addresses are taken: it may run Python code
  NEED(p >= 0 && p <= 1, "p must be from 0 to 1, got ", p);
  const Opt there = THPVariable_Check(a[2]) ? &THPVariable_Unpack(a[2]) : nullptr;
  const uint64_t seed = there != nullptr ? 0 : bits64(a[2]);
  const int64_t offset = whole(a[3]);
  NEED(offset >= 0, "offset must not be negative");
  const Device d;
  one_value(d, there, "seed", at::kLong);
  float_on(d, x, "x");
  const Matrix m(x, "x");
  const Opt residual = optional(a[4], "residual");
  if (residual != nullptr) like(d, *residual, "residual", x.scalar_type(), x.sizes());
  const Output out(a[5], "out", [&] { return d.empty(x.sizes(), x.scalar_type()); });
  like(d, *out.t, "out", x.scalar_type(), x.sizes());
  check(tide_dropout(m.rows, m.cols, x.data_ptr(), m.stride, code(x.scalar_type()), p, seed,
                     static_cast<const int64_t*>(at_of(there)), offset, at_of(residual),
                     residual != nullptr ? Matrix(*residual, "residual").stride : m.cols, out.t->data_ptr(),
                     Matrix(*out.t, "out").stride, d.stream()),
        "tide_dropout");
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
                          method<expert_sort>("expert_sort"),
                          method<expert_dispatch>("expert_dispatch"),
                          method<expert_combine>("expert_combine"),
                          method<expert_combine_bwd>("expert_combine_bwd"),
                          method<rotary>("rotary"),
                          method<dropout>("dropout"),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_step", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__step(void) { return PyModule_Create(&kModule); }
