// Python binding of the block join, the expert permutation and routing, the
// token embedding and the head's cross entropy: checks of the tensors, new
// outputs, the current stream, the C call of include/zero.h.
// train_ops.py has the functions' Python signatures and documentation.
//
// These calls are made many times a step and their kernels can take a few
// microseconds, so the marshalling is compiled. Measured in turn with the same
// calls through ctypes, us a pass: a join of one row of 4096 6.5-6.9 (ctypes
// 16.8-18.4), sort, dispatch and combine of 8 tokens 15-16 (31-35); forward and
// backward of a join keep the host 21-27 us (48-61).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <string>
#include <vector>

#include "zero.h"

namespace {

using at::Tensor;

PyObject* g_zero_error = nullptr;  // zero.ZeroError, set by train_ops

// A Python error is set; unwinds to the call's end.
struct PythonError {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw PythonError();
}
[[noreturn]] void value_error(const char* what, const std::string& text) {
  raise(PyExc_ValueError, std::string(what) + ": " + text);
}

void check(zero_status st) {
  if (st == ZERO_OK) return;
  PyObject* e = PyObject_CallFunction(g_zero_error, "is", static_cast<int>(st), zero_last_error());
  if (e) {
    PyErr_SetObject(g_zero_error, e);
    Py_DECREF(e);
  }
  throw PythonError();
}

// An argument that has to be a tensor, or may be None.
Tensor tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(what) + ": expected a torch.Tensor");
  return THPVariable_Unpack(o);
}
Tensor maybe(PyObject* o, const char* what) { return o == Py_None ? Tensor() : tensor(o, what); }

int type_of(at::ScalarType t, const char* what) {
  if (t == at::kHalf) return ZERO_FP16;
  if (t == at::kBFloat16) return ZERO_BF16;
  if (t == at::kFloat) return ZERO_FP32;
  raise(PyExc_TypeError, std::string(what) + ": expected float16, bfloat16 or float32");
}
int type_of(const Tensor& t, const char* what) { return type_of(t.scalar_type(), what); }

const char* name_of(at::ScalarType t) { return c10::toString(t); }
std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (int64_t n : s) r += std::to_string(n) + ", ";
  return r + ")";
}

// The device of the call's first tensor, which has to be the current one.
int device_of(const Tensor& t, const char* what) {
  if (!t.is_cuda()) value_error(what, "tensor must be on a CUDA device");
  const int dev = t.get_device();
  if (dev != c10::cuda::current_device())
    value_error(what, "on cuda:" + std::to_string(dev) + ", which is not the current device");
  return dev;
}
void on(const Tensor& t, const char* what, int dev) {
  if (!t.is_cuda() || t.get_device() != dev) value_error(what, "not on cuda:" + std::to_string(dev));
}

// Elements between rows of a tensor [..., hidden] whose rows are contiguous
// and evenly spaced.
int64_t row_stride(const Tensor& t, const char* what, at::IntArrayRef shape, int dev) {
  on(t, what, dev);
  if (t.sizes() != shape) value_error(what, "shape " + shape_of(t.sizes()) + ", expected " + shape_of(shape));
  const int64_t hidden = shape.back();
  if (t.is_contiguous()) return hidden;
  int64_t row = -1, next = -1;
  bool even = t.stride(-1) == 1 || hidden == 1;
  for (int64_t d = t.dim() - 2; d >= 0 && even; --d) {
    if (t.size(d) == 1) continue;
    if (row < 0)
      row = t.stride(d);
    else
      even = t.stride(d) == next;
    next = t.stride(d) * t.size(d);
  }
  if (!even) value_error(what, "rows must be contiguous and evenly spaced (use .contiguous())");
  return row < 0 ? hidden : row;
}

// A caller's output, checked, or a new one.
Tensor result(const Tensor& t, const char* what, at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  if (!t.defined()) return at::empty(shape, like.options().dtype(type));
  on(t, what, like.get_device());
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
    value_error(what, std::string("expected a contiguous ") + name_of(type) + " tensor of shape " + shape_of(shape) +
                          ", got " + name_of(t.scalar_type()) + " " + shape_of(t.sizes()) +
                          (t.is_contiguous() ? "" : ", not contiguous"));
  return t;
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }
int64_t number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError();
  return v != 0;
}
int small(PyObject* o, const char* what) {
  const int64_t v = number(o);
  if (v < INT32_MIN || v > INT32_MAX) value_error(what, "out of range");
  return static_cast<int>(v);
}

// Runs a C call without the interpreter's lock, as ctypes does.
template <class F>
void unlocked(F call) {
  zero_status st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  check(st);
}

PyObject* wrapped(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* tuple_of(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw PythonError();
  Py_ssize_t k = 0;
  for (const Tensor& t : ts) {
    PyObject* o = wrapped(t);
    if (!o) {
      Py_DECREF(r);
      throw PythonError();
    }
    PyTuple_SET_ITEM(r, k++, o);
  }
  return r;
}

Tensor workspace_of(PyObject* o, int64_t need, const Tensor& like) {
  if (o == Py_None) return at::empty({need}, like.options().dtype(at::kByte));
  Tensor t = tensor(o, "workspace");
  on(t, "workspace", like.get_device());
  if (!t.is_contiguous() || static_cast<int64_t>(t.nbytes()) < need)
    value_error("workspace", "needs " + std::to_string(need) + " contiguous bytes");
  return t;
}

// Runs a call's body; Python and torch errors become Python errors.
template <class F>
PyObject* guarded(F body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const PythonError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
void expect_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) raise(PyExc_TypeError, "expected " + std::to_string(want) + " arguments");
}

// ---------------------------------------------------------------------------
// block join

struct Join {
  Tensor x, b, w_post, bias_post, w_pre, bias_pre, gate;
  zero_join_desc d = {};
  zero_join_inputs in = {};
  int dev = 0;
  at::ScalarType act;

  // a: x, b, w_post, bias_post, w_pre, bias_pre, gate, kind, scale, eps;
  // act_like: whose type n has when there is no b (None: see below), and its name
  Join(PyObject* const* a, const Tensor& act_like, const char* act_name) {
    x = tensor(a[0], "x");
    dev = device_of(x, "x");
    if (x.dim() < 1) value_error("x", "expected [..., hidden]");
    const at::IntArrayRef shape = x.sizes();
    const int64_t hidden = shape.back();
    b = maybe(a[1], "b"), w_post = maybe(a[2], "w_post"), bias_post = maybe(a[3], "bias_post");
    w_pre = maybe(a[4], "w_pre"), bias_pre = maybe(a[5], "bias_pre"), gate = maybe(a[6], "gate");
    d.hidden = hidden;
    d.rows = hidden ? x.numel() / hidden : 0;
    d.res_dtype = type_of(x, "x");
    d.x_stride = row_stride(x, "x", shape, dev);
    act = x.scalar_type();
    const char* act_of = "x";
    if (b.defined()) {
      act = b.scalar_type(), act_of = "b";
      d.b_stride = row_stride(b, "b", shape, dev);
    } else if (act_like.defined()) {
      act = act_like.scalar_type(), act_of = act_name;
    } else if (act == at::kFloat && w_pre.defined()) {
      act = w_pre.scalar_type(), act_of = "w_pre";
    }
    d.act_dtype = d.param_dtype = d.gate_dtype = type_of(act, act_of);
    const Tensor* first = nullptr;
    vector(w_post, "w_post", hidden, first);
    vector(bias_post, "bias_post", hidden, first);
    vector(w_pre, "w_pre", hidden, first);
    vector(bias_pre, "bias_pre", hidden, first);
    if (first) d.param_dtype = type_of(*first, "parameters");
    if (gate.defined()) {
      on(gate, "gate", dev);
      d.gate_dtype = type_of(gate, "gate");
      if (gate.dim() == 1 && gate.size(0) == hidden && x.dim() != 1) {
        if (!gate.is_contiguous()) value_error("gate", "expected a contiguous vector");
        d.gate_kind = ZERO_GATE_CHANNEL;
      } else if (gate.sizes() == shape) {
        d.gate_kind = ZERO_GATE_FULL;
        d.gate_stride = row_stride(gate, "gate", shape, dev);
      } else {
        std::vector<int64_t> rows(shape.begin(), shape.end());
        rows.back() = 1;
        if (gate.sizes() != at::IntArrayRef(rows))
          value_error("gate", "shape " + shape_of(gate.sizes()) + ", expected a channel's, a row's or " +
                                  shape_of(shape));
        d.gate_kind = ZERO_GATE_ROW;
        d.gate_stride = row_stride(gate, "gate", rows, dev);
      }
    }
    if (PyUnicode_Check(a[7]) && PyUnicode_CompareWithASCIIString(a[7], "rms") == 0)
      d.kind = ZERO_JOIN_RMS;
    else if (PyUnicode_Check(a[7]) && PyUnicode_CompareWithASCIIString(a[7], "layer") == 0)
      d.kind = ZERO_JOIN_LAYER;
    else
      value_error("kind", "must be 'rms' or 'layer'");
    d.scale = real(a[8]);
    d.eps = real(a[9]);
    in = {ptr(x), ptr(b), ptr(gate), ptr(w_post), ptr(bias_post), ptr(w_pre), ptr(bias_pre)};
  }

  void vector(const Tensor& t, const char* what, int64_t hidden, const Tensor*& first) {
    if (!t.defined()) return;
    on(t, what, dev);
    if (t.dim() != 1 || t.size(0) != hidden || !t.is_contiguous())
      value_error(what, "expected a contiguous vector of " + std::to_string(hidden));
    if (!first)
      first = &t;
    else if (t.scalar_type() != first->scalar_type())
      raise(PyExc_TypeError, std::string(what) + ": another type than another parameter's");
  }
};

// x, b, w_post, bias_post, w_pre, bias_pre, gate, kind, scale, eps, o, n,
// want_o, want_stats -> (o, n, stats)
PyObject* block_join(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 14);
    Tensor o = maybe(a[10], "o"), n = maybe(a[11], "n"), stats;
    Join j(a, n, "n");
    if (n.defined() && !j.w_pre.defined()) value_error("n", "needs w_pre");
    const bool want_o = truth(a[12]) && (j.b.defined() || o.defined());
    if (want_o)
      o = result(o, "o", j.x.sizes(), j.x.scalar_type(), j.x);
    else
      o = Tensor();
    if (j.w_pre.defined()) n = result(n, "n", j.x.sizes(), j.act, j.x);
    if (truth(a[13])) stats = at::empty({j.d.rows, 4}, j.x.options().dtype(at::kFloat));
    void* stream = stream_of(j.dev);
    unlocked([&] { return zero_block_join(&j.d, &j.in, ptr(o), ptr(n), static_cast<float*>(ptr(stats)), stream); });
    if (!want_o && !j.b.defined()) o = j.x;
    return tuple_of({o, n, stats});
  });
}

// x, b, w_post, bias_post, w_pre, bias_pre, gate, kind, scale, eps -> bytes
PyObject* block_join_workspace_bytes(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 10);
    Join j(a, Tensor(), "");
    int64_t need = 0;
    check(zero_block_join_workspace_bytes(&j.d, &need));
    return PyLong_FromLongLong(need);
  });
}

constexpr int kGrads = 7;
PyObject* g_names[kGrads];  // "dx", "db", ...

// x, b, w_post, bias_post, w_pre, bias_pre, gate, kind, scale, eps, d_o, d_n,
// stats, want, workspace -> {"dx": ..., ...}
PyObject* block_join_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 15);
    const Tensor d_o = maybe(a[10], "d_o"), d_n = maybe(a[11], "d_n"), stats = maybe(a[12], "stats");
    Join j(a, d_n, "d_n");
    if (d_o.defined()) {
      if (d_o.scalar_type() != j.x.scalar_type()) raise(PyExc_TypeError, "d_o: another type than x");
      j.d.do_stride = row_stride(d_o, "d_o", j.x.sizes(), j.dev);
    }
    if (d_n.defined()) {
      if (d_n.scalar_type() != j.act) raise(PyExc_TypeError, "d_n: another type than b");
      j.d.dn_stride = row_stride(d_n, "d_n", j.x.sizes(), j.dev);
    }
    if (stats.defined()) result(stats, "stats", {j.d.rows, 4}, at::kFloat, j.x);
    const Tensor* like[kGrads] = {&j.x, &j.b, &j.gate, &j.w_post, &j.bias_post, &j.w_pre, &j.bias_pre};
    Tensor out[kGrads];
    void* at_[kGrads] = {};
    bool asked = false, sums = false, unused = false;
    for (int k = 0; k < kGrads; ++k) {
      if (!like[k]->defined()) continue;
      if (a[13] != Py_None) {
        const int has = PySequence_Contains(a[13], g_names[k]);
        if (has < 0) throw PythonError();
        if (!has) continue;
      }
      if (k >= 5 && !d_n.defined()) {  // n was not used
        out[k] = at::zeros(like[k]->sizes(), like[k]->options());
        unused = true;
        continue;
      }
      out[k] = at::empty(like[k]->sizes(), like[k]->options());
      at_[k] = out[k].data_ptr();
      asked = asked || at_[k];
      sums = sums || k >= 3 || (k == 2 && j.d.gate_kind == ZERO_GATE_CHANNEL);
    }
    if (!(unused && !asked)) {
      Tensor ws;
      int64_t need = 0;
      if (sums) {
        check(zero_block_join_workspace_bytes(&j.d, &need));
        ws = workspace_of(a[14], need, j.x);
      }
      const zero_join_grads g = {at_[0], at_[1], at_[2], at_[3], at_[4], at_[5], at_[6]};
      void* stream = stream_of(j.dev);
      unlocked([&] {
        return zero_block_join_backward(&j.d, &j.in, ptr(d_o), ptr(d_n), static_cast<const float*>(ptr(stats)), &g,
                                        ptr(ws), need, stream);
      });
    }
    PyObject* r = PyDict_New();
    if (!r) throw PythonError();
    for (int k = 0; k < kGrads; ++k) {
      PyObject* o = wrapped(out[k]);
      if (!o || PyDict_SetItem(r, g_names[k], o) < 0) {
        Py_XDECREF(o);
        Py_DECREF(r);
        throw PythonError();
      }
      Py_DECREF(o);
    }
    return r;
  });
}

// ---------------------------------------------------------------------------
// expert permutation

// ids, n_experts, workspace -> (offsets, rows, pairs)
PyObject* expert_sort(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 3);
    const Tensor ids = tensor(a[0], "ids");
    const int dev = device_of(ids, "ids");
    if (ids.dim() != 2 || !ids.is_contiguous()) value_error("ids", "expected a contiguous [tokens, topk] tensor");
    if (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong)
      raise(PyExc_TypeError, "ids: expected int32 or int64");
    const int64_t tokens = ids.size(0), topk = ids.size(1);
    if (topk < 1 || topk > INT32_MAX) value_error("ids", "topk must be at least 1");
    const int n_experts = small(a[1], "n_experts");
    int64_t need = 0;
    check(zero_expert_sort_workspace_bytes(tokens, static_cast<int32_t>(topk), n_experts, &need));
    const at::TensorOptions as = ids.options().dtype(at::kInt);
    const Tensor offsets = at::empty({static_cast<int64_t>(n_experts) + 1}, as), rows = at::empty(ids.sizes(), as),
                 pairs = at::empty({tokens * topk}, as);
    const Tensor ws = need ? workspace_of(a[2], need, ids) : Tensor();
    void* stream = stream_of(dev);
    unlocked([&] { return zero_expert_sort(ptr(ids), static_cast<int32_t>(ids.element_size()), tokens, static_cast<int32_t>(topk),
                           n_experts, static_cast<int32_t*>(ptr(offsets)), static_cast<int32_t*>(ptr(rows)),
                           static_cast<int32_t*>(ptr(pairs)), ptr(ws), need, stream); });
    return tuple_of({offsets, rows, pairs});
  });
}

struct Order {
  Tensor offsets, rows;
  int n_experts, topk;
  int64_t tokens;
  // a: offsets, rows, n_experts, tokens, topk
  Order(PyObject* const* a, int dev) {
    offsets = tensor(a[0], "order.offsets"), rows = tensor(a[1], "order.rows");
    n_experts = small(a[2], "n_experts"), tokens = number(a[3]), topk = small(a[4], "topk");
    on(offsets, "order", dev);
    on(rows, "order", dev);
    if (offsets.scalar_type() != at::kInt || rows.scalar_type() != at::kInt || !offsets.is_contiguous() ||
        !rows.is_contiguous() || rows.dim() != 2 || rows.size(0) != tokens || rows.size(1) != topk ||
        offsets.numel() != static_cast<int64_t>(n_experts) + 1)
      value_error("order", "not what zero_expert_sort returns");
  }
  const int32_t* first() const { return static_cast<const int32_t*>(ptr(offsets)); }
  const int32_t* places() const { return static_cast<const int32_t*>(ptr(rows)); }
  // [tokens * topk, hidden] in expert order
  void sorted(const Tensor& t, const char* what) const {
    if (t.dim() != 2 || t.size(0) != tokens * topk || !t.is_contiguous())
      value_error(what, "expected a contiguous [" + std::to_string(tokens * topk) + ", hidden] tensor");
  }
  // [tokens, hidden]; its row stride
  int64_t by_token(const Tensor& t, const char* what, int dev) const {
    if (t.dim() != 2 || t.size(0) != tokens)
      value_error(what, "expected [" + std::to_string(tokens) + ", hidden], got " + shape_of(t.sizes()));
    return row_stride(t, what, t.sizes(), dev);
  }
  int weights(const Tensor& t, int dev) const {
    on(t, "weights", dev);
    if (t.sizes() != rows.sizes() || !t.is_contiguous())
      value_error("weights", "expected a contiguous " + shape_of(rows.sizes()) + " tensor");
    return type_of(t, "weights");
  }
};

// x, (order's five), out -> xs
PyObject* expert_dispatch(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 7);
    const Tensor x = tensor(a[0], "x");
    const int dev = device_of(x, "x"), type = type_of(x, "x");
    const Order order(a + 1, dev);
    const int64_t stride = order.by_token(x, "x", dev), hidden = x.size(1);
    const Tensor xs = result(maybe(a[6], "out"), "out", {order.tokens * order.topk, hidden}, x.scalar_type(), x);
    void* stream = stream_of(dev);
    unlocked([&] { return zero_expert_dispatch(ptr(x), stride, static_cast<zero_dtype>(type), order.tokens, order.topk, hidden,
                               order.first(), order.n_experts, order.places(), ptr(xs), stream); });
    return wrapped(xs);
  });
}

// dxs, (order's five), out -> dx
PyObject* expert_dispatch_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 7);
    const Tensor dxs = tensor(a[0], "dxs");
    const int dev = device_of(dxs, "dxs"), type = type_of(dxs, "dxs");
    const Order order(a + 1, dev);
    order.sorted(dxs, "dxs");
    const int64_t hidden = dxs.size(1);
    const Tensor dx = result(maybe(a[6], "out"), "out", {order.tokens, hidden}, dxs.scalar_type(), dxs);
    void* stream = stream_of(dev);
    unlocked([&] { return zero_expert_dispatch_backward(ptr(dxs), static_cast<zero_dtype>(type), order.tokens, order.topk, hidden,
                                        order.places(), ptr(dx), stream); });
    return wrapped(dx);
  });
}

// ys, weights, (order's five), out -> y
PyObject* expert_combine(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 8);
    const Tensor ys = tensor(a[0], "ys"), weights = tensor(a[1], "weights");
    const int dev = device_of(ys, "ys"), type = type_of(ys, "ys");
    const Order order(a + 2, dev);
    order.sorted(ys, "ys");
    const int64_t hidden = ys.size(1);
    const int wtype = order.weights(weights, dev);
    const Tensor y = result(maybe(a[7], "out"), "out", {order.tokens, hidden}, ys.scalar_type(), ys);
    void* stream = stream_of(dev);
    unlocked([&] { return zero_expert_combine(ptr(ys), static_cast<zero_dtype>(type), ptr(weights), static_cast<zero_dtype>(wtype),
                              order.tokens, order.topk, hidden, order.places(), ptr(y), stream); });
    return wrapped(y);
  });
}

// dy, ys, weights, (order's five), want_weights -> (dys, dweights)
PyObject* expert_combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 9);
    const Tensor dy = tensor(a[0], "dy"), ys = tensor(a[1], "ys"), weights = tensor(a[2], "weights");
    const int dev = device_of(ys, "ys"), type = type_of(ys, "ys");
    const Order order(a + 3, dev);
    order.sorted(ys, "ys");
    const int64_t hidden = ys.size(1);
    on(dy, "dy", dev);
    const int64_t stride = order.by_token(dy, "dy", dev);
    if (dy.scalar_type() != ys.scalar_type() || dy.size(1) != hidden)
      raise(PyExc_TypeError, "dy: another type or row length than ys");
    const int wtype = order.weights(weights, dev);
    const Tensor dys = at::empty(ys.sizes(), ys.options());
    const Tensor dw = truth(a[8]) ? at::empty(weights.sizes(), weights.options()) : Tensor();
    void* stream = stream_of(dev);
    unlocked([&] { return zero_expert_combine_backward(ptr(dy), stride, ptr(ys), static_cast<zero_dtype>(type), ptr(weights),
                                       static_cast<zero_dtype>(wtype), order.tokens, order.topk, hidden,
                                       order.first(), order.n_experts, order.places(), ptr(dys), ptr(dw),
                                       stream); });
    return tuple_of({dys, dw});
  });
}

// ---------------------------------------------------------------------------
// router

at::ScalarType scalar_of(int type) {
  return type == ZERO_FP16 ? at::kHalf : type == ZERO_BF16 ? at::kBFloat16 : at::kFloat;
}

// Elements between rows of a matrix whose rows are contiguous.
int64_t matrix_stride(const Tensor& t, const char* what, int dev) {
  on(t, what, dev);
  if (t.dim() != 2) value_error(what, "expected a matrix, got " + shape_of(t.sizes()));
  return row_stride(t, what, t.sizes(), dev);
}

int id_bytes_of(const Tensor& t, const char* what, int dev) {
  on(t, what, dev);
  if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)
    raise(PyExc_TypeError, std::string(what) + ": expected int32 or int64");
  if (!t.is_contiguous()) value_error(what, "expected a contiguous tensor");
  return static_cast<int>(t.element_size());
}

// The logits' shape and stride.
struct Scores {
  Tensor z;
  int dev, type;
  int64_t tokens, stride;
  int experts;
  explicit Scores(PyObject* o) {
    z = tensor(o, "logits");
    dev = device_of(z, "logits"), type = type_of(z, "logits");
    stride = matrix_stride(z, "logits", dev);
    tokens = z.size(0);
    if (z.size(1) > INT32_MAX) value_error("logits", "too many experts");
    experts = static_cast<int>(z.size(1));
    if (tokens <= 1) stride = std::max(stride, z.size(1));
  }
};

// logits, topk, normalize, workspace -> (ids, weights, counts, losses, stats)
PyObject* expert_route(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 4);
    const Scores s(a[0]);
    const int topk = small(a[1], "topk");
    const bool normalize = truth(a[2]);
    int64_t need = 0;
    check(zero_expert_route_workspace_bytes(s.tokens, s.experts, &need));
    if (topk < 1 || topk > s.experts) value_error("topk", "must lie in [1, n_experts]");
    const at::TensorOptions f = s.z.options().dtype(at::kFloat), i = s.z.options().dtype(at::kInt);
    const Tensor ids = at::empty({s.tokens, topk}, i), weights = at::empty({s.tokens, topk}, f),
                 counts = at::empty({s.experts}, i), losses = at::empty({2}, f), stats = at::empty({s.tokens + 1}, f);
    const Tensor ws = need ? workspace_of(a[3], need, s.z) : Tensor();
    void* stream = stream_of(s.dev);
    unlocked([&] {
      return zero_expert_route(ptr(s.z), s.stride, static_cast<zero_dtype>(s.type), s.tokens, s.experts, topk, normalize,
                               static_cast<int32_t*>(ptr(ids)), static_cast<float*>(ptr(weights)),
                               static_cast<int32_t*>(ptr(counts)), static_cast<float*>(ptr(losses)),
                               static_cast<float*>(ptr(stats)), ptr(ws), need, stream);
    });
    return tuple_of({ids, weights, counts, losses, stats});
  });
}

// logits, normalize, ids, weights, counts, stats, d_weights, d_losses, out -> d_logits
PyObject* expert_route_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 9);
    const Scores s(a[0]);
    const bool normalize = truth(a[1]);
    const Tensor ids = tensor(a[2], "ids"), weights = tensor(a[3], "weights"), counts = tensor(a[4], "counts"),
                 stats = tensor(a[5], "stats"), dw = maybe(a[6], "d_weights"), dl = maybe(a[7], "d_losses");
    if (ids.dim() != 2 || ids.size(1) > INT32_MAX) value_error("ids", "expected [tokens, topk]");
    const int topk = static_cast<int>(ids.size(1));
    result(ids, "ids", {s.tokens, topk}, at::kInt, s.z);
    result(weights, "weights", {s.tokens, topk}, at::kFloat, s.z);
    result(counts, "counts", {s.experts}, at::kInt, s.z);
    result(stats, "stats", {s.tokens + 1}, at::kFloat, s.z);
    if (dw.defined()) result(dw, "d_weights", {s.tokens, topk}, at::kFloat, s.z);
    if (dl.defined()) result(dl, "d_losses", {2}, at::kFloat, s.z);
    const Tensor out = result(maybe(a[8], "out"), "out", s.z.sizes(), s.z.scalar_type(), s.z);
    void* stream = stream_of(s.dev);
    unlocked([&] {
      return zero_expert_route_backward(ptr(s.z), s.stride, static_cast<zero_dtype>(s.type), s.tokens, s.experts, topk,
                                        normalize, static_cast<const int32_t*>(ptr(ids)),
                                        static_cast<const float*>(ptr(weights)),
                                        static_cast<const int32_t*>(ptr(counts)),
                                        static_cast<const float*>(ptr(stats)), static_cast<const float*>(ptr(dw)),
                                        static_cast<const float*>(ptr(dl)), ptr(out), stream);
    });
    return wrapped(out);
  });
}

// ---------------------------------------------------------------------------
// token embedding

// ids, table, scale, type (-1: the table's), out -> y
PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 5);
    const Tensor ids = tensor(a[0], "ids"), table = tensor(a[1], "table");
    const int dev = device_of(table, "table"), from = type_of(table, "table");
    const int id_bytes = id_bytes_of(ids, "ids", dev);
    int64_t stride = matrix_stride(table, "table", dev);
    if (table.size(0) <= 1) stride = std::max(stride, table.size(1));
    const double scale = real(a[2]);
    Tensor y = maybe(a[4], "out");
    int type = small(a[3], "dtype");
    if (type < 0) type = y.defined() ? type_of(y, "out") : from;
    std::vector<int64_t> shape(ids.sizes().begin(), ids.sizes().end());
    shape.push_back(table.size(1));
    y = result(y, "out", shape, scalar_of(type), table);
    void* stream = stream_of(dev);
    unlocked([&] {
      return zero_embedding(ptr(ids), id_bytes, ids.numel(), ptr(table), stride, static_cast<zero_dtype>(from),
                            table.size(0), table.size(1), scale, ptr(y), static_cast<zero_dtype>(type), stream);
    });
    return wrapped(y);
  });
}

// dy, ids, vocab, scale, type (-1: dy's), out, accumulate, workspace -> dtable
PyObject* embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 8);
    const Tensor dy = tensor(a[0], "dy"), ids = tensor(a[1], "ids");
    const int dev = device_of(dy, "dy"), from = type_of(dy, "dy");
    const int id_bytes = id_bytes_of(ids, "ids", dev);
    if (dy.dim() < 1 || dy.sizes().slice(0, static_cast<size_t>(dy.dim() - 1)) != ids.sizes())
      value_error("dy", "shape " + shape_of(dy.sizes()) + ", expected " + shape_of(ids.sizes()) + " and the hidden size");
    const int64_t tokens = ids.numel(), hidden = dy.size(-1), vocab = number(a[2]);
    int64_t stride = row_stride(dy, "dy", dy.sizes(), dev);
    if (tokens <= 1) stride = std::max(stride, hidden);
    const double scale = real(a[3]);
    Tensor out = maybe(a[5], "out");
    const bool accumulate = truth(a[6]);
    if (accumulate && !out.defined()) value_error("accumulate", "needs out");
    int type = small(a[4], "dtype");
    if (type < 0) type = out.defined() ? type_of(out, "out") : from;
    int64_t need = 0;
    check(zero_embedding_workspace_bytes(tokens, vocab, hidden, &need));
    out = result(out, "out", {vocab, hidden}, scalar_of(type), dy);
    const Tensor ws = workspace_of(a[7], need, dy);
    void* stream = stream_of(dev);
    unlocked([&] {
      return zero_embedding_backward(ptr(dy), stride, static_cast<zero_dtype>(from), ptr(ids), id_bytes, tokens, vocab,
                                     hidden, scale, accumulate, ptr(out), static_cast<zero_dtype>(type), ptr(ws), need,
                                     stream);
    });
    return wrapped(out);
  });
}

// ---------------------------------------------------------------------------
// linear softmax cross entropy

struct Head {
  Tensor x, w, targets;
  zero_linear_ce_desc d = {};
  int dev;
  // a: x, w, targets, scale
  explicit Head(PyObject* const* a) {
    x = tensor(a[0], "x"), w = tensor(a[1], "w"), targets = tensor(a[2], "targets");
    dev = device_of(x, "x");
    if (x.dim() < 1) value_error("x", "expected [..., hidden]");
    if (x.scalar_type() != at::kHalf && x.scalar_type() != at::kBFloat16)
      raise(PyExc_TypeError, "x: expected float16 or bfloat16");
    d.hidden = x.size(-1);
    d.x_stride = row_stride(x, "x", x.sizes(), dev);
    d.w_stride = matrix_stride(w, "w", dev);
    if (w.size(1) != d.hidden)
      value_error("w", "shape " + shape_of(w.sizes()) + ", expected rows of " + std::to_string(d.hidden));
    if (w.scalar_type() != x.scalar_type()) raise(PyExc_TypeError, "w: another type than x");
    d.vocab = w.size(0);
    d.tokens = d.hidden ? x.numel() / d.hidden : 0;
    d.id_bytes = id_bytes_of(targets, "targets", dev);
    if (targets.sizes() != x.sizes().slice(0, static_cast<size_t>(x.dim() - 1)))
      value_error("targets", "shape " + shape_of(targets.sizes()) + ", expected that of x's rows");
    // one row or none: any stride
    if (d.tokens <= 1) d.x_stride = std::max(d.x_stride, d.hidden);
    if (d.vocab <= 1) d.w_stride = std::max(d.w_stride, d.hidden);
    d.dtype = d.dw_dtype = static_cast<zero_dtype>(type_of(x, "x"));
    d.scale = real(a[3]);
  }
  // type of dw, -1: that of a given one, or of w
  void dw_type(int type, const Tensor& dw) {
    if (type < 0) type = dw.defined() ? type_of(dw, "dw") : static_cast<int>(d.dtype);
    if (type != d.dtype && type != ZERO_FP32) raise(PyExc_TypeError, "dw: expected the type of w or float32");
    d.dw_dtype = static_cast<zero_dtype>(type);
  }
  Tensor workspace(PyObject* o, bool backward, int64_t* need) const {
    check(zero_linear_cross_entropy_workspace_bytes(&d, ptr(w), backward, need));
    return workspace_of(o, *need, x);
  }
};

// x, w, targets, scale, backward, dw_type -> bytes
PyObject* linear_cross_entropy_workspace_bytes(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 6);
    Head h(a);
    h.dw_type(small(a[5], "dw_dtype"), Tensor());
    int64_t need = 0;
    check(zero_linear_cross_entropy_workspace_bytes(&h.d, ptr(h.w), truth(a[4]), &need));
    return PyLong_FromLongLong(need);
  });
}

// x, w, targets, scale, workspace -> (losses, lse, total, rows, rest)
PyObject* linear_cross_entropy(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 5);
    const Head h(a);
    int64_t need = 0;
    const Tensor ws = h.workspace(a[4], false, &need);
    const at::TensorOptions f = h.x.options().dtype(at::kFloat);
    const Tensor losses = at::empty(h.targets.sizes(), f), lse = at::empty(h.targets.sizes(), f),
                 total = at::empty({3}, f), rows = at::empty({h.d.tokens + 1}, f.dtype(at::kInt)),
                 rest = at::empty(h.targets.sizes(), f);
    void* stream = stream_of(h.dev);
    unlocked([&] {
      return zero_linear_cross_entropy_rest(&h.d, ptr(h.x), ptr(h.w), ptr(h.targets), static_cast<float*>(ptr(losses)),
                                            static_cast<float*>(ptr(lse)), static_cast<float*>(ptr(rest)),
                                            static_cast<int32_t*>(ptr(rows)), static_cast<float*>(ptr(total)), ptr(ws),
                                            need, stream);
    });
    return tuple_of({losses, lse, total, rows, rest});
  });
}

// x, w, targets, scale, lse, rows, d_loss, reduction, want_dx, want_dw, dx, dw,
// dw_type (-1: w's), workspace, rest (None: from lse) -> (dx, dw)
PyObject* linear_cross_entropy_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    expect_args(n_args, 15);
    Head h(a);
    const Tensor lse = tensor(a[4], "lse"), rows = tensor(a[5], "rows"), d_loss = tensor(a[6], "d_loss"),
                 rest = maybe(a[14], "rest");
    const int reduction = small(a[7], "reduction");
    result(lse, "lse", h.targets.sizes(), at::kFloat, h.x);
    if (rest.defined()) result(rest, "rest", h.targets.sizes(), at::kFloat, h.x);
    result(rows, "rows", {h.d.tokens + 1}, at::kInt, h.x);
    if (reduction == ZERO_LOSS_NONE) {
      result(d_loss, "d_loss", h.targets.sizes(), at::kFloat, h.x);
    } else {
      on(d_loss, "d_loss", h.dev);
      if (d_loss.scalar_type() != at::kFloat || d_loss.numel() != 1)
        value_error("d_loss", "expected one float32 number");
    }
    Tensor dx = maybe(a[10], "dx"), dw = maybe(a[11], "dw");
    const bool want_dx = truth(a[8]), want_dw = truth(a[9]);
    if ((dx.defined() && !want_dx) || (dw.defined() && !want_dw)) value_error("want", "an output that is not wanted");
    h.dw_type(small(a[12], "dw_dtype"), dw);
    int64_t need = 0;
    const Tensor ws = h.workspace(a[13], true, &need);
    if (want_dx) dx = result(dx, "dx", h.x.sizes(), h.x.scalar_type(), h.x);
    if (want_dw) dw = result(dw, "dw", h.w.sizes(), scalar_of(h.d.dw_dtype), h.w);
    void* stream = stream_of(h.dev);
    unlocked([&] {
      const float *of_lse = static_cast<const float*>(ptr(lse)), *d = static_cast<const float*>(ptr(d_loss));
      const int32_t* list = static_cast<const int32_t*>(ptr(rows));
      if (!rest.defined())
        return zero_linear_cross_entropy_backward(&h.d, ptr(h.x), ptr(h.w), ptr(h.targets), of_lse, list, d, reduction,
                                                  ptr(dx), ptr(dw), ptr(ws), need, stream);
      return zero_linear_cross_entropy_rest_backward(&h.d, ptr(h.x), ptr(h.w), ptr(h.targets), of_lse,
                                                     static_cast<const float*>(ptr(rest)), list, d, reduction, ptr(dx),
                                                     ptr(dw), ptr(ws), need, stream);
    });
    return tuple_of({dx, dw});
  });
}

// The class of errors that the C calls' statuses raise.
PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_zero_error);
  g_zero_error = type;
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef g_methods[] = {
    {"set_error", set_error, METH_O, nullptr},
    {"block_join", fast(block_join), METH_FASTCALL, nullptr},
    {"block_join_workspace_bytes", fast(block_join_workspace_bytes), METH_FASTCALL, nullptr},
    {"block_join_backward", fast(block_join_backward), METH_FASTCALL, nullptr},
    {"expert_sort", fast(expert_sort), METH_FASTCALL, nullptr},
    {"expert_dispatch", fast(expert_dispatch), METH_FASTCALL, nullptr},
    {"expert_dispatch_backward", fast(expert_dispatch_backward), METH_FASTCALL, nullptr},
    {"expert_combine", fast(expert_combine), METH_FASTCALL, nullptr},
    {"expert_combine_backward", fast(expert_combine_backward), METH_FASTCALL, nullptr},
    {"expert_route", fast(expert_route), METH_FASTCALL, nullptr},
    {"expert_route_backward", fast(expert_route_backward), METH_FASTCALL, nullptr},
    {"embedding", fast(embedding), METH_FASTCALL, nullptr},
    {"embedding_backward", fast(embedding_backward), METH_FASTCALL, nullptr},
    {"linear_cross_entropy", fast(linear_cross_entropy), METH_FASTCALL, nullptr},
    {"linear_cross_entropy_workspace_bytes", fast(linear_cross_entropy_workspace_bytes), METH_FASTCALL, nullptr},
    {"linear_cross_entropy_backward", fast(linear_cross_entropy_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_train_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__train_ops() {
  static const char* const names[kGrads] = {"dx", "db", "dgate", "dw_post", "dbias_post", "dw_pre", "dbias_pre"};
  for (int k = 0; k < kGrads; ++k)
    if (!(g_names[k] = PyUnicode_InternFromString(names[k]))) return nullptr;
  return PyModule_Create(&g_module);
}
