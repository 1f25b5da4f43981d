// block_binding.cpp -- the Python calls of block.py and optim.py for plain
// arguments: contiguous CUDA tensors of one device, the current one, with no
// gradient to record and no forward-mode tangent.  A function here checks its tensors, allocates the
// results, packs hcb_args and calls the library; where anything is not plain,
// or the library refuses, it returns None and has done nothing, and the Python
// code goes through the same call in full (views, errors, other devices).
// Call by call this takes a third of the time of the Python code, which for
// few tokens is longer than the kernel.
#define PY_SSIZE_T_CLEAN
#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <vector>

#include "adamw.h"
#include "hc_block.h"

namespace {

using Entry = int (*)(const hcb_args*, birkhoff4_stream_t);
using WorkspaceEntry = size_t (*)(int64_t, int32_t, int32_t);
Entry f_enter, f_enter_backward, f_leave, f_leave_backward;
WorkspaceEntry f_workspace;

int32_t code(at::ScalarType t) {
  return t == at::kFloat ? B4_F32 : t == at::kBFloat16 ? B4_BF16 : -1;
}

// What a call knows of its streams, and the checks of everything beside them.
struct Call {
  hcb_args args;
  const at::Tensor* x = nullptr;
  at::IntArrayRef lead;  // x's leading dimensions
  int64_t S = 0, C = 0, T = 0;
  c10::DeviceIndex dev = -1;
  bool plain = true, learns = false;

  static const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

  bool fits(const at::Tensor* t) {
    if (t == nullptr || !t->is_cuda() || !t->is_contiguous() || t->layout() != at::kStrided) return plain = false;
    if (t->get_device() != dev) return plain = false;
    if (t->_fw_grad(/*level=*/0).defined()) return plain = false;  // refused by the Python code, whatever the grad mode
    learns = learns || t->requires_grad();
    return true;
  }
  Call(PyObject* o) {
    memset(&args, 0, sizeof(args));
    args.norm = 1;
    x = tensor(o);
    if (x == nullptr || !x->is_cuda() || code(x->scalar_type()) < 0 || x->dim() < 2) {
      plain = false;
      return;
    }
    dev = x->get_device();
    if (dev != c10::cuda::current_device() || !fits(x)) {
      plain = false;
      return;
    }
    S = x->size(-2), C = x->size(-1);
    if (S < 1 || S > HCB_MAX_STREAMS || C < 1 || C > HCB_MAX_CHANNELS || x->numel() == 0) {
      plain = false;
      return;
    }
    T = x->numel() / (S * C);
    lead = x->sizes().slice(0, x->dim() - 2);
    args.T = T, args.S = static_cast<int32_t>(S), args.C = static_cast<int32_t>(C);
    args.x_dtype = code(x->scalar_type());
  }
  // lead followed by n (and m)
  std::vector<int64_t> shape(int64_t n, int64_t m = -1) const {
    std::vector<int64_t> s(lead.begin(), lead.end());
    s.push_back(n);
    if (m >= 0) s.push_back(m);
    return s;
  }
  bool leads(const at::Tensor& t, int64_t n, int64_t m = -1) const {
    const int64_t d = static_cast<int64_t>(lead.size());
    if (t.dim() != d + (m < 0 ? 1 : 2) || t.size(d) != n || (m >= 0 && t.size(d + 1) != m)) return false;
    return t.sizes().slice(0, d) == lead;
  }
  void streams(PyObject* o, const void** at, int64_t* ts, int64_t* ss) {
    if (!plain) return;
    const at::Tensor* t = tensor(o);
    if (!fits(t)) return;
    if (t->scalar_type() != x->scalar_type() || t->sizes() != x->sizes()) {
      plain = false;
      return;
    }
    *at = t->data_ptr(), *ts = S * C, *ss = C;
  }
  void row(PyObject* o, const void** at, int64_t* ts, bool sets_type = false) {
    if (!plain) return;
    const at::Tensor* t = tensor(o);
    if (!fits(t)) return;
    const int32_t k = code(t->scalar_type());
    if (sets_type) args.y_dtype = k;
    if (k < 0 || k != args.y_dtype || (k == B4_F32 && args.x_dtype == B4_BF16) || !leads(*t, C)) {
      plain = false;
      return;
    }
    *at = t->data_ptr(), *ts = C;
  }
  void few(PyObject* o, const void** at, int32_t* type, int64_t* ts, int64_t n, int64_t m = -1) {
    if (!plain || o == Py_None) return;
    const at::Tensor* t = tensor(o);
    if (!fits(t)) return;
    *type = code(t->scalar_type());
    if (*type < 0 || !leads(*t, n, m)) {
      plain = false;
      return;
    }
    *at = t->data_ptr(), *ts = m < 0 ? n : n * m;
  }
  void weight(PyObject* o, const void** at, int32_t* type) {
    if (!plain || o == Py_None) return;
    const at::Tensor* t = tensor(o);
    if (!fits(t)) return;
    *type = code(t->scalar_type());
    if (*type < 0 || t->dim() != 1 || t->size(0) != C) {
      plain = false;
      return;
    }
    *at = t->data_ptr();
  }
  // Nothing in the way of the library call.
  bool ready() const { return plain && !(learns && at::GradMode::is_enabled()); }

  at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, void** at) const {
    at::Tensor t = at::empty(sizes, x->options().dtype(type).requires_grad(false));
    *at = t.data_ptr();
    return t;
  }
  at::Tensor like(PyObject* o, void** at, bool wanted = true) const {
    if (o == Py_None || !wanted) return {};
    const at::Tensor& t = THPVariable_Unpack(o);
    return make(t.sizes(), t.scalar_type(), at);
  }
  at::Tensor scratch(int weights) {
    const size_t need = weights ? f_workspace(T, args.C, weights) : 0;
    if (need == 0) return {};
    at::Tensor t = make({static_cast<int64_t>(need)}, at::kByte, &args.workspace);
    args.workspace_bytes = need;
    return t;
  }
  bool run(Entry f) const {
    return f(&args, reinterpret_cast<birkhoff4_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream())) == B4_OK;
  }
};

PyObject* wrapped(at::Tensor t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(t));
}
template <size_t N>
PyObject* tuple(at::Tensor (&t)[N]) {
  PyObject* r = PyTuple_New(N);
  if (r == nullptr) return nullptr;
  for (size_t i = 0; i < N; ++i) {
    PyObject* o = wrapped(std::move(t[i]));
    if (o == nullptr) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// A number argument; anything else is not plain.
bool number(PyObject* o, float* v) {
  if (!PyFloat_CheckExact(o)) return false;
  *v = static_cast<float>(PyFloat_AS_DOUBLE(o));
  return true;
}
long whole(PyObject* o) { return PyLong_CheckExact(o) ? PyLong_AsLong(o) : -1; }
// Which of a gradient's results are wanted, from the argument behind the
// first n if there is one: bit k stands for result k.
struct Wanted {
  unsigned long bits;
  Wanted(PyObject* const* o, Py_ssize_t n, Py_ssize_t given) : bits(given > n ? whole(o[n]) : ~0ul) {}
  bool operator[](int k) const { return bits >> k & 1; }
};

// enter(x, a, weight, eps, y type or -1) -> h
PyObject* enter_impl(PyObject* const* o, Py_ssize_t) {
  Call c(o[0]);
  if (!c.plain || !number(o[3], &c.args.eps)) Py_RETURN_NONE;
  const long type = whole(o[4]);
  if (type > B4_BF16) Py_RETURN_NONE;
  c.args.y_dtype = type < 0 ? c.args.x_dtype : static_cast<int32_t>(type);
  if (c.args.y_dtype == B4_F32 && c.args.x_dtype == B4_BF16) Py_RETURN_NONE;
  c.streams(o[0], &c.args.x, &c.args.x_ts, &c.args.x_ss);
  c.few(o[1], &c.args.a, &c.args.a_dtype, &c.args.a_ts, c.S);
  c.weight(o[2], &c.args.w, &c.args.w_dtype);
  if (!c.ready()) Py_RETURN_NONE;
  at::Tensor h = c.make(c.shape(c.C), c.args.y_dtype == B4_BF16 ? at::kBFloat16 : at::kFloat, &c.args.h);
  if (!c.run(f_enter)) Py_RETURN_NONE;
  return wrapped(std::move(h));
}

// enter_backward(dh, x, a, weight, eps, dres[, wanted]) -> (dx, da, dweight)
PyObject* enter_backward_impl(PyObject* const* o, Py_ssize_t n) {
  const Wanted want(o, 6, n);
  Call c(o[1]);
  if (!c.plain || !number(o[4], &c.args.eps)) Py_RETURN_NONE;
  c.streams(o[1], &c.args.x, &c.args.x_ts, &c.args.x_ss);
  c.row(o[0], &c.args.dh, &c.args.dh_ts, true);
  c.few(o[2], &c.args.a, &c.args.a_dtype, &c.args.a_ts, c.S);
  c.weight(o[3], &c.args.w, &c.args.w_dtype);
  if (o[5] != Py_None) c.streams(o[5], &c.args.dres, &c.args.dres_ts, &c.args.dres_ss);
  if (!c.plain) Py_RETURN_NONE;
  at::Tensor out[3] = {c.like(o[1], &c.args.dx, want[0]), c.like(o[2], &c.args.da, want[1]),
                       c.like(o[3], &c.args.dw, want[2])};
  const at::Tensor ws = c.scratch(c.args.dw != nullptr);
  if (!c.run(f_enter_backward)) Py_RETURN_NONE;
  return tuple(out);
}

// What leave and its gradient have in common, from o[0] on:
// x, y, P, b, gate, act, weight, norm, scale, eps
bool leave_inputs(Call& c, PyObject* const* o) {
  const long act = whole(o[5]);
  if (!c.plain || act < 0 || !PyBool_Check(o[7]) || !number(o[8], &c.args.scale) || !number(o[9], &c.args.eps))
    return false;
  c.args.norm = o[7] == Py_True;
  c.row(o[1], &c.args.y, &c.args.y_ts, true);
  c.few(o[2], &c.args.P, &c.args.p_dtype, &c.args.P_ts, c.S, c.S);
  c.few(o[3], &c.args.b, &c.args.b_dtype, &c.args.b_ts, c.S);
  if (o[4] != Py_None) {
    c.args.act = static_cast<int32_t>(act);
    c.row(o[4], &c.args.gate, &c.args.gate_ts);
  }
  c.weight(o[6], &c.args.w, &c.args.w_dtype);
  return c.plain;
}

// leave(x, y, P, b, gate, act, weight, norm, scale, eps, want_h, a_next, weight_next, eps_next) -> (out, h)
PyObject* leave_impl(PyObject* const* o, Py_ssize_t) {
  Call c(o[0]);
  if (!leave_inputs(c, o) || !number(o[13], &c.args.eps_next)) Py_RETURN_NONE;
  c.streams(o[0], &c.args.x, &c.args.x_ts, &c.args.x_ss);
  const bool want_h = o[10] == Py_True;
  if (want_h) {
    c.few(o[11], &c.args.a, &c.args.a_dtype, &c.args.a_ts, c.S);
    c.weight(o[12], &c.args.w_next, &c.args.wn_dtype);
  }
  if (!c.ready()) Py_RETURN_NONE;
  at::Tensor out[2] = {c.like(o[0], &c.args.out), {}};
  if (want_h) out[1] = c.like(o[1], &c.args.h);
  if (!c.run(f_leave)) Py_RETURN_NONE;
  return tuple(out);
}

// leave_backward(x, y, P, b, gate, act, weight, norm, scale, eps, dout, dh, out, a_next, weight_next, eps_next[, wanted])
// -> (dx, dy, dP, db, dgate, dweight, da_next, dweight_next); dh None: leave's alone, and otherwise always dx
PyObject* leave_backward_impl(PyObject* const* o, Py_ssize_t n) {
  const Wanted want(o, 16, n);
  Call c(o[0]);
  if (!leave_inputs(c, o) || !number(o[15], &c.args.eps_next)) Py_RETURN_NONE;
  const bool mix = o[2] != Py_None, next = o[11] != Py_None;
  c.streams(o[10], &c.args.dout, &c.args.dout_ts, &c.args.dout_ss);
  if (mix) c.streams(o[0], &c.args.x, &c.args.x_ts, &c.args.x_ss);
  if (next) {
    c.row(o[11], &c.args.dh, &c.args.dh_ts);
    c.streams(o[12], &c.args.out_in, &c.args.out_ts, &c.args.out_ss);
    c.few(o[13], &c.args.a, &c.args.a_dtype, &c.args.a_ts, c.S);
    c.weight(o[14], &c.args.w_next, &c.args.wn_dtype);
  }
  if (!c.plain) Py_RETURN_NONE;
  at::Tensor out[8];
  // without a mixing matrix dx is dout, unless h's gradient is added to it
  out[0] = mix || next ? c.like(o[0], &c.args.dx, next || want[0]) : THPVariable_Unpack(o[10]);
  out[1] = c.like(o[1], &c.args.dy, want[1]);
  out[2] = c.like(o[2], &c.args.dP, want[2]);
  out[3] = c.like(o[3], &c.args.db, want[3]);
  out[4] = c.like(o[4], &c.args.dgate, want[4]);
  out[5] = c.like(o[6], &c.args.dw, want[5]);
  if (next) {
    out[6] = c.like(o[13], &c.args.da, want[6]);
    out[7] = c.like(o[14], &c.args.dw_next, want[7]);
  }
  const at::Tensor ws = c.scratch((c.args.dw != nullptr) + (c.args.dw_next != nullptr));
  if (!c.run(f_leave_backward)) Py_RETURN_NONE;
  return tuple(out);
}

// adamw_table(params, table, p type, device) -> (table, g type): the table is
// that of adamw_tensor with the addresses of p and g open.
PyObject* adamw_table_impl(PyObject* const* o, Py_ssize_t) {
  if (!PyList_CheckExact(o[0]) || !PyBytes_CheckExact(o[1])) Py_RETURN_NONE;
  const Py_ssize_t n = PyList_GET_SIZE(o[0]);
  const long type = whole(o[2]), dev = whole(o[3]);
  if (n == 0 || PyBytes_GET_SIZE(o[1]) != static_cast<Py_ssize_t>(n * sizeof(adamw_tensor))) Py_RETURN_NONE;
  std::vector<adamw_tensor> rows(n);
  memcpy(rows.data(), PyBytes_AS_STRING(o[1]), n * sizeof(adamw_tensor));
  int32_t kind = -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor* p = Call::tensor(PyList_GET_ITEM(o[0], i));
    if (p == nullptr || !p->is_cuda() || !p->is_contiguous() || p->get_device() != dev || p->numel() != rows[i].n ||
        code(p->scalar_type()) != type)
      Py_RETURN_NONE;
    const at::Tensor& g = p->grad();
    if (!g.defined() || g.layout() != at::kStrided || !g.is_cuda() || !g.is_contiguous() || g.get_device() != dev ||
        g.numel() != rows[i].n)
      Py_RETURN_NONE;
    const int32_t k = code(g.scalar_type());
    if (k < 0 || (i > 0 && k != kind)) Py_RETURN_NONE;
    kind = k;
    rows[i].p = p->data_ptr();
    rows[i].g = g.data_ptr();
  }
  return Py_BuildValue("(y#i)", reinterpret_cast<const char*>(rows.data()),
                       static_cast<Py_ssize_t>(n * sizeof(adamw_tensor)), static_cast<int>(kind));
}

// Calls IMPL with N arguments, or up to MORE more; C++ exceptions become Python's, with the types that torch gives them.
template <PyObject* (*IMPL)(PyObject* const*, Py_ssize_t), Py_ssize_t N, Py_ssize_t MORE = 0>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < N || n > N + MORE) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return IMPL(args, n);
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// init(addresses of hcb_enter, hcb_enter_backward, hcb_leave, hcb_leave_backward, hcb_workspace_bytes)
PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "expected 5 addresses");
    return nullptr;
  }
  void* f[5];
  for (int i = 0; i < 5; ++i) {
    f[i] = PyLong_AsVoidPtr(args[i]);
    if (f[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  f_enter = reinterpret_cast<Entry>(f[0]);
  f_enter_backward = reinterpret_cast<Entry>(f[1]);
  f_leave = reinterpret_cast<Entry>(f[2]);
  f_leave_backward = reinterpret_cast<Entry>(f[3]);
  f_workspace = reinterpret_cast<WorkspaceEntry>(f[4]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {
    {"init", FAST(init)},
    {"enter", FAST((entry<enter_impl, 5>))},
    {"enter_backward", FAST((entry<enter_backward_impl, 6, 1>))},
    {"leave", FAST((entry<leave_impl, 14>))},
    {"leave_backward", FAST((entry<leave_backward_impl, 16, 1>))},
    {"adamw_table", FAST((entry<adamw_table_impl, 4>))},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_binding() { return PyModule_Create(&module); }
