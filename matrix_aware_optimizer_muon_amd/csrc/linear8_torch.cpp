// Python binding of the 8-bit linear layer (module _linear8): argument
// checks, allocation from torch's caching allocator, the current stream, and
// the calls of the C ABI (include/muon_linear8.h).  Written against CPython's
// vector call rather than ctypes because a call on one token is host bound:
// measured on the norm of one 3584-wide row, 15.1 us per call with ctypes and
// torch.empty from Python, 4.8 us here, of which the launch itself is 3.4 us.
//
// No work is done here: every result comes from libmuon.so's kernels.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "muon_linear8.h"

namespace {

PyObject* g_q8 = nullptr;     // class linear8.Q8
PyObject* g_error = nullptr;  // class MuonError(status, where)

// A Python exception that is already set.
struct Raised {};

[[noreturn]] void bad(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Raised();
}

void check(muon_status st, const char* where) {
  if (st == MUON_OK) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, where)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) bad(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// A tensor taken as rows of its last dimension.
struct Rows {
  int64_t r, c, ld;
};
Rows rows(const at::Tensor& t, const char* what) {
  const int64_t d = t.dim();
  if (d == 2) {
    const int64_t r = t.size(0), c = t.size(1), sr = t.stride(0), sc = t.stride(1);
    if (sc != 1 && c > 1 && r > 0) bad(std::string(what) + " must have unit stride in its last dimension");
    if (r > 1 && sr < c) bad(std::string(what) + " must have rows that do not overlap");
    return {r, c, sr > c ? sr : c};
  }
  if (d == 0) bad(std::string(what) + " must have at least one dimension");
  if (!t.is_contiguous()) bad(std::string(what) + " must be contiguous (or 2-D with any row stride)");
  int64_t r = 1;
  for (int64_t i = 0; i + 1 < d; ++i) r *= t.size(i);
  const int64_t c = t.size(d - 1);
  return {r, c, c};
}

muon_dtype typed(at::ScalarType t, const char* what) {
  if (t == at::kFloat) return MUON_F32;
  if (t == at::kBFloat16) return MUON_BF16;
  bad(std::string(what) + " must be fp32 or bf16");
}

void vector(const at::Tensor& t, int64_t n, const char* what) {
  if (t.scalar_type() != at::kFloat || t.numel() != n || !t.is_contiguous())
    bad(std::string(what) + " must be contiguous fp32 with " + std::to_string(n) + " elements");
}

struct Q8 {
  const at::Tensor& q;
  const at::Tensor& scale;
  Rows s;
};
Q8 q8(PyObject* o, const char* what) {
  if (!PyObject_TypeCheck(o, (PyTypeObject*)g_q8) || PyTuple_GET_SIZE(o) != 2)
    bad(std::string(what) + " must be a Q8");
  const at::Tensor& q = tensor(PyTuple_GET_ITEM(o, 0), what);
  const at::Tensor& s = tensor(PyTuple_GET_ITEM(o, 1), what);
  if (q.scalar_type() != at::kChar) bad(std::string(what) + ".q must be int8");
  const Rows r = rows(q, what);
  vector(s, r.r, (std::string(what) + ".scale").c_str());
  return {q, s, r};
}

at::ScalarType dtype(PyObject* o) {
  if (!THPDtype_Check(o)) bad("dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

void device(const at::Tensor& a) {
  if (!a.is_cuda()) bad("tensors must be CUDA tensors");
}
void device(const at::Tensor& a, const at::Tensor& b) {
  device(b);
  if (a.device() != b.device()) bad("tensors must be on one device");
}

void same(const at::Tensor& t, const at::Tensor& x, const char* what, const char* as) {
  if (t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type())
    bad(std::string(what) + " must have " + as + "'s shape and type");
}

// (past the dispatcher: at::empty took 0.25 us more, four times for a norm to
// 8 bits, 6.2 -> 5.2 us a call)
at::Tensor make(at::IntArrayRef size, at::ScalarType t, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(size, t, like.device(), std::nullopt));
}
at::IntArrayRef leading(const at::Tensor& t) { return t.sizes().slice(0, t.dim() - 1); }

// What a forward operator leaves for autograd, if it records and an input
// requires a gradient: a node that raises when a backward pass reaches it.  Of
// 8-bit rows the scale carries it.  (The backward operators leave nothing:
// their results are gradients already.)
template <typename... In> std::shared_ptr<torch::autograd::Node> undifferentiated(const char* name, const In&... in) {
  using namespace torch::autograd;
  if (!compute_requires_grad(in...)) return nullptr;
  return std::shared_ptr<Node>(new NotImplemented(name, collect_next_edges(in...)), deleteNode);
}
void mark(const at::Tensor& out, const std::shared_ptr<torch::autograd::Node>& node) {
  if (node) torch::autograd::set_history(out, node);
}

hipStream_t stream(const at::Tensor& t) {
  return c10::hip::getCurrentHIPStream(t.device().index()).stream();
}
template <typename T = void> T* ptr(const at::Tensor& t) { return (T*)t.data_ptr(); }

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* wrap8(at::Tensor q, at::Tensor s) {
  PyObject* a = wrap(std::move(q));
  PyObject* b = wrap(std::move(s));
  PyObject* r = PyObject_CallFunctionObjArgs(g_q8, a, b, nullptr);
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}
PyObject* tuple(std::initializer_list<PyObject*> v) {
  PyObject* t = PyTuple_New((Py_ssize_t)v.size());
  Py_ssize_t i = 0;
  for (PyObject* o : v) PyTuple_SET_ITEM(t, i++, o);
  return t;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) bad("wrong number of arguments");
}

PyObject* do_quantize(PyObject* const* a, Py_ssize_t n) {
  count(n, 1);
  const at::Tensor& x = tensor(a[0], "x");
  const muon_dtype t = typed(x.scalar_type(), "x");
  const Rows s = rows(x, "x");
  device(x);
  const c10::DeviceGuard guard(x.device());
  at::Tensor q = make(x.sizes(), at::kChar, x), scale = make(leading(x), at::kFloat, x);
  check(muon_q8_quantize(ptr(x), s.ld, t, s.r, s.c, ptr<int8_t>(q), s.c, ptr<float>(scale), stream(x)),
        "muon_q8_quantize");
  mark(scale, undifferentiated("linear8.quantize", x));
  return wrap8(std::move(q), std::move(scale));
}

PyObject* do_dequantize(PyObject* const* a, Py_ssize_t n) {
  count(n, 2);
  const Q8 x = q8(a[0], "x");
  const at::ScalarType st = dtype(a[1]);
  const muon_dtype t = typed(st, "dtype");
  device(x.q);
  device(x.q, x.scale);
  const c10::DeviceGuard guard(x.q.device());
  at::Tensor out = make(x.q.sizes(), st, x.q);
  check(muon_q8_dequantize(ptr<int8_t>(x.q), x.s.ld, ptr<float>(x.scale), x.s.r, x.s.c, ptr(out), x.s.c, t,
                           stream(x.q)),
        "muon_q8_dequantize");
  mark(out, undifferentiated("linear8.dequantize", x.scale));
  return wrap(std::move(out));
}

// x, weight, residual or None, eps, q8
PyObject* do_rmsnorm(PyObject* const* a, Py_ssize_t n) {
  count(n, 5);
  const at::Tensor& x = tensor(a[0], "x");
  const at::Tensor& w = tensor(a[1], "weight");
  const muon_dtype t = typed(x.scalar_type(), "x");
  const Rows s = rows(x, "x");
  vector(w, s.c, "weight");
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised();
  const int eight = PyObject_IsTrue(a[4]);
  if (eight < 0) throw Raised();
  const void* res = nullptr;
  int64_t ldr = 0;
  const at::Tensor* residual = nullptr;
  if (a[2] != Py_None) {
    const at::Tensor& r = tensor(a[2], "residual");
    same(r, x, "residual", "x");
    ldr = rows(r, "residual").ld;
    device(x, r);
    res = ptr(r);
    residual = &r;
  }
  device(x);
  device(x, w);
  const c10::DeviceGuard guard(x.device());
  // (a residual with no elements has no address either)
  at::Tensor h = a[2] != Py_None ? make(x.sizes(), x.scalar_type(), x) : x;
  at::Tensor rstd = make(leading(x), at::kFloat, x);
  at::Tensor y = make(x.sizes(), eight ? at::kChar : x.scalar_type(), x);
  at::Tensor scale;
  if (eight) scale = make(leading(x), at::kFloat, x);
  check(muon_rmsnorm_forward(ptr(x), s.ld, res, ldr, ptr<float>(w), t, s.r, s.c, (float)eps,
                             res ? ptr(h) : nullptr, s.c, eight ? nullptr : ptr(y), s.c,
                             eight ? ptr<int8_t>(y) : nullptr, s.c, eight ? ptr<float>(scale) : nullptr,
                             ptr<float>(rstd), stream(x)),
        "muon_rmsnorm_forward");
  if (const auto node = undifferentiated("linear8.rmsnorm", x, w, residual ? *residual : x)) {
    mark(eight ? scale : y, node);
    mark(rstd, node);
    if (residual) mark(h, node);
  }
  PyObject* first = eight ? wrap8(std::move(y), std::move(scale)) : wrap(std::move(y));
  if (!first) throw Raised();
  PyObject* second;
  if (a[2] != Py_None) {
    second = wrap(std::move(h));
  } else {
    second = a[0];
    Py_INCREF(second);
  }
  return tuple({first, second, wrap(std::move(rstd))});
}

// dy, h (tensor or Q8), rstd, weight, dh or None
PyObject* do_rmsnorm_backward(PyObject* const* a, Py_ssize_t n) {
  count(n, 5);
  const at::Tensor& dy = tensor(a[0], "dy");
  const muon_dtype t = typed(dy.scalar_type(), "dy");
  const Rows s = rows(dy, "dy");
  const void* h;
  const float* hs = nullptr;
  int64_t ldh;
  const at::Tensor* on[3] = {nullptr, nullptr, nullptr};
  if (PyObject_TypeCheck(a[1], (PyTypeObject*)g_q8)) {
    const Q8 v = q8(a[1], "h");
    if (v.s.r != s.r || v.s.c != s.c) bad("h must have dy's shape");
    h = ptr(v.q);
    hs = ptr<float>(v.scale);
    ldh = v.s.ld;
    on[0] = &v.q;
    on[1] = &v.scale;
  } else {
    const at::Tensor& v = tensor(a[1], "h");
    same(v, dy, "h", "dy");
    h = ptr(v);
    ldh = rows(v, "h").ld;
    on[0] = &v;
  }
  const at::Tensor& rstd = tensor(a[2], "rstd");
  const at::Tensor& w = tensor(a[3], "weight");
  vector(rstd, s.r, "rstd");
  vector(w, s.c, "weight");
  const void* dh = nullptr;
  int64_t lddh = 0;
  if (a[4] != Py_None) {
    const at::Tensor& v = tensor(a[4], "dh");
    same(v, dy, "dh", "dy");
    lddh = rows(v, "dh").ld;
    dh = ptr(v);
    on[2] = &v;
  }
  device(dy);
  for (const at::Tensor* v : on)
    if (v) device(dy, *v);
  device(dy, rstd);
  device(dy, w);
  const c10::DeviceGuard guard(dy.device());
  size_t need = 0;
  check(muon_rmsnorm_backward_workspace(s.r, s.c, &need), "muon_rmsnorm_backward_workspace");
  at::Tensor dx = make(dy.sizes(), dy.scalar_type(), dy), dw = make({s.c}, at::kFloat, dy), ws;
  if (need) ws = make({(int64_t)need}, at::kByte, dy);
  check(muon_rmsnorm_backward(ptr(dy), s.ld, h, ldh, hs, ptr<float>(rstd), ptr<float>(w), dh, lddh, t, s.r,
                              s.c, ptr(dx), s.c, ptr<float>(dw), need ? ptr(ws) : nullptr, need, stream(dy)),
        "muon_rmsnorm_backward");
  return tuple({wrap(std::move(dx)), wrap(std::move(dw))});
}

at::Tensor scratch(muon_q8_product kind, const void* a, int64_t lda, const void* b, int64_t ldb, int64_t t,
                   int64_t n, int64_t k, const at::Tensor& like, size_t* need) {
  *need = 0;
  check(muon_q8_workspace(kind, a, lda, b, ldb, t, n, k, need), "muon_q8_workspace");
  return *need ? make({(int64_t)*need}, at::kByte, like) : at::Tensor();
}

c10::SmallVector<int64_t, 6> shaped(const at::Tensor& t, int64_t last) {
  c10::SmallVector<int64_t, 6> v(t.sizes().begin(), t.sizes().end());
  v.back() = last;
  return v;
}

// x (Q8), w (Q8), dtype
PyObject* do_matmul(PyObject* const* a, Py_ssize_t n) {
  count(n, 3);
  const Q8 x = q8(a[0], "x"), w = q8(a[1], "w");
  const at::ScalarType st = dtype(a[2]);
  const muon_dtype t = typed(st, "dtype");
  if (w.s.c != x.s.c || w.q.dim() != 2) bad("w must be (n, k) with x's last dimension k");
  device(x.q);
  device(x.q, x.scale);
  device(x.q, w.q);
  device(x.q, w.scale);
  const c10::DeviceGuard guard(x.q.device());
  at::Tensor y = make(shaped(x.q, w.s.r), st, x.q);
  size_t need;
  const at::Tensor ws = scratch(MUON_Q8_MATMUL, ptr(x.q), x.s.ld, ptr(w.q), w.s.ld, x.s.r, w.s.r, x.s.c, x.q, &need);
  check(muon_q8_matmul(ptr<int8_t>(x.q), x.s.ld, ptr<float>(x.scale), ptr<int8_t>(w.q), w.s.ld,
                       ptr<float>(w.scale), x.s.r, w.s.r, x.s.c, ptr(y), w.s.r, t, need ? ptr(ws) : nullptr,
                       need, stream(x.q)),
        "muon_q8_matmul");
  mark(y, undifferentiated("linear8.matmul", x.scale, w.scale));
  return wrap(std::move(y));
}

const at::Tensor& gradient(PyObject* o) {
  const at::Tensor& dy = tensor(o, "dy");
  if (dy.scalar_type() != at::kBFloat16) bad("dy must be bf16");
  return dy;
}

// dy, w (Q8), dtype
PyObject* do_grad_input(PyObject* const* a, Py_ssize_t n) {
  count(n, 3);
  const at::Tensor& dy = gradient(a[0]);
  const Rows s = rows(dy, "dy");
  const Q8 w = q8(a[1], "w");
  const at::ScalarType st = dtype(a[2]);
  const muon_dtype t = typed(st, "dtype");
  if (w.s.r != s.c || w.q.dim() != 2) bad("w must be (n, k) with dy's last dimension n");
  device(dy);
  device(dy, w.q);
  device(dy, w.scale);
  const c10::DeviceGuard guard(dy.device());
  at::Tensor dx = make(shaped(dy, w.s.c), st, dy);
  size_t need;
  const at::Tensor ws = scratch(MUON_Q8_GRAD_INPUT, ptr(dy), s.ld, ptr(w.q), w.s.ld, s.r, s.c, w.s.c, dy, &need);
  check(muon_q8_grad_input(ptr(dy), s.ld, ptr<int8_t>(w.q), w.s.ld, ptr<float>(w.scale), s.r, s.c, w.s.c,
                           ptr(dx), w.s.c, t, need ? ptr(ws) : nullptr, need, stream(dy)),
        "muon_q8_grad_input");
  return wrap(std::move(dx));
}

// dy, x (Q8), dtype, out or None, accumulate
PyObject* do_grad_weight(PyObject* const* a, Py_ssize_t n) {
  count(n, 5);
  const at::Tensor& dy = gradient(a[0]);
  const Rows s = rows(dy, "dy");
  const Q8 x = q8(a[1], "x");
  if (x.s.r != s.r) bad("dy and x must have the same number of rows");
  const int accumulate = PyObject_IsTrue(a[4]);
  if (accumulate < 0) throw Raised();
  at::Tensor out;
  if (a[3] != Py_None) {
    out = tensor(a[3], "out");
    if (out.dim() != 2 || out.size(0) != s.c || out.size(1) != x.s.c) bad("out must be (n, k)");
  } else if (accumulate) {
    bad("accumulate needs out");
  }
  const at::ScalarType st = out.defined() ? out.scalar_type() : dtype(a[2]);
  const muon_dtype t = typed(st, out.defined() ? "out" : "dtype");
  device(dy);
  device(dy, x.q);
  device(dy, x.scale);
  if (out.defined()) device(dy, out);
  const c10::DeviceGuard guard(dy.device());
  if (!out.defined()) out = make({s.c, x.s.c}, st, dy);
  const int64_t ldo = rows(out, "out").ld;
  size_t need;
  const at::Tensor ws = scratch(MUON_Q8_GRAD_WEIGHT, ptr(dy), s.ld, ptr(x.q), x.s.ld, s.r, s.c, x.s.c, dy, &need);
  check(muon_q8_grad_weight(ptr(dy), s.ld, ptr<int8_t>(x.q), x.s.ld, ptr<float>(x.scale), s.r, s.c, x.s.c,
                            ptr(out), ldo, t, accumulate, need ? ptr(ws) : nullptr, need, stream(dy)),
        "muon_q8_grad_weight");
  if (a[3] != Py_None) {
    if (!out.is_inference()) torch::autograd::impl::bump_version(out);  // (autograd sees the write)
    Py_INCREF(a[3]);
    return a[3];
  }
  return wrap(std::move(out));
}

// (Q8 class, error class): what the functions build and raise.
PyObject* do_classes(PyObject* const* a, Py_ssize_t n) {
  count(n, 2);
  if (!PyType_Check(a[0]) || !PyType_IsSubtype((PyTypeObject*)a[0], &PyTuple_Type)) bad("Q8 must be a tuple class");
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XDECREF(g_q8);
  Py_XDECREF(g_error);
  g_q8 = a[0];
  g_error = a[1];
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (!g_q8 && F != do_classes) bad("_linear8 is used through linear8");
    return F(a, n);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void (*)())entry<F>, METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<do_quantize>("quantize"),
                           method<do_dequantize>("dequantize"),
                           method<do_rmsnorm>("rmsnorm"),
                           method<do_rmsnorm_backward>("rmsnorm_backward"),
                           method<do_matmul>("matmul"),
                           method<do_grad_input>("grad_input"),
                           method<do_grad_weight>("grad_weight"),
                           method<do_classes>("set_classes"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_linear8", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__linear8() { return PyModule_Create(&g_module); }
