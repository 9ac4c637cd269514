// Python binding of the 8-bit floating-point layer (module _float8): argument
// checks, allocation, the current stream, and the calls of the C ABI
// (include/muon_float8.h).  No work is done here.
#include "binding.hpp"
#include "muon_float8.h"

namespace {

constexpr at::ScalarType kE4M3 = at::kFloat8_e4m3fn, kE8M0 = at::kFloat8_e8m0fnu;

PyObject* g_f8 = nullptr;  // class float8.F8

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }
int64_t blocks(int64_t v) { return (v + 127) / 128; }

// Matrices of a tensor's last two dimensions, `stride` elements apart.
struct Stack {
  int64_t count, r, c, ld, stride;
};
Stack stack(const at::Tensor& t, const char* what, bool written = false) {
  const int64_t d = t.dim();
  if (d != 2 && d != 3) bad(std::string(what) + " must have two or three dimensions");
  const int64_t count = d == 3 ? t.size(0) : 1, r = t.size(d - 2), c = t.size(d - 1);
  int64_t ld = t.stride(d - 2), stride = d == 3 ? t.stride(0) : 0;
  if (t.numel() > 0) {
    if (t.stride(d - 1) != 1 && c > 1) bad(std::string(what) + " must have unit stride in its last dimension");
    if (r > 1 && ld < c) bad(std::string(what) + " must have rows that do not overlap");
    if (r <= 1) ld = c;
    if (count <= 1) stride = 0;
    else if (stride < (written ? (r - 1) * ld + c : 0)) bad(std::string(what) + " must have matrices that do not overlap");
  }
  return {count, r, c, ld, stride};
}

// 8-bit rows start at multiples of 16 bytes and can be read to the next one
// behind their last column.
void readable(const at::Tensor& q, int64_t rows, int64_t c, int64_t ld, int64_t count, int64_t stride, const char* what) {
  if (q.numel() == 0) return;
  if ((uintptr_t)q.data_ptr() % 16 || (rows > 1 && ld % 16) || (count > 1 && stride % 16))
    bad(std::string(what) + ".q must start its rows at multiples of 16 bytes, as quantize lays them out");
  const int64_t last = q.storage_offset() + (count - 1) * stride + (rows - 1) * ld + up16(c);
  if (last > (int64_t)q.storage().nbytes())
    bad(std::string(what) + ".q must have room for 16 bytes at the end of its last row, as quantize leaves it");
}

struct F8 {
  const at::Tensor& q;
  const at::Tensor& scale;
};
F8 f8(PyObject* o, const char* what) {
  if (!PyObject_TypeCheck(o, (PyTypeObject*)g_f8) || PyTuple_GET_SIZE(o) != 2) bad(std::string(what) + " must be an F8");
  const F8 v = {tensor(PyTuple_GET_ITEM(o, 0), what), tensor(PyTuple_GET_ITEM(o, 1), what)};
  if (v.q.scalar_type() != kE4M3) bad(std::string(what) + ".q must be float8_e4m3fn");
  if (v.scale.scalar_type() != kE8M0) bad(std::string(what) + ".scale must be float8_e8m0fnu");
  if (!v.scale.is_contiguous()) bad(std::string(what) + ".scale must be contiguous");
  if (v.q.dim() < 1) bad(std::string(what) + ".q must have at least one dimension");
  return v;
}
// Whether an F8's scales are per 128 values of a row, or per 128 x 128.
bool of_rows(const F8& v) {
  const int64_t d = v.q.dim();
  return v.scale.dim() == d && v.scale.sizes().slice(0, d - 1) == v.q.sizes().slice(0, d - 1) &&
         v.scale.size(d - 1) == blocks(v.q.size(d - 1));
}
bool of_squares(const F8& v) {
  const int64_t d = v.q.dim();
  return d >= 2 && v.scale.dim() == d && v.scale.sizes().slice(0, d - 2) == v.q.sizes().slice(0, d - 2) &&
         v.scale.size(d - 2) == blocks(v.q.size(d - 2)) && v.scale.size(d - 1) == blocks(v.q.size(d - 1));
}

// Rows (..., c) of any row distance that all leading dimensions share.
Rows rows8(const F8& v, const char* what) {
  if (!of_rows(v)) bad(std::string(what) + ".scale must have a scale for each 128 values of a row");
  const at::Tensor& q = v.q;
  const int64_t d = q.dim(), c = q.size(d - 1);
  int64_t r = 1, ld = up16(c);
  bool found = false;
  if (q.numel() > 0) {
    if (q.stride(d - 1) != 1 && c > 1) bad(std::string(what) + ".q must have unit stride in its last dimension");
    for (int64_t i = d - 2; i >= 0; --i) {
      if (q.size(i) > 1) {
        if (!found) ld = q.stride(i);
        else if (q.stride(i) != ld * r) bad(std::string(what) + ".q must have one row distance in all its dimensions");
        found = true;
      }
      r *= q.size(i);
    }
    if (r > 1 && ld < c) bad(std::string(what) + ".q must have rows that do not overlap");
    readable(q, r, c, ld, 1, 0, what);
  } else {
    for (int64_t i = 0; i + 1 < d; ++i) r *= q.size(i);
  }
  return {r, c, ld};
}
Stack weights8(const F8& v, const char* what) {
  const Stack s = stack(v.q, what, true);
  if (!of_squares(v)) bad(std::string(what) + ".scale must have a scale for each 128 x 128 values of a matrix");
  readable(v.q, s.r, s.c, s.ld, s.count, s.stride, what);
  return s;
}

// A tensor of 8-bit rows, each starting at a multiple of 16 bytes.
at::Tensor make8(at::IntArrayRef sizes, const at::Tensor& like) {
  const int64_t d = (int64_t)sizes.size(), c = sizes[d - 1], ld = up16(c);
  if (c == ld || d == 0) return make(sizes, kE4M3, like);
  c10::SmallVector<int64_t, 6> room(sizes.begin(), sizes.end()), strides((size_t)d, 1);
  room.back() = ld;
  at::Tensor t = make(room, kE4M3, like);
  int64_t s = ld;
  for (int64_t i = d - 2; i >= 0; --i) {
    strides[i] = s;
    s *= std::max<int64_t>(sizes[i], 1);
  }
  t.unsafeGetTensorImpl()->set_sizes_and_strides(sizes, strides);
  return t;
}
at::Tensor scales(at::IntArrayRef sizes, bool squares, const at::Tensor& like) {
  c10::SmallVector<int64_t, 6> v(sizes.begin(), sizes.end());
  v.back() = blocks(v.back());
  if (squares) v[v.size() - 2] = blocks(v[v.size() - 2]);
  return make(v, kE8M0, like);
}

PyObject* wrap8(at::Tensor q, at::Tensor s) {
  PyObject* a = wrap(std::move(q));
  PyObject* b = wrap(std::move(s));
  PyObject* r = PyObject_CallFunctionObjArgs(g_f8, a, b, nullptr);
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

// x
PyObject* do_quantize(PyObject* const* a, Py_ssize_t n) {
  count(n, 1);
  const at::Tensor& x = tensor(a[0], "x");
  const muon_dtype t = typed(x.scalar_type(), "x");
  const Rows s = rows(x, "x");
  device(x);
  const c10::DeviceGuard guard(x.device());
  at::Tensor q = make8(x.sizes(), x), scale = scales(x.sizes(), false, x);
  check(muon_f8_quantize(ptr(x), s.ld, 0, t, 1, s.r, s.c, 1, ptr<uint8_t>(q), up16(s.c), 0, ptr<uint8_t>(scale), stream(x)),
        "muon_f8_quantize");
  mark(scale, undifferentiated("float8.quantize", x));
  return wrap8(std::move(q), std::move(scale));
}

// w
PyObject* do_quantize_weight(PyObject* const* a, Py_ssize_t n) {
  count(n, 1);
  const at::Tensor& w = tensor(a[0], "w");
  const muon_dtype t = typed(w.scalar_type(), "w");
  const Stack s = stack(w, "w");
  device(w);
  const c10::DeviceGuard guard(w.device());
  at::Tensor q = make8(w.sizes(), w), scale = scales(w.sizes(), true, w);
  check(muon_f8_quantize(ptr(w), s.ld, s.stride, t, s.count, s.r, s.c, 128, ptr<uint8_t>(q), up16(s.c), s.r * up16(s.c),
                         ptr<uint8_t>(scale), stream(w)),
        "muon_f8_quantize");
  mark(scale, undifferentiated("float8.quantize_weight", w));
  return wrap8(std::move(q), std::move(scale));
}

// x (F8), dtype
PyObject* do_dequantize(PyObject* const* a, Py_ssize_t n) {
  count(n, 2);
  const F8 x = f8(a[0], "x");
  const at::ScalarType st = dtype(a[1]);
  const muon_dtype t = typed(st, "dtype");
  device(x.q);
  device(x.q, x.scale);
  const c10::DeviceGuard guard(x.q.device());
  at::Tensor out;
  if (of_rows(x)) {
    const Rows s = rows8(x, "x");
    out = make(x.q.sizes(), st, x.q);
    check(muon_f8_dequantize(ptr<uint8_t>(x.q), s.ld, 0, ptr<uint8_t>(x.scale), 1, s.r, s.c, 1, ptr(out), s.c, 0, t,
                             stream(x.q)),
          "muon_f8_dequantize");
  } else {
    const Stack s = weights8(x, "x");
    out = make(x.q.sizes(), st, x.q);
    check(muon_f8_dequantize(ptr<uint8_t>(x.q), s.ld, s.stride, ptr<uint8_t>(x.scale), s.count, s.r, s.c, 128, ptr(out),
                             s.c, s.r * s.c, t, stream(x.q)),
          "muon_f8_dequantize");
  }
  mark(out, undifferentiated("float8.dequantize", x.q, x.scale));
  return wrap(std::move(out));
}

// ends or None: where each expert's rows end.
struct Ends {
  const int32_t* at = nullptr;
  int64_t experts = 1;
};
Ends ends_of(PyObject* o, const at::Tensor& like) {
  Ends e;
  if (o == Py_None) return e;
  const at::Tensor& t = tensor(o, "ends");
  if (t.scalar_type() != at::kInt || t.dim() != 1 || !t.is_contiguous() || t.numel() < 1)
    bad("ends must be contiguous int32 with an end for each expert");
  device(like, t);
  e.at = ptr<int32_t>(t);
  e.experts = t.numel();
  return e;
}

at::Tensor scratch(muon_f8_product kind, const void* a, int64_t lda, const Ends& e, int64_t t, int64_t n, int64_t k,
                   muon_dtype dtype, const at::Tensor& like, size_t* need) {
  *need = 0;
  check(muon_f8_workspace(kind, a, lda, e.at != nullptr, e.experts, t, n, k, dtype, need), "muon_f8_workspace");
  return *need ? make({(int64_t)*need}, at::kByte, like) : at::Tensor();
}

c10::SmallVector<int64_t, 6> shaped(const at::Tensor& t, int64_t last) {
  c10::SmallVector<int64_t, 6> v(t.sizes().begin(), t.sizes().end());
  v.back() = last;
  return v;
}

// The weights of a product: one matrix, or with ends one per expert.
Stack weights_of(const F8& w, const Ends& e) {
  const Stack s = weights8(w, "w");
  if (e.at ? w.q.dim() != 3 || s.count != e.experts : w.q.dim() != 2)
    bad(e.at ? "w must be (experts, n, k) with an expert for each of ends" : "w must be (n, k)");
  return s;
}

// x (F8), w (F8), ends or None, dtype
PyObject* do_matmul(PyObject* const* a, Py_ssize_t n) {
  count(n, 4);
  const F8 x = f8(a[0], "x"), w = f8(a[1], "w");
  const at::ScalarType st = dtype(a[3]);
  const muon_dtype t = typed(st, "dtype");
  const Rows s = rows8(x, "x");
  device(x.q);
  device(x.q, x.scale);
  device(x.q, w.q);
  device(x.q, w.scale);
  const Ends e = ends_of(a[2], x.q);
  const Stack m = weights_of(w, e);
  if (m.c != s.c) bad("w must be (n, k) with x's last dimension k");
  const c10::DeviceGuard guard(x.q.device());
  at::Tensor y = make(shaped(x.q, m.r), st, x.q);
  size_t need;
  const at::Tensor ws = scratch(MUON_F8_MATMUL, ptr(x.q), s.ld, e, s.r, m.r, s.c, t, x.q, &need);
  check(muon_f8_matmul(ptr<uint8_t>(x.q), s.ld, ptr<uint8_t>(x.scale), ptr<uint8_t>(w.q), m.ld, m.stride,
                       ptr<uint8_t>(w.scale), e.at, e.experts, s.r, m.r, s.c, ptr(y), m.r, t, need ? ptr(ws) : nullptr,
                       need, stream(x.q)),
        "muon_f8_matmul");
  mark(y, undifferentiated("float8.matmul", x.q, x.scale, w.q, w.scale));
  return wrap(std::move(y));
}

const at::Tensor& gradient(PyObject* o) {
  const at::Tensor& dy = tensor(o, "dy");
  if (dy.scalar_type() != at::kBFloat16) bad("dy must be bf16");
  return dy;
}

// dy, w (F8), ends or None, dtype
PyObject* do_grad_input(PyObject* const* a, Py_ssize_t n) {
  count(n, 4);
  const at::Tensor& dy = gradient(a[0]);
  const Rows s = rows(dy, "dy");
  const F8 w = f8(a[1], "w");
  const at::ScalarType st = dtype(a[3]);
  const muon_dtype t = typed(st, "dtype");
  device(dy);
  device(dy, w.q);
  device(dy, w.scale);
  no_tangents("float8.grad_input", dy, w.q, w.scale);
  const Ends e = ends_of(a[2], dy);
  const Stack m = weights_of(w, e);
  if (m.r != s.c) bad("w must be (n, k) with dy's last dimension n");
  const c10::DeviceGuard guard(dy.device());
  at::Tensor dx = make(shaped(dy, m.c), st, dy);
  size_t need;
  const at::Tensor ws = scratch(MUON_F8_GRAD_INPUT, ptr(dy), s.ld, e, s.r, s.c, m.c, t, dy, &need);
  check(muon_f8_grad_input(ptr(dy), s.ld, ptr<uint8_t>(w.q), m.ld, m.stride, ptr<uint8_t>(w.scale), e.at, e.experts, s.r,
                           s.c, m.c, ptr(dx), m.c, t, need ? ptr(ws) : nullptr, need, stream(dy)),
        "muon_f8_grad_input");
  return wrap(std::move(dx));
}

// dy, x (F8), ends or None, dtype, out or None, accumulate
PyObject* do_grad_weight(PyObject* const* a, Py_ssize_t n) {
  count(n, 6);
  const at::Tensor& dy = gradient(a[0]);
  const Rows s = rows(dy, "dy");
  const F8 x = f8(a[1], "x");
  const Rows r = rows8(x, "x");
  if (r.r != s.r) bad("dy and x must have the same number of rows");
  const int accumulate = PyObject_IsTrue(a[5]);
  if (accumulate < 0) throw Raised();
  if (a[4] != Py_None && c10::GradMode::is_enabled() && tensor(a[4], "out").requires_grad())
    bad("grad_weight records nothing for autograd: out must not require a gradient, or be written under no_grad");
  device(dy);
  device(dy, x.q);
  device(dy, x.scale);
  const Ends e = ends_of(a[2], dy);
  at::Tensor out;
  if (a[4] != Py_None) {
    out = tensor(a[4], "out");
    device(dy, out);
    if (out.dim() != (e.at ? 3 : 2) || (e.at && out.size(0) != e.experts) || out.size(-2) != s.c || out.size(-1) != r.c)
      bad(e.at ? "out must be (experts, n, k)" : "out must be (n, k)");
  } else if (accumulate) {
    bad("accumulate needs out");
  }
  const at::ScalarType st = out.defined() ? out.scalar_type() : dtype(a[3]);
  const muon_dtype t = typed(st, out.defined() ? "out" : "dtype");
  no_tangents("float8.grad_weight", dy, x.q, x.scale, out);
  const c10::DeviceGuard guard(dy.device());
  if (!out.defined()) out = e.at ? make({e.experts, s.c, r.c}, st, dy) : make({s.c, r.c}, st, dy);
  const Stack o = stack(out, "out", true);
  size_t need;
  const at::Tensor ws = scratch(MUON_F8_GRAD_WEIGHT, ptr(dy), s.ld, e, s.r, s.c, r.c, t, dy, &need);
  check(muon_f8_grad_weight(ptr(dy), s.ld, ptr<uint8_t>(x.q), r.ld, ptr<uint8_t>(x.scale), e.at, e.experts, s.r, s.c, r.c,
                            ptr(out), o.ld, o.stride, t, accumulate, need ? ptr(ws) : nullptr, need, stream(dy)),
        "muon_f8_grad_weight");
  if (a[4] != Py_None) {
    if (!out.is_inference()) torch::autograd::impl::bump_version(out);  // (autograd sees the write)
    Py_INCREF(a[4]);
    return a[4];
  }
  return wrap(std::move(out));
}

// (F8 class, error class): what the functions build and raise.
PyObject* do_classes(PyObject* const* a, Py_ssize_t n) {
  count(n, 2);
  if (!PyType_Check(a[0]) || !PyType_IsSubtype((PyTypeObject*)a[0], &PyTuple_Type)) bad("F8 must be a tuple class");
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XDECREF(g_f8);
  Py_XDECREF(g_error);
  g_f8 = a[0];
  g_error = a[1];
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (!g_f8 && F != do_classes) bad("_float8 is used through float8");
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
                           method<do_quantize_weight>("quantize_weight"),
                           method<do_dequantize>("dequantize"),
                           method<do_matmul>("matmul"),
                           method<do_grad_input>("grad_input"),
                           method<do_grad_weight>("grad_weight"),
                           method<do_classes>("set_classes"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_float8", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__float8() { return PyModule_Create(&g_module); }
