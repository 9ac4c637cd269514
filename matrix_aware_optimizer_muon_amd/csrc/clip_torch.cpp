// Python binding of gradient clipping (module _clip): argument checks,
// allocation, the current stream, and the calls of the C ABI
// (include/muon_clip.h).  No work is done here.
#include "binding.hpp"
#include "muon_clip.h"

#include <cmath>
#include <vector>

namespace {

// A sequence's tensors as flat runs, all on one device.
struct Tensors {
  std::vector<at::Tensor> t;
  std::vector<void*> at;
  std::vector<int64_t> n;
  std::vector<muon_dtype> type;
};
Tensors tensors(PyObject* o, const char* what, const char* each) {
  PyObject* s = PySequence_Fast(o, (std::string(what) + " must be a sequence of tensors").c_str());
  if (!s) {
    PyErr_Clear();
    bad(std::string(what) + " must be a sequence of tensors");
  }
  Tensors v;
  try {
    const Py_ssize_t num = PySequence_Fast_GET_SIZE(s);
    if (num < 1) bad(std::string(what) + " must hold at least one tensor");
    for (Py_ssize_t i = 0; i < num; ++i) {
      const at::Tensor& t = tensor(PySequence_Fast_GET_ITEM(s, i), each);
      v.type.push_back(typed(t.scalar_type(), each));
      if (!t.is_non_overlapping_and_dense())
        bad(std::string(each) + " must be dense (its elements without gaps, in any order)");
      device(v.t.empty() ? t : v.t[0], t);
      v.t.push_back(t);
      v.at.push_back(t.data_ptr());
      v.n.push_back(t.numel());
    }
  } catch (...) {
    Py_DECREF(s);
    throw;
  }
  Py_DECREF(s);
  return v;
}

at::Tensor scratch(const Tensors& g, size_t* need) {
  *need = 0;
  check(muon_clip_workspace((int)g.t.size(), g.n.data(), g.type.data(), need), "muon_clip_workspace");
  return *need ? make({(int64_t)*need}, at::kByte, g.t[0]) : at::Tensor();
}

std::shared_ptr<torch::autograd::Node> not_recorded(const char* name, const std::vector<at::Tensor>& in) {
  using namespace torch::autograd;
  for (const at::Tensor& t : in) no_tangents(name, t);
  bool any = false;
  for (const at::Tensor& t : in) any = any || t.requires_grad();
  if (!any || !c10::GradMode::is_enabled()) return nullptr;
  edge_list edges;
  for (const at::Tensor& t : in)
    if (t.requires_grad()) edges.push_back(impl::gradient_edge(t));
  return std::shared_ptr<Node>(new NotImplemented(name, std::move(edges)), deleteNode);
}

// grads
PyObject* do_grad_norm(PyObject* const* a, Py_ssize_t n) {
  count(n, 1);
  const Tensors g = tensors(a[0], "grads", "a gradient");
  const c10::DeviceGuard guard(g.t[0].device());
  at::Tensor norm = make({}, at::kFloat, g.t[0]);
  size_t need;
  const at::Tensor ws = scratch(g, &need);
  check(muon_grad_norm((int)g.t.size(), (const void* const*)g.at.data(), g.n.data(), g.type.data(), ptr<float>(norm),
                       need ? ptr(ws) : nullptr, need, stream(g.t[0])),
        "muon_grad_norm");
  mark(norm, not_recorded("clip.grad_norm", g.t));
  return wrap(std::move(norm));
}

// grads, max_norm, out or None
PyObject* do_clip(PyObject* const* a, Py_ssize_t n) {
  count(n, 3);
  const double max_norm = PyFloat_AsDouble(a[1]);
  if (max_norm == -1.0 && PyErr_Occurred()) throw Raised();
  if (!(max_norm >= 0.0)) bad("max_norm must not be negative");
  if (std::isinf((float)max_norm) && !std::isinf(max_norm)) bad("max_norm must be infinite or in fp32's range");
  const Tensors g = tensors(a[0], "grads", "a gradient");
  Tensors made;
  const bool in_place = a[2] == Py_None;
  if (!in_place) {
    made = tensors(a[2], "out", "an output");
    if (made.t.size() != g.t.size()) bad("out must hold an output for each gradient");
    for (size_t i = 0; i < g.t.size(); ++i) {
      if (made.t[i].sizes() != g.t[i].sizes() || made.t[i].strides() != g.t[i].strides())
        bad("an output must have its gradient's shape and strides");
      device(g.t[0], made.t[i]);
    }
  }
  const Tensors& out = in_place ? g : made;
  if (c10::GradMode::is_enabled())
    for (size_t i = 0; i < g.t.size(); ++i)
      if (g.t[i].requires_grad() || out.t[i].requires_grad())
        bad("clipping records nothing for autograd: call it without gradients that require one, or under no_grad");
  for (size_t i = 0; i < g.t.size(); ++i) no_tangents("clip.clip_grad_norm", g.t[i], out.t[i]);
  const c10::DeviceGuard guard(g.t[0].device());
  at::Tensor norm = make({}, at::kFloat, g.t[0]);
  size_t need;
  const at::Tensor ws = scratch(g, &need);
  check(muon_clip_grads((int)g.t.size(), (const void* const*)g.at.data(), g.n.data(), g.type.data(), out.at.data(),
                        out.type.data(), (float)max_norm, ptr<float>(norm), need ? ptr(ws) : nullptr, need,
                        stream(g.t[0])),
        "muon_clip_grads");
  for (const at::Tensor& t : out.t)
    if (!t.is_inference()) torch::autograd::impl::bump_version(t);  // (autograd sees the write)
  return wrap(std::move(norm));
}

// (error class): what the functions raise.
PyObject* do_classes(PyObject* const* a, Py_ssize_t n) {
  count(n, 1);
  Py_INCREF(a[0]);
  Py_XDECREF(g_error);
  g_error = a[0];
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (!g_error && F != do_classes) bad("_clip is used through clip");
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

PyMethodDef g_methods[] = {method<do_grad_norm>("grad_norm"), method<do_clip>("clip_grad_norm"),
                           method<do_classes>("set_classes"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_clip", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__clip() { return PyModule_Create(&g_module); }
