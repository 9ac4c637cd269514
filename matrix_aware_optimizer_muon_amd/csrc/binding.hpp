// What the Python bindings share: argument checks, allocation from torch's
// caching allocator, the current stream, and errors.  Each module has a copy of
// its own.
#pragma once

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

#include "muon.h"

namespace {

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

// Forward mode is not implemented: a tangent, which no result would carry, raises.
template <typename... In> void no_tangents(const char* name, const In&... in) {
  const bool any = (... || (in.defined() && in.unsafeGetTensorImpl()->_fw_grad(/*level=*/0, in).defined()));
  TORCH_CHECK_NOT_IMPLEMENTED(!any, "forward-mode derivative for ", name, " is not implemented");
}

// What a forward operator leaves for autograd, if it records and an input
// requires a gradient: a node that raises when a backward pass reaches it.  Of
// 8-bit rows the scale carries it.  (The backward operators leave nothing:
// their results are gradients already; they only refuse tangents.)
template <typename... In> std::shared_ptr<torch::autograd::Node> undifferentiated(const char* name, const In&... in) {
  using namespace torch::autograd;
  no_tangents(name, in...);
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
PyObject* tuple(std::initializer_list<PyObject*> v) {
  PyObject* t = PyTuple_New((Py_ssize_t)v.size());
  Py_ssize_t i = 0;
  for (PyObject* o : v) PyTuple_SET_ITEM(t, i++, o);
  return t;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) bad("wrong number of arguments");
}

}  // namespace
