// The short way from Python to the calls of include/fp8bq_step.h.
//
// At a few tokens the kernels take 3 to 8 us, less than ctypes and Python's
// own argument checks and allocations do (5 to 8 us a call). These functions
// take the tensors as they are, and where every argument is what the call
// expects, on the current device, they allocate the outputs, enqueue, and
// return them; a nonzero status is returned as a number. In every other case
// they return None without having done anything, and the Python of step.py
// says what is wrong, or makes the call on the other device.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp8bq_step.h"

namespace {

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool is(const at::Tensor* t, at::ScalarType type, int64_t dim, int device) {
  return t != nullptr && t->scalar_type() == type && t->dim() == dim && t->is_cuda() && t->get_device() == device &&
         t->is_contiguous();
}

bool shaped(const at::Tensor* t, at::ScalarType type, at::IntArrayRef sizes, int device) {
  return is(t, type, static_cast<int64_t>(sizes.size()), device) && t->sizes() == sizes;
}

// A tensor or None: false where it is neither, or not what is expected.
bool optional(PyObject* o, const at::Tensor** out, at::ScalarType type, at::IntArrayRef sizes, int device) {
  *out = nullptr;
  if (o == Py_None) return true;
  *out = tensor(o);
  return shaped(*out, type, sizes, device);
}

void* data(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
  return at::empty(sizes, like.options().dtype(type).requires_grad(false));
}

PyObject* pair_of(PyObject* a, PyObject* b) {
  PyObject* out = a != nullptr && b != nullptr ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return out;
}

// A C++ exception becomes the Python one that torch makes of it: an output that
// does not fit the device raises torch.OutOfMemoryError, as in the Python of
// step.py.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// The device and the stream a call ends with.
bool place(PyObject* const* args, int* device, void** stream) {
  *device = static_cast<int>(PyLong_AsLong(args[0]));
  *stream = PyLong_AsVoidPtr(args[1]);
  return PyErr_Occurred() == nullptr;
}

bool counted(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// (x, weight, residual | None, eps, out_residual | None, i8, device, stream)
// -> (codes, scales, h)
PyObject* rmsnorm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  int device;
  void* stream;
  if (!counted(n, 8) || !place(args + 6, &device, &stream)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor* x = tensor(args[0]);
    if (!is(x, at::kBFloat16, 2, device) || !PyFloat_Check(args[3])) Py_RETURN_NONE;
    const int64_t m = x->size(0), k = x->size(1);
    const at::Tensor *r, *h;
    if (!shaped(tensor(args[1]), at::kBFloat16, {k}, device) ||
        !optional(args[2], &r, at::kBFloat16, x->sizes(), device) ||
        !optional(args[4], &h, at::kBFloat16, x->sizes(), device) || (h != nullptr && r == nullptr))
      Py_RETURN_NONE;
    const bool i8 = args[5] == Py_True;
    if (i8 && k == 0) Py_RETURN_NONE;  // the call writes no scales then: step.py does
    at::Tensor h_new;
    if (r != nullptr && h == nullptr) {
      h_new = empty(x->sizes(), at::kBFloat16, *x);
      h = &h_new;
    }
    const at::Tensor codes = empty(x->sizes(), i8 ? at::kChar : at::kByte, *x);
    const at::Tensor scales = i8 ? empty({m}, at::kFloat, *x) : empty({m, k / 128}, at::kFloat, *x);
    const int st = (i8 ? fp8bq_rmsnorm_quant_i8 : fp8bq_rmsnorm_quant)(
        m, k, data(x), data(r), data(tensor(args[1])), PyFloat_AS_DOUBLE(args[3]), data(h), codes.data_ptr(),
        scales.data_ptr<float>(), stream);
    if (st != FP8BQ_OK) return PyLong_FromLong(st);
    PyObject* third = h_new.defined() ? THPVariable_Wrap(h_new) : Py_NewRef(r != nullptr ? args[4] : args[0]);
    PyObject *first = THPVariable_Wrap(codes), *second = THPVariable_Wrap(scales);
    PyObject* out = first != nullptr && second != nullptr && third != nullptr ? PyTuple_Pack(3, first, second, third)
                                                                              : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    Py_XDECREF(third);
    return out;
  });
}

// (a_q, a_s, w_q, w_s, out | None, workspace | None, device, stream) -> c
PyObject* gemm_i8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  int device;
  void* stream;
  if (!counted(n, 8) || !place(args + 6, &device, &stream)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor *aq = tensor(args[0]), *wq = tensor(args[2]);
    if (!is(aq, at::kChar, 2, device) || !is(wq, at::kChar, 2, device)) Py_RETURN_NONE;
    const int64_t m = aq->size(0), k = aq->size(1), rows = wq->size(0);
    const at::Tensor *as = tensor(args[1]), *ws = tensor(args[3]), *out, *space = nullptr;
    if (wq->size(1) != k || !shaped(as, at::kFloat, {m}, device) || !shaped(ws, at::kFloat, {rows}, device) ||
        !optional(args[4], &out, at::kBFloat16, {m, rows}, device))
      Py_RETURN_NONE;
    if (args[5] != Py_None) {
      space = tensor(args[5]);
      if (!is(space, at::kByte, 1, device)) Py_RETURN_NONE;
    }
    at::Tensor c_new, scratch;
    if (out == nullptr) {
      c_new = empty({m, rows}, at::kBFloat16, *aq);
      out = &c_new;
    }
    if (space == nullptr) {
      const int64_t need = fp8bq_gemm_i8_workspace_bytes(m, rows, k);
      if (need < 0) return PyLong_FromLong(static_cast<long>(need));
      if (need > 0) {
        scratch = empty({need}, at::kByte, *aq);
        space = &scratch;
      }
    }
    const int st = fp8bq_gemm_i8(m, rows, k, data(aq), as->data_ptr<float>(), data(wq), ws->data_ptr<float>(),
                                 data(out), data(space), space == nullptr ? 0 : space->numel(), stream);
    if (st != FP8BQ_OK) return PyLong_FromLong(st);
    return c_new.defined() ? THPVariable_Wrap(c_new) : Py_NewRef(args[4]);
  });
}

// (target_p, drafts, u_accept, u_sample, draft_p | None, draft_len | None,
// workspace | None, device, stream) -> (tokens, accepted)
PyObject* verify_drafts(PyObject*, PyObject* const* args, Py_ssize_t n) {
  int device;
  void* stream;
  if (!counted(n, 9) || !place(args + 7, &device, &stream)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor *target = tensor(args[0]), *drafts = tensor(args[1]);
    if (!is(drafts, at::kInt, 2, device) || target == nullptr) Py_RETURN_NONE;
    const at::ScalarType kind = target->scalar_type();
    if ((kind != at::kFloat && kind != at::kBFloat16) || !is(target, kind, 3, device)) Py_RETURN_NONE;
    const int64_t b = drafts->size(0), k = drafts->size(1), v = target->size(2);
    const at::Tensor *ua = tensor(args[2]), *us = tensor(args[3]), *q, *lens, *space = nullptr;
    if (target->size(0) != b || target->size(1) != k + 1 || !shaped(ua, at::kFloat, {b, k}, device) ||
        !shaped(us, at::kFloat, {b}, device) || !optional(args[4], &q, kind, {b, k, v}, device) ||
        !optional(args[5], &lens, at::kInt, {b}, device))
      Py_RETURN_NONE;
    if (args[6] != Py_None) {
      space = tensor(args[6]);
      if (!is(space, at::kByte, 1, device)) Py_RETURN_NONE;
    }
    at::Tensor scratch;
    if (space == nullptr) {
      const int64_t need = fp8bq_verify_workspace_bytes(b, k, v);
      if (need < 0) return PyLong_FromLong(static_cast<long>(need));
      if (need > 0) {
        scratch = empty({need}, at::kByte, *target);
        space = &scratch;
      }
    }
    const at::Tensor tokens = empty({b, k + 1}, at::kInt, *target), accepted = empty({b}, at::kInt, *target);
    const int st = fp8bq_verify_drafts(b, k, v, kind == at::kFloat ? FP8BQ_F32 : FP8BQ_BF16, data(target),
                                       k > 0 ? data(q) : nullptr, drafts->data_ptr<int>(),
                                       lens == nullptr ? nullptr : lens->data_ptr<int>(), ua->data_ptr<float>(),
                                       us->data_ptr<float>(), data(space), space == nullptr ? 0 : space->numel(),
                                       tokens.data_ptr<int>(), accepted.data_ptr<int>(), stream);
    if (st != FP8BQ_OK) return PyLong_FromLong(st);
    return pair_of(THPVariable_Wrap(tokens), THPVariable_Wrap(accepted));
  });
}

using FastCall = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction method(FastCall f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {
    {"rmsnorm", method(rmsnorm), METH_FASTCALL, nullptr},
    {"gemm_i8", method(gemm_i8), METH_FASTCALL, nullptr},
    {"verify_drafts", method(verify_drafts), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
