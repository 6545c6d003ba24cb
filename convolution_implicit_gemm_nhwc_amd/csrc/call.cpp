// The short way through a call of the output-layer operators (mx.py, xent.py).
//
// Their smallest calls take 2 to 5 us on the GPU; through ctypes the host took
// 6.5 us for a quantisation and 32 us for a loss with its gradient.  Here a call
// checks its tensors, allocates what it returns and its workspace from torch's
// allocator on the current stream, and enters the C ABI, whose functions it is
// given by address (the library that _abi.py has loaded).
//
// Every function returns None, with nothing done, for anything out of the
// ordinary (another type, shape, device, a tensor subclass with a dispatch of
// its own): the binding then takes its full way, which checks each argument
// with a message.  A status other than FCONV_OK is returned as an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fconv_mx.h"
#include "fconv_xent.h"

namespace {

using at::ScalarType;

// The arguments of a call: tensors, then whole numbers.
struct Call {
  PyObject* const* args;
  c10::DeviceIndex device = -1;
  bool ok = true;

  int64_t whole(int i) {
    const long long v = PyLong_AsLongLong(args[i]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  template <typename F>
  F function(int i) {
    void* p = PyLong_AsVoidPtr(args[i]);
    if (!p) {
      PyErr_Clear();
      ok = false;
    }
    return reinterpret_cast<F>(p);
  }
  // The tensor at i, if it lives on the call's device (that of the first one) and is of the type.
  const at::Tensor* tensor(int i, ScalarType type) {
    if (!THPVariable_Check(args[i])) return fail();
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    if (!t.defined() || !t.is_cuda() || t.scalar_type() != type || t.layout() != at::kStrided ||
        t.unsafeGetTensorImpl()->is_python_dispatch())
      return fail();
    if (device < 0) device = t.device().index();
    if (t.device().index() != device) return fail();
    return &t;
  }
  // Address of a [rows, cols] matrix with dense rows, ld elements apart.
  void* matrix(int i, ScalarType type, int64_t rows, int64_t cols, int64_t* ld) {
    const at::Tensor* t = tensor(i, type);
    if (!t) return nullptr;
    if (t->dim() == 2 && t->size(0) == rows && t->size(1) == cols) {
      *ld = rows > 1 ? t->stride(0) : cols;
      if ((t->stride(1) != 1 && cols > 1) || *ld < cols) return fail(), nullptr;
    } else if (t->numel() == rows * cols && t->is_contiguous()) {
      *ld = cols;
    } else {
      return fail(), nullptr;
    }
    return t->data_ptr();
  }
  void* vector(int i, ScalarType type, int64_t numel) {
    const at::Tensor* t = tensor(i, type);
    if (!t) return nullptr;
    if (t->numel() != numel || !t->is_contiguous()) return fail(), nullptr;
    return t->data_ptr();
  }
  // After the tensors: whether the call can go on, on the current device.
  bool ready() const { return ok && device >= 0 && device == c10::hip::current_device(); }

 private:
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
};

ScalarType type_of(int64_t dtype) { return dtype == FCONV_BF16 ? at::kBFloat16 : at::kFloat; }

at::TensorBase make(at::IntArrayRef size, ScalarType type, c10::DeviceIndex device) {
  return at::detail::empty_cuda(size, type, at::Device(at::kCUDA, device), std::nullopt);
}

// run(stream) with the interpreter's lock let go; a status as a Python int, or
// `result` (whose tensors are wrapped only then).
template <typename R, typename F>
PyObject* launch(const Call& c, R run, F result) {
  void* stream = c10::hip::getCurrentHIPStream(c.device).stream();
  fconv_status st;
  Py_BEGIN_ALLOW_THREADS
  st = run(stream);
  Py_END_ALLOW_THREADS
  if (st != FCONV_OK) return PyLong_FromLong(st);
  return result();
}

PyObject* pair(at::TensorBase&& a, at::TensorBase&& b) {
  PyObject* x = THPVariable_Wrap(std::move(a));
  if (!x) return nullptr;
  PyObject* y = THPVariable_Wrap(std::move(b));
  if (!y) {
    Py_DECREF(x);
    return nullptr;
  }
  PyObject* t = PyTuple_New(2);
  if (!t) {
    Py_DECREF(x);
    Py_DECREF(y);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, x);
  PyTuple_SET_ITEM(t, 1, y);
  return t;
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// quantize(x, fn, rows, cols, dtype, bytes) -> codes and scales
PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 6)) return nullptr;
  Call c{args};
  const auto fn = c.function<decltype(&fconv_mx_quantize)>(1);
  const int64_t rows = c.whole(2), cols = c.whole(3), dtype = c.whole(4), bytes = c.whole(5);
  int64_t ld = 0;
  const void* x = c.matrix(0, type_of(dtype), rows, cols, &ld);
  if (!c.ready()) Py_RETURN_NONE;
  at::TensorBase mx = make({bytes}, at::kByte, c.device);
  return launch(
      c,
      [&](void* s) {
        return fn(s, x, ld, static_cast<int32_t>(rows), static_cast<int32_t>(cols), static_cast<int32_t>(dtype),
                  mx.data_ptr());
      },
      [&] { return THPVariable_Wrap(std::move(mx)); });
  END_HANDLE_TH_ERRORS
}

// dequantize(data, fn, rows, cols, dtype, bytes) -> y
PyObject* dequantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 6)) return nullptr;
  Call c{args};
  const auto fn = c.function<decltype(&fconv_mx_dequantize)>(1);
  const int64_t rows = c.whole(2), cols = c.whole(3), dtype = c.whole(4), bytes = c.whole(5);
  const at::Tensor* mx = c.tensor(0, at::kByte);
  if (!c.ready() || mx->numel() < bytes || !mx->is_contiguous()) Py_RETURN_NONE;
  at::TensorBase y = make({rows, cols}, type_of(dtype), c.device);
  return launch(
      c,
      [&](void* s) {
        return fn(s, mx->data_ptr(), static_cast<int32_t>(rows), static_cast<int32_t>(cols),
                  static_cast<int32_t>(dtype), y.data_ptr(), cols);
      },
      [&] { return THPVariable_Wrap(std::move(y)); });
  END_HANDLE_TH_ERRORS
}

// product(x, w_data, bias or None, fn, plan, M, N, K, dtype, w bytes, workspace bytes) -> y
PyObject* product(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 11)) return nullptr;
  Call c{args};
  const auto fn = c.function<decltype(&fconv_mx_plan_run)>(3);
  const auto plan = c.function<fconv_mx_plan>(4);
  const int64_t M = c.whole(5), N = c.whole(6), K = c.whole(7), dtype = c.whole(8), w_bytes = c.whole(9),
                ws_bytes = c.whole(10);
  fconv_mx_args a = {};
  a.x = c.matrix(0, type_of(dtype), M, K, &a.ldx);
  const at::Tensor* w = c.tensor(1, at::kByte);
  if (args[2] != Py_None) a.bias = static_cast<const float*>(c.vector(2, at::kFloat, N));
  if (!c.ready() || w->numel() < w_bytes || !w->is_contiguous()) Py_RETURN_NONE;
  a.w_mx = w->data_ptr();
  at::TensorBase y = make({M, N}, type_of(dtype), c.device), ws;
  a.y = y.data_ptr();
  a.ldy = N;
  if (ws_bytes) {
    ws = make({ws_bytes}, at::kByte, c.device);
    a.workspace = ws.data_ptr();
    a.workspace_bytes = static_cast<size_t>(ws_bytes);
  }
  return launch(
      c, [&](void* s) { return fn(plan, s, &a); }, [&] { return THPVariable_Wrap(std::move(y)); });
  END_HANDLE_TH_ERRORS
}

// xent_forward(h, w, target, fn, plan, T, D, V, dtype, workspace bytes) -> (loss, lse)
PyObject* xent_forward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 10)) return nullptr;
  Call c{args};
  const auto fn = c.function<decltype(&fconv_xent_plan_forward)>(3);
  const auto plan = c.function<fconv_xent_plan>(4);
  const int64_t T = c.whole(5), D = c.whole(6), V = c.whole(7), dtype = c.whole(8), ws_bytes = c.whole(9);
  fconv_xent_args a = {};
  a.h = c.matrix(0, type_of(dtype), T, D, &a.ldh);
  a.w = c.matrix(1, type_of(dtype), V, D, &a.ldw);
  a.target = static_cast<const int64_t*>(c.vector(2, at::kLong, T));
  if (!c.ready()) Py_RETURN_NONE;
  at::TensorBase loss = make({T}, at::kFloat, c.device), lse = make({T}, at::kFloat, c.device),
                 ws = make({ws_bytes}, at::kByte, c.device);
  a.loss = static_cast<float*>(loss.data_ptr());
  a.lse = static_cast<float*>(lse.data_ptr());
  a.workspace = ws.data_ptr();
  a.workspace_bytes = static_cast<size_t>(ws_bytes);
  return launch(
      c, [&](void* s) { return fn(plan, s, &a); }, [&] { return pair(std::move(loss), std::move(lse)); });
  END_HANDLE_TH_ERRORS
}

// xent_backward(h, w, target, lse, dloss, fn, plan, T, D, V, dtype, workspace bytes) -> (dh, dw)
PyObject* xent_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 12)) return nullptr;
  Call c{args};
  const auto fn = c.function<decltype(&fconv_xent_plan_backward)>(5);
  const auto plan = c.function<fconv_xent_plan>(6);
  const int64_t T = c.whole(7), D = c.whole(8), V = c.whole(9), dtype = c.whole(10), ws_bytes = c.whole(11);
  fconv_xent_args a = {};
  a.h = c.matrix(0, type_of(dtype), T, D, &a.ldh);
  a.w = c.matrix(1, type_of(dtype), V, D, &a.ldw);
  a.target = static_cast<const int64_t*>(c.vector(2, at::kLong, T));
  a.lse = static_cast<float*>(c.vector(3, at::kFloat, T));
  a.dloss = static_cast<const float*>(c.vector(4, at::kFloat, T));
  if (!c.ready()) Py_RETURN_NONE;
  at::TensorBase dh = make({T, D}, type_of(dtype), c.device), dw = make({V, D}, type_of(dtype), c.device),
                 ws = make({ws_bytes}, at::kByte, c.device);
  a.dh = dh.data_ptr();
  a.lddh = D;
  a.dw = dw.data_ptr();
  a.lddw = D;
  a.workspace = ws.data_ptr();
  a.workspace_bytes = static_cast<size_t>(ws_bytes);
  return launch(
      c, [&](void* s) { return fn(plan, s, &a); }, [&] { return pair(std::move(dh), std::move(dw)); });
  END_HANDLE_TH_ERRORS
}

#define FCONV_CALL(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr }
PyMethodDef kMethods[] = {FCONV_CALL(quantize),     FCONV_CALL(dequantize),    FCONV_CALL(product),
                          FCONV_CALL(xent_forward), FCONV_CALL(xent_backward), {nullptr, nullptr, 0, nullptr}};
#undef FCONV_CALL

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call() { return PyModule_Create(&kModule); }
