// What the calls on torch tensors share (mx_torch.cpp, fp8_torch.cpp): arguments by position and name, checked
// tensors, refusals as Python exceptions.
#pragma once
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "moe_ffn.h"

namespace torch_args {

inline PyObject* moe_error = nullptr;    // MoeError
inline PyObject* on_stream = nullptr;    // mx._on
inline PyObject* module_dict = nullptr;  // the module's, for a call handed to another stream

struct Refused {
  std::string why;
};
struct Failed {
  int status;
  const char* where;
};
struct PythonError {};  // already set

template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.why.c_str());
  } catch (const Failed& s) {
    PyObject* e = PyObject_CallFunction(moe_error, "is", s.status, s.where);
    if (e) {
      PyErr_SetObject(moe_error, e);
      Py_DECREF(e);
    }
  } catch (const PythonError&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- arguments

template <size_t N>
struct Call {
  PyObject* v[N] = {};
  Call(const char* fn, const char* const (&names)[N], size_t required, PyObject* const* args, Py_ssize_t nargs,
       PyObject* kwnames) {
    if (static_cast<size_t>(nargs) > N) {
      PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments (%d given)", fn, static_cast<int>(N),
                   static_cast<int>(nargs));
      throw PythonError{};
    }
    for (Py_ssize_t i = 0; i < nargs; ++i) v[i] = args[i];
    const Py_ssize_t kw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t j = 0; j < kw; ++j) {
      PyObject* name = PyTuple_GET_ITEM(kwnames, j);
      size_t i = 0;
      while (i < N && PyUnicode_CompareWithASCIIString(name, names[i]) != 0) ++i;
      if (i == N || v[i]) {
        PyErr_Format(PyExc_TypeError, i == N ? "%s() got an unexpected keyword argument %R"
                                             : "%s() got multiple values for argument %R", fn, name);
        throw PythonError{};
      }
      v[i] = args[nargs + j];
    }
    for (size_t i = 0; i < N; ++i) {
      if (!v[i] && i < required) {
        PyErr_Format(PyExc_TypeError, "%s() missing required argument '%s'", fn, names[i]);
        throw PythonError{};
      }
      if (v[i] == Py_None) v[i] = nullptr;
    }
  }
};

// The call again with `stream` (the last argument) current.
template <size_t N>
PyObject* hand_over(const char* fn, const Call<N>& c) {
  PyObject* self = PyDict_GetItemString(module_dict, fn);
  PyObject* args[N + 1] = {c.v[N - 1], self};
  for (size_t i = 0; i + 1 < N; ++i) args[2 + i] = c.v[i] ? c.v[i] : Py_None;
  return PyObject_Vectorcall(on_stream, args, N + 1, nullptr);
}

inline const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!o || !THPVariable_Check(o)) throw Refused{std::string(name) + ": expected a tensor"};
  return THPVariable_Unpack(o);
}

inline int64_t integer(PyObject* o, const char* name) {
  if (!o) throw Refused{std::string(name) + ": expected an integer"};
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
inline float number(PyObject* o, const char* name) {
  if (!o) throw Refused{std::string(name) + ": expected a number"};
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(v);
}

[[noreturn]] inline void refuse(const char* name, const std::string& wanted, const at::Tensor& t) {
  std::ostringstream s;
  s << name << ": expected " << wanted << ", got " << t.scalar_type() << " " << t.sizes() << " on " << t.device();
  throw Refused{s.str()};
}

// A tensor that the library reads through its pointer: dense, on the device, of this type and shape.
inline const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || t.sizes() != shape || t.get_device() != dev || !t.is_contiguous()) {
    std::ostringstream s;
    s << "a contiguous " << type << " tensor " << shape << " on device " << dev;
    refuse(name, s.str(), t);
  }
  return t;
}

// fp32 values, or null.
inline const float* values(PyObject* o, const char* name, int64_t count, int dev) {
  if (!o || o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kFloat || t.numel() != count || t.get_device() != dev || !t.is_contiguous())
    refuse(name, std::to_string(count) + " fp32 value(s) on device " + std::to_string(dev), t);
  return static_cast<const float*>(t.const_data_ptr());
}

// bf16 rows: the row stride in elements, d or more (that of a single row is not used, and torch may report any).
inline int64_t row_stride(const at::Tensor& t, const char* name, int64_t n, int64_t d, int dev) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 2 || t.size(0) != n || t.size(1) != d || t.get_device() != dev ||
      t.stride(1) != 1)
    refuse(name, "bf16 rows [" + std::to_string(n) + ", " + std::to_string(d) + "] on device " + std::to_string(dev), t);
  if (n <= 1) return d;
  // expanded rows, or a window that slides by less than a row
  if (t.stride(0) < d) refuse(name, "rows of their own, not " + std::to_string(t.stride(0)) + " elements apart", t);
  return t.stride(0);
}

inline void two_dims(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) refuse(name, "two dimensions", t);
}

// The stream to launch on; the device is made current by the caller's guard.
inline cudaStream_t stream_of(int dev) {
  if (dev < 0) throw Refused{"expected tensors on a CUDA device"};
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
}
// A library call without the interpreter's lock: a launch waits where the GPU's queue is full.  What it
// points to is held by the caller's arguments or by tensors of the call.
template <typename F>
void call(const char* where, F f) {
  moe_status st;
  {
    struct Unlocked {
      PyThreadState* state = PyEval_SaveThread();
      ~Unlocked() { PyEval_RestoreThread(state); }
    } unlocked;
    st = f();
  }
  if (st != MOE_OK) throw Failed{st, where};
}

// An attribute, None as null.
struct Field {
  PyObject* o;
  Field(PyObject* from, PyObject* name) : o(PyObject_GetAttr(from, name)) {
    if (!o) throw PythonError{};
  }
  Field(const Field&) = delete;
  ~Field() { Py_XDECREF(o); }
  PyObject* get() const { return o == Py_None ? nullptr : o; }
};

#define MOE_TORCH_CALL(name, doc) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL | METH_KEYWORDS, doc}

}  // namespace torch_args
