// The microscaled-format calls on torch tensors (moe_mx.h; mx.py adds the classes).
//
// A decode step's call is a few microseconds of GPU time.  Checked and launched
// from Python through ctypes a call takes 8 to 17 us of host time; here the
// tensors are checked in C++ and the C ABI is called directly.  The module holds
// no computation: it checks arguments, allocates what a call returns and launches
// on the current stream.
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

#include "mx_default.h"

namespace {

PyObject* rows_class = nullptr;   // mx.MxRows
PyObject* moe_error = nullptr;    // MoeError
PyObject* on_stream = nullptr;    // mx._on
PyObject* module_dict = nullptr;  // this module's, for a call handed to another stream

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

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!o || !THPVariable_Check(o)) throw Refused{std::string(name) + ": expected a tensor"};
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* name) {
  if (!o) throw Refused{std::string(name) + ": expected an integer"};
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
float number(PyObject* o, const char* name) {
  if (!o) throw Refused{std::string(name) + ": expected a number"};
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(v);
}

[[noreturn]] void refuse(const char* name, const std::string& wanted, const at::Tensor& t) {
  std::ostringstream s;
  s << name << ": expected " << wanted << ", got " << t.scalar_type() << " " << t.sizes() << " on " << t.device();
  throw Refused{s.str()};
}

// A tensor that the library reads through its pointer: dense, on the device, of this type and shape.
const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || t.sizes() != shape || t.get_device() != dev || !t.is_contiguous()) {
    std::ostringstream s;
    s << "a contiguous " << type << " tensor " << shape << " on device " << dev;
    refuse(name, s.str(), t);
  }
  return t;
}

// fp32 values, or null.
const float* values(PyObject* o, const char* name, int64_t count, int dev) {
  if (!o || o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kFloat || t.numel() != count || t.get_device() != dev || !t.is_contiguous())
    refuse(name, std::to_string(count) + " fp32 value(s) on device " + std::to_string(dev), t);
  return static_cast<const float*>(t.const_data_ptr());
}

// bf16 rows: the row stride in elements, d or more (that of a single row is not used, and torch may report any).
int64_t row_stride(const at::Tensor& t, const char* name, int64_t n, int64_t d, int dev) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 2 || t.size(0) != n || t.size(1) != d || t.get_device() != dev ||
      t.stride(1) != 1)
    refuse(name, "bf16 rows [" + std::to_string(n) + ", " + std::to_string(d) + "] on device " + std::to_string(dev), t);
  if (n <= 1) return d;
  // expanded rows, or a window that slides by less than a row
  if (t.stride(0) < d) refuse(name, "rows of their own, not " + std::to_string(t.stride(0)) + " elements apart", t);
  return t.stride(0);
}

void two_dims(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) refuse(name, "two dimensions", t);
}

// The stream to launch on; the device is made current by the caller's guard.
cudaStream_t stream_of(int dev) {
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

// ---------------------------------------------------------------- rows

struct Field {
  PyObject* o;
  Field(PyObject* from, PyObject* name) : o(PyObject_GetAttr(from, name)) {
    if (!o) throw PythonError{};
  }
  Field(const Field&) = delete;
  ~Field() { Py_XDECREF(o); }
  PyObject* get() const { return o == Py_None ? nullptr : o; }
};

PyObject* s_fmt;
PyObject* s_cols;
PyObject* s_codes;
PyObject* s_scales;
PyObject* s_global_scale;
PyObject* s_num_experts;
PyObject* s_n_out;
PyObject* s_k;
PyObject* s_packed;
PyObject* s_alpha;
PyObject* s_alpha_up;
PyObject* s_swiglu;

struct Rows {
  int32_t fmt = 0;
  int64_t n = 0, cols = 0;
  void* codes = nullptr;
  void* scales = nullptr;
  at::Tensor codes_t, scales_t;  // what is held while the call runs
};

// (Widths that the C calls' 32 bits do not hold are refused here, before they are cut to them.)
void widths(int64_t fmt, int64_t cols, int64_t* code_bytes, int64_t* pitch) {
  *code_bytes = fmt < 0 || fmt > 3 || cols > INT32_MAX
                    ? 0
                    : static_cast<int64_t>(moe_mx_code_bytes(static_cast<int32_t>(fmt), cols));
  if (*code_bytes == 0) throw Failed{MOE_ERR_UNSUPPORTED, "moe_mx_code_bytes"};
  *pitch = static_cast<int64_t>(moe_mx_scale_pitch(static_cast<int32_t>(fmt), cols));
}

// An MxRows, checked; *dev is its device, or has to be where it is not -2.
Rows rows_of(PyObject* o, int* dev) {
  Rows r;
  const Field fmt(o, s_fmt), cols(o, s_cols), codes(o, s_codes), scales(o, s_scales);
  const int64_t f = integer(fmt.get(), "fmt");
  r.cols = integer(cols.get(), "cols");
  int64_t cb, pitch;
  widths(f, r.cols, &cb, &pitch);
  r.fmt = static_cast<int32_t>(f);
  r.codes_t = tensor(codes.get(), "codes");
  two_dims(r.codes_t, "codes");
  r.n = r.codes_t.size(0);
  if (*dev == -2) *dev = static_cast<int>(r.codes_t.get_device());
  dense(codes.get(), "codes", at::kByte, {r.n, cb}, *dev);
  r.codes = r.codes_t.data_ptr();
  if (pitch) {
    if (!scales.get()) throw Refused{"scales: missing"};
    r.scales_t = dense(scales.get(), "scales", at::kByte, {r.n, pitch}, *dev);
    r.scales = r.scales_t.data_ptr();
  }
  return r;
}

const float* factor_of(PyObject* rows, int dev, at::Tensor* held) {
  const Field g(rows, s_global_scale);
  const float* p = values(g.get(), "global_scale", 1, dev);
  if (p) *held = tensor(g.get(), "global_scale");
  return p;
}

// Where a call writes its rows: a new MxRows or the caller's `out`, which gets its factor with the rows (take):
// a call that is refused leaves both as they were.
struct Target {
  Rows r;
  PyObject* object = nullptr;  // owned
  PyObject* factor = nullptr;  // of the caller's rows; the call's argument
  ~Target() { Py_XDECREF(object); }
  PyObject* take() {
    if (factor && PyObject_SetAttr(object, s_global_scale, factor) < 0) throw PythonError{};
    PyObject* o = object;
    object = nullptr;
    return o;
  }
};

// need: rows that have to be there (those of x, where no positions say which are written).
void target(Target* t, int64_t fmt, int64_t rows, int64_t cols, int64_t need, PyObject* global_scale, PyObject* out,
            const at::Tensor& like, int dev) {
  if (out) {
    t->r = rows_of(out, &dev);
    if (t->r.fmt != fmt || t->r.cols != cols) throw Refused{"out: of another format or width"};
    if (t->r.n < need) throw Refused{"out: fewer rows than x, and no positions"};
    t->object = Py_NewRef(out);
    t->factor = global_scale ? global_scale : Py_None;
    return;
  }
  int64_t cb, pitch;
  widths(fmt, cols, &cb, &pitch);
  if (rows < 0) throw Refused{"out_rows: negative"};
  if (rows < need) throw Refused{"out_rows: fewer rows than x, and no positions"};
  stream_of(dev);  // host tensors are refused before anything is allocated
  t->r.fmt = static_cast<int32_t>(fmt);
  t->r.n = rows;
  t->r.cols = cols;
  t->r.codes_t = at::empty({rows, cb}, like.options().dtype(at::kByte));
  t->r.codes = t->r.codes_t.data_ptr();
  if (pitch) {
    t->r.scales_t = at::empty({rows, pitch}, like.options().dtype(at::kByte));
    t->r.scales = t->r.scales_t.data_ptr();
  }
  PyObject* a[5] = {PyLong_FromLongLong(fmt), PyLong_FromLongLong(cols), THPVariable_Wrap(t->r.codes_t),
                    pitch ? THPVariable_Wrap(t->r.scales_t) : Py_NewRef(Py_None),
                    Py_NewRef(global_scale ? global_scale : Py_None)};
  bool ok = true;
  for (PyObject* o : a) ok &= o != nullptr;
  if (ok) t->object = PyObject_Vectorcall(rows_class, a, 5, nullptr);
  for (PyObject* o : a) Py_XDECREF(o);
  if (!t->object) throw PythonError{};
}

// positions [n, k] or null; *k its width (1).
const int32_t* positions_of(PyObject* o, int64_t n, int dev, int64_t* k) {
  *k = 1;
  if (!o) return nullptr;
  const at::Tensor& t = tensor(o, "positions");
  two_dims(t, "positions");
  *k = t.size(1);
  if (*k > INT32_MAX) throw Failed{MOE_ERR_UNSUPPORTED, "positions"};
  return static_cast<const int32_t*>(dense(o, "positions", at::kInt, {n, *k}, dev).const_data_ptr());
}

PyObject* mx_quantise(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"x", "fmt", "positions", "out_rows", "global_scale", "out", "stream"};
    const Call<7> c("mx_quantise", names, 2, args, nargs, kwnames);
    if (c.v[6]) return hand_over("mx_quantise", c);
    const at::Tensor& x = tensor(c.v[0], "x");
    two_dims(x, "x");
    const int64_t fmt = integer(c.v[1], "fmt"), n = x.size(0), d = x.size(1);
    const int dev = static_cast<int>(x.get_device());
    const int64_t ld = row_stride(x, "x", n, d, dev);
    int64_t k;
    const int32_t* pos = positions_of(c.v[2], n, dev, &k);
    const float* g = values(c.v[4], "global_scale", 1, dev);
    const c10::cuda::OptionalCUDAGuard on(dev < 0 ? std::nullopt : std::make_optional(x.device()));
    Target t;
    target(&t, fmt, c.v[3] ? integer(c.v[3], "out_rows") : n * k, d, c.v[2] ? 0 : n, c.v[4], c.v[5], x, dev);
    const cudaStream_t s = stream_of(dev);
    call("moe_mx_quantise", [&] {
      return moe_mx_quantise(t.r.fmt, n, static_cast<int32_t>(k), static_cast<int32_t>(d), x.const_data_ptr(), ld, pos, g,
                             t.r.n, t.r.codes, t.r.scales, s);
    });
    return t.take();
  });
}

PyObject* mx_add_rmsnorm(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"x",        "residual",     "gain",    "eps", "fmt",   "positions",
                                        "out_rows", "global_scale", "sum_out", "out", "stream"};
    const Call<11> c("mx_add_rmsnorm", names, 5, args, nargs, kwnames);
    if (c.v[10]) return hand_over("mx_add_rmsnorm", c);
    const at::Tensor& x = tensor(c.v[0], "x");
    two_dims(x, "x");
    const int64_t n = x.size(0), d = x.size(1);
    const int dev = static_cast<int>(x.get_device());
    const int64_t ld = row_stride(x, "x", n, d, dev);
    const void* res = nullptr;
    int64_t r_ld = 0;
    if (c.v[1]) {
      const at::Tensor& r = tensor(c.v[1], "residual");
      r_ld = row_stride(r, "residual", n, d, dev);
      res = r.const_data_ptr();
    }
    const at::Tensor& gain = dense(c.v[2], "gain", at::kBFloat16, {d}, dev);
    const float eps = number(c.v[3], "eps");
    const int64_t fmt = integer(c.v[4], "fmt");
    int64_t k;
    const int32_t* pos = positions_of(c.v[5], n, dev, &k);
    const float* g = values(c.v[7], "global_scale", 1, dev);
    const c10::cuda::OptionalCUDAGuard on(dev < 0 ? std::nullopt : std::make_optional(x.device()));
    at::Tensor sum;
    if (c.v[8]) {
      sum = tensor(c.v[8], "sum_out");
      const int64_t s_ld = row_stride(sum, "sum_out", n, d, dev);
      if (res && s_ld != r_ld) throw Refused{"sum_out: its row stride differs from residual's"};
      r_ld = s_ld;
    }
    Target t;
    target(&t, fmt, c.v[6] ? integer(c.v[6], "out_rows") : n * k, d, c.v[5] ? 0 : n, c.v[7], c.v[9], x, dev);
    const cudaStream_t s = stream_of(dev);
    if (!c.v[8]) {
      if (!res) r_ld = d;
      sum = r_ld == d ? at::empty({n, d}, x.options()) : at::empty_strided({n, d}, {r_ld, 1}, x.options());
    }
    call("moe_mx_add_rmsnorm", [&] {
      return moe_mx_add_rmsnorm(t.r.fmt, n, static_cast<int32_t>(k), static_cast<int32_t>(d), x.const_data_ptr(), ld, res,
                                r_ld, gain.const_data_ptr(), eps, pos, g, t.r.n, sum.data_ptr(), t.r.codes, t.r.scales, s);
    });
    PyObject* rows = t.take();
    PyObject* sum_o = c.v[8] ? Py_NewRef(c.v[8]) : THPVariable_Wrap(sum);
    PyObject* both = sum_o ? PyTuple_New(2) : nullptr;
    if (!both) {
      Py_DECREF(rows);
      Py_XDECREF(sum_o);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(both, 0, rows);
    PyTuple_SET_ITEM(both, 1, sum_o);
    return both;
  });
}

PyObject* mx_dequantise(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"r", "out", "stream"};
    const Call<3> c("mx_dequantise", names, 1, args, nargs, kwnames);
    if (c.v[2]) return hand_over("mx_dequantise", c);
    if (!c.v[0]) throw Refused{"r: expected rows"};
    int dev = -2;
    const Rows r = rows_of(c.v[0], &dev);
    at::Tensor g_held;
    const float* g = factor_of(c.v[0], dev, &g_held);
    const cudaStream_t s = stream_of(dev);
    const c10::cuda::CUDAGuard on(r.codes_t.device());
    at::Tensor out;
    int64_t ld = r.cols;
    if (c.v[1]) {
      out = tensor(c.v[1], "out");
      ld = row_stride(out, "out", r.n, r.cols, dev);
    } else {
      out = at::empty({r.n, r.cols}, r.codes_t.options().dtype(at::kBFloat16));
    }
    call("moe_mx_dequantise", [&] {
      return moe_mx_dequantise(r.fmt, r.n, static_cast<int32_t>(r.cols), r.codes, r.scales, g, out.data_ptr(), ld, s);
    });
    return c.v[1] ? Py_NewRef(c.v[1]) : THPVariable_Wrap(out);
  });
}

// ---------------------------------------------------------------- products

// An MxWeights, checked, and its tensors.
struct Weights {
  moe_mx_weights w{};
  at::Tensor held[3];
};
Weights weights_of(PyObject* o, int dev) {
  if (!o) throw Refused{"weights: expected MxWeights"};
  Weights all;
  moe_mx_weights& w = all.w;
  const Field fmt(o, s_fmt), experts(o, s_num_experts), n_out(o, s_n_out), k(o, s_k), swiglu(o, s_swiglu),
      packed(o, s_packed), alpha(o, s_alpha), alpha_up(o, s_alpha_up);
  const int64_t v[4] = {integer(fmt.get(), "fmt"), integer(experts.get(), "num_experts"),
                        integer(n_out.get(), "n_out"), integer(k.get(), "k")};
  for (int64_t i : v)
    if (i < 0 || i > INT32_MAX) throw Failed{MOE_ERR_UNSUPPORTED, "moe_mx_packed_bytes"};
  w.format = static_cast<int32_t>(v[0]);
  w.num_experts = static_cast<int32_t>(v[1]);
  w.n_out = static_cast<int32_t>(v[2]);
  w.k = static_cast<int32_t>(v[3]);
  w.swiglu = PyObject_IsTrue(swiglu.o) == 1;
  const size_t bytes = moe_mx_packed_bytes(&w);
  if (bytes == 0) throw Failed{MOE_ERR_UNSUPPORTED, "moe_mx_packed_bytes"};
  const at::Tensor& p = tensor(packed.get(), "packed");
  if (static_cast<size_t>(p.numel()) * p.element_size() != bytes || !p.is_contiguous() || p.get_device() != dev)
    refuse("packed", std::to_string(bytes) + " contiguous bytes on device " + std::to_string(dev), p);
  w.packed = p.const_data_ptr();
  w.alpha = values(alpha.get(), "alpha", w.num_experts, dev);
  w.alpha_up = values(alpha_up.get(), "alpha_up", w.num_experts, dev);
  all.held[0] = p;
  if (w.alpha) all.held[1] = tensor(alpha.get(), "alpha");
  if (w.alpha_up) all.held[2] = tensor(alpha_up.get(), "alpha_up");
  return all;
}

// The caller's workspace.
at::Tensor workspace_of(PyObject* o, int dev) {
  const at::Tensor& t = tensor(o, "ws");
  if (t.get_device() != dev || !t.is_contiguous()) refuse("ws", "contiguous bytes on device " + std::to_string(dev), t);
  return t;
}

// A product's: the caller's, or the one that the library keeps for the current device (mx_get_error reads its word).
struct Workspace {
  void* at;
  size_t bytes;
  at::Tensor held;
};
Workspace product_workspace(PyObject* o, int dev) {
  if (!o) return Workspace{moe_mx_default_workspace(), MOE_MX_PRODUCT_WORKSPACE, at::Tensor()};
  const at::Tensor t = workspace_of(o, dev);
  return Workspace{t.data_ptr(), t.nbytes(), t};
}

void same_operands(const Rows& x, const moe_mx_weights& w) {
  if (x.fmt != w.format || x.cols != w.k) throw Refused{"x: of another format or width than the weights"};
}

PyObject* mx_grouped_product(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"x", "w", "offsets", "out", "out_pos", "row_weight", "ws", "out_type", "stream"};
    const Call<9> c("mx_grouped_product", names, 3, args, nargs, kwnames);
    if (c.v[8]) return hand_over("mx_grouped_product", c);
    if (!c.v[0]) throw Refused{"x: expected rows"};
    int dev = -2;
    const Rows x = rows_of(c.v[0], &dev);
    at::Tensor g_held;
    const float* g = factor_of(c.v[0], dev, &g_held);
    const Weights weights = weights_of(c.v[1], dev);
    const moe_mx_weights& w = weights.w;
    same_operands(x, w);
    const at::Tensor& off = dense(c.v[2], "offsets", at::kInt, {w.num_experts + 1}, dev);
    const int64_t type = c.v[7] ? integer(c.v[7], "out_type") : MOE_MX_OUT_BF16;
    if (type != MOE_MX_OUT_BF16 && type != MOE_MX_OUT_F16) throw Failed{MOE_ERR_INVALID_ARG, "out_type"};
    const at::ScalarType dtype = type == MOE_MX_OUT_F16 ? at::kHalf : at::kBFloat16;
    int64_t out_rows = x.n, ld = w.n_out;
    if (c.v[3]) {
      const at::Tensor& o = tensor(c.v[3], "out");
      if (o.scalar_type() != dtype || o.dim() != 2 || o.size(1) != w.n_out || o.get_device() != dev ||
          (w.n_out > 1 && o.stride(1) != 1))
        throw Refused{"out: of another type, width or device"};
      out_rows = o.size(0);
      ld = out_rows > 1 ? o.stride(0) : std::max<int64_t>(o.stride(0), ld);
    }
    const int32_t* pos =
        c.v[4] ? static_cast<const int32_t*>(dense(c.v[4], "out_pos", at::kInt, {x.n}, dev).const_data_ptr()) : nullptr;
    const float* weight = values(c.v[5], "row_weight", out_rows, dev);
    const cudaStream_t s = stream_of(dev);
    const c10::cuda::CUDAGuard on(x.codes_t.device());
    const Workspace ws = product_workspace(c.v[6], dev);
    at::Tensor out;
    if (c.v[3]) {
      out = tensor(c.v[3], "out");
    } else {
      // rows on 32-byte boundaries: the kernel writes them in whole pieces (2.5 times as fast)
      ld = (ld + 15) / 16 * 16;
      out = ld == w.n_out ? at::empty({x.n, ld}, x.codes_t.options().dtype(dtype))
                          : at::empty_strided({x.n, w.n_out}, {ld, 1}, x.codes_t.options().dtype(dtype));
    }
    call("moe_mx_grouped_product", [&] {
      return moe_mx_grouped_product(&w, x.n, x.codes, x.scales, g, static_cast<const int32_t*>(off.const_data_ptr()),
                                    out.data_ptr(), static_cast<int32_t>(type), out_rows, ld, pos, weight,
                                    ws.at, ws.bytes, s);
    });
    return c.v[3] ? Py_NewRef(c.v[3]) : THPVariable_Wrap(out);
  });
}

PyObject* mx_grouped_swiglu(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"x", "w", "offsets", "h_global", "out", "ws", "stream"};
    const Call<7> c("mx_grouped_swiglu", names, 3, args, nargs, kwnames);
    if (c.v[6]) return hand_over("mx_grouped_swiglu", c);
    if (!c.v[0]) throw Refused{"x: expected rows"};
    int dev = -2;
    const Rows x = rows_of(c.v[0], &dev);
    at::Tensor g_held;
    const float* g = factor_of(c.v[0], dev, &g_held);
    const Weights weights = weights_of(c.v[1], dev);
    const moe_mx_weights& w = weights.w;
    same_operands(x, w);
    const at::Tensor& off = dense(c.v[2], "offsets", at::kInt, {w.num_experts + 1}, dev);
    const float* hg = values(c.v[3], "h_global", 1, dev);
    const cudaStream_t s = stream_of(dev);
    const c10::cuda::CUDAGuard on(x.codes_t.device());
    Target t;
    target(&t, w.format, x.n, w.n_out, 0, c.v[3], c.v[4], x.codes_t, dev);
    if (t.r.n != x.n) throw Refused{"out: of another number of rows"};
    const Workspace ws = product_workspace(c.v[5], dev);
    call("moe_mx_grouped_swiglu", [&] {
      return moe_mx_grouped_swiglu(&w, x.n, x.codes, x.scales, g, static_cast<const int32_t*>(off.const_data_ptr()), hg,
                  t.r.codes, t.r.scales, ws.at, ws.bytes, s);
    });
    return t.take();
  });
}

PyObject* mx_layer_forward(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"x",       "residual", "gain",     "eps",      "topk_ids", "topk_weight", "gate_up",
                                        "down",    "x_global", "h_global", "ws",       "out_is_fp32", "stream"};
    const Call<13> c("mx_layer_forward", names, 8, args, nargs, kwnames);
    if (c.v[12]) return hand_over("mx_layer_forward", c);
    const at::Tensor& x = tensor(c.v[0], "x");
    two_dims(x, "x");
    const int64_t n = x.size(0), d = x.size(1);
    const int dev = static_cast<int>(x.get_device());
    dense(c.v[0], "x", at::kBFloat16, {n, d}, dev);
    const void* res = c.v[1] ? dense(c.v[1], "residual", at::kBFloat16, {n, d}, dev).const_data_ptr() : nullptr;
    const void* gain = c.v[2] ? dense(c.v[2], "gain", at::kBFloat16, {d}, dev).const_data_ptr() : nullptr;
    const float eps = number(c.v[3], "eps");
    const at::Tensor& ids = tensor(c.v[4], "topk_ids");
    two_dims(ids, "topk_ids");
    const int64_t k = ids.size(1);
    if (k > INT32_MAX) throw Failed{MOE_ERR_UNSUPPORTED, "topk_ids"};
    dense(c.v[4], "topk_ids", at::kInt, {n, k}, dev);
    const at::Tensor& weight = dense(c.v[5], "topk_weight", at::kFloat, {n, k}, dev);
    const Weights gu_all = weights_of(c.v[6], dev), dn_all = weights_of(c.v[7], dev);
    const moe_mx_weights &gu = gu_all.w, &dn = dn_all.w;
    if (d != gu.k) throw Refused{"x: of another width than the experts"};
    const float* xg = values(c.v[8], "x_global", 1, dev);
    const float* hg = values(c.v[9], "h_global", 1, dev);
    const bool fp32 = c.v[11] && PyObject_IsTrue(c.v[11]) == 1;
    const cudaStream_t s = stream_of(dev);
    const c10::cuda::CUDAGuard on(x.device());
    at::Tensor ws;
    if (c.v[10]) {
      ws = workspace_of(c.v[10], dev);
    } else {
      const size_t bytes = moe_mx_layer_workspace_size(&gu, &dn, static_cast<int32_t>(k), n);
      if (bytes == 0) throw Failed{MOE_ERR_UNSUPPORTED, "moe_mx_layer_workspace_size"};
      ws = at::empty({static_cast<int64_t>(bytes)}, x.options().dtype(at::kByte));
    }
    at::Tensor sum;
    if (gain) sum = at::empty({n, d}, x.options());
    const at::Tensor out = at::empty({n, d}, fp32 ? x.options().dtype(at::kFloat) : x.options());
    call("moe_mx_layer_forward", [&] {
      return (c.v[10] ? moe_mx_layer_forward : moe_mx_layer_forward_default)(
                  &gu, &dn, static_cast<int32_t>(k), n, x.const_data_ptr(), res, gain, eps,
                  static_cast<const int32_t*>(ids.const_data_ptr()),
                  static_cast<const float*>(weight.const_data_ptr()), xg, hg, gain ? sum.data_ptr() : nullptr,
                  out.data_ptr(), fp32, ws.data_ptr(), ws.nbytes(), s);
    });
    PyObject* sum_o = gain ? THPVariable_Wrap(sum) : Py_NewRef(Py_None);
    PyObject* out_o = THPVariable_Wrap(out);
    PyObject* both = sum_o && out_o ? PyTuple_New(2) : nullptr;
    if (!both) {
      Py_XDECREF(sum_o);
      Py_XDECREF(out_o);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(both, 0, sum_o);
    PyTuple_SET_ITEM(both, 1, out_o);
    return both;
  });
}

// default_error(): moe_get_error of the current device's own workspace.
PyObject* default_error(PyObject*, PyObject*) {
  return guarded([&]() -> PyObject* {
    void* const ws = moe_mx_default_workspace();
    if (!ws) throw Failed{MOE_ERR_CUDA, "moe_mx_default_workspace"};
    const cudaStream_t s = c10::cuda::getCurrentCUDAStream().stream();
    moe_status st;
    Py_BEGIN_ALLOW_THREADS
    st = moe_get_error(ws, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
  });
}

// setup(MxRows, MoeError, on): what the calls make, raise and hand other streams to.
PyObject* setup(PyObject* self, PyObject* args) {
  PyObject *rows, *error, *on;
  if (!PyArg_ParseTuple(args, "OOO", &rows, &error, &on)) return nullptr;
  Py_XSETREF(rows_class, Py_NewRef(rows));
  Py_XSETREF(moe_error, Py_NewRef(error));
  Py_XSETREF(on_stream, Py_NewRef(on));
  module_dict = PyModule_GetDict(self);
  Py_RETURN_NONE;
}

#define MX_CALL(name, doc) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL | METH_KEYWORDS, doc}

PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, nullptr},
    {"default_error", default_error, METH_NOARGS, nullptr},
    MX_CALL(mx_quantise,
            "mx_quantise(x, fmt, positions=None, out_rows=None, global_scale=None, out=None, stream=None) -> MxRows\n\n"
            "bf16 rows x [n, d] (any row stride that is a multiple of 8) into a format; row t goes to each of\n"
            "positions[t] (int32 [n, k], entries outside the rows are skipped; default its own place, for which there\n"
            "have to be n rows or more) of `out` (out_rows rows, default n * k)."),
    MX_CALL(mx_add_rmsnorm,
            "mx_add_rmsnorm(x, residual, gain, eps, fmt, positions=None, out_rows=None, global_scale=None,\n"
            "               sum_out=None, out=None, stream=None) -> (MxRows, sum)\n\n"
            "sum = bf16(x + residual) (residual may be None), rows = Q(rmsnorm(sum)) written as by mx_quantise.\n"
            "sum_out may be x or residual."),
    MX_CALL(mx_dequantise, "mx_dequantise(r, out=None, stream=None)\n\nbf16 values of rows."),
    MX_CALL(mx_grouped_product,
            "mx_grouped_product(x, w, offsets, out=None, out_pos=None, row_weight=None, ws=None,\n"
            "                   out_type=MOE_MX_OUT_BF16, stream=None)\n\n"
            "out[p(r)] = row_weight[p(r)] * x[r] W_e^T for the rows offsets[e] .. offsets[e + 1] - 1 of each expert e;\n"
            "p = out_pos (int32 [rows], default r).  A new out has rows on 32-byte boundaries (its row stride is n_out\n"
            "rounded up to 16).  Rows of no expert are left as they are, all of them where the offsets do not ascend within\n"
            "the rows of x; in a new out they are uninitialised.  Device errors: moe_get_error(ws), mx_get_error() where no\n"
            "ws is given."),
    MX_CALL(mx_grouped_swiglu,
            "mx_grouped_swiglu(x, w, offsets, h_global=None, out=None, ws=None, stream=None) -> MxRows\n\n"
            "Rows of silu(x Wg_e^T) * (x Wu_e^T) in the format of x.  Rows of no expert and device errors as in\n"
            "mx_grouped_product."),
    MX_CALL(mx_layer_forward,
            "mx_layer_forward(x, residual, gain, eps, topk_ids, topk_weight, gate_up, down, x_global=None,\n"
            "                 h_global=None, ws=None, out_is_fp32=False, stream=None) -> (sum, out)\n\n"
            "The MoE block on microscaled experts: sum = bf16(x + residual), out = sum + the routed experts on\n"
            "rmsnorm(sum); with gain None (and residual None) (None, the routed experts on x).  Device errors (ids outside\n"
            "the experts, whose tokens' out rows are unspecified; expert rows beyond f16's range): moe_get_error(ws),\n"
            "mx_get_error() where no ws is given."),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef definition = {PyModuleDef_HEAD_INIT, "_mx_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mx_torch() {
  struct {
    PyObject** at;
    const char* name;
  } names[] = {{&s_fmt, "fmt"},         {&s_cols, "cols"},   {&s_codes, "codes"},     {&s_scales, "scales"},
               {&s_global_scale, "global_scale"}, {&s_num_experts, "num_experts"}, {&s_n_out, "n_out"},
               {&s_k, "k"},             {&s_packed, "packed"}, {&s_alpha, "alpha"},   {&s_alpha_up, "alpha_up"},
               {&s_swiglu, "swiglu"}};
  for (auto& n : names)
    if (!(*n.at = PyUnicode_InternFromString(n.name))) return nullptr;
  return PyModule_Create(&definition);
}
