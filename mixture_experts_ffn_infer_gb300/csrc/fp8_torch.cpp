// The router's and the FP8 calls on torch tensors (moe_router.h, moe_fp8.h; fp8.py adds the classes), part of the
// module of mx_torch.cpp.
#include "moe_fp8.h"
#include "moe_router.h"
#include "mx_default.h"
#include "torch_args.h"

namespace {

using namespace torch_args;

PyObject* rows_class = nullptr;  // fp8.Fp8Rows
PyObject* s_codes;
PyObject* s_scales;
PyObject* s_num_experts;
PyObject* s_n_out;
PyObject* s_k;
PyObject* s_packed;

PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* both = a && b ? PyTuple_New(2) : nullptr;
  if (!both) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    throw PythonError{};
  }
  PyTuple_SET_ITEM(both, 0, a);
  PyTuple_SET_ITEM(both, 1, b);
  return both;
}

bool truth(PyObject* o, bool otherwise) {
  if (!o) return otherwise;
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v == 1;
}

// A 32-bit argument.
int32_t small(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) throw Failed{MOE_ERR_UNSUPPORTED, name};
  return static_cast<int32_t>(v);
}

// ---------------------------------------------------------------- the router

// Rows [n, E] of logits (or their gradient): the row stride in elements.
int64_t logit_rows(const at::Tensor& t, const char* name, at::ScalarType type, int64_t n, int64_t E, int dev) {
  if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != n || t.size(1) != E || t.get_device() != dev ||
      (E > 1 && t.stride(1) != 1)) {
    std::ostringstream s;
    s << type << " rows [" << n << ", " << E << "] on device " << dev;
    refuse(name, s.str(), t);
  }
  if (n <= 1) return E;
  if (t.stride(0) < E) refuse(name, "rows of their own, not " + std::to_string(t.stride(0)) + " elements apart", t);
  return t.stride(0);
}

struct Logits {
  const at::Tensor* t;
  int64_t n, E, ld;
  int dev;
  moe_router r{};
};
Logits logits_of(PyObject* o, PyObject* score) {
  Logits l;
  l.t = &tensor(o, "logits");
  two_dims(*l.t, "logits");
  l.n = l.t->size(0);
  l.E = l.t->size(1);
  l.dev = static_cast<int>(l.t->get_device());
  if (l.t->scalar_type() != at::kFloat && l.t->scalar_type() != at::kBFloat16)
    refuse("logits", "fp32 or bf16 rows", *l.t);
  l.ld = logit_rows(*l.t, "logits", l.t->scalar_type(), l.n, l.E, l.dev);
  if (l.E > INT32_MAX) throw Failed{MOE_ERR_UNSUPPORTED, "logits"};
  l.r.num_experts = static_cast<int32_t>(l.E);
  l.r.score = small(score, "score");
  l.r.logits_type = l.t->scalar_type() == at::kFloat ? MOE_LOGITS_F32 : MOE_LOGITS_BF16;
  l.r.groups = l.r.top_groups = 1;
  l.r.scale = 1.f;
  return l;
}

const int32_t* ids_of(PyObject* o, Logits* l) {
  const at::Tensor& t = tensor(o, "ids");
  two_dims(t, "ids");
  const int64_t k = t.size(1);
  if (k > INT32_MAX) throw Failed{MOE_ERR_UNSUPPORTED, "ids"};
  l->r.top_k = static_cast<int32_t>(k);
  return static_cast<const int32_t*>(dense(o, "ids", at::kInt, {l->n, k}, l->dev).const_data_ptr());
}

const int32_t* sequences_of(PyObject* o, int dev, int64_t* count) {
  *count = 1;
  if (!o) return nullptr;
  const at::Tensor& t = tensor(o, "seq_offsets");
  if (t.dim() != 1 || t.numel() < 2) refuse("seq_offsets", "an int32 tensor of two values or more", t);
  *count = t.numel() - 1;
  return static_cast<const int32_t*>(dense(o, "seq_offsets", at::kInt, {*count + 1}, dev).const_data_ptr());
}

PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"logits",    "top_k", "score", "bias",    "groups", "top_groups",
                                        "normalise", "scale", "ids",   "weights", "stream"};
    const Call<11> c("route", names, 3, args, nargs, kwnames);
    if (c.v[10]) return hand_over("route", c);
    Logits l = logits_of(c.v[0], c.v[2]);
    l.r.top_k = small(c.v[1], "top_k");
    const float* bias = values(c.v[3], "bias", l.E, l.dev);
    if (c.v[4]) l.r.groups = small(c.v[4], "groups");
    if (c.v[5]) l.r.top_groups = small(c.v[5], "top_groups");
    l.r.normalise = truth(c.v[6], true);
    if (c.v[7]) l.r.scale = number(c.v[7], "scale");
    if (l.r.top_k < 1) throw Failed{MOE_ERR_UNSUPPORTED, "moe_route"};
    const int64_t k = l.r.top_k;
    at::Tensor ids, weights;
    if (c.v[8]) ids = dense(c.v[8], "ids", at::kInt, {l.n, k}, l.dev);
    if (c.v[9]) weights = dense(c.v[9], "weights", at::kFloat, {l.n, k}, l.dev);
    const cudaStream_t s = stream_of(l.dev);
    const c10::cuda::CUDAGuard on(l.t->device());
    if (k <= 32) {  // (a larger one is refused below, before it is allocated)
      if (!c.v[8]) ids = at::empty({l.n, k}, l.t->options().dtype(at::kInt));
      if (!c.v[9]) weights = at::empty({l.n, k}, l.t->options().dtype(at::kFloat));
    }
    call("moe_route", [&] {
      return moe_route(&l.r, l.n, l.t->const_data_ptr(), l.ld, bias,
                       k <= 32 ? static_cast<int32_t*>(ids.data_ptr()) : nullptr,
                       k <= 32 ? static_cast<float*>(weights.data_ptr()) : nullptr, s);
    });
    PyObject* a = c.v[8] ? Py_NewRef(c.v[8]) : THPVariable_Wrap(ids);
    return pair(a, c.v[9] ? Py_NewRef(c.v[9]) : THPVariable_Wrap(weights));
  });
}

PyObject* balance_loss(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"logits", "ids", "coef", "score", "seq_offsets", "ws", "stream"};
    const Call<7> c("balance_loss", names, 4, args, nargs, kwnames);
    if (c.v[6]) return hand_over("balance_loss", c);
    Logits l = logits_of(c.v[0], c.v[3]);
    const int32_t* ids = ids_of(c.v[1], &l);
    const float coef = number(c.v[2], "coef");
    int64_t sequences;
    const int32_t* offsets = sequences_of(c.v[4], l.dev, &sequences);
    const cudaStream_t s = stream_of(l.dev);
    const c10::cuda::CUDAGuard on(l.t->device());
    const size_t bytes = moe_balance_workspace_size(&l.r, l.n, sequences);
    if (bytes == 0) throw Failed{MOE_ERR_UNSUPPORTED, "moe_balance_workspace_size"};
    at::Tensor ws;
    if (c.v[5]) {
      ws = tensor(c.v[5], "ws");
      if (ws.get_device() != l.dev || !ws.is_contiguous())
        refuse("ws", "contiguous bytes on device " + std::to_string(l.dev), ws);
    } else {
      ws = at::empty({static_cast<int64_t>(bytes)}, l.t->options().dtype(at::kByte));
    }
    const at::Tensor counts = at::empty({sequences, l.E}, l.t->options().dtype(at::kInt));
    const at::Tensor loss = at::empty({}, l.t->options().dtype(at::kFloat));
    call("moe_balance_loss", [&] {
      return moe_balance_loss(&l.r, l.n, l.t->const_data_ptr(), l.ld, ids, coef, offsets, sequences,
                              static_cast<int32_t*>(counts.data_ptr()), static_cast<float*>(loss.data_ptr()),
                              ws.data_ptr(), ws.nbytes(), s);
    });
    PyObject* a = THPVariable_Wrap(loss);
    return pair(a, THPVariable_Wrap(counts));
  });
}

PyObject* route_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"logits", "ids",    "score",       "d_weights", "normalise", "scale",
                                        "counts", "coef",   "d_loss",      "seq_offsets", "out",     "stream"};
    const Call<12> c("route_backward", names, 3, args, nargs, kwnames);
    if (c.v[11]) return hand_over("route_backward", c);
    Logits l = logits_of(c.v[0], c.v[2]);
    const int32_t* ids = ids_of(c.v[1], &l);
    const float* d_weights = nullptr;
    if (c.v[3])
      d_weights = static_cast<const float*>(
          dense(c.v[3], "d_weights", at::kFloat, {l.n, static_cast<int64_t>(l.r.top_k)}, l.dev).const_data_ptr());
    l.r.normalise = truth(c.v[4], true);
    if (c.v[5]) l.r.scale = number(c.v[5], "scale");
    int64_t sequences;
    const int32_t* offsets = sequences_of(c.v[9], l.dev, &sequences);
    const int32_t* counts = nullptr;
    float coef = 0.f;
    if (c.v[6]) {
      counts = static_cast<const int32_t*>(dense(c.v[6], "counts", at::kInt, {sequences, l.E}, l.dev).const_data_ptr());
      if (!c.v[7]) throw Refused{"coef: missing, it goes with counts"};
      coef = number(c.v[7], "coef");
    }
    const float* d_loss = values(c.v[8], "d_loss", 1, l.dev);
    int64_t ld = l.E;
    at::Tensor out;
    if (c.v[10]) {
      out = tensor(c.v[10], "out");
      ld = logit_rows(out, "out", l.t->scalar_type(), l.n, l.E, l.dev);
    }
    const cudaStream_t s = stream_of(l.dev);
    const c10::cuda::CUDAGuard on(l.t->device());
    if (!c.v[10]) out = at::empty({l.n, l.E}, l.t->options());
    call("moe_route_backward", [&] {
      return moe_route_backward(&l.r, l.n, l.t->const_data_ptr(), l.ld, ids, d_weights, coef, counts, d_loss, offsets,
                                sequences, out.data_ptr(), ld, s);
    });
    return c.v[10] ? Py_NewRef(c.v[10]) : THPVariable_Wrap(out);
  });
}

// ---------------------------------------------------------------- FP8 rows

struct Rows {
  int64_t n = 0, cols = 0;
  at::Tensor codes, scales;
};

int64_t pitch_of(int64_t cols) {
  const int64_t pitch = moe_fp8_scale_pitch(cols);
  if (pitch == 0 || cols > INT32_MAX) throw Failed{MOE_ERR_UNSUPPORTED, "moe_fp8_scale_pitch"};
  return pitch;
}

// An Fp8Rows, checked; *dev is its device, or has to be where it is not -2.
Rows rows_of(PyObject* o, int* dev) {
  const Field codes(o, s_codes), scales(o, s_scales);
  Rows r;
  r.codes = tensor(codes.get(), "codes");
  two_dims(r.codes, "codes");
  r.n = r.codes.size(0);
  r.cols = r.codes.size(1);
  if (*dev == -2) *dev = static_cast<int>(r.codes.get_device());
  const int64_t pitch = pitch_of(r.cols);
  if ((r.codes.scalar_type() != at::kByte && r.codes.scalar_type() != at::kFloat8_e4m3fn) || !r.codes.is_contiguous() ||
      r.codes.get_device() != *dev)
    refuse("codes", "contiguous e4m3 codes (as bytes or float8_e4m3fn) on device " + std::to_string(*dev), r.codes);
  r.scales = dense(scales.get(), "scales", at::kFloat, {r.n, pitch}, *dev);
  return r;
}

PyObject* fp8_quantise(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"x", "positions", "out_rows", "out", "stream"};
    const Call<5> c("fp8_quantise", names, 1, args, nargs, kwnames);
    if (c.v[4]) return hand_over("fp8_quantise", c);
    const at::Tensor& x = tensor(c.v[0], "x");
    two_dims(x, "x");
    const int64_t n = x.size(0), d = x.size(1);
    int dev = static_cast<int>(x.get_device());
    const int64_t ld = row_stride(x, "x", n, d, dev);
    int64_t k = 1;
    const int32_t* pos = nullptr;
    if (c.v[1]) {
      const at::Tensor& t = tensor(c.v[1], "positions");
      two_dims(t, "positions");
      k = t.size(1);
      if (k > INT32_MAX) throw Failed{MOE_ERR_UNSUPPORTED, "positions"};
      pos = static_cast<const int32_t*>(dense(c.v[1], "positions", at::kInt, {n, k}, dev).const_data_ptr());
    }
    const int64_t pitch = pitch_of(d);
    Rows r;
    if (c.v[3]) {
      r = rows_of(c.v[3], &dev);
      if (r.cols != d) throw Refused{"out: of another width"};
    } else {
      r.n = c.v[2] ? integer(c.v[2], "out_rows") : n * k;
      if (r.n < 0) throw Refused{"out_rows: negative"};
    }
    if (!pos && r.n < n) throw Refused{std::string(c.v[3] ? "out" : "out_rows") + ": fewer rows than x, and no positions"};
    const cudaStream_t s = stream_of(dev);
    const c10::cuda::CUDAGuard on(x.device());
    if (!c.v[3]) {
      r.codes = at::empty({r.n, d}, x.options().dtype(at::kByte));
      r.scales = at::empty({r.n, pitch}, x.options().dtype(at::kFloat));
    }
    call("moe_fp8_quantise", [&] {
      return moe_fp8_quantise(n, static_cast<int32_t>(k), static_cast<int32_t>(d), x.const_data_ptr(), ld, pos, r.n,
                              r.codes.data_ptr(), static_cast<float*>(r.scales.data_ptr()), s);
    });
    if (c.v[3]) return Py_NewRef(c.v[3]);
    PyObject* a[2] = {THPVariable_Wrap(r.codes), THPVariable_Wrap(r.scales)};
    PyObject* o = a[0] && a[1] ? PyObject_Vectorcall(rows_class, a, 2, nullptr) : nullptr;
    Py_XDECREF(a[0]);
    Py_XDECREF(a[1]);
    if (!o) throw PythonError{};
    return o;
  });
}

PyObject* fp8_dequantise(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"r", "out", "stream"};
    const Call<3> c("fp8_dequantise", names, 1, args, nargs, kwnames);
    if (c.v[2]) return hand_over("fp8_dequantise", c);
    if (!c.v[0]) throw Refused{"r: expected rows"};
    int dev = -2;
    const Rows r = rows_of(c.v[0], &dev);
    at::Tensor out;
    int64_t ld = r.cols;
    if (c.v[1]) {
      out = tensor(c.v[1], "out");
      ld = row_stride(out, "out", r.n, r.cols, dev);
    }
    const cudaStream_t s = stream_of(dev);
    const c10::cuda::CUDAGuard on(r.codes.device());
    if (!c.v[1]) out = at::empty({r.n, r.cols}, r.codes.options().dtype(at::kBFloat16));
    call("moe_fp8_dequantise", [&] {
      return moe_fp8_dequantise(r.n, static_cast<int32_t>(r.cols), r.codes.const_data_ptr(),
                                static_cast<const float*>(r.scales.const_data_ptr()), out.data_ptr(), ld, s);
    });
    return c.v[1] ? Py_NewRef(c.v[1]) : THPVariable_Wrap(out);
  });
}

// ---------------------------------------------------------------- FP8 products

struct Weights {
  moe_fp8_weights w{};
  at::Tensor held[2];
};
Weights weights_of(PyObject* o, int dev) {
  if (!o) throw Refused{"w: expected Fp8Weights"};
  Weights all;
  moe_fp8_weights& w = all.w;
  const Field experts(o, s_num_experts), n_out(o, s_n_out), k(o, s_k), packed(o, s_packed), scales(o, s_scales);
  w.num_experts = small(experts.get(), "num_experts");
  w.n_out = small(n_out.get(), "n_out");
  w.k = small(k.get(), "k");
  const size_t bytes = moe_fp8_packed_bytes(&w);
  if (bytes == 0) throw Failed{MOE_ERR_UNSUPPORTED, "moe_fp8_packed_bytes"};
  const at::Tensor& p = tensor(packed.get(), "packed");
  if (p.nbytes() != bytes || !p.is_contiguous() || p.get_device() != dev)
    refuse("packed", std::to_string(bytes) + " contiguous bytes on device " + std::to_string(dev), p);
  w.packed = p.const_data_ptr();
  const int64_t nb = (static_cast<int64_t>(w.n_out) + 127) / 128, kb = (static_cast<int64_t>(w.k) + 127) / 128;
  const at::Tensor& t = dense(scales.get(), "scales", at::kFloat, {w.num_experts, nb, kb}, dev);
  w.scales = static_cast<const float*>(t.const_data_ptr());
  all.held[0] = p;
  all.held[1] = t;
  return all;
}

PyObject* fp8_grouped_product(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"x", "w", "offsets", "out", "out_pos", "row_weight", "ws", "out_type", "stream"};
    const Call<9> c("fp8_grouped_product", names, 2, args, nargs, kwnames);
    if (c.v[8]) return hand_over("fp8_grouped_product", c);
    if (!c.v[0]) throw Refused{"x: expected rows"};
    int dev = -2;
    const Rows x = rows_of(c.v[0], &dev);
    const Weights all = weights_of(c.v[1], dev);
    const moe_fp8_weights& w = all.w;
    if (x.cols != w.k) throw Refused{"x: of another width than the weights"};
    const int32_t* offsets = nullptr;
    if (c.v[2])
      offsets = static_cast<const int32_t*>(
          dense(c.v[2], "offsets", at::kInt, {static_cast<int64_t>(w.num_experts) + 1}, dev).const_data_ptr());
    else if (w.num_experts != 1)
      throw Refused{"offsets: missing, there are several experts"};
    const int64_t type = c.v[7] ? integer(c.v[7], "out_type") : MOE_FP8_OUT_BF16;
    if (type < MOE_FP8_OUT_BF16 || type > MOE_FP8_OUT_F32) throw Failed{MOE_ERR_INVALID_ARG, "out_type"};
    const at::ScalarType dtype =
        type == MOE_FP8_OUT_F32 ? at::kFloat : type == MOE_FP8_OUT_F16 ? at::kHalf : at::kBFloat16;
    int64_t out_rows = x.n, ld = w.n_out;
    at::Tensor out;
    if (c.v[3]) {
      out = tensor(c.v[3], "out");
      if (out.scalar_type() != dtype || out.dim() != 2 || out.size(1) != w.n_out || out.get_device() != dev ||
          (w.n_out > 1 && out.stride(1) != 1))
        throw Refused{"out: of another type, width or device"};
      out_rows = out.size(0);
      if (out_rows > 1) ld = out.stride(0);
      if (ld < w.n_out) throw Refused{"out: rows that overlap"};
    }
    const int32_t* pos =
        c.v[4] ? static_cast<const int32_t*>(dense(c.v[4], "out_pos", at::kInt, {x.n}, dev).const_data_ptr()) : nullptr;
    const float* weight = values(c.v[5], "row_weight", out_rows, dev);
    const cudaStream_t s = stream_of(dev);
    const c10::cuda::CUDAGuard on(x.codes.device());
    at::Tensor held;
    void* ws = nullptr;
    size_t ws_bytes = MOE_FP8_PRODUCT_WORKSPACE;
    if (c.v[6]) {
      held = tensor(c.v[6], "ws");
      if (held.get_device() != dev || !held.is_contiguous())
        refuse("ws", "contiguous bytes on device " + std::to_string(dev), held);
      ws = held.data_ptr();
      ws_bytes = held.nbytes();
    } else {
      ws = moe_mx_default_workspace();
    }
    if (!c.v[3]) {
      // rows on 32-byte boundaries: the kernel writes them in whole pieces
      const int64_t per = type == MOE_FP8_OUT_F32 ? 8 : 16;
      ld = (ld + per - 1) / per * per;
      out = ld == w.n_out ? at::empty({x.n, ld}, x.codes.options().dtype(dtype))
                          : at::empty_strided({x.n, w.n_out}, {ld, 1}, x.codes.options().dtype(dtype));
    }
    call("moe_fp8_grouped_product", [&] {
      return moe_fp8_grouped_product(&w, x.n, x.codes.const_data_ptr(), static_cast<const float*>(x.scales.const_data_ptr()),
                                     offsets, out.data_ptr(), static_cast<int32_t>(type), out_rows, ld, pos, weight, ws,
                                     ws_bytes, s);
    });
    return c.v[3] ? Py_NewRef(c.v[3]) : THPVariable_Wrap(out);
  });
}

// fp8_setup(Fp8Rows): what the calls make.
PyObject* fp8_setup(PyObject*, PyObject* rows) {
  Py_XSETREF(rows_class, Py_NewRef(rows));
  Py_RETURN_NONE;
}

}  // namespace

PyMethodDef moe_fp8_methods[] = {
    {"fp8_setup", fp8_setup, METH_O, nullptr},
    MOE_TORCH_CALL(route,
                   "route(logits, top_k, score, bias=None, groups=1, top_groups=1, normalise=True, scale=1.0, ids=None,\n"
                   "      weights=None, stream=None) -> (ids, weights)\n\n"
                   "The top_k experts of each row of logits [n, E] (fp32 or bf16, any row stride) by score + bias (fp32 [E])\n"
                   "within the top_groups best of `groups` runs of experts, in descending order, ties to the lowest index,\n"
                   "and their weights: scale * score, over the chosen scores' sum with normalise.  score: MOE_SCORE_SOFTMAX\n"
                   "or MOE_SCORE_SIGMOID.  ids int32, weights fp32, [n, top_k]: new, or the caller's.  A logit of -inf masks\n"
                   "its expert; places that stay empty get id -1 and weight 0, a row with a NaN ids -1 and weights NaN."),
    MOE_TORCH_CALL(balance_loss,
                   "balance_loss(logits, ids, coef, score, seq_offsets=None, ws=None, stream=None) -> (loss, counts)\n\n"
                   "coef times the mean over the sequences with rows of E / (k T^2) sum_e count_e sum_t q_te, with q the scores\n"
                   "over their sum: coef where all experts get the same.  Sequence s has the rows seq_offsets[s] ..\n"
                   "seq_offsets[s + 1] - 1 (int32; None: one sequence of all rows); rows behind the last add nothing.\n"
                   "loss: fp32, no dimensions; counts: int32 [sequences, E] entries of ids per expert.  ws:\n"
                   "moe_balance_workspace_size bytes that the call may overwrite (default: allocated)."),
    MOE_TORCH_CALL(route_backward,
                   "route_backward(logits, ids, score, d_weights=None, normalise=True, scale=1.0, counts=None, coef=None,\n"
                   "               d_loss=None, seq_offsets=None, out=None, stream=None) -> d_logits\n\n"
                   "The logits' gradient: of the weights of ids, given theirs (d_weights, fp32 [n, top_k]), and of the balance\n"
                   "loss, given counts, coef, seq_offsets as balance_loss had and made them and d_loss (fp32, one value,\n"
                   "default 1); either part may be left out.  out may be logits itself."),
    MOE_TORCH_CALL(fp8_quantise,
                   "fp8_quantise(x, positions=None, out_rows=None, out=None, stream=None) -> Fp8Rows\n\n"
                   "bf16 rows x [n, d] (any row stride that is a multiple of 8) as e4m3 codes with one fp32 scale per 128\n"
                   "columns; row t goes to each of positions[t] (int32 [n, k], entries outside the rows are skipped; default\n"
                   "its own place, for which there have to be n rows or more) of `out` (out_rows rows, default n * k)."),
    MOE_TORCH_CALL(fp8_dequantise, "fp8_dequantise(r, out=None, stream=None)\n\nbf16 values of rows."),
    MOE_TORCH_CALL(fp8_grouped_product,
                   "fp8_grouped_product(x, w, offsets=None, out=None, out_pos=None, row_weight=None, ws=None,\n"
                   "                    out_type=MOE_FP8_OUT_BF16, stream=None)\n\n"
                   "out[p(r)] = row_weight[p(r)] * x[r] W_e^T for the rows offsets[e] .. offsets[e + 1] - 1 of each expert e\n"
                   "(offsets may be left out where there is one expert: all rows); p = out_pos (int32 [rows], default r).  A\n"
                   "new out has rows on 32-byte boundaries.  Rows of no expert are left as they are, all of them where the\n"
                   "offsets do not ascend within the rows of x; in a new out they are uninitialised.  Device errors:\n"
                   "moe_get_error(ws), mx_get_error() where no ws is given."),
    {nullptr, nullptr, 0, nullptr}};

bool moe_fp8_names() {
  struct {
    PyObject** at;
    const char* name;
  } names[] = {{&s_codes, "codes"}, {&s_scales, "scales"}, {&s_num_experts, "num_experts"},
               {&s_n_out, "n_out"}, {&s_k, "k"},           {&s_packed, "packed"}};
  for (auto& n : names)
    if (!(*n.at = PyUnicode_InternFromString(n.name))) return false;
  return true;
}
