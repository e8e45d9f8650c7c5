// Python entry to the C ABI of the layers around the experts (block.py) and of a
// training step's losses and optimiser (step.py): the argument checks, output
// allocation and the call, in one C function each.  A decode step's calls take the
// GPU 4 to 8 us; these take the host 3.6 to 5 (the products' gradients 8 to 9), where
// the same steps in Python and ctypes took 11 to 13.5.  No computation happens here.
#include <Python.h>

#include <algorithm>
#include <initializer_list>
#include <utility>
#include <vector>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mgg.h"

namespace {

using at::ScalarType;
using at::Tensor;

// Thrown with a Python exception set.
struct Raised {};

[[noreturn]] void fail(PyObject* type, const char* fmt, const char* what, long a = 0, long b = 0) {
  PyErr_Format(type, fmt, what, a, b);
  throw Raised{};
}

const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", what);
  return THPVariable_Unpack(o);
}
mgg_dtype code(ScalarType t) {
  if (t == at::kBFloat16) return MGG_BF16;
  if (t == at::kFloat) return MGG_F32;
  PyErr_SetString(PyExc_TypeError, "unsupported dtype: bfloat16 or float32");
  throw Raised{};
}
ScalarType dtype_or(PyObject* o, ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) fail(PyExc_TypeError, "%s must be a torch.dtype", "dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
void on_gpu(const Tensor& t) {
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must live on a CUDA device", "tensors");
}

// A call's tensors live on one GPU, that of its first argument, and the call
// runs there whichever device is current: the library launches, asks for sizes
// and zeroes on the current device.  Built before anything else is read off the
// arguments (what is no tensor is refused later, by name).
struct OnDevice {
  OnDevice(const Tensor& x, std::initializer_list<std::pair<PyObject*, const char*>> others) {
    if (!x.is_cuda()) return;  // (refused by its own check)
    for (const auto& [o, what] : others)
      if (THPVariable_Check(o) && THPVariable_Unpack(o).device() != x.device())
        fail(PyExc_ValueError, "%s must be on the first argument's device", what);
    guard.set_index(x.device().index());
  }
  c10::cuda::OptionalCUDAGuard guard;
};

// A matrix with contiguous rows, rows ld elements apart.
struct Rows {
  const void* ptr;
  int rows, cols;
  int64_t ld;
};
int small(int64_t n, const char* what) {
  if (n > 0x7fffffff) fail(PyExc_ValueError, "%s has a dimension over 2^31 - 1", what);
  return static_cast<int>(n);
}
Rows rows_of(const Tensor& t, const char* what) {
  on_gpu(t);
  if (t.dim() != 2) fail(PyExc_ValueError, "%s must be a 2-D tensor", what);
  Rows r{t.data_ptr(), small(t.size(0), what), small(t.size(1), what), t.size(1)};
  if (!t.is_contiguous()) {
    if (r.cols > 1 && t.stride(1) != 1)
      fail(PyExc_ValueError, "%s: the last dimension must be contiguous", what);
    if (r.rows > 1) r.ld = t.stride(0);
    if (r.ld < r.cols) fail(PyExc_ValueError, "%s: rows must not overlap", what);
  }
  return r;
}
// A contiguous tensor of the given shape.
void* dense(const Tensor& t, std::initializer_list<int64_t> shape, const char* what) {
  if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size())) {
    if (shape.size() == 1)
      fail(PyExc_ValueError, "%s must be [%ld]", what, *shape.begin());
    fail(PyExc_ValueError, "%s must be [%ld, %ld]", what, *shape.begin(), *(shape.begin() + 1));
  }
  on_gpu(t);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", "tensors");
  return t.data_ptr();
}
float* dense_f32(const Tensor& t, std::initializer_list<int64_t> shape, const char* what) {
  if (t.scalar_type() != at::kFloat) fail(PyExc_ValueError, "%s must be float32", what);
  return static_cast<float*>(dense(t, shape, what));
}
const void* opt_bf16(PyObject* o, std::initializer_list<int64_t> shape, const char* what) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, what);
  if (t.scalar_type() != at::kBFloat16) fail(PyExc_TypeError, "%s must be bfloat16", what);
  return dense(t, shape, what);
}

Tensor empty(std::initializer_list<int64_t> shape, ScalarType t, const Tensor& like) {
  return at::detail::empty_cuda(at::IntArrayRef(shape.begin(), shape.size()), t, like.device(),
                                c10::nullopt);
}
// The caller's workspace where it is large enough, else a new one.
Tensor room(PyObject* o, size_t bytes, const Tensor& like) {
  if (o != Py_None) {
    const Tensor& t = tensor(o, "workspace");
    if (t.nbytes() >= bytes && t.is_cuda() && t.is_contiguous()) return t;
  }
  return empty({static_cast<int64_t>(bytes < 256 ? 256 : bytes)}, at::kByte, like);
}
void* stream(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }
int32_t* status_word(PyObject* o) {
  const Tensor& t = tensor(o, "status");
  if (t.scalar_type() != at::kInt || t.numel() < 1) fail(PyExc_ValueError, "%s must be int32 [1]", "status");
  on_gpu(t);
  return static_cast<int32_t*>(t.data_ptr());
}
long integer(PyObject* o, const char* what) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v != static_cast<int>(v)) fail(PyExc_ValueError, "%s is out of range", what);
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

// Raise the package's MggError for a status other than MGG_OK.
void check(mgg_status s, const char* where) {
  if (s == MGG_OK) return;
  PyObject* m = PyImport_ImportModule("variable_size_expert_gb300._lib");
  if (m) {
    PyObject* r = PyObject_CallMethod(m, "check", "is", static_cast<int>(s), where);
    Py_XDECREF(r);
    Py_DECREF(m);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
  }
  throw Raised{};
}

PyObject* none() { return Py_NewRef(Py_None); }
PyObject* wrap(const Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : none(); }
PyObject* tuple(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}

using Body = PyObject* (*)(PyObject* const*);
template <Body F, int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// x, weight, bias, eps, out_dtype
PyObject* layer_norm_forward(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const OnDevice dev(x, {{a[1], "weight"}, {a[2], "bias"}});
  const Tensor& w = tensor(a[1], "weight");
  const Rows r = rows_of(x, "x");
  const void* wp = dense(w, {r.cols}, "weight");
  const void* bp = nullptr;
  if (a[2] != Py_None) {
    const Tensor& b = tensor(a[2], "bias");
    bp = dense(b, {r.cols}, "bias");
    if (b.scalar_type() != w.scalar_type())
      fail(PyExc_TypeError, "%s must share a dtype", "weight and bias");
  }
  const double eps = number(a[3]);
  const ScalarType yt = dtype_or(a[4], x.scalar_type());
  const mgg_dtype xc = code(x.scalar_type()), yc = code(yt), wc = code(w.scalar_type());
  Tensor y = empty({r.rows, r.cols}, yt, x), mean = empty({r.rows}, at::kFloat, x),
         rstd = empty({r.rows}, at::kFloat, x);
  check(mgg_layer_norm_forward(r.ptr, xc, r.ld, wp, bp, wc, r.rows, r.cols, static_cast<float>(eps),
                               y.data_ptr(), yc, static_cast<float*>(mean.data_ptr()),
                               static_cast<float*>(rstd.data_ptr()), stream(x)),
        "mgg_layer_norm_forward");
  return tuple({y, mean, rstd});
}

// dy, x, weight, mean, rstd, bias, workspace
PyObject* layer_norm_backward(PyObject* const* a) {
  const Tensor& dy = tensor(a[0], "dy");
  const OnDevice dev(dy, {{a[1], "x"}, {a[2], "weight"}, {a[3], "mean"}, {a[4], "rstd"}, {a[6], "workspace"}});
  const Tensor &x = tensor(a[1], "x"), &w = tensor(a[2], "weight");
  const Rows r = rows_of(x, "x");
  const void* gp = dense(dy, {r.rows, r.cols}, "dy");
  const void* wp = dense(w, {r.cols}, "weight");
  const float* mp = dense_f32(tensor(a[3], "mean"), {r.rows}, "mean");
  const float* rp = dense_f32(tensor(a[4], "rstd"), {r.rows}, "rstd");
  const mgg_dtype xc = code(x.scalar_type()), wc = code(w.scalar_type()), yc = code(dy.scalar_type());
  Tensor dx = empty({r.rows, r.cols}, x.scalar_type(), x), dw = empty({r.cols}, w.scalar_type(), x), db;
  if (truth(a[5])) db = empty({r.cols}, w.scalar_type(), x);
  Tensor ws = room(a[6], mgg_workspace_bytes(MGG_OP_LAYER_NORM_BACKWARD, r.rows, 0, 0, 0, r.cols, xc), x);
  check(mgg_layer_norm_backward(gp, yc, r.ptr, xc, r.ld, wp, wc, mp, rp, r.rows, r.cols, dx.data_ptr(),
                                dw.data_ptr(), db.defined() ? db.data_ptr() : nullptr, ws.data_ptr(),
                                ws.nbytes(), stream(x)),
        "mgg_layer_norm_backward");
  return tuple({dx, dw, db});
}

// logits, k, scoring, bias, groups, topk_groups, renormalize, scale
PyObject* select_experts(PyObject* const* a) {
  const Tensor& l = tensor(a[0], "logits");
  const OnDevice dev(l, {{a[3], "bias"}});
  const Rows r = rows_of(l, "logits");
  const int k = static_cast<int>(integer(a[1], "k"));
  const float* bp = a[3] == Py_None ? nullptr : dense_f32(tensor(a[3], "bias"), {r.cols}, "bias");
  const mgg_dtype lc = code(l.scalar_type());
  if (k < 0) fail(PyExc_ValueError, "%s must be positive", "k");
  Tensor ids = empty({r.rows, k}, at::kInt, l), w = empty({r.rows, k}, at::kFloat, l);
  check(mgg_select_experts(r.ptr, lc, r.ld, r.rows, r.cols, k,
                           static_cast<mgg_scoring>(integer(a[2], "scoring")), bp,
                           static_cast<int>(integer(a[4], "groups")),
                           static_cast<int>(integer(a[5], "topk_groups")), truth(a[6]),
                           static_cast<float>(number(a[7])), static_cast<int32_t*>(ids.data_ptr()),
                           static_cast<float*>(w.data_ptr()), stream(l)),
        "mgg_select_experts");
  return tuple({ids, w});
}

// dtopk, logits, expert_ids, topk_weights, scoring, renormalize, scale, status
PyObject* select_experts_backward(PyObject* const* a) {
  const Tensor& g = tensor(a[0], "dtopk");
  const OnDevice dev(g, {{a[1], "logits"}, {a[2], "expert_ids"}, {a[3], "topk_weights"}, {a[7], "status"}});
  const Tensor &l = tensor(a[1], "logits"), &ids = tensor(a[2], "expert_ids"),
               &w = tensor(a[3], "topk_weights");
  const Rows r = rows_of(l, "logits");
  if (ids.dim() != 2 || ids.scalar_type() != at::kInt)
    fail(PyExc_ValueError, "%s must be int32 [T, k]", "expert_ids");
  const int k = small(ids.size(1), "expert_ids");
  const void* ip = dense(ids, {r.rows, k}, "expert_ids");
  const float* gp = dense_f32(g, {r.rows, k}, "dtopk");
  const float* wp = dense_f32(w, {r.rows, k}, "topk_weights");
  const mgg_dtype lc = code(l.scalar_type());
  Tensor d = empty({r.rows, r.cols}, l.scalar_type(), l);
  check(mgg_select_experts_backward(gp, r.ptr, lc, r.ld, static_cast<const int32_t*>(ip), wp, r.rows,
                                    r.cols, k, static_cast<mgg_scoring>(integer(a[4], "scoring")),
                                    truth(a[5]), static_cast<float>(number(a[6])), d.data_ptr(),
                                    status_word(a[7]), stream(l)),
        "mgg_select_experts_backward");
  return wrap(d);
}

struct LinearArgs {
  Rows x;
  int N;
  const void* W;
};
LinearArgs linear_args(const Tensor& x, const Tensor& W) {
  if (x.scalar_type() != at::kBFloat16 || W.scalar_type() != at::kBFloat16)
    fail(PyExc_TypeError, "%s must be bfloat16", "x and W");
  LinearArgs r{rows_of(x, "x"), 0, nullptr};
  r.N = W.dim() == 2 ? small(W.size(0), "W") : 0;
  r.W = dense(W, {r.N, r.x.cols}, "W");
  return r;
}

// x, W, bias, activation, residual, out_dtype, save_pre, status, out
PyObject* linear_forward(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const OnDevice dev(x, {{a[1], "W"}, {a[2], "bias"}, {a[4], "residual"}, {a[7], "status"}, {a[8], "out"}});
  const Tensor& W = tensor(a[1], "W");
  const LinearArgs l = linear_args(x, W);
  const int T = l.x.rows;
  const void* bp = nullptr;
  mgg_dtype bc = MGG_F32, rc = MGG_F32;
  if (a[2] != Py_None) {
    const Tensor& b = tensor(a[2], "bias");
    bp = dense(b, {l.N}, "bias");
    bc = code(b.scalar_type());
  }
  Rows res{nullptr, T, l.N, l.N};
  if (a[4] != Py_None) {
    const Tensor& t = tensor(a[4], "residual");
    res = rows_of(t, "residual");
    rc = code(t.scalar_type());
    if (res.rows != T || res.cols != l.N)
      fail(PyExc_ValueError, "%s must be [%ld, %ld]", "residual", T, l.N);
  }
  const int act = static_cast<int>(integer(a[3], "activation"));
  Tensor out, pre;
  if (a[8] != Py_None) {
    out = tensor(a[8], "out");
    dense(out, {T, l.N}, "out");
    if (out.scalar_type() != dtype_or(a[5], out.scalar_type()))
      fail(PyExc_TypeError, "%s must have out_dtype", "out");
  } else {
    const ScalarType t = dtype_or(a[5], at::kBFloat16);
    code(t);
    out = empty({T, l.N}, t, x);
  }
  const mgg_dtype oc = code(out.scalar_type());
  const bool save = truth(a[6]);
  if (save) pre = empty({T, l.N}, at::kBFloat16, x);
  check(mgg_linear_forward(l.x.ptr, l.x.ld, l.W, bp, bc, res.ptr, rc, res.ld, T, l.x.cols, l.N,
                           static_cast<mgg_activation>(act), out.data_ptr(), oc,
                           save ? pre.data_ptr() : nullptr, status_word(a[7]), stream(x)),
        "mgg_linear_forward");
  return save ? tuple({out, pre}) : wrap(out);
}

// dy, x, W, pre, activation, bias_dtype, need_dx, need_dW, status, workspace
PyObject* linear_backward(PyObject* const* a) {
  const Tensor& dy = tensor(a[0], "dy");
  const OnDevice dev(dy, {{a[1], "x"}, {a[2], "W"}, {a[3], "pre"}, {a[8], "status"}, {a[9], "workspace"}});
  const Tensor &x = tensor(a[1], "x"), &W = tensor(a[2], "W");
  const LinearArgs l = linear_args(x, W);
  const int T = l.x.rows, K = l.x.cols;
  const Rows g = rows_of(dy, "dy");
  if (g.rows != T || g.cols != l.N) fail(PyExc_ValueError, "%s must be [%ld, %ld]", "dy", T, l.N);
  const mgg_dtype gc = code(dy.scalar_type());
  const void* pp = opt_bf16(a[3], {T, l.N}, "pre");
  const int act = static_cast<int>(integer(a[4], "activation"));
  if (act != MGG_ACT_NONE && a[3] == Py_None) fail(PyExc_ValueError, "%s's backward needs pre", "an activation");
  Tensor dx, dW, db;
  mgg_dtype bc = MGG_F32;
  if (a[5] != Py_None) {
    const ScalarType t = dtype_or(a[5], at::kFloat);
    bc = code(t);
    db = empty({l.N}, t, x);
  }
  if (truth(a[6])) dx = empty({T, K}, at::kBFloat16, x);
  if (truth(a[7])) dW = empty({l.N, K}, at::kBFloat16, x);
  Tensor ws = room(a[9], mgg_workspace_bytes(MGG_OP_LINEAR_BACKWARD, T, 0, 0, l.N, K, MGG_BF16), x);
  auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  check(mgg_linear_backward(g.ptr, gc, g.ld, l.x.ptr, l.x.ld, l.W, pp, static_cast<mgg_activation>(act), T,
                            K, l.N, ptr(dx), ptr(dW), ptr(db), bc, status_word(a[8]), ws.data_ptr(),
                            ws.nbytes(), stream(x)),
        "mgg_linear_backward");
  return tuple({dx, dW, db});
}

// [T] bools, or none: every token counts.
const uint8_t* token_mask(PyObject* o, int T) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, "mask");
  if (t.scalar_type() != at::kBool) fail(PyExc_TypeError, "%s must be bool", "mask");
  return static_cast<const uint8_t*>(dense(t, {T}, "mask"));
}
const float* scalar_f32(const Tensor& t, const char* what) {
  if (t.scalar_type() != at::kFloat || t.numel() != 1) fail(PyExc_ValueError, "%s must be float32 [1]", what);
  on_gpu(t);
  return static_cast<const float*>(t.data_ptr());
}
int runs_of(PyObject* o, int T) {
  const long n = integer(o, "sequences");
  if (n < 1 || T % n != 0) fail(PyExc_ValueError, "%s must divide the tokens", "sequences");
  return static_cast<int>(n);
}

// logits, expert_ids, scoring, mask, sequences, status, workspace
PyObject* balance_loss_forward(PyObject* const* a) {
  const Tensor& l = tensor(a[0], "logits");
  const OnDevice dev(l, {{a[1], "expert_ids"}, {a[3], "mask"}, {a[5], "status"}, {a[6], "workspace"}});
  const Tensor& ids = tensor(a[1], "expert_ids");
  const Rows r = rows_of(l, "logits");
  if (ids.dim() != 2 || ids.scalar_type() != at::kInt)
    fail(PyExc_ValueError, "%s must be int32 [T, k]", "expert_ids");
  const int k = small(ids.size(1), "expert_ids");
  const void* ip = dense(ids, {r.rows, k}, "expert_ids");
  const uint8_t* mp = token_mask(a[3], r.rows);
  const int runs = runs_of(a[4], r.rows);
  const mgg_dtype lc = code(l.scalar_type());
  Tensor loss = empty({}, at::kFloat, l), counts = empty({runs, r.cols}, at::kInt, l),
         slope = empty({runs, r.cols}, at::kFloat, l);
  const size_t need = mgg_workspace_bytes(MGG_OP_BALANCE, r.rows, runs, r.cols, 0, 0, lc);
  Tensor ws;
  if (need) ws = room(a[6], need, l);
  check(mgg_balance_loss(r.ptr, lc, r.ld, static_cast<const int32_t*>(ip), mp, r.rows, r.cols, k, runs,
                         static_cast<mgg_scoring>(integer(a[2], "scoring")),
                         static_cast<float*>(loss.data_ptr()), static_cast<int32_t*>(counts.data_ptr()),
                         static_cast<float*>(slope.data_ptr()), status_word(a[5]), need ? ws.data_ptr() : nullptr,
                         need ? ws.nbytes() : 0, stream(l)),
        "mgg_balance_loss");
  return tuple({loss, counts, slope});
}

// dloss, logits, slope, scoring, mask
PyObject* balance_loss_backward(PyObject* const* a) {
  const Tensor& g = tensor(a[0], "dloss");
  const OnDevice dev(g, {{a[1], "logits"}, {a[2], "slope"}, {a[4], "mask"}});
  const Tensor &l = tensor(a[1], "logits"), &slope = tensor(a[2], "slope");
  const Rows r = rows_of(l, "logits");
  const float* gp = scalar_f32(g, "dloss");
  const int runs = slope.dim() == 2 ? small(slope.size(0), "slope") : 0;
  const float* sp = dense_f32(slope, {runs, r.cols}, "slope");
  if (runs < 1 || r.rows % runs != 0) fail(PyExc_ValueError, "%s must be [sequences, E]", "slope");
  const uint8_t* mp = token_mask(a[4], r.rows);
  const mgg_dtype lc = code(l.scalar_type());
  Tensor d = empty({r.rows, r.cols}, l.scalar_type(), l);
  check(mgg_balance_loss_backward(gp, r.ptr, lc, r.ld, sp, mp, r.rows, r.cols, runs,
                                  static_cast<mgg_scoring>(integer(a[3], "scoring")), d.data_ptr(), stream(l)),
        "mgg_balance_loss_backward");
  return wrap(d);
}

// The tokens' targets: int64 or int32 [T].
const void* targets_of(const Tensor& t, int T, bool* i64) {
  *i64 = t.scalar_type() == at::kLong;
  if (!*i64 && t.scalar_type() != at::kInt) fail(PyExc_TypeError, "%s must be int64 or int32", "targets");
  return dense(t, {T}, "targets");
}
long long wide_integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

// x, W, targets, ignore_index, reduction, z_loss, status, workspace
PyObject* linear_cross_entropy_forward(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const OnDevice dev(x, {{a[1], "W"}, {a[2], "targets"}, {a[6], "status"}, {a[7], "workspace"}});
  const LinearArgs l = linear_args(x, tensor(a[1], "W"));
  const int T = l.x.rows;
  bool i64;
  const void* tp = targets_of(tensor(a[2], "targets"), T, &i64);
  const int reduction = static_cast<int>(integer(a[4], "reduction"));
  Tensor loss = reduction == MGG_REDUCE_NONE ? empty({T}, at::kFloat, x) : empty({}, at::kFloat, x);
  Tensor lse = empty({T}, at::kFloat, x), weight = empty({1}, at::kFloat, x);
  Tensor ws = room(a[7], mgg_workspace_bytes(MGG_OP_VOCAB_FORWARD, T, 0, 0, l.N, l.x.cols, MGG_BF16), x);
  check(mgg_linear_cross_entropy(l.x.ptr, l.x.ld, l.W, tp, i64, wide_integer(a[3]), T, l.x.cols, l.N,
                                 static_cast<mgg_reduction>(reduction), static_cast<float>(number(a[5])),
                                 static_cast<float*>(loss.data_ptr()), static_cast<float*>(lse.data_ptr()),
                                 static_cast<float*>(weight.data_ptr()), status_word(a[6]), ws.data_ptr(),
                                 ws.nbytes(), stream(x)),
        "mgg_linear_cross_entropy");
  return tuple({loss, lse, weight});
}

// dloss, x, W, targets, lse, weight, ignore_index, z_loss, need_dx, need_dW, status, workspace
PyObject* linear_cross_entropy_backward(PyObject* const* a) {
  const Tensor& g = tensor(a[0], "dloss");
  const OnDevice dev(g, {{a[1], "x"}, {a[2], "W"}, {a[3], "targets"}, {a[4], "lse"}, {a[5], "weight"},
                         {a[10], "status"}, {a[11], "workspace"}});
  const Tensor& x = tensor(a[1], "x");
  const LinearArgs l = linear_args(x, tensor(a[2], "W"));
  const int T = l.x.rows, K = l.x.cols;
  bool i64;
  const void* tp = targets_of(tensor(a[3], "targets"), T, &i64);
  const float* lp = dense_f32(tensor(a[4], "lse"), {T}, "lse");
  const float* wp = scalar_f32(tensor(a[5], "weight"), "weight");
  const bool per_token = g.dim() == 1 && g.size(0) == T;
  const float* gp = per_token ? dense_f32(g, {T}, "dloss") : scalar_f32(g, "dloss");
  Tensor dx, dW;
  if (truth(a[8])) dx = empty({T, K}, at::kBFloat16, x);
  if (truth(a[9])) dW = empty({l.N, K}, at::kBFloat16, x);
  Tensor ws = room(a[11], mgg_workspace_bytes(MGG_OP_VOCAB_BACKWARD, T, 0, 0, l.N, K, MGG_BF16), x);
  check(mgg_linear_cross_entropy_backward(gp, per_token, wp, l.x.ptr, l.x.ld, l.W, tp, i64, wide_integer(a[6]),
                                          lp, T, K, l.N, static_cast<float>(number(a[7])),
                                          dx.defined() ? dx.data_ptr() : nullptr,
                                          dW.defined() ? dW.data_ptr() : nullptr, status_word(a[10]),
                                          ws.data_ptr(), ws.nbytes(), stream(x)),
        "mgg_linear_cross_entropy_backward");
  return tuple({dx, dW});
}

// A list or tuple of n tensors (n < 0: of any length), or none where that is allowed.
struct List {
  List(PyObject* o, const char* name, Py_ssize_t n, bool optional) : what(name) {
    if (optional && o == Py_None) return;
    fast = PySequence_Fast(o, "tensors come in lists");
    if (!fast) throw Raised{};
    count = PySequence_Fast_GET_SIZE(fast);
    if (n >= 0 && count != n) {
      Py_DECREF(fast);
      fail(PyExc_ValueError, "%s must hold a tensor for each of params", what);
    }
  }
  ~List() { Py_XDECREF(fast); }
  List(const List&) = delete;
  List& operator=(const List&) = delete;
  bool given() const { return fast != nullptr; }
  const Tensor& get(Py_ssize_t i) const { return tensor(PySequence_Fast_ITEMS(fast)[i], what); }
  // the i-th: of this dtype and number of elements, dense, on the device (a
  // training step checks a thousand of these: one look at the tensor's own fields)
  void* at(Py_ssize_t i, caffe2::TypeMeta t, int64_t n, c10::Device dev) const {
    const Tensor& x = get(i);
    const c10::TensorImpl* p = x.unsafeGetTensorImpl();
    if (p->dtype() != t) fail(PyExc_TypeError, "%s: the tensors' dtype differs or is not supported", what);
    if (p->numel() != n) fail(PyExc_ValueError, "%s: a tensor has %ld elements, not %ld", what, x.numel(), n);
    if (p->device() != dev) fail(PyExc_ValueError, "%s must be on the first parameter's device", what);
    if (!p->is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", what);
    return x.data_ptr();
  }
  PyObject* fast = nullptr;
  Py_ssize_t count = 0;
  const char* what;
};

void written(const Tensor& t) {
  c10::TensorImpl* p = t.unsafeGetTensorImpl();
  if (!p->is_inference()) p->bump_version();
}

// params, grads, exp_avg, exp_avg_sq, step, lr, beta1, beta2, eps, weight_decay, masters,
// exp_avg_scale, exp_avg_sq_scale, grad_scale.  `only_check`: everything but the step,
// whose refusals are then known before any of several calls has updated anything.
PyObject* adamw(PyObject* const* a, bool only_check) {
  const List params(a[0], "params", -1, false);
  const Py_ssize_t n = params.count;
  const List grads(a[1], "grads", n, false), m(a[2], "exp_avg", n, false), v(a[3], "exp_avg_sq", n, false),
      masters(a[10], "masters", n, true), ms(a[11], "exp_avg_scale", n, true), vs(a[12], "exp_avg_sq_scale", n, true);
  if (ms.given() != vs.given()) fail(PyExc_ValueError, "%s go together", "exp_avg_scale and exp_avg_sq_scale");
  const double lr = THPVariable_Check(a[5]) ? 0.0 : number(a[5]);
  const long long step = THPVariable_Check(a[4]) ? 0 : wide_integer(a[4]);
  if (n == 0) return none();
  const Tensor& first = params.get(0);
  on_gpu(first);
  const c10::Device dev = first.device();
  const OnDevice on(first, {{a[4], "step"}, {a[5], "lr"}, {a[13], "grad_scale"}});
  const float* lr_dev = THPVariable_Check(a[5]) ? scalar_f32(tensor(a[5], "lr"), "lr") : nullptr;
  const int32_t* step_dev = nullptr;
  if (THPVariable_Check(a[4])) {
    const Tensor& s = tensor(a[4], "step");
    if (s.scalar_type() != at::kInt || s.numel() != 1) fail(PyExc_ValueError, "%s must be int32 [1]", "step");
    on_gpu(s);
    step_dev = static_cast<const int32_t*>(s.data_ptr());
  }
  const float* gs = a[13] == Py_None ? nullptr : scalar_f32(tensor(a[13], "grad_scale"), "grad_scale");
  const ScalarType pt = first.scalar_type(),
                   gt = grads.get(0).scalar_type();
  const mgg_dtype pc = code(pt), gc = code(gt);
  const caffe2::TypeMeta state = c10::scalarTypeToTypeMeta(ms.given() ? at::kFloat8_e4m3fn : at::kFloat),
                         f32 = c10::scalarTypeToTypeMeta(at::kFloat), pm = c10::scalarTypeToTypeMeta(pt),
                         gm = c10::scalarTypeToTypeMeta(gt);
  std::vector<mgg_adamw_tensor> t(static_cast<size_t>(n));
  std::vector<std::pair<const char*, int64_t>> spans;
  spans.reserve(t.size());
  for (Py_ssize_t i = 0; i < n; ++i) {
    const int64_t size = params.get(i).numel();
    const int64_t blocks = (size + MGG_ADAMW_BLOCK - 1) / MGG_ADAMW_BLOCK;
    mgg_adamw_tensor& e = t[static_cast<size_t>(i)];
    e.n = size;
    e.param = params.at(i, pm, size, dev);
    e.grad = grads.at(i, gm, size, dev);
    e.exp_avg = m.at(i, state, size, dev);
    e.exp_avg_sq = v.at(i, state, size, dev);
    e.master = masters.given() ? static_cast<float*>(masters.at(i, f32, size, dev)) : nullptr;
    e.exp_avg_scale = ms.given() ? static_cast<float*>(ms.at(i, f32, blocks, dev)) : nullptr;
    e.exp_avg_sq_scale = ms.given() ? static_cast<float*>(vs.at(i, f32, blocks, dev)) : nullptr;
    if (size) spans.emplace_back(static_cast<const char*>(e.param), size * (pt == at::kFloat ? 4 : 2));
  }
  if (!std::is_sorted(spans.begin(), spans.end())) std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i - 1].first + spans[i - 1].second > spans[i].first)
      fail(PyExc_ValueError, "%s must not overlap (is one of them listed twice?)", "params");
  // (with no tensors the library checks the numbers alone)
  check(mgg_adamw_step(t.data(), only_check ? 0 : static_cast<int>(n), pc, gc, ms.given() ? 8 : 32, lr, lr_dev,
                       number(a[6]), number(a[7]), number(a[8]), number(a[9]), step, step_dev, gs, stream(first)),
        "mgg_adamw_step");
  if (only_check) return none();
  // written in place: a backward pass that kept the old values has to notice (15 ns
  // a tensor; masters are in no graph)
  for (Py_ssize_t i = 0; i < n; ++i) written(params.get(i));
  return none();
}
PyObject* adamw_step(PyObject* const* a) { return adamw(a, false); }
PyObject* adamw_check(PyObject* const* a) { return adamw(a, true); }

#define MGG_ENTRY(f, n)                                                               \
  {                                                                                   \
    #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)),    \
        METH_FASTCALL, nullptr                                                        \
  }
PyMethodDef methods[] = {MGG_ENTRY(layer_norm_forward, 5),
                         MGG_ENTRY(layer_norm_backward, 7),
                         MGG_ENTRY(select_experts, 8),
                         MGG_ENTRY(select_experts_backward, 8),
                         MGG_ENTRY(linear_forward, 9),
                         MGG_ENTRY(linear_backward, 10),
                         MGG_ENTRY(balance_loss_forward, 7),
                         MGG_ENTRY(balance_loss_backward, 5),
                         MGG_ENTRY(linear_cross_entropy_forward, 8),
                         MGG_ENTRY(linear_cross_entropy_backward, 12),
                         MGG_ENTRY(adamw_step, 14),
                         MGG_ENTRY(adamw_check, 14),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__host() { return PyModule_Create(&module); }
