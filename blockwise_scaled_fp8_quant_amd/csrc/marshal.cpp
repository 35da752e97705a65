// Argument marshalling of the operators of puro_ops.h for Python (module _marshal, used by ops.py): checks tensors by
// the package's rules, allocates outputs and workspaces with torch, passes pointers, sizes and the current
// stream to the C ABI, and raises what the package raises (TypeError, ValueError; PuroError for a non-zero status).
// It computes nothing.  Native because these calls are short: of a few microseconds on the GPU the interpreter took
// ten (measured, one token: norm 11.6 us a call, product 8.9).
//
// Functions take positional arguments only, None for what is not given; ops.py has the names, defaults and
// documentation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>

#include <limits>
#include <memory>
#include <string>
#include <unordered_set>
#include <vector>

#include "../../include/puro_ops.h"

namespace {

PyObject* get_device = nullptr;   // () -> the current GPU
PyObject* get_stream = nullptr;   // (GPU) -> its current stream's handle
PyObject* raise_status = nullptr; // (status, where): raises PuroError

struct Refused {   // an argument error: the Python exception to raise
  PyObject* type;
  std::string text;
};
// the Python error is set already
struct Raised {};

[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }

using Shape = std::vector<int64_t>;

std::string text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

int64_t as_int(PyObject* o, const char* what) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(what) + ": expected an integer");
  }
  return v;
}

double as_float(PyObject* o, const char* what) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(what) + ": expected a number");
  }
  return v;
}

bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

// One call: the current GPU, its stream, and the checks against it.
class Call {
 public:
  Call() {
    PyObject* d = PyObject_CallNoArgs(get_device);
    if (!d) throw Raised{};
    dev_ = PyLong_AsLong(d);
    Py_DECREF(d);
  }

  hipStream_t stream() const {
    PyObject* i = PyLong_FromLong(dev_);
    PyObject* s = i ? PyObject_CallOneArg(get_stream, i) : nullptr;
    Py_XDECREF(i);
    if (!s) throw Raised{};
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!p && PyErr_Occurred()) throw Raised{};
    return static_cast<hipStream_t>(p);
  }

  // A tensor on the current GPU, of `dtype` and, where given, `shape`.
  const at::Tensor& tensor(PyObject* o, const std::string& what, c10::optional<at::ScalarType> dtype,
                           const Shape* shape) const {
    if (!THPVariable_Check(o)) type_error(what + ": expected a torch.Tensor, got " + Py_TYPE(o)->tp_name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) value_error(what + ": must be a GPU tensor, not on " + t.device().str());
    if (t.get_device() != dev_)
      value_error(what + ": must live on the current GPU (cuda:" + std::to_string(dev_) + "), not on " + t.device().str());
    if (dtype && t.scalar_type() != *dtype)
      type_error(what + ": dtype " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(*dtype));
    if (t.layout() != at::kStrided) type_error(what + ": expected a dense tensor");
    if (shape && t.sizes() != at::IntArrayRef(*shape))
      value_error(what + ": shape " + text(t.sizes()) + ", expected " + text(*shape));
    return t;
  }

  // ... that is contiguous (a dimension of one element may carry any stride).
  const at::Tensor& whole(PyObject* o, const std::string& what, c10::optional<at::ScalarType> dtype,
                          const Shape* shape) const {
    const at::Tensor& t = tensor(o, what, dtype, shape);
    if (!t.is_contiguous()) value_error(what + ": must be contiguous");
    return t;
  }

  // ... or a matrix with unit element stride in its rows; `ld` gets the row stride.
  const at::Tensor& rows(PyObject* o, const char* what, c10::optional<at::ScalarType> dtype, const Shape* shape,
                         int64_t& ld) const {
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 2) value_error(std::string(what) + ": expected a 2-D tensor");
    const at::Tensor& t = tensor(o, what, dtype, shape);
    const int64_t T = t.size(0), C = t.size(1);
    if (t.stride(1) != 1 && C > 1 && T > 0)
      value_error(std::string(what) + ": rows must have unit element stride (got strides " + text(t.strides()) + ")");
    if (T <= 1 || C == 0) {
      ld = C > 0 ? C : 1;   // a single row's stride says nothing
    } else {
      ld = t.stride(0);
      if (ld < C)
        value_error(std::string(what) + ": row stride " + std::to_string(ld) + " is smaller than a row of " + std::to_string(C));
    }
    return t;
  }

  // Whether an object is a tensor that `tensor` and `whole` would take (of `dtype`, where it is named), at less cost.
  bool plain(PyObject* o, at::ScalarType dtype) const {
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.is_cuda() && t.get_device() == dev_ && t.layout() == at::kStrided && t.scalar_type() == dtype;
  }

  at::Tensor make(const Shape& shape, at::ScalarType dtype) const {
    // torch.empty without its dispatch, which costs as much as the allocation
    return at::Tensor(at::detail::empty_cuda(shape, dtype, at::Device(at::kCUDA, (c10::DeviceIndex)dev_), c10::nullopt));
  }

  at::Tensor out_rows(PyObject* o, const char* what, at::ScalarType dtype, const Shape& shape, int64_t& ld) const {
    if (o != Py_None) return rows(o, what, dtype, &shape, ld);
    ld = shape[1] > 0 ? shape[1] : 1;
    return make(shape, dtype);
  }

  at::Tensor out_whole(PyObject* o, const char* what, at::ScalarType dtype, const Shape& shape) const {
    return o != Py_None ? whole(o, what, dtype, &shape) : make(shape, dtype);
  }

  at::Tensor workspace(PyObject* o, size_t need, size_t& bytes) const {
    at::Tensor t;
    if (o != Py_None)
      t = whole(o, "workspace", c10::nullopt, nullptr);
    else if (need)
      t = make({(int64_t)need}, at::kByte);
    bytes = t.defined() ? t.nbytes() : 0;
    return t;
  }

 private:
  int64_t dev_;
};

// The scaled types of puro_fp8.h.
int dtype_code(PyObject* o, const std::string& what, at::ScalarType& st) {
  if (THPVariable_Check(o)) {
    st = THPVariable_Unpack(o).scalar_type();
    if (st == at::kBFloat16) return PURO_OUT_BF16;
    if (st == at::kFloat) return PURO_OUT_FP32;
  }
  type_error(what + ": expected a bf16 or fp32 torch.Tensor");
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
float* fptr(const at::Tensor& t) { return static_cast<float*>(ptr(t)); }

// Runs a C entry point without the interpreter's lock.
template <typename F>
void enqueue(const char* where, F f) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  if (status != PURO_OK) {
    PyObject* r = PyObject_CallFunction(raise_status, "is", status, where);
    Py_XDECREF(r);
    throw Raised{};
  }
}

// A tensor of the caller's (o, None if the call made its own) has been written: raises its version, by which autograd
// notices that one it has saved is not what it was.  (Those made in inference mode have none.)
void written(PyObject* o) {
  if (o == Py_None) return;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

template <typename... T>
PyObject* wrap_all(const T&... t) {
  PyObject* tuple = PyTuple_New(sizeof...(t));
  if (!tuple) throw Raised{};
  Py_ssize_t i = 0;
  bool ok = true;
  auto put = [&](const at::Tensor& x) {
    PyObject* o = ok ? wrap(x) : nullptr;
    ok = ok && o;
    PyTuple_SET_ITEM(tuple, i++, o);
  };
  (put(t), ...);
  if (!ok) {
    Py_DECREF(tuple);
    throw Raised{};
  }
  return tuple;
}

template <int N, PyObject* (*F)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    return F(args);
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.text.c_str());
    return nullptr;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

int norm_kind(PyObject* o) {
  const int64_t kind = as_int(o, "kind");
  if (kind != PURO_NORM_LAYER && kind != PURO_NORM_RMS)
    value_error("kind " + std::to_string(kind) + ": expected LAYER_NORM or RMS_NORM");
  return (int)kind;
}

// x, weight, bias, eps, kind: what every forward form takes.
struct NormIn {
  int kind, xd, wd = 0;
  float eps;
  int64_t T, C, ldx;
  at::ScalarType xt;
  at::Tensor x, weight, bias;
  NormIn(const Call& c, PyObject* const* a) {
    kind = norm_kind(a[4]);
    eps = (float)as_float(a[3], "eps");
    xd = dtype_code(a[0], "x", xt);
    x = c.rows(a[0], "x", xt, nullptr, ldx);
    T = x.size(0);
    C = x.size(1);
    at::ScalarType wt;
    const Shape v{C};
    wd = dtype_code(a[1], "weight", wt);
    weight = c.whole(a[1], "weight", wt, &v);
    if (a[2] != Py_None) bias = c.whole(a[2], "bias", wt, &v);
  }
};

struct Stats {
  at::Tensor mean, rstd;
  Stats(const Call& c, PyObject* m, PyObject* r, const NormIn& n, bool make) {
    const Shape v{n.T};
    const int kind = n.kind;
    if (m != Py_None) {
      if (kind == PURO_NORM_RMS) value_error("mean: an RMS norm has none");
      mean = c.whole(m, "mean", at::kFloat, &v);
    } else if (make && kind == PURO_NORM_LAYER) {
      mean = c.make(v, at::kFloat);
    }
    if (r != Py_None)
      rstd = c.whole(r, "rstd", at::kFloat, &v);
    else if (make)
      rstd = c.make(v, at::kFloat);
    columns = n.C > 0;
  }

  // Rows of no columns: the library writes nothing, and their statistics are 0 / 0.
  void of_nothing() const {
    if (columns) return;
    for (const at::Tensor& t : {mean, rstd})
      if (t.defined()) t.fill_(std::numeric_limits<float>::quiet_NaN());
  }

 private:
  bool columns;
};

// x, weight, bias, eps, kind, y, mean, rstd, stats
PyObject* layer_norm(PyObject* const* a) {
  Call c;
  NormIn n(c, a);
  int64_t ldy;
  const at::Tensor y = c.out_rows(a[5], "y", n.xt, {n.T, n.C}, ldy);
  const Stats s(c, a[6], a[7], n, as_bool(a[8]));
  const hipStream_t st = c.stream();
  enqueue("puro_layer_norm", [&] {
    return puro_layer_norm(n.kind, n.xd, ptr(n.x), n.T, n.C, n.ldx, n.wd, ptr(n.weight), ptr(n.bias), n.eps, ptr(y), ldy,
                           fptr(s.mean), fptr(s.rstd), st);
  });
  s.of_nothing();
  for (int i : {5, 6, 7}) written(a[i]);
  return wrap_all(y, s.mean, s.rstd);
}

// x, weight, bias, eps, kind, q, s, mean, rstd
PyObject* layer_norm_quant(PyObject* const* a) {
  Call c;
  NormIn n(c, a);
  int64_t ldq;
  const at::Tensor q = c.out_rows(a[5], "q", at::kByte, {n.T, n.C}, ldq);
  const at::Tensor s = c.out_whole(a[6], "s", at::kFloat, {n.C / 128, n.T});
  const Stats k(c, a[7], a[8], n, false);
  const hipStream_t st = c.stream();
  enqueue("puro_layer_norm_quant", [&] {
    return puro_layer_norm_quant(n.kind, n.xd, ptr(n.x), n.T, n.C, n.ldx, n.wd, ptr(n.weight), ptr(n.bias), n.eps,
                                 static_cast<uint8_t*>(ptr(q)), ldq, fptr(s), fptr(k.mean), fptr(k.rstd), st);
  });
  k.of_nothing();
  for (int i : {5, 6, 7, 8}) written(a[i]);
  return wrap_all(q, s);
}

// x, weight, bias, eps, kind, q, s, qT, sT, mean, rstd
PyObject* layer_norm_quant_dual(PyObject* const* a) {
  Call c;
  NormIn n(c, a);
  int64_t ldq, ldqT;
  const at::Tensor q = c.out_rows(a[5], "q", at::kByte, {n.T, n.C}, ldq);
  const at::Tensor s = c.out_whole(a[6], "s", at::kFloat, {n.C / 128, n.T});
  const at::Tensor qT = c.out_rows(a[7], "qT", at::kByte, {n.C, n.T}, ldqT);
  const at::Tensor sT = c.out_whole(a[8], "sT", at::kFloat, {n.T / 128, n.C});
  const Stats k(c, a[9], a[10], n, true);
  const hipStream_t st = c.stream();
  enqueue("puro_layer_norm_quant_dual", [&] {
    return puro_layer_norm_quant_dual(n.kind, n.xd, ptr(n.x), n.T, n.C, n.ldx, n.wd, ptr(n.weight), ptr(n.bias), n.eps,
                                      static_cast<uint8_t*>(ptr(q)), ldq, fptr(s), static_cast<uint8_t*>(ptr(qT)), ldqT,
                                      fptr(sT), fptr(k.mean), fptr(k.rstd), st);
  });
  k.of_nothing();
  for (int i : {5, 6, 7, 8, 9, 10}) written(a[i]);
  return wrap_all(q, s, qT, sT, k.mean, k.rstd);
}

// dy, x, weight, mean, rstd, kind, dx, dweight, dbias, with_bias, accumulate, workspace
PyObject* layer_norm_backward(PyObject* const* a) {
  Call c;
  const int kind = norm_kind(a[5]);
  at::ScalarType xt, wt;
  int64_t ldx, lddy, lddx;
  const int xd = dtype_code(a[1], "x", xt);
  const at::Tensor x = c.rows(a[1], "x", xt, nullptr, ldx);
  const int64_t T = x.size(0), C = x.size(1);
  const Shape shape{T, C}, vec{C}, stat{T};
  const at::Tensor dy = c.rows(a[0], "dy", xt, &shape, lddy);
  const int wd = dtype_code(a[2], "weight", wt);
  const at::Tensor weight = c.whole(a[2], "weight", wt, &vec);
  at::Tensor mean;
  if (kind == PURO_NORM_LAYER)
    mean = c.whole(a[3], "mean", at::kFloat, &stat);
  else if (a[3] != Py_None)
    value_error("mean: an RMS norm has none");
  const at::Tensor rstd = c.whole(a[4], "rstd", at::kFloat, &stat);
  const bool with_bias = as_bool(a[9]) || a[8] != Py_None, accumulate = as_bool(a[10]);
  if (accumulate && (a[7] == Py_None || (with_bias && a[8] == Py_None)))
    value_error("accumulate: needs the gradients it adds to");
  const at::Tensor dx = c.out_rows(a[6], "dx", xt, shape, lddx);
  const at::Tensor dw = c.out_whole(a[7], "dweight", at::kFloat, vec);
  at::Tensor db;
  if (with_bias) db = c.out_whole(a[8], "dbias", at::kFloat, vec);
  size_t bytes;
  const at::Tensor ws = c.workspace(a[11], puro_layer_norm_backward_workspace_size(T, C), bytes);
  const hipStream_t st = c.stream();
  enqueue("puro_layer_norm_backward", [&] {
    return puro_layer_norm_backward(kind, xd, ptr(dy), lddy, ptr(x), ldx, T, C, wd, ptr(weight), fptr(mean), fptr(rstd),
                                    ptr(dx), lddx, fptr(dw), fptr(db), accumulate ? 1 : 0, ptr(ws), bytes, st);
  });
  for (int i : {6, 7, 8}) written(a[i]);
  return wrap_all(dx, dw, db);
}

// The jobs of a list of gradients and, where given, of their outputs.  (The lists are the caller's and hold the tensors.)
// A gradient fills its range of memory in any order of its dimensions (contiguous, or the transpose of that), which
// is all that its norm and scaling need; its output then has the same strides.
std::vector<puro_grad_job> grad_jobs(const Call& c, PyObject* grads, PyObject* outs) {
  if (!PyList_Check(grads) && !PyTuple_Check(grads)) type_error("grads: expected a list of tensors");
  if (outs != Py_None && !PyList_Check(outs) && !PyTuple_Check(outs)) type_error("outs: expected a list of tensors");
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(grads);
  if (outs != Py_None && PySequence_Fast_GET_SIZE(outs) != n)
    value_error("outs: " + std::to_string(PySequence_Fast_GET_SIZE(outs)) + " tensors for " + std::to_string(n) + " gradients");
  std::vector<puro_grad_job> jobs((size_t)n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PySequence_Fast_GET_ITEM(grads, i);
    const auto name = [i](const char* list) { return std::string(list) + "[" + std::to_string(i) + "]"; };
    at::ScalarType st;
    const std::string what = name("grads");
    const int code = dtype_code(o, what, st);
    const at::Tensor& g = c.tensor(o, what, st, nullptr);
    const bool whole = g.is_contiguous();
    if (!whole && !g.is_non_overlapping_and_dense()) value_error(what + ": must be contiguous");
    puro_grad_job& j = jobs[(size_t)i];
    j.src = g.data_ptr();
    j.dst = g.data_ptr();
    j.n = g.numel();
    j.dtype = code;
    if (outs != Py_None) {
      const Shape shape = g.sizes().vec();
      const at::Tensor& d = c.tensor(PySequence_Fast_GET_ITEM(outs, i), name("outs"), st, &shape);
      if (whole ? !d.is_contiguous() : d.strides() != g.strides()) value_error(name("outs") + ": must have the gradient's layout");
      j.dst = d.data_ptr();
    }
  }
  return jobs;
}

// The gradients, or their outputs, have been scaled.
void scaled(PyObject* grads, PyObject* outs) {
  PyObject* list = outs == Py_None ? grads : outs;
  for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(list); ++i) written(PySequence_Fast_GET_ITEM(list, i));
}

at::Tensor norm_value(const Call& c, PyObject* o) {
  if (o == Py_None) return c.make({}, at::kFloat);
  const at::Tensor t = c.whole(o, "norm", at::kFloat, nullptr);
  if (t.numel() != 1) value_error("norm: expected one value");
  return t;
}

// grads, max_norm (None: the norm alone), outs, norm, workspace
PyObject* clip_grad_norm(PyObject* const* a) {
  Call c;
  const auto jobs = grad_jobs(c, a[0], a[2]);
  const int n = (int)jobs.size();
  const bool clip = a[1] != Py_None;
  const float max_norm = clip ? (float)as_float(a[1], "max_norm") : 0.f;
  const at::Tensor norm = norm_value(c, a[3]);
  size_t bytes;
  const at::Tensor ws = c.workspace(a[4], puro_grad_norm_workspace_size(jobs.data(), n), bytes);
  const hipStream_t st = c.stream();
  if (clip)
    enqueue("puro_clip_grad_norm", [&] { return puro_clip_grad_norm(jobs.data(), n, max_norm, fptr(norm), ptr(ws), bytes, st); });
  else
    enqueue("puro_grad_norm", [&] { return puro_grad_norm(jobs.data(), n, fptr(norm), ptr(ws), bytes, st); });
  if (clip) scaled(a[0], a[2]);
  written(a[3]);
  return wrap(norm);
}

// grads, max_norm, norm, outs
PyObject* scale_by_norm(PyObject* const* a) {
  if (a[2] == Py_None) value_error("norm: the scaling needs the norm's tensor");
  Call c;
  const auto jobs = grad_jobs(c, a[0], a[3]);
  const float max_norm = (float)as_float(a[1], "max_norm");
  const at::Tensor norm = norm_value(c, a[2]);
  const hipStream_t st = c.stream();
  enqueue("puro_scale_by_norm", [&] { return puro_scale_by_norm(jobs.data(), (int)jobs.size(), max_norm, fptr(norm), st); });
  scaled(a[0], a[3]);
  Py_RETURN_NONE;
}

// A, sA, B, sB, C, out_dtype, workspace
PyObject* gemm_rows(PyObject* const* a) {
  Call c;
  int64_t lda, ldb, ldc;
  const at::Tensor A = c.rows(a[0], "A", at::kByte, nullptr, lda), B = c.rows(a[2], "B", at::kByte, nullptr, ldb);
  const int64_t M = A.size(0), K = A.size(1), N = B.size(0);
  if (B.size(1) != K)
    value_error("A " + text(A.sizes()) + " and B " + text(B.sizes()) + " differ in the contraction length");
  const Shape ssa{K / 128, M}, ssb{N / 128, K / 128};
  const at::Tensor sA = c.whole(a[1], "sA", at::kFloat, &ssa), sB = c.whole(a[3], "sB", at::kFloat, &ssb);
  const int64_t od = as_int(a[5], "out_dtype");
  if (od != PURO_OUT_BF16 && od != PURO_OUT_FP32)
    value_error("out_dtype " + std::to_string(od) + ": expected OUT_BF16 or OUT_FP32");
  const bool bf16 = od == PURO_OUT_BF16;
  const at::Tensor C = c.out_rows(a[4], "C", bf16 ? at::kBFloat16 : at::kFloat, {M, N}, ldc);
  size_t bytes;
  const at::Tensor ws = c.workspace(a[6], bf16 ? puro_gemm_rows_workspace_size(M, N, K) : 0, bytes);
  const hipStream_t st = c.stream();
  enqueue("puro_gemm_rows", [&] {
    return puro_gemm_rows(M, N, K, static_cast<const uint8_t*>(ptr(A)), lda, fptr(sA), static_cast<const uint8_t*>(ptr(B)), ldb,
                          fptr(sB), ptr(C), ldc, (int)od, ptr(ws), bytes, st);
  });
  written(a[4]);
  return wrap(C);
}

// ---- residual sum and norm ---------------------------------------------------------------------------
constexpr int kResidualIn = 14;

// h, x, weight, bias, eps, kind, gate, post_weight, scale, h_out, mean, rstd, post_mean, post_rstd: what every forward form
// takes.  make: statistics that are not given are allocated.
struct ResidualIn {
  puro_residual r = {};
  at::ScalarType xt;
  at::Tensor h, x, weight, bias, gate, post, h_out, mean, rstd, post_mean, post_rstd;
  ResidualIn(const Call& c, PyObject* const* a, bool make) {
    r.kind = norm_kind(a[5]);
    r.eps = (float)as_float(a[4], "eps");
    r.scale = (float)as_float(a[8], "scale");
    r.x_dtype = dtype_code(a[0], "h", xt);
    h = c.rows(a[0], "h", xt, nullptr, r.ldh);
    const Shape shape{h.size(0), h.size(1)}, vec{shape[1]}, stat{shape[0]};
    r.T = shape[0];
    r.C = shape[1];
    x = c.rows(a[1], "x", xt, &shape, r.ldx);
    at::ScalarType wt;
    r.w_dtype = dtype_code(a[2], "weight", wt);
    weight = c.whole(a[2], "weight", wt, &vec);
    if (a[3] != Py_None) bias = c.whole(a[3], "bias", wt, &vec);
    if (a[6] != Py_None) gate = c.whole(a[6], "gate", wt, &vec);
    if (a[7] != Py_None) post = c.whole(a[7], "post_weight", wt, &vec);
    h_out = c.out_rows(a[9], "h_out", xt, shape, r.ldh_out);
    const bool layer = r.kind == PURO_NORM_LAYER;
    const auto statistic = [&](PyObject* o, const char* what, bool there, const char* why) {
      if (o != Py_None && !there) value_error(std::string(what) + why);
      if (o != Py_None) return at::Tensor(c.whole(o, what, at::kFloat, &stat));
      return make && there ? c.make(stat, at::kFloat) : at::Tensor();
    };
    mean = statistic(a[10], "mean", layer, ": an RMS norm has none");
    rstd = statistic(a[11], "rstd", true, "");
    post_mean = statistic(a[12], "post_mean", layer && post.defined(), ": an RMS norm, or no norm of x, has none");
    post_rstd = statistic(a[13], "post_rstd", post.defined(), ": without post_weight there is no norm of x");
    r.h = ptr(h);
    r.x = ptr(x);
    r.weight = ptr(weight);
    r.bias = ptr(bias);
    r.gate = ptr(gate);
    r.post_weight = ptr(post);
    r.h_out = ptr(h_out);
    r.mean = fptr(mean);
    r.rstd = fptr(rstd);
    r.post_mean = fptr(post_mean);
    r.post_rstd = fptr(post_rstd);
  }

  // After the call: rows of no columns have statistics of 0 / 0, and the caller's tensors are new.
  void done(PyObject* const* a) const {
    if (r.C == 0)
      for (const at::Tensor& t : {mean, rstd, post_mean, post_rstd})
        if (t.defined()) t.fill_(std::numeric_limits<float>::quiet_NaN());
    for (int i = 9; i < kResidualIn; ++i) written(a[i]);
  }
};

// the above, y, stats
PyObject* residual_norm(PyObject* const* a) {
  Call c;
  const ResidualIn n(c, a, as_bool(a[kResidualIn + 1]));
  int64_t ldy;
  const at::Tensor y = c.out_rows(a[kResidualIn], "y", n.xt, {n.r.T, n.r.C}, ldy);
  const hipStream_t st = c.stream();
  enqueue("puro_residual_norm", [&] { return puro_residual_norm(&n.r, ptr(y), ldy, st); });
  n.done(a);
  written(a[kResidualIn]);
  return wrap_all(y, n.h_out, n.mean, n.rstd, n.post_mean, n.post_rstd);
}

// the above, q, s
PyObject* residual_norm_quant(PyObject* const* a) {
  Call c;
  const ResidualIn n(c, a, false);
  int64_t ldq;
  const at::Tensor q = c.out_rows(a[kResidualIn], "q", at::kByte, {n.r.T, n.r.C}, ldq);
  const at::Tensor s = c.out_whole(a[kResidualIn + 1], "s", at::kFloat, {n.r.C / 128, n.r.T});
  const hipStream_t st = c.stream();
  enqueue("puro_residual_norm_quant", [&] { return puro_residual_norm_quant(&n.r, static_cast<uint8_t*>(ptr(q)), ldq, fptr(s), st); });
  n.done(a);
  for (int i : {0, 1}) written(a[kResidualIn + i]);
  return wrap_all(q, s, n.h_out);
}

// the above, q, s, qT, sT
PyObject* residual_norm_quant_dual(PyObject* const* a) {
  Call c;
  const ResidualIn n(c, a, true);
  PyObject* const* o = a + kResidualIn;
  int64_t ldq, ldqT;
  const at::Tensor q = c.out_rows(o[0], "q", at::kByte, {n.r.T, n.r.C}, ldq);
  const at::Tensor s = c.out_whole(o[1], "s", at::kFloat, {n.r.C / 128, n.r.T});
  const at::Tensor qT = c.out_rows(o[2], "qT", at::kByte, {n.r.C, n.r.T}, ldqT);
  const at::Tensor sT = c.out_whole(o[3], "sT", at::kFloat, {n.r.T / 128, n.r.C});
  const hipStream_t st = c.stream();
  enqueue("puro_residual_norm_quant_dual", [&] {
    return puro_residual_norm_quant_dual(&n.r, static_cast<uint8_t*>(ptr(q)), ldq, fptr(s), static_cast<uint8_t*>(ptr(qT)), ldqT,
                                         fptr(sT), st);
  });
  n.done(a);
  for (int i : {0, 1, 2, 3}) written(o[i]);
  return wrap_all(q, s, qT, sT, n.h_out, n.mean, n.rstd, n.post_mean, n.post_rstd);
}

// dy, h_out, weight, mean, rstd, x, gate, post_weight, post_mean, post_rstd, dh_out, scale, kind, dh, dx, dweight, dbias,
// dgate, dpost_weight, with_bias, accumulate, workspace
PyObject* residual_norm_backward(PyObject* const* a) {
  Call c;
  puro_residual_grad r = {};
  r.kind = norm_kind(a[12]);
  const bool layer = r.kind == PURO_NORM_LAYER;
  at::ScalarType xt, wt;
  r.x_dtype = dtype_code(a[1], "h_out", xt);
  const at::Tensor h = c.rows(a[1], "h_out", xt, nullptr, r.ldh_out);
  const Shape shape{h.size(0), h.size(1)}, vec{shape[1]}, stat{shape[0]};
  r.T = shape[0];
  r.C = shape[1];
  r.scale = (float)as_float(a[11], "scale");
  const at::Tensor dy = c.rows(a[0], "dy", xt, &shape, r.lddy);
  r.w_dtype = dtype_code(a[2], "weight", wt);
  const at::Tensor weight = c.whole(a[2], "weight", wt, &vec);
  at::Tensor gate, post, x, mean, post_mean, post_rstd, dho;
  if (a[6] != Py_None) gate = c.whole(a[6], "gate", wt, &vec);
  if (a[7] != Py_None) post = c.whole(a[7], "post_weight", wt, &vec);
  const bool gated = gate.defined() || post.defined();
  if (layer)
    mean = c.whole(a[3], "mean", at::kFloat, &stat);
  else if (a[3] != Py_None || a[8] != Py_None)
    value_error("mean: an RMS norm has none");
  const at::Tensor rstd = c.whole(a[4], "rstd", at::kFloat, &stat);
  if (post.defined()) {
    if (layer) post_mean = c.whole(a[8], "post_mean", at::kFloat, &stat);
    post_rstd = c.whole(a[9], "post_rstd", at::kFloat, &stat);
  } else if (a[8] != Py_None || a[9] != Py_None) {
    value_error("post_rstd: without post_weight there is no norm of x");
  }
  if (a[5] != Py_None) x = c.rows(a[5], "x", xt, &shape, r.ldx);
  if (gated && !x.defined()) value_error("x: a gate or a norm of it needs the block's output");
  if (a[10] != Py_None) dho = c.rows(a[10], "dh_out", xt, &shape, r.lddh_out);
  const bool with_bias = as_bool(a[19]) || a[16] != Py_None, accumulate = as_bool(a[20]);
  if (a[17] != Py_None && !gate.defined()) value_error("dgate: there is no gate");
  if (a[18] != Py_None && !post.defined()) value_error("dpost_weight: there is no post_weight");
  if (accumulate && (a[15] == Py_None || (with_bias && a[16] == Py_None) || (gate.defined() && a[17] == Py_None) ||
                     (post.defined() && a[18] == Py_None)))
    value_error("accumulate: needs the gradients it adds to");
  const at::Tensor dh = c.out_rows(a[13], "dh", xt, shape, r.lddh);
  at::Tensor dx, db, dg, dp;
  // (without gate, norm and scale it is dh's equal: dh stands for it)
  const bool own_dx = gated || r.scale != 1.f || a[14] != Py_None;
  if (own_dx) dx = c.out_rows(a[14], "dx", xt, shape, r.lddx);
  const at::Tensor dw = c.out_whole(a[15], "dweight", at::kFloat, vec);
  if (with_bias) db = c.out_whole(a[16], "dbias", at::kFloat, vec);
  if (gate.defined()) dg = c.out_whole(a[17], "dgate", at::kFloat, vec);
  if (post.defined()) dp = c.out_whole(a[18], "dpost_weight", at::kFloat, vec);
  size_t bytes;
  const at::Tensor ws = c.workspace(a[21], puro_residual_norm_backward_workspace_size(r.T, r.C, gated ? 1 : 0), bytes);
  r.dy = ptr(dy);
  r.h_out = ptr(h);
  r.dh_out = ptr(dho);
  r.x = gated ? ptr(x) : nullptr;
  r.weight = ptr(weight);
  r.gate = ptr(gate);
  r.post_weight = ptr(post);
  r.mean = fptr(mean);
  r.rstd = fptr(rstd);
  r.post_mean = fptr(post_mean);
  r.post_rstd = fptr(post_rstd);
  r.dh = ptr(dh);
  r.dx = ptr(dx);
  r.dweight = fptr(dw);
  r.dbias = fptr(db);
  r.dgate = fptr(dg);
  r.dpost_weight = fptr(dp);
  r.accumulate = accumulate ? 1 : 0;
  const hipStream_t st = c.stream();
  enqueue("puro_residual_norm_backward", [&] { return puro_residual_norm_backward(&r, ptr(ws), bytes, st); });
  for (int i = 13; i <= 18; ++i) written(a[i]);
  return wrap_all(dh, own_dx ? dx : dh, dw, db, dg, dp);
}

// ---- rotary positions --------------------------------------------------------------------------------

// [T, H, D] with unit stride in its heads; the strides of tokens and heads (natural ones where they say nothing).
const at::Tensor& heads(const Call& c, PyObject* o, const char* what, at::ScalarType dtype, const Shape* shape, int64_t& ld_t,
                        int64_t& ld_h) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 3) value_error(std::string(what) + ": expected a 3-D tensor");
  const at::Tensor& t = c.tensor(o, what, dtype, shape);
  if (t.stride(2) != 1 && t.size(2) > 1 && t.numel() > 0)
    value_error(std::string(what) + ": heads must have unit element stride (got strides " + text(t.strides()) + ")");
  ld_h = t.size(1) > 1 ? t.stride(1) : t.size(2);
  ld_t = t.size(0) > 1 ? t.stride(0) : t.size(1) * ld_h;
  return t;
}

// x, freqs, positions, start, layout, scale, inverse, y
PyObject* rotary(PyObject* const* a) {
  Call c;
  at::ScalarType xt;
  int64_t ld_t, ld_h, ldy_t, ldy_h;
  const int xd = dtype_code(a[0], "x", xt);
  const at::Tensor x = heads(c, a[0], "x", xt, nullptr, ld_t, ld_h);
  const Shape shape = x.sizes().vec(), tokens{shape[0]};
  const at::Tensor freqs = c.whole(a[1], "freqs", at::kDouble, nullptr);
  if (freqs.dim() != 1 || 2 * freqs.numel() > shape[2])
    value_error("freqs: expected one value for each pair of at most " + std::to_string(shape[2]) + " columns, got shape " +
                text(freqs.sizes()));
  at::Tensor positions;
  if (a[2] != Py_None) positions = c.whole(a[2], "positions", at::kLong, &tokens);
  const int64_t start = as_int(a[3], "start"), layout = as_int(a[4], "layout");
  if (layout != PURO_ROTARY_HALF && layout != PURO_ROTARY_INTERLEAVED)
    value_error("layout " + std::to_string(layout) + ": expected ROTARY_HALF or ROTARY_INTERLEAVED");
  const float scale = (float)as_float(a[5], "scale");
  const bool inverse = as_bool(a[6]);
  at::Tensor y;
  if (a[7] != Py_None) {
    y = heads(c, a[7], "y", xt, &shape, ldy_t, ldy_h);
  } else {
    y = c.make(shape, xt);
    ldy_h = shape[2];
    ldy_t = shape[1] * shape[2];
  }
  const hipStream_t st = c.stream();
  enqueue("puro_rotary", [&] {
    return puro_rotary(xd, (int)layout, inverse ? 1 : 0, ptr(x), ld_t, ld_h, shape[0], shape[1], shape[2],
                       static_cast<const int64_t*>(ptr(positions)), start, static_cast<const double*>(ptr(freqs)), freqs.numel(),
                       scale, ptr(y), ldy_t, ldy_h, st);
  });
  written(a[7]);
  return wrap(y);
}

// ---- AdamW -------------------------------------------------------------------------------------------

// A list of `n` tensors (None: there is none).
bool list_of(PyObject* o, const char* what, Py_ssize_t n) {
  if (o == Py_None) return false;
  if (!PyList_Check(o) && !PyTuple_Check(o)) type_error(std::string(what) + ": expected a list of tensors");
  if (n >= 0 && PySequence_Fast_GET_SIZE(o) != n)
    value_error(std::string(what) + ": " + std::to_string(PySequence_Fast_GET_SIZE(o)) + " tensors for " + std::to_string(n) +
                " parameters");
  return true;
}

// A number, or a tensor of one value on the GPU (then `dev` points to it).
template <typename T>
const T* scalar_tensor(const Call& c, PyObject* o, const char* what, at::ScalarType dtype) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = c.whole(o, what, dtype, nullptr);
  if (t.numel() != 1) value_error(std::string(what) + ": expected one value");
  return static_cast<const T*>(t.data_ptr());
}

// params, grads, exp_avg, exp_avg_sq, step, lr, beta1, beta2, eps, weight_decay, masters, avg_scales, sq_scales, norm,
// max_norm, seed
PyObject* adamw(PyObject* const* a) {
  Call c;
  if (!list_of(a[0], "params", -1)) type_error("params: expected a list of tensors");
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(a[0]);
  const char* names[] = {"params", "grads", "exp_avg", "exp_avg_sq"};
  for (int i = 1; i < 4; ++i)
    if (!list_of(a[i], names[i], n)) type_error(std::string(names[i]) + ": expected a list of tensors");
  const bool masters = list_of(a[10], "masters", n);
  const bool eight = list_of(a[11], "avg_scales", n);
  if (list_of(a[12], "sq_scales", n) != eight) value_error("avg_scales and sq_scales: both, or neither");
  std::vector<puro_adamw_job> jobs((size_t)n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const auto item = [&](int list) { return PySequence_Fast_GET_ITEM(a[list], i); };
    const auto name = [i](const char* list) { return std::string(list) + "[" + std::to_string(i) + "]"; };
    // (names are made for errors alone: a list has hundreds of tensors)
    const auto type_of = [&](int list, const char* what, at::ScalarType& st) {
      if (THPVariable_Check(item(list))) {
        st = THPVariable_Unpack(item(list)).scalar_type();
        if (st == at::kBFloat16) return (int)PURO_OUT_BF16;
        if (st == at::kFloat) return (int)PURO_OUT_FP32;
      }
      return dtype_code(item(list), name(what), st);
    };
    const auto take = [&](int list, const char* what, at::ScalarType dtype) -> const at::Tensor& {
      return c.plain(item(list), dtype) ? THPVariable_Unpack(item(list)) : c.tensor(item(list), name(what), dtype, nullptr);
    };
    puro_adamw_job& j = jobs[(size_t)i];
    at::ScalarType pt, gt;
    j.param_dtype = type_of(0, "params", pt);
    const at::Tensor& p = take(0, "params", pt);
    const bool whole = p.is_contiguous();
    if (!whole && !p.is_non_overlapping_and_dense()) value_error(name("params") + ": must be contiguous");
    // one that goes with it, element by element in memory
    const auto same = [&](int list, const char* what, at::ScalarType dtype) {
      const at::Tensor& t = take(list, what, dtype);
      if (t.sizes() != p.sizes()) value_error(name(what) + ": shape " + text(t.sizes()) + ", expected " + text(p.sizes()));
      if (whole ? !t.is_contiguous() : t.strides() != p.strides()) value_error(name(what) + ": must have the parameter's layout");
      return t.data_ptr();
    };
    j.param = p.data_ptr();
    j.n = p.numel();
    j.grad_dtype = type_of(1, "grads", gt);
    j.grad = same(1, "grads", gt);
    bool codes = false;
    if (eight) {
      codes = item(11) != Py_None;
      if (codes != (item(12) != Py_None)) value_error(name("sq_scales") + ": both scales, or neither");
    }
    j.exp_avg = same(2, "exp_avg", codes ? at::kByte : at::kFloat);
    j.exp_avg_sq = same(3, "exp_avg_sq", codes ? at::kByte : at::kFloat);
    if (codes) {
      const Shape blocks{(j.n + 127) / 128};
      const auto scale = [&](int list, const char* what) {
        const at::Tensor& t = take(list, what, at::kFloat);
        if (t.sizes() != at::IntArrayRef(blocks) || !t.is_contiguous()) return fptr(c.whole(item(list), name(what), at::kFloat, &blocks));
        return fptr(t);
      };
      j.avg_scale = scale(11, "avg_scales");
      j.sq_scale = scale(12, "sq_scales");
    }
    if (masters && item(10) != Py_None) {
      if (pt != at::kBFloat16) value_error(name("masters") + ": an fp32 parameter is its own");
      j.master = static_cast<float*>(same(10, "masters", at::kFloat));
    }
  }
  puro_adamw_hyper h = {};
  h.step_dev = scalar_tensor<int64_t>(c, a[4], "step", at::kLong);
  if (!h.step_dev) h.step = as_int(a[4], "step");
  h.lr_dev = scalar_tensor<float>(c, a[5], "lr", at::kFloat);
  if (!h.lr_dev) h.lr = as_float(a[5], "lr");
  h.beta1 = as_float(a[6], "beta1");
  h.beta2 = as_float(a[7], "beta2");
  h.eps = as_float(a[8], "eps");
  h.weight_decay = as_float(a[9], "weight_decay");
  at::Tensor norm;
  if (a[13] != Py_None) norm = norm_value(c, a[13]);
  h.norm = fptr(norm);
  h.max_norm = (float)as_float(a[14], "max_norm");
  h.seed = PyLong_Check(a[15]) ? PyLong_AsUnsignedLongLong(a[15]) : 0;
  if (!PyLong_Check(a[15])) type_error("seed: expected an integer");
  if (PyErr_Occurred()) {
    PyErr_Clear();
    value_error("seed: expected an integer of 0 to 2^64 - 1");
  }
  const hipStream_t st = c.stream();
  enqueue("puro_adamw", [&] { return puro_adamw(jobs.data(), (int)n, &h, st); });
  for (int list : {0, 2, 3, 10, 11, 12})
    if (a[list] != Py_None)
      for (Py_ssize_t i = 0; i < n; ++i) written(PySequence_Fast_GET_ITEM(a[list], i));
  Py_RETURN_NONE;
}

// tensors: for the forward pass of a step that is being captured into a graph (the current stream records).  A leaf's
// gradient belongs to the stream that was current when the first graph that reaches it was built, for as long as one of
// those graphs lives, and the autograd engine joins that stream to the backward pass.  One that does not record breaks
// the capture from inside the engine, which ends the process: refused here, before the pass starts.  The leaves are the
// tensors themselves and those that the graphs behind them end in (a view of a leaf, what an earlier layer made of one).
PyObject* check_capture(PyObject* const* a) {
  if (!PyTuple_Check(a[0])) type_error("expected a tuple of tensors");
  std::vector<std::shared_ptr<torch::autograd::Node>> todo;
  std::unordered_set<torch::autograd::Node*> seen;
  const auto visit = [&](const std::shared_ptr<torch::autograd::Node>& node) {
    if (node && seen.insert(node.get()).second) todo.push_back(node);
  };
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(a[0]); ++i) {
    PyObject* o = PyTuple_GET_ITEM(a[0], i);
    if (!THPVariable_Check(o)) continue;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || !t.requires_grad()) continue;
    visit(t.is_leaf() ? torch::autograd::impl::try_get_grad_accumulator(t) : t.grad_fn());
  }
  while (!todo.empty()) {
    const auto node = todo.back();
    todo.pop_back();
    if (dynamic_cast<const torch::autograd::AccumulateGrad*>(node.get())) {
      const auto st = node->stream();
      if (st && *st != c10::impl::VirtualGuardImpl(st->device_type()).getStream(st->device()))
        throw Refused{PyExc_RuntimeError,
                      "a step is being captured while the autograd graph of another stream reaches the same parameter or "
                      "input: delete the outputs of the earlier passes first"};
    }
    for (const auto& edge : node->next_edges()) visit(edge.function);
  }
  Py_RETURN_NONE;
}

// get_device, get_stream, raise_status: called once, before any of the above
PyObject* init(PyObject* const* a) {
  PyObject** slots[] = {&get_device, &get_stream, &raise_status};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(a[i]);
    Py_XDECREF(*slots[i]);
    *slots[i] = a[i];
  }
  Py_RETURN_NONE;
}

#define PURO_ENTRY(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<n, name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    PURO_ENTRY(init, 3),
    PURO_ENTRY(check_capture, 1),
    PURO_ENTRY(layer_norm, 9),
    PURO_ENTRY(layer_norm_quant, 9),
    PURO_ENTRY(layer_norm_quant_dual, 11),
    PURO_ENTRY(layer_norm_backward, 12),
    PURO_ENTRY(clip_grad_norm, 5),
    PURO_ENTRY(scale_by_norm, 4),
    PURO_ENTRY(gemm_rows, 7),
    PURO_ENTRY(residual_norm, 16),
    PURO_ENTRY(residual_norm_quant, 16),
    PURO_ENTRY(residual_norm_quant_dual, 18),
    PURO_ENTRY(residual_norm_backward, 22),
    PURO_ENTRY(rotary, 8),
    PURO_ENTRY(adamw, 16),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Argument marshalling of the operators of puro_ops.h.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
