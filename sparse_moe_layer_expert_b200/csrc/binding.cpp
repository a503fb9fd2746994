// binding.cpp -- the Python side of the operators around the layer, natively:
// argument checks (type, shape, device, strides), outputs and workspaces where
// none are given, and the call into libmoefp8's C ABI.
//
// A decode step makes these calls back to back, and in Python the checks of
// eight tensors and the ctypes marshalling took longer than the launch (10 us a
// call, 3 of them the launch's).  The module holds no state but the addresses
// of the C entry points and the exception class, both given once by
// _binding.py.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "moe_fp8.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Api {
  decltype(&fp8_add_rmsnorm_quant_1x128) norm_fwd = nullptr;
  decltype(&add_rmsnorm_backward_workspace_size) norm_bwd_ws = nullptr;
  decltype(&add_rmsnorm_backward) norm_bwd = nullptr;
  decltype(&moe_balance_loss_workspace_size) balance_ws = nullptr;
  decltype(&moe_balance_loss) balance = nullptr;
  decltype(&moe_router_backward_workspace_size) router_ws = nullptr;
  decltype(&moe_router_backward) router_bwd = nullptr;
} api;
PyObject *moe_error = nullptr;  // MoeError(status, where)

// A refused argument or a status other than MOE_OK: the Python error is set.
struct Raised {};

[[noreturn]] void raise(int status, const std::string &where) {
  if (PyObject *e = PyObject_CallFunction(moe_error, "is", status, where.c_str())) {
    PyErr_SetObject(moe_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}
[[noreturn]] void refuse(const char *where, const std::string &what) {
  raise(MOE_ERR_INVALID_ARG, std::string(where) + ": " + what);
}

std::string describe(PyObject *o) {
  if (!THPVariable_Check(o)) return Py_TYPE(o)->tp_name;
  const Tensor &t = THPVariable_Unpack(o);
  std::string s = c10::toString(t.scalar_type());
  s += " [";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "] on " + t.device().str() + (t.is_contiguous() ? "" : ", not contiguous");
}
std::string dims(std::initializer_list<int64_t> shape) {
  std::string s = "[";
  for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
  return s + "]";
}

const Tensor &tensor(PyObject *o, const char *where, const char *name) {
  if (!THPVariable_Check(o)) refuse(where, std::string(name) + " is " + describe(o) + ", wanted a tensor");
  return THPVariable_Unpack(o);
}

// The pointer of a contiguous `type` tensor of that shape on CUDA device `dev`.
void *want(PyObject *o, const char *where, const char *name, ScalarType type, std::initializer_list<int64_t> shape,
           int dev) {
  if (THPVariable_Check(o)) {
    const Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() == type && t.is_cuda() && t.get_device() == dev &&
        t.sizes().equals(c10::IntArrayRef(shape.begin(), shape.size())) && t.is_contiguous())
      return t.data_ptr();
  }
  refuse(where, std::string(name) + " is " + describe(o) + ", wanted a contiguous " + c10::toString(type) + " " +
                    dims(shape) + " on CUDA device " + std::to_string(dev));
}
void *want_or_null(PyObject *o, const char *where, const char *name, ScalarType type,
                   std::initializer_list<int64_t> shape, int dev) {
  return o == Py_None ? nullptr : want(o, where, name, type, shape, dev);
}
// The same, of any shape; the elements in *n.
void *want_any(PyObject *o, const char *where, const char *name, ScalarType type, int dev, int64_t *n) {
  if (THPVariable_Check(o)) {
    const Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.is_contiguous()) {
      *n = t.numel();
      return t.data_ptr();
    }
  }
  refuse(where, std::string(name) + " is " + describe(o) + ", wanted a contiguous " + c10::toString(type) +
                    " tensor on CUDA device " + std::to_string(dev));
}

int stream_type(const Tensor &t, const char *where, const char *name) {
  if (t.scalar_type() == ScalarType::BFloat16) return MOE_DTYPE_BF16;
  if (t.scalar_type() != ScalarType::Float)
    refuse(where, std::string(name) + " is " + c10::toString(t.scalar_type()) + ", wanted bf16 or float32");
  return MOE_DTYPE_F32;
}
int device_of(const Tensor &t, const char *where, const char *name) {
  if (!t.is_cuda()) refuse(where, std::string(name) + " is not on a CUDA device");
  return t.get_device();
}

// A new reference to `o`, or where it is None (or True) to a new tensor.
struct Out {
  PyObject *o = nullptr;
  Out(PyObject *given, bool make, at::IntArrayRef shape, ScalarType type, int dev) {
    if (make)
      o = THPVariable_Wrap(at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev)));
    else
      o = Py_NewRef(given);
    if (!o) throw Raised{};
  }
  Out(Out &&b) noexcept : o(b.o) { b.o = nullptr; }
  ~Out() { Py_XDECREF(o); }
  Out(const Out &) = delete;
  Out &operator=(const Out &) = delete;
};
Out workspace(PyObject *given, size_t bytes, int dev) {
  const int64_t n = bytes < 256 ? 256 : static_cast<int64_t>(bytes);
  return Out(given, given == Py_None, {n}, ScalarType::Byte, dev);
}
Out error_flag(PyObject *given, int dev) {
  Out e(given, given == Py_None, {1}, ScalarType::Int, dev);
  if (given == Py_None) THPVariable_Unpack(e.o).zero_();
  return e;
}

void done(int status, const char *where) {
  if (status != MOE_OK) raise(status, where);
}

long as_long(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
void *as_ptr(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised{};
  return p;
}
float as_float(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

// Every function: (arguments...) positional, as _binding.py passes them.
template <PyObject *(*F)(PyObject *const *)>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n, Py_ssize_t want_n) {
  if (n != want_n) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, wanted %zd", n, want_n);
    return nullptr;
  }
  // torch's errors become its Python exceptions (torch.OutOfMemoryError and the like)
  HANDLE_TH_ERRORS
  try {
    return F(a);
  } catch (const Raised &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// stream, x, resid, weight, eps, h, y, q, scales, rstd, pow2
PyObject *norm_fwd(PyObject *const *a) {
  const char *w = "fp8_add_rmsnorm_quant_1x128";
  const Tensor &x = tensor(a[1], w, "x");
  const int code = stream_type(x, w, "x"), dev = device_of(x, w, "x");
  const ScalarType type = x.scalar_type();
  if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1)) refuse(w, "x is [rows, cols] with unit stride along cols");
  const int64_t rows = x.size(0), cols = x.size(1);
  // a single row has no row stride
  const int64_t ld = rows > 1 ? x.stride(0) : cols;
  int64_t ld_r = cols;
  const void *rp = nullptr;
  const bool has_r = a[2] != Py_None;
  if (has_r) {
    const Tensor &r = tensor(a[2], w, "resid");
    if (r.scalar_type() != type || !r.is_cuda() || r.get_device() != dev || !r.sizes().equals(x.sizes()) ||
        (cols > 1 && r.stride(1) != 1))
      refuse(w, "resid is " + describe(a[2]) + ", wanted x's type, shape and device with unit stride along cols");
    if (rows > 1) ld_r = r.stride(0);
    rp = r.data_ptr();
  }
  Out h(a[5] == Py_None && !has_r ? a[1] : a[5], a[5] == Py_None && has_r, {rows, cols}, type, dev);
  Out y(a[6], a[6] == Py_None, {rows, cols}, ScalarType::BFloat16, dev);
  Out q(a[7], a[7] == Py_None, {rows, cols}, ScalarType::Byte, dev);
  Out s(a[8], a[8] == Py_None, {rows, cols / 128}, ScalarType::Float, dev);
  Out rstd(a[9], a[9] == Py_None, {rows}, ScalarType::Float, dev);
  const void *xp = x.data_ptr();
  const auto *wp = static_cast<const float *>(want_or_null(a[3], w, "weight", ScalarType::Float, {cols}, dev));
  const float eps = as_float(a[4]);
  void *hp = a[5] == Py_None && !has_r ? nullptr : want(h.o, w, "h", type, {rows, cols}, dev);
  void *yp = want(y.o, w, "y", ScalarType::BFloat16, {rows, cols}, dev);
  auto *qp = static_cast<uint8_t *>(want(q.o, w, "q", ScalarType::Byte, {rows, cols}, dev));
  auto *sp = static_cast<float *>(want(s.o, w, "scales", ScalarType::Float, {rows, cols / 128}, dev));
  auto *rsp = static_cast<float *>(want(rstd.o, w, "rstd", ScalarType::Float, {rows}, dev));
  const int pow2 = PyObject_IsTrue(a[10]);
  if (pow2 < 0) throw Raised{};
  void *st = as_ptr(a[0]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = api.norm_fwd(xp, ld, rp, ld_r, code, wp, eps, rows, cols, hp, yp, qp, sp, rsp,
                        pow2 ? MOE_SCALE_POW2 : MOE_SCALE_AMAX, st);
  Py_END_ALLOW_THREADS
  done(status, w);
  return PyTuple_Pack(5, h.o, y.o, q.o, s.o, rstd.o);
}

// stream, dy, h, rstd, weight, dres, dx, dw, dx_dtype (a torch dtype or None), ws
PyObject *norm_bwd(PyObject *const *a) {
  const char *w = "add_rmsnorm_backward";
  const Tensor &h = tensor(a[2], w, "h");
  const int code = stream_type(h, w, "h"), dev = device_of(h, w, "h");
  const ScalarType type = h.scalar_type();
  if (h.dim() != 2) refuse(w, "h is [rows, cols]");
  const int64_t rows = h.size(0), cols = h.size(1);
  const Tensor &dy = tensor(a[1], w, "dy");
  const int ycode = stream_type(dy, w, "dy");
  ScalarType xtype = type;
  if (a[8] != Py_None) {
    if (!THPDtype_Check(a[8])) refuse(w, "dx_dtype is a torch dtype");
    xtype = reinterpret_cast<THPDtype *>(a[8])->scalar_type;
  }
  if (a[6] != Py_None) {
    const ScalarType given = tensor(a[6], w, "dx").scalar_type();
    if (a[8] != Py_None && given != xtype) refuse(w, "dx is " + describe(a[6]) + ", not of dx_dtype");
    xtype = given;
  }
  if (xtype != ScalarType::Float && xtype != ScalarType::BFloat16) refuse(w, "dx is bf16 or float32");
  Out dx(a[6], a[6] == Py_None, {rows, cols}, xtype, dev);
  Out dw(a[7], a[7] == Py_None, {cols}, ScalarType::Float, dev);
  Out ws = workspace(a[9], a[9] == Py_None ? api.norm_bwd_ws(rows, cols) : 0, dev);
  const void *yp = want(a[1], w, "dy", dy.scalar_type(), {rows, cols}, dev);
  const void *hp = want(a[2], w, "h", type, {rows, cols}, dev);
  const void *dp = want_or_null(a[5], w, "dres", type, {rows, cols}, dev);
  const auto *wp = static_cast<const float *>(want_or_null(a[4], w, "weight", ScalarType::Float, {cols}, dev));
  const auto *rp = static_cast<const float *>(want(a[3], w, "rstd", ScalarType::Float, {rows}, dev));
  void *xp = want(dx.o, w, "dx", xtype, {rows, cols}, dev);
  auto *dwp = static_cast<float *>(want(dw.o, w, "dw", ScalarType::Float, {cols}, dev));
  int64_t bytes = 0;
  void *wsp = want_any(ws.o, w, "ws", ScalarType::Byte, dev, &bytes);
  void *st = as_ptr(a[0]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = api.norm_bwd(yp, ycode, hp, dp, code, wp, rp, rows, cols, xp,
                        xtype == ScalarType::Float ? MOE_DTYPE_F32 : MOE_DTYPE_BF16, dwp, wsp,
                        static_cast<size_t>(bytes), st);
  Py_END_ALLOW_THREADS
  done(status, w);
  return PyTuple_Pack(2, dx.o, dw.o);
}

struct RouterState {
  int64_t splits, T;
  int dev;
  const float *logits;
  const int32_t *idx;
};
RouterState router_state(const moe_config *cfg, PyObject *logits, PyObject *idx, const char *w) {
  const Tensor &z = tensor(logits, w, "logits");
  RouterState r{};
  r.dev = device_of(z, w, "logits");
  if (z.dim() != 3 || z.size(0) < 1 || z.size(2) != cfg->n_routed)
    refuse(w, "logits is " + describe(logits) + ", wanted [n_splits, T, " + std::to_string(cfg->n_routed) + "]");
  r.splits = z.size(0);
  r.T = z.size(1);
  r.logits = static_cast<const float *>(want(logits, w, "logits", ScalarType::Float, {r.splits, r.T, z.size(2)}, r.dev));
  r.idx = static_cast<const int32_t *>(want(idx, w, "idx", ScalarType::Int, {r.T, cfg->top_k}, r.dev));
  if (r.splits > INT32_MAX) refuse(w, "too many splits");
  return r;
}
const int32_t *sequences(PyObject *off, const char *w, int dev, int64_t *n_seq) {
  int64_t n = 0;
  const auto *p = static_cast<const int32_t *>(want_any(off, w, "seq_offsets", ScalarType::Int, dev, &n));
  if (THPVariable_Unpack(off).dim() != 1 || n < 1 || n - 1 > INT32_MAX) refuse(w, "seq_offsets is [n_seq + 1]");
  *n_seq = n - 1;
  return p;
}

// stream, cfg address, logits, idx, seq_offsets, alpha, loss, counts, ws, err
PyObject *balance_loss(PyObject *const *a) {
  const char *w = "moe_balance_loss";
  const auto *cfg = static_cast<const moe_config *>(as_ptr(a[1]));
  const RouterState r = router_state(cfg, a[2], a[3], w);
  int64_t n_seq = 0, bytes = 0, one = 0;
  const int32_t *off = sequences(a[4], w, r.dev, &n_seq);
  Out loss(a[6], a[6] == Py_None, {n_seq}, ScalarType::Float, r.dev);
  Out counts(a[7], a[7] == Py_None, {n_seq, cfg->n_routed}, ScalarType::Int, r.dev);
  Out ws = workspace(a[8], a[8] == Py_None ? api.balance_ws(cfg, r.T, n_seq) : 0, r.dev);
  Out err = error_flag(a[9], r.dev);
  auto *lp = static_cast<float *>(want(loss.o, w, "loss", ScalarType::Float, {n_seq}, r.dev));
  auto *cp = static_cast<int32_t *>(want(counts.o, w, "counts", ScalarType::Int, {n_seq, cfg->n_routed}, r.dev));
  void *wsp = want_any(ws.o, w, "ws", ScalarType::Byte, r.dev, &bytes);
  auto *ep = static_cast<int32_t *>(want_any(err.o, w, "err", ScalarType::Int, r.dev, &one));
  if (one < 1) refuse(w, "err holds an int32");
  const float alpha = as_float(a[5]);
  void *st = as_ptr(a[0]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = api.balance(cfg, r.logits, static_cast<int32_t>(r.splits), r.idx, r.T, off, n_seq, alpha, lp, cp, wsp,
                       static_cast<size_t>(bytes), ep, st);
  Py_END_ALLOW_THREADS
  done(status, w);
  return PyTuple_Pack(2, loss.o, counts.o);
}

PyObject *dict_get(PyObject *d, const char *key) {  // borrowed, or null
  return PyDict_GetItemString(d, key);
}

// The balance gradient of dict(seq_offsets, counts, dloss, alpha).
moe_balance_grad balance_grad(const moe_config *cfg, PyObject *d, const char *w, int dev) {
  if (!PyDict_Check(d)) refuse(w, "balance is a dict(seq_offsets, counts, dloss, alpha)");
  PyObject *off = dict_get(d, "seq_offsets"), *counts = dict_get(d, "counts"), *dloss = dict_get(d, "dloss"),
           *alpha = dict_get(d, "alpha");
  if (!off || !counts) refuse(w, "balance holds seq_offsets and counts");
  moe_balance_grad g{};
  int64_t n_seq = 0;
  g.seq_offsets_dev = sequences(off, w, dev, &n_seq);
  g.n_seq = static_cast<int32_t>(n_seq);
  g.alpha = alpha ? as_float(alpha) : 1e-4f;
  g.counts_dev = static_cast<const int32_t *>(want(counts, w, "counts", ScalarType::Int, {n_seq, cfg->n_routed}, dev));
  if (dloss && dloss != Py_None)
    g.dloss_dev = static_cast<const float *>(want(dloss, w, "dloss", ScalarType::Float, {n_seq}, dev));
  return g;
}

// stream, cfg address, logits, idx, x, wr, dgate, balance, dlogits, dx, dx_accumulate, dwr, ws, err
PyObject *router_backward(PyObject *const *a) {
  const char *w = "moe_router_backward";
  const auto *cfg = static_cast<const moe_config *>(as_ptr(a[1]));
  const RouterState r = router_state(cfg, a[2], a[3], w);
  const int64_t H = cfg->hidden, Nr = cfg->n_routed;
  const int acc = PyObject_IsTrue(a[10]);
  if (acc < 0) throw Raised{};
  auto asked = [](PyObject *o) { return o != Py_None && o != Py_False; };
  if (acc && (!asked(a[9]) || a[9] == Py_True)) refuse(w, "dx_accumulate needs a dx to add to");
  // None, False: not wanted; True: a new tensor; else the caller's
  auto out = [&](PyObject *o, std::initializer_list<int64_t> shape) {
    return Out(asked(o) ? o : Py_None, o == Py_True, at::IntArrayRef(shape.begin(), shape.size()), ScalarType::Float,
               r.dev);
  };
  Out dlogits = out(a[8], {r.T, Nr}), dx = out(a[9], {r.T, H}), dwr = out(a[11], {Nr, H});
  auto *lp = static_cast<float *>(want_or_null(dlogits.o, w, "dlogits", ScalarType::Float, {r.T, Nr}, r.dev));
  auto *xp = static_cast<float *>(want_or_null(dx.o, w, "dx", ScalarType::Float, {r.T, H}, r.dev));
  auto *wp = static_cast<float *>(want_or_null(dwr.o, w, "dwr", ScalarType::Float, {Nr, H}, r.dev));
  const auto *gp = static_cast<const float *>(want_or_null(a[6], w, "dgate", ScalarType::Float, {r.T, cfg->top_k}, r.dev));
  const void *xin = wp || a[4] != Py_None ? want(a[4], w, "x", ScalarType::BFloat16, {r.T, H}, r.dev) : nullptr;
  const void *wr = xp || a[5] != Py_None ? want(a[5], w, "wr", ScalarType::BFloat16, {Nr, H}, r.dev) : nullptr;
  moe_balance_grad bal{};
  if (a[7] != Py_None) bal = balance_grad(cfg, a[7], w, r.dev);
  const bool products = xp || wp;
  Out ws = products ? workspace(a[12], a[12] == Py_None ? api.router_ws(cfg, r.T) : 0, r.dev)
                    : Out(a[12], false, {}, ScalarType::Byte, r.dev);
  Out err = error_flag(a[13], r.dev);
  int64_t bytes = 0, one = 0;
  void *wsp = ws.o == Py_None ? nullptr : want_any(ws.o, w, "ws", ScalarType::Byte, r.dev, &bytes);
  auto *ep = static_cast<int32_t *>(want_any(err.o, w, "err", ScalarType::Int, r.dev, &one));
  if (one < 1) refuse(w, "err holds an int32");
  void *st = as_ptr(a[0]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = api.router_bwd(cfg, r.logits, static_cast<int32_t>(r.splits), r.idx, r.T, gp,
                          a[7] != Py_None ? &bal : nullptr, xin, wr, lp, xp, acc, wp, wsp, static_cast<size_t>(bytes),
                          ep, st);
  Py_END_ALLOW_THREADS
  done(status, w);
  return PyTuple_Pack(3, dlogits.o, dx.o, dwr.o);
}

// MoeError, then the addresses of the C entry points in Api's order.
PyObject *init(PyObject *const *a) {
  moe_error = Py_NewRef(a[0]);
  auto get = [&](int i, auto &f) { f = reinterpret_cast<std::decay_t<decltype(f)>>(as_ptr(a[i])); };
  get(1, api.norm_fwd);
  get(2, api.norm_bwd_ws);
  get(3, api.norm_bwd);
  get(4, api.balance_ws);
  get(5, api.balance);
  get(6, api.router_ws);
  get(7, api.router_bwd);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *method(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  return entry<F>(self, a, n, N);
}
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyMethodDef def(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&method<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {def<init, 8>("init"),
                         def<norm_fwd, 11>("norm_fwd"),
                         def<norm_bwd, 10>("norm_bwd"),
                         def<balance_loss, 10>("balance_loss"),
                         def<router_backward, 14>("router_backward"),
                         {nullptr, nullptr, 0, nullptr}};
// The doc string says which Python and torch the module was built against; build.py looks for it.
#ifndef MOE_MADE_FOR
#define MOE_MADE_FOR ""
#endif
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", MOE_MADE_FOR, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
