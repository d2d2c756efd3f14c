// Python binding of the operators around the block (mx4.py, norms.py,
// experts.py).  Their kernels take a few microseconds, and checking tensors and
// converting arguments in Python took as long again: a call through this
// module costs 5 to 6 us on the host where the same through ctypes cost 7 to
// 10, 3 of them the launch.  It holds argument checks and output allocation
// only; every step of an operator runs in libcfr.so.
//
// A tensor that does not fit raises ValueError; an error of the library raises
// what the `check` callable given to init() raises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/cfr.h"

namespace {

PyObject* g_stream = nullptr;  // device ordinal -> raw handle of its current stream
PyObject* g_check = nullptr;   // raises the library's error for a return code

// Thrown after a Python error has been set.
struct Raised {};

template <typename... A>
[[noreturn]] void refuse(const char* format, A... a) {
  PyErr_Format(PyExc_ValueError, format, a...);
  throw Raised();
}

int code_of(at::ScalarType t) {
  return t == at::kFloat ? CFR_F32 : t == at::kBFloat16 ? CFR_BF16 : t == at::kHalf ? CFR_F16 : -1;
}

// The operators have no backward pass: a tensor that needs a gradient is
// refused where one would be recorded, unless the result has none by its type
// (no_grad_lost).
const at::Tensor* optional(PyObject* o, const char* name, bool no_grad_lost = false) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse("%s: expected a tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!no_grad_lost && t.requires_grad() && at::GradMode::is_enabled())
    refuse("%s: needs a gradient, which this operator does not have: detach it, or call under torch.no_grad()", name);
  if (t.is_neg()) refuse("%s: its memory holds the negative of its values: call resolve_neg()", name);
  return &t;
}

const at::Tensor& tensor(PyObject* o, const char* name, bool no_grad_lost = false) {
  const at::Tensor* t = optional(o, name, no_grad_lost);
  if (!t) refuse("%s: expected a tensor", name);
  return *t;
}

int dtype_code(const at::Tensor& t, const char* name) {
  const int c = code_of(t.scalar_type());
  if (c < 0) refuse("%s: expected a float32, bfloat16 or float16 tensor", name);
  return c;
}

at::ScalarType dtype_arg(PyObject* o, at::ScalarType otherwise, const char* name) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o) || code_of(reinterpret_cast<THPDtype*>(o)->scalar_type) < 0)
    refuse("%s must be float32, bfloat16 or float16", name);
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

void on_device(const at::Tensor& t, int device, const char* name) {
  if (!t.is_cuda() || t.get_device() != device) refuse("%s: expected a tensor on device %d", name, device);
}

// A device tensor [..., cols] whose rows are contiguous: two dimensions with
// any row stride, or any number of them without gaps.
struct Rows {
  int64_t n, cols, stride;
  Rows(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse("%s: expected a device tensor", name);
    if (t.dim() == 2) {
      n = t.size(0), cols = t.size(1), stride = t.stride(0);
      if (t.stride(1) != 1 && cols > 1) refuse("%s: the last dimension must be contiguous", name);
      if (n <= 1) stride = cols;
      if (stride < cols) refuse("%s: rows must not overlap", name);
    } else {
      if (t.dim() == 0 || !t.is_contiguous())
        refuse("%s: expected two dimensions, or a contiguous tensor of more", name);
      cols = stride = t.size(-1);
      n = cols ? t.numel() / cols : 0;
    }
  }
};

void same_shape(const at::Tensor& t, at::IntArrayRef shape, int device, const char* name) {
  if (t.sizes() != shape) refuse("%s: unexpected shape", name);
  on_device(t, device, name);
}

void plain(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, int device, const char* name, const char* what) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) refuse("%s: expected %s", name, what);
  on_device(t, device, name);
}

at::Tensor new_like(const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type) {
  return at::empty(shape, t.options().dtype(type));
}

void* stream_of(int device) {
  PyObject* d = PyLong_FromLong(device);
  PyObject* s = d ? PyObject_CallOneArg(g_stream, d) : nullptr;
  Py_XDECREF(d);
  if (!s) throw Raised();
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!p && PyErr_Occurred()) throw Raised();
  return p;
}

void check(int rc) {
  if (rc == CFR_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "i", rc);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "cfr error %d", rc);
  throw Raised();
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v;
}

at::DimVector lead_and(const at::Tensor& t, int64_t last) {
  at::DimVector s(t.sizes().begin(), t.sizes().end());
  s.back() = last;
  return s;
}

// The result as Python sees it.  It may be a caller's tensor: autograd has to
// find it changed, as after any in-place operation.
PyObject* written(at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  return THPVariable_Wrap(std::move(t));
}

PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

// (x, out) -> (codes, scales)
PyObject* quantize(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x", true);  // codes are whole numbers
  const int dt = dtype_code(x, "x");
  const Rows r(x, "x");
  const int dev = x.get_device();
  const at::DimVector cs = lead_and(x, (r.cols + 1) / 2), ss = lead_and(x, (r.cols + 31) / 32);
  at::Tensor codes, scales;
  if (a[1] == Py_None) {
    codes = new_like(x, cs, at::kByte), scales = new_like(x, ss, at::kByte);
  } else {
    if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 2) refuse("out: expected a (codes, scales) pair");
    codes = tensor(PyTuple_GET_ITEM(a[1], 0), "codes"), scales = tensor(PyTuple_GET_ITEM(a[1], 1), "scales");
    plain(codes, at::kByte, cs, dev, "codes", "contiguous uint8 [..., ceil(cols/2)]");
    plain(scales, at::kByte, ss, dev, "scales", "contiguous uint8 [..., ceil(cols/32)]");
  }
  check(cfr_mx4_quantize(x.data_ptr(), dt, r.n, r.cols, r.stride, static_cast<uint8_t*>(codes.data_ptr()),
                         static_cast<uint8_t*>(scales.data_ptr()), dev, stream_of(dev)));
  return pair(written(codes), written(scales));
}

// (codes, scales, cols, dtype, out) -> y
PyObject* dequantize(PyObject* const* a) {
  const at::Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales");
  if (!codes.is_cuda() || codes.dim() == 0) refuse("codes: expected a uint8 device tensor");
  const int64_t cols = integer(a[2]);
  if (cols < 0) refuse("cols must be >= 0");
  const int dev = codes.get_device();
  plain(codes, at::kByte, lead_and(codes, (cols + 1) / 2), dev, "codes", "contiguous uint8 [..., ceil(cols/2)]");
  plain(scales, at::kByte, lead_and(codes, (cols + 31) / 32), dev, "scales", "contiguous uint8 [..., ceil(cols/32)]");
  const at::DimVector shape = lead_and(codes, cols);
  at::Tensor out;
  if (a[4] == Py_None) {
    out = new_like(codes, shape, dtype_arg(a[3], at::kFloat, "dtype"));
  } else {
    out = tensor(a[4], "out");
    same_shape(out, shape, dev, "out");
  }
  const int dt = dtype_code(out, "out");
  const Rows r(out, "out");
  check(cfr_mx4_dequantize(static_cast<const uint8_t*>(codes.data_ptr()), static_cast<const uint8_t*>(scales.data_ptr()),
                           r.n, r.cols, out.data_ptr(), dt, r.stride, dev, stream_of(dev)));
  return written(out);
}

// Leading sizes (all but the last) without the ones before them.
at::IntArrayRef lead(const at::Tensor& t) {
  const at::IntArrayRef s = t.sizes().slice(0, t.dim() ? t.dim() - 1 : 0);
  size_t i = 0;
  while (i < s.size() && s[i] == 1) ++i;
  return s.slice(i);
}

// Pointer and type code of a [cols] weight, or none.
struct Weight {
  const void* p = nullptr;
  int dt = 0;
  Weight(PyObject* o, int64_t cols, int device, const char* name) {
    const at::Tensor* t = optional(o, name);
    if (!t) return;
    dt = dtype_code(*t, name);
    if (t->dim() != 1 || t->size(0) != cols || !t->is_contiguous()) refuse("%s: expected a contiguous [cols] tensor", name);
    on_device(*t, device, name);
    p = t->data_ptr();
  }
};

// (x, weight, eps, offset, out, dtype) -> u
PyObject* norm_in(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const int xd = dtype_code(x, "x");
  const Rows rx(x, "x");
  const int dev = x.get_device();
  const Weight w(a[1], rx.cols, dev, "weight");
  at::Tensor out;
  if (a[4] == Py_None) {
    out = new_like(x, x.sizes(), dtype_arg(a[5], x.scalar_type(), "dtype"));
  } else {
    out = tensor(a[4], "out");
    same_shape(out, x.sizes(), dev, "out");
  }
  const int ud = dtype_code(out, "out");
  const Rows ru(out, "out");
  check(cfr_block_norm_in(x.data_ptr(), xd, rx.stride, w.p, w.dt, (float)number(a[3]), (float)number(a[2]), rx.n, rx.cols,
                          out.data_ptr(), ud, ru.stride, dev, stream_of(dev)));
  return written(out);
}

// (y, x, post_weight, post_norm, gate, gate_act, out_scale, resid_scale,
//  next_weight, next_norm, eps, offset, out, next_out, next_dtype) -> s or (s, u)
PyObject* norm_out(PyObject* const* a) {
  const at::Tensor &y = tensor(a[0], "y"), &x = tensor(a[1], "x");
  cfr_norm_out_args n = {};
  n.y_dtype = dtype_code(y, "y"), n.x_dtype = dtype_code(x, "x");
  const Rows ry(y, "y");
  const int dev = n.device = y.get_device();
  same_shape(x, y.sizes(), dev, "x");
  const Rows rx(x, "x");
  n.post_norm = truth(a[3]);
  const bool next = truth(a[9]);
  if (a[2] != Py_None && !n.post_norm) refuse("post_weight without post_norm");
  if ((a[8] != Py_None || a[13] != Py_None) && !next) refuse("next_weight or next_out without next_norm");
  const Weight wp(a[2], ry.cols, dev, "post_weight"), wn(a[8], ry.cols, dev, "next_weight");
  if (wp.p && wn.p && wp.dt != wn.dt) refuse("post_weight and next_weight must have one type");
  if (const at::Tensor* g = optional(a[4], "gate")) {
    if (dtype_code(*g, "gate") != n.y_dtype) refuse("gate: expected y's type");
    on_device(*g, dev, "gate");
    if (g->dim() != 2 && !g->is_contiguous()) refuse("gate: expected two dimensions, or a contiguous tensor");
    const bool two = g->dim() == 2;
    const int64_t gc = g->dim() ? g->size(-1) : 1, gr = two ? g->size(0) : gc ? g->numel() / gc : 1;
    // one row or y's rows: the same leading sizes, not only as many rows
    if ((!lead(*g).empty() && lead(*g) != lead(y)) || (gc != 1 && gc != ry.cols))
      refuse("gate: its shape does not broadcast to y's");
    n.gate = g->data_ptr();
    n.gate_row_stride = gr > 1 ? two ? g->stride(0) : gc : 0, n.gate_col_stride = gc > 1 ? two ? g->stride(1) : 1 : 0;
  }
  at::Tensor out, u;
  if (a[12] == Py_None) {
    out = new_like(y, y.sizes(), x.scalar_type());
  } else {
    out = tensor(a[12], "out");
    same_shape(out, y.sizes(), dev, "out");
    if (out.scalar_type() != x.scalar_type()) refuse("out: expected x's type");
  }
  const Rows ro(out, "out");
  if (next) {
    if (a[13] == Py_None) {
      u = new_like(y, y.sizes(), dtype_arg(a[14], y.scalar_type(), "next_dtype"));
    } else {
      u = tensor(a[13], "next_out");
      same_shape(u, y.sizes(), dev, "next_out");
    }
    n.u_dtype = dtype_code(u, "next_out"), n.u_stride = Rows(u, "next_out").stride, n.u_out = u.data_ptr();
  }
  n.y = y.data_ptr(), n.x = x.data_ptr(), n.x_out = out.data_ptr();
  n.post_weight = wp.p, n.next_weight = wn.p, n.w_dtype = wp.p ? wp.dt : wn.dt;
  n.rows = ry.n, n.cols = ry.cols, n.y_stride = ry.stride, n.x_stride = rx.stride, n.x_out_stride = ro.stride;
  n.gate_act = (int)integer(a[5]);
  n.out_scale = (float)number(a[6]), n.resid_scale = (float)number(a[7]);
  n.eps = (float)number(a[10]), n.offset = (float)number(a[11]);
  check(cfr_block_norm_out(&n, stream_of(dev)));
  PyObject* s = written(out);
  return next ? pair(s, written(u)) : s;
}

// (handle, hidden, top, device, x, expert_ids, gate_w, out) -> y
PyObject* experts_forward(PyObject* const* a) {
  void* h = a[0] == Py_None ? nullptr : PyLong_AsVoidPtr(a[0]);
  if (PyErr_Occurred()) throw Raised();
  const int64_t H = integer(a[1]), top = integer(a[2]);
  const int dev = (int)integer(a[3]);
  const at::Tensor &x = tensor(a[4], "x"), &ids = tensor(a[5], "expert_ids"), &w = tensor(a[6], "gate_w");
  const int dt = dtype_code(x, "x");
  if (x.dim() != 2 || x.size(1) != H) refuse("x: expected a tensor [tokens, %lld]", (long long)H);
  on_device(x, dev, "x");
  const Rows rx(x, "x");
  const int64_t slots[2] = {rx.n, top};
  plain(ids, at::kInt, slots, dev, "expert_ids", "contiguous int32 [tokens, top]");
  plain(w, at::kFloat, slots, dev, "gate_w", "contiguous float32 [tokens, top]");
  at::Tensor out;
  if (a[7] == Py_None) {
    out = new_like(x, x.sizes(), x.scalar_type());
  } else {
    out = tensor(a[7], "out");
    same_shape(out, x.sizes(), dev, "out");
    if (out.scalar_type() != x.scalar_type()) refuse("out: expected x's type");
  }
  const Rows ro(out, "out");
  if (rx.n > INT32_MAX) refuse("x: too many tokens");
  check(cfr_experts_forward(static_cast<cfr_experts*>(h), x.data_ptr(), dt, rx.stride,
                            static_cast<const int32_t*>(ids.data_ptr()), static_cast<const float*>(w.data_ptr()),
                            (int32_t)rx.n, out.data_ptr(), ro.stride, stream_of(dev)));
  return written(out);
}

// A function of N positional arguments; nothing it throws leaves this module.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (stream, check): see above; kept for the life of the module.
PyObject* init(PyObject* const* a) {
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XSETREF(g_stream, a[0]);
  Py_XSETREF(g_check, a[1]);
  Py_RETURN_NONE;
}

#define OP(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(call<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {OP(init, 2),    OP(quantize, 2),  OP(dequantize, 5),      OP(norm_in, 6),
                         OP(norm_out, 15), OP(experts_forward, 8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch: the version whose headers, and so whose layout of tensors, this was built for.
PyMODINIT_FUNC PyInit__ops() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch", CFR_TORCH) < 0) Py_CLEAR(m);
  return m;
}
