// CPython binding of include/moe_ops.h for torch tensors: checks types, shapes, layouts and devices, allocates
// outputs that are not given and scratch (on torch's current stream, which is the call's), and forwards to the C ABI. (The same checks written in Python cost a call seven to ten
// microseconds, several times what the smallest kernels take.) Every function returns the call's status code.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe_ops.h"

namespace {

constexpr int64_t kBlock = 128;
int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

struct Refused {};   // a Python error is set

[[noreturn]] void refuse(PyObject* type, const char* what, const char* why) {
  PyErr_Format(type, "%s: %s", what, why);
  throw Refused();
}
[[noreturn]] void refuse_shape(const char* what, const at::Tensor& t, at::IntArrayRef want) {
  std::ostringstream s;
  s << what << ": shape " << want << " expected, got " << t.sizes();
  PyErr_SetString(PyExc_ValueError, s.str().c_str());
  throw Refused();
}

// A function's arguments: moe_ops handle, device index, stream, then its own.
struct Args {
  PyObject* const* a;
  int64_t device;
  moe_ops ops;
  void* stream;
  at::TensorOptions opts;
  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : a(args) {
    if (n != want) refuse(PyExc_TypeError, "binding", "wrong number of arguments");
    ops = (moe_ops)PyLong_AsVoidPtr(a[0]);
    device = PyLong_AsLongLong(a[1]);
    stream = PyLong_AsVoidPtr(a[2]);
    if (PyErr_Occurred()) throw Refused();
    opts = at::TensorOptions().device(at::kCUDA, (c10::DeviceIndex)device);
  }
  int64_t integer(int i) const {
    const int64_t v = PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
  }
  double number(int i) const {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
  }
  const at::Tensor& tensor(PyObject* o, const char* what) const {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, what, "a tensor expected");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device) refuse(PyExc_ValueError, what, "not on the handle's device");
    return t;
  }
  const at::Tensor& tensor(int i, const char* what) const { return tensor(a[i], what); }
  bool given(int i) const { return a[i] != Py_None; }
  // of this type and shape, dense
  void dense(const at::Tensor& t, const char* what, at::ScalarType type, at::IntArrayRef shape) const {
    if (t.scalar_type() != type) {
      PyErr_Format(PyExc_TypeError, "%s: %s expected, got %s", what, c10::toString(type), c10::toString(t.scalar_type()));
      throw Refused();
    }
    if (t.sizes() != shape) refuse_shape(what, t, shape);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, what, "has to be contiguous");
  }
  const at::Tensor& dense(int i, const char* what, at::ScalarType type, at::IntArrayRef shape) const {
    const at::Tensor& t = tensor(i, what);
    dense(t, what, type, shape);
    return t;
  }
  // Entry `key` of the dict `out`: its address; allocated where it is None or (always) missing; null if missing.
  void* output(PyObject* out, PyObject* key, const char* what, at::ScalarType type, at::IntArrayRef shape,
               bool always = false) const {
    PyObject* o = PyDict_GetItemWithError(out, key);
    if (!o && PyErr_Occurred()) throw Refused();
    if (o && o != Py_None) {
      const at::Tensor& t = tensor(o, what);
      dense(t, what, type, shape);
      return t.data_ptr();
    }
    if (!o && !always) return nullptr;
    at::Tensor t = at::empty(shape, opts.dtype(type));
    void* p = t.data_ptr();
    PyObject* made = THPVariable_Wrap(std::move(t));
    const int bad = !made || PyDict_SetItem(out, key, made);
    Py_XDECREF(made);
    if (bad) throw Refused();
    return p;
  }
  PyObject* dict(int i) const {
    if (!PyDict_Check(a[i])) refuse(PyExc_TypeError, "out", "a dict expected");
    return a[i];
  }
};

// Row stride of a matrix whose rows are dense. (A single row has none: it may be a part of an array of any width.)
long long row_stride(const at::Tensor& t, const char* what) {
  if (t.dim() != 2) refuse(PyExc_ValueError, what, "two dimensions expected");
  if (t.size(1) > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, what, "the values of a row have to be neighbours");
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}
int dtype_of(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return MOE_BF16;
  if (t.scalar_type() == at::kFloat) return MOE_FP32;
  refuse(PyExc_TypeError, what, "bf16 or fp32 expected");
}
int to_int(int64_t v, const char* what) {
  if (v > INT32_MAX) refuse(PyExc_ValueError, what, "too large");
  return (int)v;
}
const void* address(const Args& a, int i, const char* what) { return a.given(i) ? a.tensor(i, what).data_ptr() : nullptr; }

PyObject *k_h, *k_y, *k_q, *k_scale, *k_rstd, *k_dx, *k_dw, *k_idx, *k_gate, *k_cnt, *k_off, *k_perm, *k_inv,
    *k_dlogits, *k_qt, *k_scale_t, *k_codes, *k_zero, *k_group,
    *k_act, *k_save, *k_save_scale, *k_dgu, *k_dq, *k_dq_scale, *k_dqt, *k_dqt_scale, *k_actt, *k_actt_scale, *k_dgate;

template <class F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return PyLong_FromLong((long)f());
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// x, weight, residual, eps, out
PyObject* norm_forward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 8);
    const at::Tensor& x = a.tensor(3, "x");
    const long long ld_x = row_stride(x, "x");
    const int dt = dtype_of(x, "x");
    const at::ScalarType type = x.scalar_type();
    const int64_t T = x.size(0), d = x.size(1);
    a.dense(4, "weight", type, {d});
    const void* res = nullptr;
    long long ld_res = 0;
    if (a.given(5)) {
      const at::Tensor& r = a.tensor(5, "residual");
      if (r.scalar_type() != type || r.sizes() != x.sizes()) refuse(PyExc_ValueError, "residual", "type and shape of x expected");
      ld_res = row_stride(r, "residual");
      res = r.data_ptr();
    }
    PyObject* out = a.dict(7);
    Py_ssize_t found = 0;
    const auto get = [&](PyObject* key, const char* what, at::ScalarType ty, at::IntArrayRef shape) {
      found += PyDict_Contains(out, key) == 1;
      return a.output(out, key, what, ty, shape);
    };
    void* h = get(k_h, "h", type, {T, d});
    void* y = get(k_y, "y", type, {T, d});
    void* q = get(k_q, "q", at::kFloat8_e4m3fn, {T, d});
    void* scale = get(k_scale, "scale", at::kFloat, {T, blocks(d)});
    void* rstd = get(k_rstd, "rstd", at::kFloat, {T});
    if (found != PyDict_Size(out)) refuse(PyExc_ValueError, "out", "holds unknown outputs");
    return moe_norm_forward(a.ops, dt, x.data_ptr(), ld_x, res, ld_res, a.tensor(4, "weight").data_ptr(),
                            to_int(T, "x"), to_int(d, "x"), (float)a.number(6), h, y, q, (float*)scale, (float*)rstd,
                            a.stream);
  });
}

// dy, h, weight, rstd, dh, out
PyObject* norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 9);
    const at::Tensor& dy = a.tensor(3, "dy");
    if (dy.dim() != 2) refuse(PyExc_ValueError, "dy", "two dimensions expected");
    const int dt = dtype_of(dy, "dy");
    const at::ScalarType type = dy.scalar_type();
    const int64_t T = dy.size(0), d = dy.size(1);
    a.dense(dy, "dy", type, {T, d});
    const void* h = a.dense(4, "h", type, {T, d}).data_ptr();
    const void* w = a.dense(5, "weight", type, {d}).data_ptr();
    const void* rstd = a.dense(6, "rstd", at::kFloat, {T}).data_ptr();
    const void* dh = a.given(7) ? a.dense(7, "dh", type, {T, d}).data_ptr() : nullptr;
    PyObject* out = a.dict(8);
    void* dx = a.output(out, k_dx, "dx", type, {T, d});
    void* dw = a.output(out, k_dw, "dw", at::kFloat, {d});
    at::Tensor ws;
    void* scratch = nullptr;
    if (dw) {
      size_t bytes = 0;
      const moe_status st = moe_norm_workspace_size(to_int(T, "dy"), to_int(d, "dy"), &bytes);
      if (st != MOE_OK) return st;
      ws = at::empty({(int64_t)bytes}, a.opts.dtype(at::kByte));
      scratch = ws.data_ptr();
    }
    return moe_norm_backward(a.ops, dt, dy.data_ptr(), dh, h, w, (const float*)rstd, to_int(T, "dy"), to_int(d, "dy"),
                             dx, (float*)dw, scratch, a.stream);
  });
}

moe_gate_config gate_config(const Args& a, int i, int64_t E, int64_t k) {
  moe_gate_config c;
  c.E = to_int(E, "logits");
  c.k = to_int(k, "k");
  c.router = (int)a.integer(i);
  c.renorm = PyObject_IsTrue(a.a[i + 1]);
  c.route_scale = (float)a.number(i + 2);
  c.n_groups = c.topk_groups = 1;
  return c;
}

// logits, k, bias, router, renorm, route_scale, n_groups, topk_groups, dispatch, out
PyObject* gate(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 13);
    const at::Tensor& l = a.tensor(3, "logits");
    if (l.dim() != 2) refuse(PyExc_ValueError, "logits", "two dimensions expected");
    const int64_t T = l.size(0), E = l.size(1), k = a.integer(4);
    a.dense(l, "logits", at::kFloat, {T, E});
    if (k < 0) refuse(PyExc_ValueError, "k", "negative");
    const void* bias = a.given(5) ? a.dense(5, "bias", at::kFloat, {E}).data_ptr() : nullptr;
    moe_gate_config c = gate_config(a, 6, E, k);
    c.n_groups = to_int(a.integer(9), "n_groups");
    c.topk_groups = to_int(a.integer(10), "topk_groups");
    PyObject* out = a.dict(12);
    void* idx = a.output(out, k_idx, "idx", at::kInt, {T, k}, true);
    void* g = a.output(out, k_gate, "gate", at::kFloat, {T, k}, true);
    void *cnt = nullptr, *off = nullptr, *perm = nullptr, *inv = nullptr, *scratch = nullptr;
    at::Tensor ws;
    if (PyObject_IsTrue(a.a[11])) {
      cnt = a.output(out, k_cnt, "cnt", at::kInt, {E}, true);
      off = a.output(out, k_off, "off", at::kInt, {E + 1}, true);
      perm = a.output(out, k_perm, "perm", at::kInt, {T * k}, true);
      inv = a.output(out, k_inv, "inv", at::kInt, {T * k}, true);
      size_t bytes = 0;
      const moe_status st = moe_gate_workspace_size(&c, to_int(T, "logits"), &bytes);
      if (st != MOE_OK) return st;
      if (bytes) {
        ws = at::empty({(int64_t)bytes}, a.opts.dtype(at::kByte));
        scratch = ws.data_ptr();
      }
    }
    return moe_gate_forward(a.ops, &c, (const float*)l.data_ptr(), (const float*)bias, to_int(T, "logits"),
                            (int32_t*)idx, (float*)g, (int32_t*)cnt, (int32_t*)off, (int32_t*)perm, (int32_t*)inv,
                            scratch, a.stream);
  });
}

// logits, idx, dgate, router, renorm, route_scale, out
PyObject* gate_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 10);
    const at::Tensor &l = a.tensor(3, "logits"), &idx = a.tensor(4, "idx");
    if (l.dim() != 2 || idx.dim() != 2) refuse(PyExc_ValueError, "logits, idx", "two dimensions expected");
    const int64_t T = l.size(0), E = l.size(1), k = idx.size(1);
    a.dense(l, "logits", at::kFloat, {T, E});
    a.dense(idx, "idx", at::kInt, {T, k});
    const void* dg = a.dense(5, "dgate", at::kFloat, {T, k}).data_ptr();
    const moe_gate_config c = gate_config(a, 6, E, k);
    void* dl = a.output(a.dict(9), k_dlogits, "dlogits", at::kFloat, {T, E}, true);
    return moe_gate_backward(a.ops, &c, (const float*)l.data_ptr(), (const int32_t*)idx.data_ptr(), (const float*)dg,
                             to_int(T, "logits"), (float*)dl, a.stream);
  });
}

const at::Tensor& bf16_rows(const Args& a, int i, const char* what, long long* ld) {
  const at::Tensor& t = a.tensor(i, what);
  *ld = row_stride(t, what);
  if (t.scalar_type() != at::kBFloat16) refuse(PyExc_TypeError, what, "bf16 expected");
  return t;
}

// src, swiglu, out
PyObject* quant_rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 6);
    long long ld;
    const at::Tensor& src = bf16_rows(a, 3, "src", &ld);
    const int swiglu = PyObject_IsTrue(a.a[4]);
    int64_t T = src.size(0), C = src.size(1);
    if (swiglu) {
      if (C % 2) refuse(PyExc_ValueError, "src", "an even number of columns expected");
      C /= 2;
    }
    PyObject* out = a.dict(5);
    void* q = a.output(out, k_q, "q", at::kFloat8_e4m3fn, {T, C}, true);
    void* s = a.output(out, k_scale, "scale", at::kFloat, {T, blocks(C)}, true);
    return moe_quant_rows(a.ops, src.data_ptr(), ld, to_int(T, "src"), to_int(C, "src"), swiglu, q, (float*)s,
                          a.stream);
  });
}

// Segments that off (None: one) tells, and rows that an index gathers.
int segments(const Args& a, int i) {
  if (!a.given(i)) return 1;
  const at::Tensor& off = a.tensor(i, "off");
  a.dense(off, "off", at::kInt, {off.numel()});
  if (off.numel() < 2) refuse(PyExc_ValueError, "off", "one more value than segments expected");
  return to_int(off.numel() - 1, "off");
}
int64_t indexed(const Args& a, int i, int64_t rows) {
  if (!a.given(i)) return rows;
  const at::Tensor& t = a.tensor(i, "row_index");
  a.dense(t, "row_index", at::kInt, {t.numel()});
  return t.numel();
}

// src, off, row_index, out
PyObject* quant_cols(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 7);
    long long ld;
    const at::Tensor& src = bf16_rows(a, 3, "src", &ld);
    const int64_t rows = src.size(0), C = src.size(1);
    const int G = segments(a, 4), T = to_int(indexed(a, 5, rows), "row_index");
    int Tp = 0;
    const moe_status st = moe_quant_cols_rows(T, G, &Tp);
    if (st != MOE_OK) return st;
    PyObject* out = a.dict(6);
    void* q = a.output(out, k_q, "q", at::kFloat8_e4m3fn, {C, Tp}, true);
    void* s = a.output(out, k_scale, "scale", at::kFloat, {Tp / kBlock, C}, true);
    return moe_quant_cols(a.ops, src.data_ptr(), ld, to_int(rows, "src"), T, to_int(C, "src"),
                          (const int32_t*)address(a, 4, "off"), G, (const int32_t*)address(a, 5, "row_index"), q,
                          (float*)s, a.stream);
  });
}

// w, transpose, out
PyObject* quant_blocks(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 6);
    const at::Tensor& w = a.tensor(3, "w");
    if (w.dim() != 2 && w.dim() != 3) refuse(PyExc_ValueError, "w", "two or three dimensions expected");
    a.dense(w, "w", at::kBFloat16, w.sizes());
    const bool many = w.dim() == 3;
    const int64_t G = many ? w.size(0) : 1, N = w.size(-2), K = w.size(-1);
    PyObject* out = a.dict(5);
    const auto get = [&](PyObject* key, const char* what, at::ScalarType type, int64_t r, int64_t c) {
      return many ? a.output(out, key, what, type, {G, r, c}, true) : a.output(out, key, what, type, {r, c}, true);
    };
    void* q = get(k_q, "q", at::kFloat8_e4m3fn, N, K);
    void* s = get(k_scale, "scale", at::kFloat, blocks(N), blocks(K));
    void *qt = nullptr, *st = nullptr;
    if (PyObject_IsTrue(a.a[4])) {
      qt = get(k_qt, "qt", at::kFloat8_e4m3fn, K, N);
      st = get(k_scale_t, "scale_t", at::kFloat, blocks(K), blocks(N));
    }
    return moe_quant_blocks(a.ops, w.data_ptr(), to_int(G, "w"), to_int(N, "w"), to_int(K, "w"), q, (float*)s, qt,
                            (float*)st, a.stream);
  });
}

// a, a_scale, b, b_scale, off, row_index, out
PyObject* fp8_matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 10);
    const at::Tensor &x = a.tensor(3, "a"), &b = a.tensor(5, "b");
    const bool many = a.given(7);
    if (x.dim() != 2 || b.dim() != (many ? 3 : 2))
      refuse(PyExc_ValueError, "a, b", "a: two dimensions, b: two, with off three, expected");
    const int64_t rows = x.size(0), K = x.size(1), N = b.size(-2);
    const int G = segments(a, 7);
    a.dense(x, "a", at::kFloat8_e4m3fn, {rows, K});
    const void* sa = a.dense(4, "a_scale", at::kFloat, {rows, blocks(K)}).data_ptr();
    const at::Tensor& sb = a.tensor(6, "b_scale");
    if (many) {
      a.dense(b, "b", at::kFloat8_e4m3fn, {G, N, K});
      a.dense(sb, "b_scale", at::kFloat, {G, blocks(N), blocks(K)});
    } else {
      a.dense(b, "b", at::kFloat8_e4m3fn, {N, K});
      a.dense(sb, "b_scale", at::kFloat, {blocks(N), blocks(K)});
    }
    const int M = to_int(indexed(a, 8, rows), "row_index");
    const at::Tensor& out = a.tensor(9, "out");
    const int dt = dtype_of(out, "out");
    a.dense(out, "out", out.scalar_type(), {M, N});
    at::Tensor ws;
    void* scratch = nullptr;
    if (a.given(8)) {
      size_t bytes = 0;
      const moe_status st = moe_fp8_matmul_workspace_size(M, G, to_int(K, "a"), 1, &bytes);
      if (st != MOE_OK) return st;
      if (bytes) {
        ws = at::empty({(int64_t)bytes}, a.opts.dtype(at::kByte));
        scratch = ws.data_ptr();
      }
    }
    return moe_fp8_matmul(a.ops, x.data_ptr(), (const float*)sa, to_int(rows, "a"),
                          (const int32_t*)address(a, 8, "row_index"), M, b.data_ptr(), (const float*)sb.data_ptr(),
                          (const int32_t*)address(a, 7, "off"), G, to_int(N, "b"), to_int(K, "a"), out.data_ptr(), dt,
                          scratch, a.stream);
  });
}

// dct, dct_scale, xt, xt_scale, off, tokens (None: the most), out
PyObject* fp8_wgrad(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 10);
    const at::Tensor &d = a.tensor(3, "dct"), &x = a.tensor(5, "xt");
    if (d.dim() != 2 || x.dim() != 2) refuse(PyExc_ValueError, "dct, xt", "two dimensions expected");
    const int64_t N = d.size(0), Tp = d.size(1), K = x.size(0);
    const int G = segments(a, 7);
    const int64_t T = a.given(8) ? a.integer(8) : Tp - (G > 1 ? G * kBlock : 0);
    int want = 0;
    if (T < 0 || moe_quant_cols_rows(to_int(T, "tokens"), G, &want) != MOE_OK || want != Tp)
      refuse(PyExc_ValueError, "dct", "padded tokens of another number of tokens or segments");
    a.dense(d, "dct", at::kFloat8_e4m3fn, {N, Tp});
    a.dense(x, "xt", at::kFloat8_e4m3fn, {K, Tp});
    const void* sd = a.dense(4, "dct_scale", at::kFloat, {Tp / kBlock, N}).data_ptr();
    const void* sx = a.dense(6, "xt_scale", at::kFloat, {Tp / kBlock, K}).data_ptr();
    const at::Tensor& out = a.tensor(9, "out");
    const int dt = dtype_of(out, "out");
    if (a.given(7)) a.dense(out, "out", out.scalar_type(), {G, N, K});
    else a.dense(out, "out", out.scalar_type(), {N, K});
    return moe_fp8_wgrad(a.ops, d.data_ptr(), (const float*)sd, x.data_ptr(), (const float*)sx, (int)T,
                         (const int32_t*)address(a, 7, "off"), G, to_int(N, "dct"), to_int(K, "xt"), out.data_ptr(),
                         dt, a.stream);
  });
}

// Outputs that a dict names: all of its entries have to be known.
struct Outputs {
  const Args& a;
  PyObject* out;
  Py_ssize_t found = 0;
  void* get(PyObject* key, const char* what, at::ScalarType type, at::IntArrayRef shape) {
    found += PyDict_Contains(out, key) == 1;
    return a.output(out, key, what, type, shape);
  }
  void done() const {
    if (found != PyDict_Size(out)) refuse(PyExc_ValueError, "out", "holds unknown outputs");
  }
};

// gu, out
PyObject* swiglu(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 5);
    long long ld;
    const at::Tensor& gu = bf16_rows(a, 3, "gu", &ld);
    const int64_t T = gu.size(0), f = gu.size(1) / 2, nb = blocks(f);
    if (gu.size(1) % 2 || f == 0) refuse(PyExc_ValueError, "gu", "an even number of columns expected");
    Outputs o{a, a.dict(4)};
    void* act = o.get(k_act, "act", at::kBFloat16, {T, f});
    void* q = o.get(k_q, "q", at::kFloat8_e4m3fn, {T, f});
    void* scale = o.get(k_scale, "scale", at::kFloat, {T, nb});
    void* save = o.get(k_save, "save", at::kFloat8_e4m3fn, {T, 2 * f});
    void* ss = o.get(k_save_scale, "save_scale", at::kFloat, {T, 2 * nb});
    o.done();
    return moe_swiglu_forward(a.ops, gu.data_ptr(), ld, to_int(T, "gu"), to_int(f, "gu"), act, q, (float*)scale, save,
                              (float*)ss, a.stream);
  });
}

// dact, save, save_scale, gate, off, out
PyObject* swiglu_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 9);
    long long ld;
    const at::Tensor& d = bf16_rows(a, 3, "dact", &ld);
    const int64_t T = d.size(0), f = d.size(1), nb = blocks(f);
    const void* save = a.dense(4, "save", at::kFloat8_e4m3fn, {T, 2 * f}).data_ptr();
    const void* ss = a.dense(5, "save_scale", at::kFloat, {T, 2 * nb}).data_ptr();
    const void* gate = a.given(6) ? a.dense(6, "gate", at::kFloat, {T}).data_ptr() : nullptr;
    const int G = segments(a, 7);
    int Tp = 0;
    moe_status st = moe_quant_cols_rows(to_int(T, "dact"), G, &Tp);
    if (st != MOE_OK) return st;
    Outputs o{a, a.dict(8)};
    const at::ScalarType f8 = at::kFloat8_e4m3fn;
    void* dgu = o.get(k_dgu, "dgu", at::kBFloat16, {T, 2 * f});
    void* dq = o.get(k_dq, "dq", f8, {T, 2 * f});
    void* dqs = o.get(k_dq_scale, "dq_scale", at::kFloat, {T, 2 * nb});
    void* dqt = o.get(k_dqt, "dqt", f8, {2 * f, Tp});
    void* dqts = o.get(k_dqt_scale, "dqt_scale", at::kFloat, {Tp / kBlock, 2 * f});
    void* actt = o.get(k_actt, "actt", f8, {f, Tp});
    void* actts = o.get(k_actt_scale, "actt_scale", at::kFloat, {Tp / kBlock, f});
    void* dgate = o.get(k_dgate, "dgate", at::kFloat, {T});
    o.done();
    at::Tensor ws;
    void* scratch = nullptr;
    if (dgate) {
      size_t bytes = 0;
      st = moe_swiglu_workspace_size((int)T, to_int(f, "dact"), &bytes);
      if (st != MOE_OK) return st;
      if (bytes) {
        ws = at::empty({(int64_t)bytes}, a.opts.dtype(at::kByte));
        scratch = ws.data_ptr();
      }
    }
    return moe_swiglu_backward(a.ops, save, (const float*)ss, d.data_ptr(), ld, (const float*)gate, (int)T,
                               to_int(f, "dact"), (const int32_t*)address(a, 7, "off"), G, dgu, dq, (float*)dqs, dqt,
                               (float*)dqts, actt, (float*)actts, (float*)dgate, scratch, a.stream);
  });
}

// q, scale, off, row_index, out
PyObject* requant_cols(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 8);
    const at::Tensor& q = a.tensor(3, "q");
    if (q.dim() != 2) refuse(PyExc_ValueError, "q", "two dimensions expected");
    const int64_t rows = q.size(0), C = q.size(1);
    a.dense(q, "q", at::kFloat8_e4m3fn, {rows, C});
    const void* scale = a.dense(4, "scale", at::kFloat, {rows, blocks(C)}).data_ptr();
    const int G = segments(a, 5), T = to_int(indexed(a, 6, rows), "row_index");
    int Tp = 0;
    const moe_status st = moe_quant_cols_rows(T, G, &Tp);
    if (st != MOE_OK) return st;
    PyObject* out = a.dict(7);
    void* qt = a.output(out, k_q, "q", at::kFloat8_e4m3fn, {C, Tp}, true);
    void* s = a.output(out, k_scale, "scale", at::kFloat, {Tp / kBlock, C}, true);
    return moe_requant_cols(a.ops, q.data_ptr(), (const float*)scale, to_int(rows, "q"), T, to_int(C, "q"),
                            (const int32_t*)address(a, 5, "off"), G, (const int32_t*)address(a, 6, "row_index"), qt,
                            (float*)s, a.stream);
  });
}

// Entry `key` of a dict of 4-bit weights (null if missing or None).
PyObject* entry(PyObject* w, PyObject* key) {
  PyObject* o = PyDict_GetItemWithError(w, key);
  if (!o && PyErr_Occurred()) throw Refused();
  return o == Py_None ? nullptr : o;
}

// 4-bit weights as quant_w4 returns them: [N, K], or (many) [G, N, K].
moe_w4 weights4(const Args& a, int i, const char* what, bool many, int64_t* G, int64_t* N, int64_t* K) {
  if (!PyDict_Check(a.a[i])) refuse(PyExc_TypeError, what, "a dict of codes, scale and group expected");
  PyObject *codes = entry(a.a[i], k_codes), *scale = entry(a.a[i], k_scale), *zero = entry(a.a[i], k_zero),
           *group = entry(a.a[i], k_group);
  if (!codes || !scale || !group) refuse(PyExc_ValueError, what, "codes, scale and group expected");
  const at::Tensor &c = a.tensor(codes, "codes"), &s = a.tensor(scale, "scale");
  if (c.dim() != (many ? 3 : 2)) refuse(PyExc_ValueError, what, many ? "three dimensions expected" : "two dimensions expected");
  moe_w4 w = {};
  const int64_t g = PyLong_AsLongLong(group);
  if (g == -1 && PyErr_Occurred()) throw Refused();
  if (g != 32 && g != 64 && g != 128) refuse(PyExc_ValueError, what, "groups of 32, 64 or 128 expected");
  w.group = (int)g;
  *G = many ? c.size(0) : 1;
  *N = c.size(-2);
  *K = c.size(-1) * 8;
  const int64_t KG = (*K + g - 1) / g;
  const auto check = [&](const at::Tensor& t, const char* name, at::ScalarType type, int64_t r, int64_t q) {
    if (many) a.dense(t, name, type, {*G, r, q});
    else a.dense(t, name, type, {r, q});
    return t.data_ptr();
  };
  w.codes = (const uint32_t*)check(c, "codes", at::kInt, *N, c.size(-1));
  w.scale = check(s, "scale", at::kBFloat16, KG, *N);
  if (zero) w.zero = (const uint8_t*)check(a.tensor(zero, "zero"), "zero", at::kByte, KG, *N);
  return w;
}

// w, group, zero, out
PyObject* quant_w4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 7);
    const at::Tensor& w = a.tensor(3, "w");
    if (w.dim() != 2 && w.dim() != 3) refuse(PyExc_ValueError, "w", "two or three dimensions expected");
    a.dense(w, "w", at::kBFloat16, w.sizes());
    const bool many = w.dim() == 3;
    const int64_t G = many ? w.size(0) : 1, N = w.size(-2), K = w.size(-1), g = a.integer(4);
    if (g != 32 && g != 64 && g != 128) refuse(PyExc_ValueError, "group", "32, 64 or 128 expected");
    if (K % 32) refuse(PyExc_ValueError, "w", "a multiple of 32 columns expected");
    PyObject* out = a.dict(6);
    const auto get = [&](PyObject* key, const char* what, at::ScalarType type, int64_t r, int64_t c) {
      return many ? a.output(out, key, what, type, {G, r, c}, true) : a.output(out, key, what, type, {r, c}, true);
    };
    const int64_t KG = (K + g - 1) / g;
    void* codes = get(k_codes, "codes", at::kInt, N, K / 8);
    void* scale = get(k_scale, "scale", at::kBFloat16, KG, N);
    const int points = PyObject_IsTrue(a.a[5]);
    if (points < 0) throw Refused();
    if (!points && entry(out, k_zero)) refuse(PyExc_ValueError, "out", "holds zero points that the weights would not have");
    void* zero = points ? get(k_zero, "zero", at::kByte, KG, N) : nullptr;
    return moe_quant_w4(a.ops, w.data_ptr(), to_int(G, "w"), to_int(N, "w"), to_int(K, "w"), (int)g, (uint32_t*)codes,
                        scale, (uint8_t*)zero, a.stream);
  });
}

// x, w, off, row_index, out
PyObject* w4_matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 8);
    long long ld;
    const at::Tensor& x = bf16_rows(a, 3, "x", &ld);
    const bool many = a.given(5);
    int64_t G, N, K;
    const moe_w4 w = weights4(a, 4, "w", many, &G, &N, &K);
    const int64_t rows = x.size(0);
    if (x.size(1) != K) refuse_shape("x", x, {rows, K});
    if (many && segments(a, 5) != G) refuse(PyExc_ValueError, "off", "one more value than matrices expected");
    const int M = to_int(indexed(a, 6, rows), "row_index");
    const at::Tensor& out = a.tensor(7, "out");
    const int dt = dtype_of(out, "out");
    a.dense(out, "out", out.scalar_type(), {M, N});
    return moe_w4_matmul(a.ops, x.data_ptr(), ld, to_int(rows, "x"), (const int32_t*)address(a, 6, "row_index"), M, &w,
                         (const int32_t*)address(a, 5, "off"), to_int(G, "w"), to_int(N, "w"), to_int(K, "w"),
                         out.data_ptr(), dt, a.stream);
  });
}

// x, idx, gate, w13, wd, n_shared, out
PyObject* w4_experts(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 10);
    long long ld;
    const at::Tensor &x = bf16_rows(a, 3, "x", &ld), &idx = a.tensor(4, "idx");
    if (idx.dim() != 2) refuse(PyExc_ValueError, "idx", "two dimensions expected");
    const int64_t T = x.size(0), k = idx.size(1), shared = a.integer(8);
    int64_t G, N, d, Gd, Nd, f;
    const moe_w4 w13 = weights4(a, 6, "w13", true, &G, &N, &d), wd = weights4(a, 7, "wd", true, &Gd, &Nd, &f);
    if (x.size(1) != d) refuse_shape("x", x, {T, d});
    if (Gd != G || Nd != d || N != 2 * f) refuse(PyExc_ValueError, "w13, wd", "matrices [E, 2f, d] and [E, d, f] expected");
    if (shared < 0 || shared >= G) refuse(PyExc_ValueError, "n_shared", "fewer than the experts expected");
    a.dense(idx, "idx", at::kInt, {T, k});
    const void* gate = a.dense(5, "gate", at::kFloat, {T, k}).data_ptr();
    const at::Tensor& out = a.tensor(9, "out");
    const int dt = dtype_of(out, "out");
    a.dense(out, "out", out.scalar_type(), {T, d});
    const moe_w4_config c = {to_int(G - shared, "w13"), (int)shared, to_int(k, "idx"), to_int(d, "w13"), to_int(f, "wd")};
    size_t bytes = 0;
    const moe_status st = moe_w4_experts_workspace_size(&c, to_int(T, "x"), &bytes);
    if (st != MOE_OK) return st;
    at::Tensor ws = at::empty({(int64_t)bytes}, a.opts.dtype(at::kByte));
    return moe_w4_experts(a.ops, &c, x.data_ptr(), ld, (int)T, (const int32_t*)idx.data_ptr(), (const float*)gate, &w13,
                          &wd, out.data_ptr(), dt, ws.data_ptr(), a.stream);
  });
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(norm_forward), METHOD(norm_backward), METHOD(gate),         METHOD(gate_backward),
                         METHOD(quant_rows),   METHOD(quant_cols),    METHOD(quant_blocks), METHOD(fp8_matmul),
                         METHOD(fp8_wgrad),    METHOD(quant_w4),      METHOD(w4_matmul),    METHOD(w4_experts),
                         METHOD(swiglu),       METHOD(swiglu_backward), METHOD(requant_cols), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_ops_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops_binding() {
  const struct { PyObject** key; const char* name; } keys[] = {
      {&k_h, "h"}, {&k_y, "y"}, {&k_q, "q"}, {&k_scale, "scale"}, {&k_rstd, "rstd"}, {&k_dx, "dx"}, {&k_dw, "dw"},
      {&k_idx, "idx"}, {&k_gate, "gate"}, {&k_cnt, "cnt"}, {&k_off, "off"}, {&k_perm, "perm"}, {&k_inv, "inv"},
      {&k_dlogits, "dlogits"}, {&k_qt, "qt"}, {&k_scale_t, "scale_t"}, {&k_codes, "codes"},
      {&k_zero, "zero"}, {&k_group, "group"}, {&k_act, "act"}, {&k_save, "save"}, {&k_save_scale, "save_scale"},
      {&k_dgu, "dgu"}, {&k_dq, "dq"}, {&k_dq_scale, "dq_scale"}, {&k_dqt, "dqt"}, {&k_dqt_scale, "dqt_scale"},
      {&k_actt, "actt"}, {&k_actt_scale, "actt_scale"}, {&k_dgate, "dgate"}};
  for (const auto& k : keys)
    if (!(*k.key = PyUnicode_InternFromString(k.name))) return nullptr;
  return PyModule_Create(&module_def);
}
