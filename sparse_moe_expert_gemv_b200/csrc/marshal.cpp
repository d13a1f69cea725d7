// marshal.cpp -- argument marshalling of the attention calls (binding.py).
//
// A window's append or attention takes a few microseconds on the GPU; reading
// the shapes, strides and addresses of its tensors through Python attributes
// and a ctypes call takes twice that.  These functions check the tensors
// against the context's geometry (the library sees addresses only) and make
// the call.  The entry points' addresses come from binding.py (set_calls), so
// nothing here links against libmoe.so.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "../../include/moe.h"

namespace {

decltype(&moe_qk_norm_rope) p_qk_norm_rope;
decltype(&moe_kv_append) p_kv_append;
decltype(&moe_attn_forward) p_attn[2];

struct Rows {
  void *p = nullptr;
  int64_t stride = 0;
};

// Rows [n, heads, dim] (or [n, heads * dim]) of bf16 on `device`,
// dense within a row.  False with a Python error set otherwise.
bool rows(const char *name, PyObject *o, long n, long heads, long dim, long device, Rows *out) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_ValueError, "%s: a torch tensor", name);
    return false;
  }
  const at::Tensor &t = THPVariable_Unpack(o);
  const int64_t k = t.dim();
  bool ok = (k == 2 || k == 3) && t.is_cuda() && t.scalar_type() == at::kBFloat16 && t.size(0) >= n &&
            t.stride(k - 1) == 1;
  if (ok)
    ok = k == 3 ? t.size(1) == heads && t.size(2) == dim && (heads == 1 || t.stride(1) == dim)
                : t.size(1) == heads * dim;
  if (!ok) {
    PyErr_Format(PyExc_ValueError, "%s: bf16 rows [%ld, %ld, %ld] on the GPU, dense within a row", name, n, heads,
                 dim);
    return false;
  }
  if (t.get_device() != device) {
    PyErr_Format(PyExc_ValueError, "%s: a tensor on the context's device (cuda:%ld)", name, device);
    return false;
  }
  out->p = t.data_ptr();
  out->stride = t.size(0) > 1 ? t.stride(0) : heads * dim;  // the stride of a single row means nothing
  return true;
}

struct Args {
  PyObject *const *a;
  bool bad = false;
  long num(int i) {
    const long v = PyLong_AsLong(a[i]);
    if (v == -1 && PyErr_Occurred()) bad = true;
    return v;
  }
  int num32(int i) {
    const long v = num(i);
    if (v != (int)v) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "an argument does not fit 32 bits");
      bad = true;
    }
    return (int)v;
  }
  void *ptr(int i) {  // None: null
    if (a[i] == Py_None) return nullptr;
    void *v = PyLong_AsVoidPtr(a[i]);
    if (!v && PyErr_Occurred()) bad = true;
    return v;
  }
  float real(int i) {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) bad = true;
    return (float)v;
  }
};

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
  return false;
}

// A tensor whose sizes or memory are not plain numbers (symbolic, nested,
// without storage) throws when it is asked for them: a Python error, since
// nothing may be thrown through the interpreter's C frames.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  try {
    return F(self, a, na);
  } catch (const std::exception &e) {
    PyErr_Format(PyExc_ValueError, "not a plain CUDA tensor: %s", e.what());
  } catch (...) {
    PyErr_SetString(PyExc_ValueError, "not a plain CUDA tensor");
  }
  return nullptr;
}

// (n_q, n_kv, dim, device, ctx, n_rows, q, k, pos, norm, rope, q_out, k_out, stream)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t na) {
  if (!count(na, 14)) return nullptr;
  Args g{a};
  const long n_q = g.num(0), n_kv = g.num(1), dim = g.num(2), dev = g.num(3);
  auto *ctx = (moe_ctx *)g.ptr(4);
  const int n = g.num32(5);
  auto *norm = (const moe_qk_norm *)g.ptr(9);
  auto *rope = (const moe_rope *)g.ptr(10);
  void *stream = g.ptr(13);
  if (g.bad) return nullptr;
  const int32_t *pos = nullptr;
  if (a[8] != Py_None) {
    bool ok = THPVariable_Check(a[8]);
    if (ok) {
      const at::Tensor &t = THPVariable_Unpack(a[8]);
      ok = t.is_cuda() && t.scalar_type() == at::kInt && t.is_contiguous() && t.numel() >= n && t.get_device() == dev;
      if (ok) pos = (const int32_t *)t.data_ptr();
    }
    if (!ok) return PyErr_Format(PyExc_ValueError, "pos: contiguous int32 [%d] on cuda:%ld", n, dev);
  }
  Rows q, k, qo, ko;
  if (!rows("q", a[6], n, n_q, dim, dev, &q) || !rows("k", a[7], n, n_kv, dim, dev, &k) ||
      !rows("q_out", a[11], n, n_q, dim, dev, &qo) || !rows("k_out", a[12], n, n_kv, dim, dev, &ko))
    return nullptr;
  return PyLong_FromLong(p_qk_norm_rope(ctx, n, q.p, q.stride, k.p, k.stride, pos, norm, rope, qo.p, qo.stride, ko.p,
                                        ko.stride, stream));
}

// (n_q, n_kv, dim, device, ctx, n_rows, batch, q, k, v, norm, rope, q_out, stream)
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t na) {
  if (!count(na, 14)) return nullptr;
  Args g{a};
  const long n_q = g.num(0), n_kv = g.num(1), dim = g.num(2), dev = g.num(3);
  auto *ctx = (moe_ctx *)g.ptr(4);
  const int n = g.num32(5);
  auto *batch = (const moe_kv_batch *)g.ptr(6);
  auto *norm = (const moe_qk_norm *)g.ptr(10);
  auto *rope = (const moe_rope *)g.ptr(11);
  void *stream = g.ptr(13);
  if (g.bad) return nullptr;
  Rows q, k, v, qo;
  if ((a[7] != Py_None && !rows("q", a[7], n, n_q, dim, dev, &q)) || !rows("k", a[8], n, n_kv, dim, dev, &k) ||
      !rows("v", a[9], n, n_kv, dim, dev, &v) || (a[12] != Py_None && !rows("q_out", a[12], n, n_q, dim, dev, &qo)))
    return nullptr;
  return PyLong_FromLong(p_kv_append(ctx, batch, q.p, q.stride, k.p, k.stride, v.p, v.stride, norm, rope, qo.p,
                                     qo.stride, stream));
}

// (chunk, n_q, dim, device, ctx, n_rows, batch, q, max_T, scale, window, n_sink, out, stream)
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t na) {
  if (!count(na, 14)) return nullptr;
  Args g{a};
  const long chunk = g.num(0), n_q = g.num(1), dim = g.num(2), dev = g.num(3);
  auto *ctx = (moe_ctx *)g.ptr(4);
  const int n = g.num32(5);
  auto *batch = (const moe_kv_batch *)g.ptr(6);
  const int max_T = g.num32(8);
  const float scale = g.real(9);
  const int window = g.num32(10), n_sink = g.num32(11);
  void *stream = g.ptr(13);
  if (g.bad) return nullptr;
  Rows q, out;
  if (!rows("q", a[7], n, n_q, dim, dev, &q) || !rows("out", a[12], n, n_q, dim, dev, &out)) return nullptr;
  return PyLong_FromLong(p_attn[chunk != 0](ctx, batch, q.p, q.stride, max_T, scale, window, n_sink, out.p,
                                            out.stride, stream));
}

// (moe_qk_norm_rope, moe_kv_append, moe_attn_forward, moe_attn_prefill): their addresses
PyObject *set_calls(PyObject *, PyObject *const *a, Py_ssize_t na) {
  if (!count(na, 4)) return nullptr;
  Args g{a};
  void *f[4];
  for (int i = 0; i < 4; ++i) f[i] = g.ptr(i);
  if (g.bad) return nullptr;
  p_qk_norm_rope = (decltype(p_qk_norm_rope))f[0];
  p_kv_append = (decltype(p_kv_append))f[1];
  p_attn[0] = (decltype(p_attn[0]))f[2];
  p_attn[1] = (decltype(p_attn[1]))f[3];
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"qk_norm_rope", (PyCFunction)(void *)guarded<qk_norm_rope>, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void *)guarded<kv_append>, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void *)guarded<attend>, METH_FASTCALL, nullptr},
    {"set_calls", (PyCFunction)(void *)set_calls, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
