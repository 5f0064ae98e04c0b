// Python calls of the serving operators (module _serve): argument checks,
// outputs and the library call in one native function each. A decode step
// makes these calls every few microseconds, which is what their checks would
// take in Python. Every arithmetic step runs in the library; torch provides
// device memory and streams.
//
// Arguments come by position from the functions of the package's
// __init__.py, which document them. Errors: TypeError, ValueError, and the
// package's LqmmError for a status of the library (through the callable that
// `setup` is given).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "lqmm.h"

namespace {

PyObject *g_raise_status = nullptr;  // raises the package's error for a status
PyObject *g_raw_stream = nullptr;    // current stream's handle of a device index
PyObject *g_workspace_on = nullptr;  // workspace for (device index, stream, bytes)

struct Failed {};  // a Python error is set

[[noreturn]] void type_error(const char *format, const char *name) {
  PyErr_Format(PyExc_TypeError, format, name);
  throw Failed();
}
[[noreturn]] void value_error(const char *format, const char *name) {
  PyErr_Format(PyExc_ValueError, format, name);
  throw Failed();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) type_error("%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

const at::Tensor &on_device(const at::Tensor &t, const char *name) {
  if (!t.is_cuda()) value_error("%s must be a device tensor", name);
  return t;
}

// A contiguous device tensor of the given element type.
const at::Tensor &whole(PyObject *o, at::ScalarType type, const char *name) {
  const at::Tensor &t = on_device(tensor(o, name), name);
  if (t.scalar_type() != type) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, at::toString(type),
                 at::toString(t.scalar_type()));
    throw Failed();
  }
  if (!t.is_contiguous()) value_error("%s must be contiguous", name);
  return t;
}

int type_code(const at::Tensor &t, const char *name, bool f32) {
  switch (t.scalar_type()) {
    case at::kFloat: if (f32) return LQMM_F32; break;
    case at::kHalf: return LQMM_F16;
    case at::kBFloat16: return LQMM_BF16;
    default: break;
  }
  PyErr_Format(PyExc_TypeError, "%s has element type %s, which this call does not take", name,
               at::toString(t.scalar_type()));
  throw Failed();
}

void same_device(const at::Tensor &a, const at::Tensor &b) {
  if (a.get_device() != b.get_device()) {
    PyErr_SetString(PyExc_ValueError, "all tensors must be on the same device");
    throw Failed();
  }
}

// (tokens, heads, dim) with contiguous rows: its row stride in elements.
int64_t row_stride(const at::Tensor &t, int64_t heads, int64_t dim, const char *name) {
  on_device(t, name);
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != dim) {
    PyErr_Format(PyExc_ValueError, "%s must be (tokens, %lld, %lld)", name, (long long)heads,
                 (long long)dim);
    throw Failed();
  }
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != dim))
    value_error("the heads of one token of %s must be contiguous", name);
  return t.size(0) > 1 ? t.stride(0) : heads * dim;
}

struct Caches {
  const at::Tensor &k, &v;
  int64_t pages, heads, page_size, dim;
  int type;
};

Caches caches(PyObject *ko, PyObject *vo) {
  const at::Tensor &kt = tensor(ko, "k_cache");
  const at::Tensor &k = whole(ko, kt.scalar_type(), "k_cache");
  const at::Tensor &v = whole(vo, kt.scalar_type(), "v_cache");
  if (k.dim() != 4) value_error("%s must be (num_pages, n_kv_heads, page_size, head_dim)", "k_cache");
  const int64_t p = k.size(0), h = k.size(1), ps = k.size(2), d = k.size(3);
  if (ps % 8 != 0 || v.dim() != 5 || v.size(0) != p || v.size(1) != h || v.size(2) != ps / 8 ||
      v.size(3) != d || v.size(4) != 8)
    value_error("%s must be (num_pages, n_kv_heads, page_size / 8, head_dim, 8)", "v_cache");
  same_device(k, v);
  return {k, v, p, h, ps, d, type_code(k, "k_cache", false)};
}

bool has_shape(const at::Tensor &t, std::initializer_list<int64_t> want) {
  return t.sizes() == at::IntArrayRef(want.begin(), want.size());
}

int64_t integer(PyObject *o, const char *name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    PyObject *i = PyNumber_Index(o);
    if (!i) {
      PyErr_Clear();
      type_error("%s must be an integer", name);
    }
    const long long w = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (w == -1 && PyErr_Occurred()) throw Failed();
    return w;
  }
  return v;
}

// The stream's handle: of the argument (None: the device's current one).
void *stream_of(PyObject *o, const at::Tensor &t) {
  PyObject *v;
  if (o == Py_None) {
    PyObject *i = PyLong_FromLong(t.get_device());
    if (!i) throw Failed();
    v = PyObject_CallFunctionObjArgs(g_raw_stream, i, nullptr);
    Py_DECREF(i);
  } else if (PyLong_Check(o)) {
    const unsigned long long h = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) throw Failed();  // (no handle: negative or too wide)
    return reinterpret_cast<void *>((uintptr_t)h);
  } else {
    v = PyObject_GetAttrString(o, "cuda_stream");
  }
  if (!v) throw Failed();
  void *p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!p && PyErr_Occurred()) throw Failed();
  return p;
}

void check(lqmm_status st) {
  if (st == LQMM_OK) return;
  PyObject *r = PyObject_CallFunction(g_raise_status, "i", (int)st);
  if (r) {
    Py_DECREF(r);
    PyErr_SetString(PyExc_RuntimeError, "the library reported an error");
  }
  throw Failed();
}

// The library call without the interpreter's lock, on the tensors' device.
template <class F>
lqmm_status call(F f) {
  PyThreadState *s = PyEval_SaveThread();
  const lqmm_status st = f();
  PyEval_RestoreThread(s);
  return st;
}

// Runs a binding's body; C++ errors (torch's allocation among them) become
// Python's.
template <class F>
PyObject *guarded(F f) {
  try {
    return f();
  } catch (const Failed &) {
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject * {
    PyObject *qo = a[0], *po = a[3], *turns_o = a[7], *out_o = a[9];
    const Caches c = caches(a[5], a[6]);
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const int64_t ldk = row_stride(k, c.heads, c.dim, "k"), ldv = row_stride(v, c.heads, c.dim, "v");
    const int64_t tokens = k.size(0);
    const int type = type_code(k, "k", true);
    if (v.scalar_type() != k.scalar_type() || v.size(0) != tokens)
      value_error("%s must have the same element type and tokens", "k and v");
    const at::Tensor &slots = whole(a[4], at::kLong, "slots");
    if (slots.numel() != tokens) value_error("%s must have one entry per token", "slots");
    same_device(k, v);
    same_device(k, slots);
    same_device(k, c.k);
    int64_t rot = 0;
    const void *positions = nullptr, *turns = nullptr;
    if (turns_o != Py_None) {
      const at::Tensor &tt = whole(turns_o, at::kLong, "rope_turns");
      const at::Tensor &pt = whole(po, at::kInt, "positions");
      if (pt.numel() != tokens) value_error("%s must have one entry per token", "positions");
      same_device(k, tt);
      same_device(k, pt);
      rot = 2 * tt.numel();
      positions = pt.data_ptr();
      turns = tt.data_ptr();
    }
    const int interleaved = PyObject_IsTrue(a[8]);
    if (interleaved < 0) throw Failed();
    const c10::DeviceGuard guard(k.device());
    int64_t heads = 0, ldq = 0;
    const void *qp = nullptr;
    at::Tensor out;
    if (qo != Py_None) {
      const at::Tensor &q = tensor(qo, "q");
      if (q.dim() != 3) value_error("%s must be (tokens, n_q_heads, head_dim)", "q");
      heads = q.size(1);
      ldq = row_stride(q, heads, c.dim, "q");
      if (q.scalar_type() != k.scalar_type() || q.size(0) != tokens)
        value_error("%s must have the same element type and tokens", "q and k");
      same_device(k, q);
      if (out_o == Py_None) {
        out = at::empty({tokens, heads, c.dim}, c.k.options());
      } else {
        out = whole(out_o, c.k.scalar_type(), "q_out");
        if (!has_shape(out, {tokens, heads, c.dim})) value_error("%s has the wrong shape", "q_out");
        same_device(k, out);
      }
      qp = q.data_ptr();
    } else if (out_o != Py_None) {
      value_error("%s without q", "q_out");
    }
    void *stream = stream_of(a[10], k);
    void *outp = out.defined() ? out.data_ptr() : nullptr;
    check(call([&] {
      return lqmm_kv_append(qp, k.data_ptr(), v.data_ptr(), type, ldq, ldk, ldv,
                            static_cast<const int32_t *>(positions),
                            static_cast<const int64_t *>(slots.data_ptr()),
                            static_cast<const uint64_t *>(turns), rot, interleaved, outp,
                            c.k.data_ptr(), c.v.data_ptr(), c.type, tokens, heads, c.heads, c.dim,
                            c.page_size, c.pages, stream);
    }));
    if (!out.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(out);
  });
}

PyObject *attn_prefix(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 15)) return nullptr;
  return guarded([&]() -> PyObject * {
    const at::Tensor &q = tensor(a[0], "q");
    const Caches c = caches(a[1], a[2]);
    if (q.dim() != 3) value_error("%s must be (tokens, n_q_heads, head_dim)", "q");
    const int64_t tokens = q.size(0), heads = q.size(1);
    const int64_t ldq = row_stride(q, heads, c.dim, "q");
    if (q.scalar_type() != c.k.scalar_type()) type_error("%s must have the caches' element type", "q");
    const at::Tensor &pages = whole(a[3], at::kInt, "pages");
    const at::Tensor &lens = whole(a[4], at::kInt, "seq_lens");
    if (pages.dim() != 2 || lens.dim() != 1 || pages.size(0) != lens.size(0))
      value_error("%s must be (batch, max_pages) and seq_lens (batch,)", "pages");
    const int64_t batch = pages.size(0), max_pages = pages.size(1);
    same_device(q, c.k);
    same_device(q, pages);
    same_device(q, lens);
    const int64_t prefix_len = integer(a[6], "prefix_len"), max_q = integer(a[8], "max_q");
    const int32_t *prefix = nullptr, *start = nullptr;
    if (prefix_len != 0) {
      const at::Tensor &p = whole(a[5], at::kInt, "prefix_pages");
      if (p.numel() * c.page_size < prefix_len)
        value_error("%s hold fewer than prefix_len tokens", "prefix_pages");
      same_device(q, p);
      prefix = static_cast<const int32_t *>(p.data_ptr());
    }
    if (a[7] != Py_None) {
      const at::Tensor &s = whole(a[7], at::kInt, "q_start");
      if (s.numel() != batch + 1) value_error("%s must have batch + 1 entries", "q_start");
      same_device(q, s);
      start = static_cast<const int32_t *>(s.data_ptr());
    }
    double scale;
    if (a[9] == Py_None) {
      scale = 1.0 / std::sqrt((double)c.dim);
    } else {
      scale = PyFloat_AsDouble(a[9]);
      if (scale == -1.0 && PyErr_Occurred()) throw Failed();
    }
    const c10::DeviceGuard guard(q.device());
    at::Tensor out, lse;
    if (a[10] == Py_None) {
      out = at::empty({tokens, heads, c.dim}, q.options());
    } else {
      out = whole(a[10], q.scalar_type(), "out");
      if (!has_shape(out, {tokens, heads, c.dim})) value_error("%s has the wrong shape", "out");
      same_device(q, out);
    }
    const int want_lse = PyObject_IsTrue(a[11]);
    if (want_lse < 0) throw Failed();
    if (a[12] != Py_None) {
      lse = whole(a[12], at::kFloat, "lse");
      if (lse.numel() != tokens * heads) value_error("%s has the wrong size", "lse");
      same_device(q, lse);
    } else if (want_lse) {
      lse = at::empty({tokens, heads}, q.options().dtype(at::kFloat));
    }
    void *stream = stream_of(a[14], q);
    void *ws = nullptr;
    size_t ws_bytes = 0;
    at::Tensor scratch;
    if (a[13] != Py_None) {
      const at::Tensor &w = whole(a[13], at::kByte, "workspace");
      same_device(q, w);
      ws = w.data_ptr();
      ws_bytes = (size_t)w.numel();
    } else {
      const size_t need = lqmm_attn_prefix_workspace_bytes(prefix_len, max_pages, max_q, tokens, batch,
                                                           heads, c.heads, c.dim, c.page_size);
      // Its own workspace for every call, from the allocator's memory of the
      // stream it runs on: freed behind the launches, it is handed out again in
      // stream order, to whatever thread, and a graph under capture has its own.
      if (need && (a[14] == Py_None || stream == stream_of(Py_None, q))) {
        scratch = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
      } else if (need) {
        PyObject *w = PyObject_CallFunction(g_workspace_on, "iOK", (int)q.get_device(), a[14],
                                            (unsigned long long)need);
        if (!w) throw Failed();
        scratch = THPVariable_Unpack(w);
        Py_DECREF(w);
      }
      if (need) {
        ws = scratch.data_ptr();
        ws_bytes = (size_t)scratch.numel();
      }
    }
    float *lse_p = lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr;
    check(call([&] {
      return lqmm_attn_prefix(q.data_ptr(), ldq, c.k.data_ptr(), c.v.data_ptr(), c.type, prefix,
                              prefix_len, static_cast<const int32_t *>(pages.data_ptr()), max_pages,
                              static_cast<const int32_t *>(lens.data_ptr()), start, max_q,
                              out.data_ptr(), lse_p, (float)scale, tokens, batch, heads, c.heads,
                              c.dim, c.page_size, c.pages, ws, ws_bytes, stream);
    }));
    PyObject *r = THPVariable_Wrap(out);
    if (!r || !lse.defined()) return r;
    PyObject *l = THPVariable_Wrap(lse);
    PyObject *both = l ? PyTuple_Pack(2, r, l) : nullptr;
    Py_DECREF(r);
    Py_XDECREF(l);
    return both;
  });
}

// A 2-D contiguous device tensor of e4m3 codes (float8_e4m3fn or raw bytes).
const at::Tensor &codes(PyObject *o, const char *name) {
  if (!THPVariable_Check(o) || (THPVariable_Unpack(o).scalar_type() != at::kFloat8_e4m3fn &&
                                THPVariable_Unpack(o).scalar_type() != at::kByte))
    type_error("%s must be a float8_e4m3fn (or uint8) torch.Tensor", name);
  const at::Tensor &t = whole(o, THPVariable_Unpack(o).scalar_type(), name);
  if (t.dim() != 2) value_error("%s must be 2-D", name);
  return t;
}

PyObject *quant_f8b128(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 4)) return nullptr;
  return guarded([&]() -> PyObject * {
    const at::Tensor &x = on_device(tensor(a[0], "X"), "X");
    if (x.dim() != 2) value_error("%s must be (M, K)", "X");
    const int64_t M = x.size(0), K = x.size(1), blocks = (K + 127) / 128;
    if (K > 1 && x.stride(1) != 1) value_error("the rows of %s must be contiguous", "X");
    const int type = type_code(x, "X", true);
    const c10::DeviceGuard guard(x.device());
    at::Tensor out, scales;
    if (a[1] == Py_None) {
      out = at::empty({M, K}, x.options().dtype(at::kFloat8_e4m3fn));
    } else {
      out = codes(a[1], "out");
      if (!has_shape(out, {M, K})) value_error("%s has the wrong shape", "out");
      same_device(x, out);
    }
    if (a[2] == Py_None) {
      scales = at::empty({blocks, M}, x.options().dtype(at::kFloat));
    } else {
      scales = whole(a[2], at::kFloat, "scales");
      if (!has_shape(scales, {blocks, M})) value_error("%s has the wrong shape", "scales");
      same_device(x, scales);
    }
    void *stream = stream_of(a[3], x);
    check(call([&] {
      return lqmm_quant_f8b128(x.data_ptr(), type, M > 1 ? x.stride(0) : K,
                               static_cast<uint8_t *>(out.data_ptr()),
                               static_cast<float *>(scales.data_ptr()), M, K, stream);
    }));
    PyObject *p = THPVariable_Wrap(out), *s = THPVariable_Wrap(scales);
    PyObject *both = p && s ? PyTuple_Pack(2, p, s) : nullptr;
    Py_XDECREF(p);
    Py_XDECREF(s);
    return both;
  });
}

PyObject *gemm_f8b128(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 7)) return nullptr;
  return guarded([&]() -> PyObject * {
    const at::Tensor &w = codes(a[0], "W"), &x = codes(a[2], "Xq");
    const at::Tensor &ws = whole(a[1], at::kFloat, "wscale"), &xs = whole(a[3], at::kFloat, "xscale");
    const int64_t N = w.size(0), K = w.size(1), M = x.size(0), blocks = (K + 127) / 128;
    if (x.size(1) != K) value_error("%s and Xq differ in K", "W");
    if (!has_shape(ws, {(N + 127) / 128, blocks}) || !has_shape(xs, {blocks, M}))
      value_error("%s has the wrong shape", "wscale or xscale");
    same_device(w, ws);
    same_device(w, x);
    same_device(w, xs);
    const c10::DeviceGuard guard(w.device());
    at::Tensor out;
    // out_dtype: a torch.dtype, or None for the output's (float16)
    at::ScalarType type = at::kHalf;
    if (a[5] != Py_None) {
      if (!THPDtype_Check(a[5])) type_error("%s must be a torch.dtype", "out_dtype");
      type = reinterpret_cast<THPDtype *>(a[5])->scalar_type;
    } else if (a[4] != Py_None) {
      type = tensor(a[4], "out").scalar_type();
    }
    if (a[4] == Py_None) {
      out = at::empty({M, N}, w.options().dtype(type));
    } else {
      out = whole(a[4], type, "out");
      if (!has_shape(out, {M, N})) value_error("%s has the wrong shape", "out");
      same_device(w, out);
    }
    const int code = type_code(out, "out", true);
    void *stream = stream_of(a[6], w);
    check(call([&] {
      return lqmm_gemm_f8b128(static_cast<const uint8_t *>(w.data_ptr()),
                              static_cast<const float *>(ws.data_ptr()),
                              static_cast<const uint8_t *>(x.data_ptr()),
                              static_cast<const float *>(xs.data_ptr()), out.data_ptr(), code, M, N, K,
                              stream);
    }));
    return THPVariable_Wrap(out);
  });
}

PyObject *setup(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 3)) return nullptr;
  PyObject **to[] = {&g_raise_status, &g_raw_stream, &g_workspace_on};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(a[i]);
    Py_XDECREF(*to[i]);
    *to[i] = a[i];
  }
  Py_RETURN_NONE;
}

#define FASTCALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef kMethods[] = {
    {"setup", FASTCALL(setup), "setup(raise_status, raw_stream, workspace_on)"},
    {"kv_append", FASTCALL(kv_append), nullptr},
    {"attn_prefix", FASTCALL(attn_prefix), nullptr},
    {"quant_f8b128", FASTCALL(quant_f8b128), nullptr},
    {"gemm_f8b128", FASTCALL(gemm_f8b128), nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_serve", "Native calls of the serving operators.", -1,
                       kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) { return PyModule_Create(&kModule); }
