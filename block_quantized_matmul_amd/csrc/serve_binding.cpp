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

bool is_f8(const at::Tensor &t) {
  return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte;
}

// f8: the 8-bit caches' codes (type 0); else 16-bit caches.
Caches caches(PyObject *ko, PyObject *vo, bool f8 = false) {
  const at::Tensor &kt = tensor(ko, "k_cache");
  if (f8 && !is_f8(kt)) type_error("%s must be float8_e4m3fn (or uint8)", "k_cache");
  const at::Tensor &k = whole(ko, kt.scalar_type(), "k_cache");
  const at::Tensor &v = whole(vo, kt.scalar_type(), "v_cache");
  if (k.dim() != 4) value_error("%s must be (num_pages, n_kv_heads, page_size, head_dim)", "k_cache");
  const int64_t p = k.size(0), h = k.size(1), ps = k.size(2), d = k.size(3);
  if (ps % 8 != 0 || v.dim() != 5 || v.size(0) != p || v.size(1) != h || v.size(2) != ps / 8 ||
      v.size(3) != d || v.size(4) != 8)
    value_error("%s must be (num_pages, n_kv_heads, page_size / 8, head_dim, 8)", "v_cache");
  same_device(k, v);
  return {k, v, p, h, ps, d, f8 ? 0 : type_code(k, "k_cache", false)};
}

bool has_shape(const at::Tensor &t, std::initializer_list<int64_t> want) {
  return t.sizes() == at::IntArrayRef(want.begin(), want.size());
}

// A contiguous device tensor of e8m0 scales (float8_e8m0fnu or raw bytes).
const at::Tensor &scale_bytes(PyObject *o, std::initializer_list<int64_t> shape, const char *name) {
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != at::kFloat8_e8m0fnu && t.scalar_type() != at::kByte)
    type_error("%s must be float8_e8m0fnu (or uint8)", name);
  whole(o, t.scalar_type(), name);
  if (!has_shape(t, shape)) value_error("%s has the wrong shape", name);
  return t;
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

at::ScalarType dtype_of(PyObject *o, const char *name) {
  if (!THPDtype_Check(o)) type_error("%s must be a torch.dtype", name);
  return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

// What an append with norms takes beside lqmm_kv_append's arguments.
struct Norms {
  PyObject *k_scales, *v_scales, *q_norm, *k_norm, *eps, *dtype;
};

const float *norm_weight(PyObject *o, const at::Tensor &like, int64_t dim, const char *name) {
  if (o == Py_None) return nullptr;
  const at::Tensor &t = whole(o, at::kFloat, name);
  if (!has_shape(t, {dim})) value_error("%s must be (head_dim,)", name);
  same_device(like, t);
  return static_cast<const float *>(t.data_ptr());
}

// a: the arguments of lqmm_kv_append in order; norms: null for that call.
PyObject *append(PyObject *const *a, const Norms *norms) {
  return guarded([&]() -> PyObject * {
    PyObject *qo = a[0], *po = a[3], *turns_o = a[7], *out_o = a[9];
    const bool f8 = norms && is_f8(tensor(a[5], "k_cache"));
    const Caches c = caches(a[5], a[6], f8);
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
    uint8_t *k_scales = nullptr, *v_scales = nullptr;
    const float *q_norm = nullptr, *k_norm = nullptr;
    double eps = 0.0;
    if (norms) {
      if (f8) {
        const at::Tensor &ks = scale_bytes(norms->k_scales, {c.pages, c.heads, c.page_size}, "k_scales");
        const at::Tensor &vs = scale_bytes(norms->v_scales, {c.pages, c.heads, c.page_size}, "v_scales");
        same_device(k, ks);
        same_device(k, vs);
        k_scales = static_cast<uint8_t *>(ks.data_ptr());
        v_scales = static_cast<uint8_t *>(vs.data_ptr());
      } else if (norms->k_scales != Py_None || norms->v_scales != Py_None) {
        value_error("%s belong to 8-bit caches", "scales");
      }
      if (qo != Py_None) q_norm = norm_weight(norms->q_norm, k, c.dim, "q_norm");
      else if (norms->q_norm != Py_None) value_error("%s without q", "q_norm");
      k_norm = norm_weight(norms->k_norm, k, c.dim, "k_norm");
      eps = PyFloat_AsDouble(norms->eps);
      if (eps == -1.0 && PyErr_Occurred()) throw Failed();
    }
    // the type of q_out, and of an 8-bit cache's readers: the 16-bit caches'; beside
    // 8-bit ones as asked for, or q_out's, or k's
    at::ScalarType q_type = f8 ? (type == LQMM_F32 ? at::kHalf : k.scalar_type()) : c.k.scalar_type();
    if (norms && norms->dtype != Py_None) {
      const at::ScalarType asked = dtype_of(norms->dtype, "dtype");
      if (f8 ? asked != at::kHalf && asked != at::kBFloat16 : asked != q_type)
        type_error("%s must be float16 or bfloat16, and 16-bit caches' own", "dtype");
      q_type = asked;
    } else if (f8 && out_o != Py_None) {
      q_type = tensor(out_o, "q_out").scalar_type();
    }
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
        out = at::empty({tokens, heads, c.dim}, c.k.options().dtype(q_type));
      } else {
        out = whole(out_o, q_type, "q_out");
        if (!has_shape(out, {tokens, heads, c.dim})) value_error("%s has the wrong shape", "q_out");
        same_device(k, out);
      }
      qp = q.data_ptr();
    } else if (out_o != Py_None) {
      value_error("%s without q", "q_out");
    }
    void *stream = stream_of(a[10], k);
    void *outp = out.defined() ? out.data_ptr() : nullptr;
    int cache_type = c.type;
    if (f8) cache_type = out.defined() ? type_code(out, "q_out", false) : q_type == at::kHalf ? LQMM_F16 : LQMM_BF16;
    check(call([&] {
      if (norms)
        return lqmm_kv_append_norm(qp, k.data_ptr(), v.data_ptr(), type, ldq, ldk, ldv,
                                   static_cast<const int32_t *>(positions),
                                   static_cast<const int64_t *>(slots.data_ptr()),
                                   static_cast<const uint64_t *>(turns), rot, interleaved, q_norm,
                                   k_norm, (float)eps, outp, c.k.data_ptr(), c.v.data_ptr(), k_scales,
                                   v_scales, cache_type, tokens, heads, c.heads, c.dim, c.page_size,
                                   c.pages, stream);
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

PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return append(a, nullptr);
}

PyObject *kv_append_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 17)) return nullptr;
  // (a norm's arguments stand between the caches and the rotation's table)
  PyObject *plain[11] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[12], a[13], a[14], a[15]};
  const Norms norms = {a[7], a[8], a[9], a[10], a[11], a[16]};
  return append(plain, &norms);
}

// A pair of tensors as a Python tuple.
PyObject *both_of(const at::Tensor &a, const at::Tensor &b) {
  PyObject *p = THPVariable_Wrap(a), *s = THPVariable_Wrap(b);
  PyObject *both = p && s ? PyTuple_Pack(2, p, s) : nullptr;
  Py_XDECREF(p);
  Py_XDECREF(s);
  return both;
}

// A torch.dtype argument, or the given output's type, or float16.
at::ScalarType out_type(PyObject *dtype, PyObject *out, const char *name) {
  if (dtype != Py_None) return dtype_of(dtype, name);
  return out != Py_None ? tensor(out, "out").scalar_type() : at::kHalf;
}

PyObject *kv_read_f8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject * {
    const Caches c = caches(a[0], a[1], true);
    const at::Tensor &ks = scale_bytes(a[2], {c.pages, c.heads, c.page_size}, "k_scales");
    const at::Tensor &vs = scale_bytes(a[3], {c.pages, c.heads, c.page_size}, "v_scales");
    const at::Tensor &pages = whole(a[4], at::kInt, "pages"), &starts = whole(a[5], at::kInt, "starts");
    if (pages.dim() != 2 || starts.numel() != pages.size(0) + 1)
      value_error("%s must be (batch, max_pages) and starts (batch + 1,)", "pages");
    const int64_t tokens = integer(a[6], "tokens");
    if (tokens <= 0) value_error("%s must be positive", "tokens");
    same_device(c.k, ks);
    same_device(c.k, vs);
    same_device(c.k, pages);
    same_device(c.k, starts);
    const c10::DeviceGuard guard(c.k.device());
    const at::ScalarType type = out_type(a[7], a[8], "dtype");
    at::Tensor out[2];
    const char *names[2] = {"k_out", "v_out"};
    for (int i = 0; i < 2; ++i) {
      if (a[8 + i] == Py_None) {
        out[i] = at::empty({tokens, c.heads, c.dim}, c.k.options().dtype(type));
      } else {
        out[i] = whole(a[8 + i], type, names[i]);
        if (!has_shape(out[i], {tokens, c.heads, c.dim})) value_error("%s has the wrong shape", names[i]);
        same_device(c.k, out[i]);
      }
    }
    const int code = type_code(out[0], "dtype", true);
    void *stream = stream_of(a[10], c.k);
    auto bytes = [](const at::Tensor &t) { return static_cast<const uint8_t *>(t.data_ptr()); };
    check(call([&] {
      return lqmm_kv_read_f8(bytes(c.k), bytes(c.v), bytes(ks), bytes(vs),
                             static_cast<const int32_t *>(pages.data_ptr()), pages.size(1),
                             static_cast<const int32_t *>(starts.data_ptr()), out[0].data_ptr(),
                             out[1].data_ptr(), code, tokens, pages.size(0), c.heads, c.dim, c.page_size,
                             c.pages, stream);
    }));
    return both_of(out[0], out[1]);
  });
}

// Attention over 16-bit caches, or over 8-bit ones with their scales. a: the
// arguments of lqmm_attn_prefix in order.
PyObject *attention(PyObject *const *a, bool f8, PyObject *k_scales, PyObject *v_scales) {
  return guarded([&]() -> PyObject * {
    const at::Tensor &q = tensor(a[0], "q");
    const Caches c = caches(a[1], a[2], f8);
    if (q.dim() != 3) value_error("%s must be (tokens, n_q_heads, head_dim)", "q");
    const int64_t tokens = q.size(0), heads = q.size(1);
    const int64_t ldq = row_stride(q, heads, c.dim, "q");
    if (!f8 && q.scalar_type() != c.k.scalar_type())
      type_error("%s must have the caches' element type", "q");
    const int type = f8 ? type_code(q, "q", false) : c.type;
    const uint8_t *ks = nullptr, *vs = nullptr;
    if (f8) {
      const at::Tensor &kt = scale_bytes(k_scales, {c.pages, c.heads, c.page_size}, "k_scales");
      const at::Tensor &vt = scale_bytes(v_scales, {c.pages, c.heads, c.page_size}, "v_scales");
      same_device(q, kt);
      same_device(q, vt);
      ks = static_cast<const uint8_t *>(kt.data_ptr());
      vs = static_cast<const uint8_t *>(vt.data_ptr());
    }
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
      const size_t need = (f8 ? lqmm_attn_prefix_f8_workspace_bytes : lqmm_attn_prefix_workspace_bytes)(
          prefix_len, max_pages, max_q, tokens, batch, heads, c.heads, c.dim, c.page_size);
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
      if (f8)
        return lqmm_attn_prefix_f8(q.data_ptr(), ldq, static_cast<const uint8_t *>(c.k.data_ptr()),
                                   static_cast<const uint8_t *>(c.v.data_ptr()), ks, vs, type, prefix,
                                   prefix_len, static_cast<const int32_t *>(pages.data_ptr()), max_pages,
                                   static_cast<const int32_t *>(lens.data_ptr()), start, max_q,
                                   out.data_ptr(), lse_p, (float)scale, tokens, batch, heads, c.heads,
                                   c.dim, c.page_size, c.pages, ws, ws_bytes, stream);
      return lqmm_attn_prefix(q.data_ptr(), ldq, c.k.data_ptr(), c.v.data_ptr(), type, prefix,
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

PyObject *attn_prefix(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 15)) return nullptr;
  return attention(a, false, nullptr, nullptr);
}

PyObject *attn_prefix_f8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 17)) return nullptr;
  PyObject *plain[15] = {a[0], a[1], a[2]};
  for (int i = 3; i < 15; ++i) plain[i] = a[i + 2];
  return attention(plain, true, a[3], a[4]);
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

// A 2-D contiguous device tensor of pairs of e2m1 codes.
const at::Tensor &codes4(PyObject *o, const char *name) {
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != at::kByte && t.scalar_type() != at::kFloat4_e2m1fn_x2)
    type_error("%s must be a uint8 (or float4_e2m1fn_x2) torch.Tensor", name);
  whole(o, t.scalar_type(), name);
  if (t.dim() != 2) value_error("%s must be 2-D", name);
  return t;
}

PyObject *quant_mxfp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 4)) return nullptr;
  return guarded([&]() -> PyObject * {
    const at::Tensor &x = on_device(tensor(a[0], "X"), "X");
    if (x.dim() != 2) value_error("%s must be (M, K)", "X");
    const int64_t M = x.size(0), K = x.size(1);
    if (K % 32 != 0) value_error("K of %s must be a multiple of 32", "X");
    if (K > 1 && x.stride(1) != 1) value_error("the rows of %s must be contiguous", "X");
    const int type = type_code(x, "X", true);
    const c10::DeviceGuard guard(x.device());
    at::Tensor out, scales;
    if (a[1] == Py_None) {
      out = at::empty({M, K / 2}, x.options().dtype(at::kByte));
    } else {
      out = codes4(a[1], "out");
      if (!has_shape(out, {M, K / 2})) value_error("%s has the wrong shape", "out");
      same_device(x, out);
    }
    if (a[2] == Py_None) {
      scales = at::empty({M, K / 32}, x.options().dtype(at::kFloat8_e8m0fnu));
    } else {
      scales = scale_bytes(a[2], {M, K / 32}, "scales");
      same_device(x, scales);
    }
    void *stream = stream_of(a[3], x);
    check(call([&] {
      return lqmm_quant_mxfp4(x.data_ptr(), type, M > 1 ? x.stride(0) : K,
                              static_cast<uint8_t *>(out.data_ptr()),
                              static_cast<uint8_t *>(scales.data_ptr()), M, K, stream);
    }));
    return both_of(out, scales);
  });
}

PyObject *gemm_mxfp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!arity(n, 7)) return nullptr;
  return guarded([&]() -> PyObject * {
    const at::Tensor &w = codes4(a[0], "W"), &x = codes4(a[2], "Xq");
    const int64_t N = w.size(0), K = 2 * w.size(1), M = x.size(0);
    if (2 * x.size(1) != K) value_error("%s and Xq differ in K", "W");
    const at::Tensor &ws = scale_bytes(a[1], {N, K / 32}, "wscale");
    const at::Tensor &xs = scale_bytes(a[3], {M, K / 32}, "xscale");
    same_device(w, ws);
    same_device(w, x);
    same_device(w, xs);
    const c10::DeviceGuard guard(w.device());
    const at::ScalarType type = out_type(a[5], a[4], "out_dtype");
    at::Tensor out;
    if (a[4] == Py_None) {
      out = at::empty({M, N}, w.options().dtype(type));
    } else {
      out = whole(a[4], type, "out");
      if (!has_shape(out, {M, N})) value_error("%s has the wrong shape", "out");
      same_device(w, out);
    }
    const int code = type_code(out, "out", true);
    void *stream = stream_of(a[6], w);
    auto bytes = [](const at::Tensor &t) { return static_cast<const uint8_t *>(t.data_ptr()); };
    check(call([&] {
      return lqmm_gemm_mxfp4(bytes(w), bytes(ws), bytes(x), bytes(xs), out.data_ptr(), code, M, N, K, stream);
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
    {"kv_append_norm", FASTCALL(kv_append_norm), nullptr},
    {"kv_read_f8", FASTCALL(kv_read_f8), nullptr},
    {"attn_prefix_f8", FASTCALL(attn_prefix_f8), nullptr},
    {"quant_mxfp4", FASTCALL(quant_mxfp4), nullptr},
    {"gemm_mxfp4", FASTCALL(gemm_mxfp4), nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_serve", "Native calls of the serving operators.", -1,
                       kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) { return PyModule_Create(&kModule); }
