// Argument marshalling of the attention block's calls for the Python binding
// (CPython C API): tensors are described by their own methods, checked, and
// handed to the C ABI. These calls run a few microseconds on the GPU in a
// decode step; the same marshalling through ctypes took 20 to 30 on the host,
// here it takes 5 to 9.
//
// Every function works on the current device and its current stream, and
// returns NotImplemented for tensors of another device; the Python functions
// around them (binding.py) then change over, and hold the documentation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdarg>
#include <cstdint>

#include "../../include/mnb.h"

namespace {

// Names and objects of torch, looked up when the module is set up.
PyObject *s_data_ptr, *s_stride, *s_shape, *s_dtype, *s_get_device, *s_new_empty, *s_cos, *s_sin,
    *s_k, *s_v, *s_starts, *s_lengths, *s_table;
PyObject *t_f32, *t_bf16, *t_i32, *t_u8, *raw_stream, *current_device, *check_status, *kw_u8;

struct Ref {  // an owned reference
  PyObject *p;
  explicit Ref(PyObject *o = nullptr) : p(o) {}
  Ref(const Ref &) = delete;
  Ref &operator=(const Ref &) = delete;
  ~Ref() { Py_XDECREF(p); }
  PyObject *take() {
    PyObject *o = p;
    p = nullptr;
    return o;
  }
};

bool refuse(const char *format, ...) {
  va_list ap;
  va_start(ap, format);
  PyErr_FormatV(PyExc_ValueError, format, ap);
  va_end(ap);
  return false;
}

struct Tensor {
  uint64_t ptr = 0;
  long device = -1;
  int dims = 0;
  int64_t shape[4] = {}, stride[4] = {};
  PyObject *dtype = nullptr;  // (torch's dtypes live as long as torch)
};

bool call_long(PyObject *o, PyObject *name, int64_t &v) {
  Ref r(PyObject_CallMethodNoArgs(o, name));
  if (!r.p) return false;
  v = static_cast<int64_t>(PyLong_AsUnsignedLongLongMask(r.p));
  return !PyErr_Occurred();
}

bool ints_of(PyObject *t, int64_t (&out)[4], int &n) {
  if (!PyTuple_Check(t)) return refuse("not a tensor");
  const Py_ssize_t k = PyTuple_GET_SIZE(t);
  n = static_cast<int>(k);
  for (Py_ssize_t i = 0; i < k && i < 4; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (out[i] == -1 && PyErr_Occurred()) return false;
  }
  return true;
}

bool describe(PyObject *o, const char *name, Tensor &t) {
  Ref shape(PyObject_GetAttr(o, s_shape));
  if (!shape.p) {
    PyErr_Clear();
    return refuse("%s must be a tensor", name);
  }
  Ref stride(PyObject_CallMethodNoArgs(o, s_stride)), dtype(PyObject_GetAttr(o, s_dtype));
  if (!stride.p || !dtype.p) return false;
  int n = 0;
  int64_t at = 0, dev = 0;
  if (!ints_of(shape.p, t.shape, t.dims) || !ints_of(stride.p, t.stride, n) ||
      !call_long(o, s_data_ptr, at) || !call_long(o, s_get_device, dev))
    return false;
  t.ptr = static_cast<uint64_t>(at);
  t.device = static_cast<long>(dev);
  t.dtype = dtype.p;
  return true;
}

int dtype_code(PyObject *d) {
  if (d == t_f32) return MNB_F32;
  if (d == t_bf16) return MNB_BF16;
  PyErr_Format(PyExc_TypeError, "unsupported dtype %R: fp32 or bf16", d);
  return -1;
}

bool on_device(const Tensor &t, const char *name, long device) {
  if (t.device < 0) return refuse("%s must be a CUDA tensor", name);
  if (t.device != device)
    return refuse("%s is on cuda:%ld, the call runs on cuda:%ld", name, t.device, device);
  return true;
}

bool contiguous(const Tensor &t) {
  int64_t want = 1;
  for (int i = t.dims - 1; i >= 0; --i) {
    if (t.shape[i] != 1 && t.stride[i] != want) return false;
    want *= t.shape[i];
  }
  return true;
}

// Rows of heads [T, heads, head_dim]; like: the rows, head size and dtype that
// they share.
struct Rows {
  Tensor t;
  mnb_heads h;
};
bool rows_of(PyObject *o, const char *name, long device, const Rows *like, Rows &r) {
  if (!describe(o, name, r.t)) return false;
  const Tensor &t = r.t;
  if (t.dims != 3) return refuse("%s must be a [T, heads, head_dim] tensor", name);
  if (!on_device(t, name, device < 0 ? t.device : device)) return false;
  if (t.stride[2] != 1 && t.shape[2] != 1) return refuse("%s's heads must be contiguous", name);
  if (like && (t.dtype != like->t.dtype || t.shape[0] != like->t.shape[0] ||
               t.shape[2] != like->t.shape[2]))
    return refuse("%s must have the rows, head size and dtype of the call's others", name);
  if (t.shape[1] > INT32_MAX) return refuse("%s has too many heads", name);
  r.h = mnb_heads{reinterpret_cast<void *>(t.ptr), t.stride[0], t.stride[1],
                  static_cast<int32_t>(t.shape[1]), 0};
  return true;
}

// An output: the caller's tensor, or a new one of `like`'s shape.
PyObject *output(PyObject *given, PyObject *like, const char *name, const Rows &in, Rows &r) {
  Ref made;
  if (given == Py_None) {
    Ref shape(PyObject_GetAttr(like, s_shape));
    if (!shape.p) return nullptr;
    made.p = PyObject_CallMethodOneArg(like, s_new_empty, shape.p);
    if (!made.p) return nullptr;
    int64_t at = 0;
    if (!call_long(made.p, s_data_ptr, at)) return nullptr;
    r.t = in.t;
    r.t.ptr = static_cast<uint64_t>(at);
    r.h = mnb_heads{reinterpret_cast<void *>(at), in.t.shape[1] * in.t.shape[2], in.t.shape[2],
                    in.h.heads, 0};
  } else {
    Py_INCREF(given);
    made.p = given;
    if (!rows_of(given, name, in.t.device, &in, r)) return nullptr;
  }
  return made.take();
}

bool gamma_of(PyObject *o, const char *name, int64_t D, long device, const float *&p) {
  p = nullptr;
  if (o == Py_None) return true;
  Tensor t;
  if (!describe(o, name, t) || !on_device(t, name, device)) return false;
  if (t.dtype != t_f32 || t.dims != 1 || t.shape[0] != D || !contiguous(t))
    return refuse("%s must be a contiguous fp32 [%lld] tensor", name, (long long)D);
  p = reinterpret_cast<const float *>(t.ptr);
  return true;
}

bool rope_of(PyObject *o, int interleaved, long device, mnb_rope &r) {
  Ref c(PyObject_GetAttr(o, s_cos)), s(PyObject_GetAttr(o, s_sin));
  if (!c.p || !s.p) return false;
  Tensor tc, ts;
  if (!describe(c.p, "cos", tc) || !describe(s.p, "sin", ts) || !on_device(tc, "cos", device) ||
      !on_device(ts, "sin", device))
    return false;
  if (tc.dims != 2 || ts.dims != 2 || tc.shape[0] != ts.shape[0] || tc.shape[1] != ts.shape[1] ||
      tc.dtype != t_f32 || ts.dtype != t_f32 || !contiguous(tc) || !contiguous(ts))
    return refuse("cos and sin must be contiguous fp32 [positions, rot_dim / 2] tensors");
  if (tc.shape[1] > (1 << 20)) return refuse("cos and sin are too wide");
  r = mnb_rope{reinterpret_cast<const float *>(tc.ptr), reinterpret_cast<const float *>(ts.ptr),
               tc.shape[0], static_cast<int32_t>(2 * tc.shape[1]), interleaved ? 1 : 0};
  return true;
}

struct Cache {
  Tensor k;
  mnb_kv_cache c;
};
bool cache_of(PyObject *o, long device, Cache &out) {
  Ref k(PyObject_GetAttr(o, s_k)), v(PyObject_GetAttr(o, s_v));
  if (!k.p || !v.p) return false;
  Tensor tv;
  Tensor &tk = out.k;
  if (!describe(k.p, "the cache's k", tk) || !describe(v.p, "the cache's v", tv)) return false;
  if (tk.dims != 4 || tv.dims != 4 || tk.dtype != tv.dtype || tk.shape[0] != tv.shape[0] ||
      tk.shape[1] != tv.shape[1] || tk.shape[2] != tv.shape[2] || tk.shape[3] != tv.shape[3])
    return refuse("k and v must be [pages, heads, page_size, head_dim] tensors of one dtype");
  if (!on_device(tk, "the cache's k", device) || !on_device(tv, "the cache's v", device))
    return false;
  if (tk.stride[3] != 1 || tv.stride[3] != 1)
    return refuse("the rows of k and v must be contiguous");
  for (int i = 1; i < 4; ++i)
    if (tk.shape[i] > INT32_MAX) return refuse("the cache is too large");
  const int code = dtype_code(tk.dtype);
  if (code < 0) return false;
  out.c = mnb_kv_cache{reinterpret_cast<void *>(tk.ptr),
                       reinterpret_cast<void *>(tv.ptr),
                       tk.shape[0],
                       tk.stride[0], tk.stride[1], tk.stride[2],
                       tv.stride[0], tv.stride[1], tv.stride[2],
                       static_cast<int32_t>(tk.shape[2]),
                       static_cast<int32_t>(tk.shape[1]),
                       static_cast<int32_t>(tk.shape[3]),
                       code};
  return true;
}

bool batch_of(PyObject *o, long device, mnb_kv_batch &b) {
  Ref s(PyObject_GetAttr(o, s_starts)), l(PyObject_GetAttr(o, s_lengths)),
      t(PyObject_GetAttr(o, s_table));
  if (!s.p || !l.p || !t.p) return false;
  Tensor ts, tl, tt;
  if (!describe(s.p, "starts", ts) || !describe(l.p, "lengths", tl) ||
      !describe(t.p, "table", tt))
    return false;
  if (ts.dims != 1 || tl.dims != 1 || tt.dims != 2 || ts.shape[0] != tl.shape[0] + 1 ||
      tt.shape[0] != tl.shape[0])
    return refuse("a batch of n sequences has starts [n + 1], lengths [n] and table [n, pages]");
  const Tensor *all[] = {&ts, &tl, &tt};
  const char *names[] = {"starts", "lengths", "table"};
  for (int i = 0; i < 3; ++i) {
    if (!on_device(*all[i], names[i], device)) return false;
    if (all[i]->dtype != t_i32) return refuse("%s must be int32", names[i]);
    const int last = all[i]->dims - 1;
    if (all[i]->stride[last] != 1 && all[i]->shape[last] > 1)
      return refuse("%s must be contiguous", names[i]);
  }
  b = mnb_kv_batch{reinterpret_cast<const int32_t *>(ts.ptr),
                   reinterpret_cast<const int32_t *>(tl.ptr),
                   reinterpret_cast<const int32_t *>(tt.ptr),
                   tl.shape[0],
                   tt.shape[1],
                   tl.shape[0] > 1 ? tt.stride[0] : tt.shape[1]};
  return true;
}

// 1: `device` is the current one, 0: another is, -1: an error.
int is_current(long device) {
  Ref d(PyObject_CallNoArgs(current_device));
  if (!d.p) return -1;
  const long now = PyLong_AsLong(d.p);
  return PyErr_Occurred() ? -1 : now == device;
}
#define MNB_CURRENT_OR_RETURN(device)                     \
  do {                                                    \
    const int here_ = is_current(device);                 \
    if (here_ < 0) return nullptr;                        \
    if (here_ == 0) return Py_NewRef(Py_NotImplemented);  \
  } while (0)

bool stream_of(long device, mnb_stream_t &s) {
  Ref d(PyLong_FromLong(device));
  if (!d.p) return false;
  Ref r(PyObject_CallOneArg(raw_stream, d.p));
  if (!r.p) return false;
  s = reinterpret_cast<mnb_stream_t>(PyLong_AsUnsignedLongLongMask(r.p));
  return !PyErr_Occurred();
}

bool status_ok(mnb_status st, const char *where) {
  if (st == MNB_OK) return true;
  Ref r(PyObject_CallFunction(check_status, "is", static_cast<int>(st), where));
  if (r.p) PyErr_SetString(PyExc_RuntimeError, where);  // (it raises)
  return false;
}

// q, k, rope, positions, gamma_q, gamma_k, eps, interleaved, out_q, out_k
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 10) return PyErr_Format(PyExc_TypeError, "10 arguments, not %zd", n);
  Rows q, k, oq, ok;
  if (!rows_of(a[0], "q", -1, nullptr, q)) return nullptr;
  const long dev = q.t.device;
  MNB_CURRENT_OR_RETURN(dev);
  const bool has_k = a[1] != Py_None;
  if (has_k && !rows_of(a[1], "k", dev, &q, k)) return nullptr;
  mnb_rope rope;
  const double eps = PyFloat_AsDouble(a[6]);
  const int inter = PyObject_IsTrue(a[7]);
  if ((eps == -1.0 && PyErr_Occurred()) || inter < 0) return nullptr;
  if (a[2] != Py_None && !rope_of(a[2], inter, dev, rope)) return nullptr;
  const int32_t *pos = nullptr;
  if (a[3] != Py_None) {
    Tensor t;
    if (!describe(a[3], "positions", t) || !on_device(t, "positions", dev)) return nullptr;
    if (t.dtype != t_i32 || t.dims != 1 || t.shape[0] != q.t.shape[0] || !contiguous(t))
      return refuse("positions must be a contiguous int32 [T] tensor"), nullptr;
    pos = reinterpret_cast<const int32_t *>(t.ptr);
  }
  if (!has_k && a[9] != Py_None) return refuse("out_k without k"), nullptr;
  const float *gq, *gk;
  if (!gamma_of(a[4], "gamma_q", q.t.shape[2], dev, gq) ||
      !gamma_of(a[5], "gamma_k", q.t.shape[2], dev, gk))
    return nullptr;
  const int code = dtype_code(q.t.dtype);
  if (code < 0) return nullptr;
  if (q.t.shape[2] > INT32_MAX) return refuse("q's heads are too long"), nullptr;
  Ref yq(output(a[8], a[0], "out_q", q, oq));
  if (!yq.p) return nullptr;
  Ref yk;
  if (has_k) {
    yk.p = output(a[9], a[1], "out_k", k, ok);
    if (!yk.p) return nullptr;
  } else {
    yk.p = Py_NewRef(Py_None);
  }
  mnb_stream_t s;
  if (!stream_of(dev, s)) return nullptr;
  if (!status_ok(mnb_qk_norm_rope(&q.h, has_k ? &k.h : nullptr, q.t.shape[0],
                                  static_cast<int>(q.t.shape[2]), static_cast<mnb_dtype>(code),
                                  gq, gk, static_cast<float>(eps),
                                  a[2] == Py_None ? nullptr : &rope, pos, &oq.h,
                                  has_k ? &ok.h : nullptr, s),
                 "mnb_qk_norm_rope"))
    return nullptr;
  return PyTuple_Pack(2, yq.p, yk.p);
}

// q, k, v, cache, batch, rope, gamma_q, gamma_k, eps, interleaved, out
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 11) return PyErr_Format(PyExc_TypeError, "11 arguments, not %zd", n);
  Rows q, k, v, oq;
  Cache c;
  mnb_kv_batch b;
  mnb_rope rope;
  if (!rows_of(a[1], "k", -1, nullptr, k)) return nullptr;
  const long dev = k.t.device;
  MNB_CURRENT_OR_RETURN(dev);
  if (!rows_of(a[2], "v", dev, &k, v) || !cache_of(a[3], dev, c)) return nullptr;
  if (k.t.dtype != c.k.dtype || k.t.shape[2] != c.k.shape[3] || k.t.shape[1] != c.k.shape[1])
    return refuse("k must have the heads, head size and dtype of the cache"), nullptr;
  const bool has_q = a[0] != Py_None;
  if (has_q && !rows_of(a[0], "q", dev, &k, q)) return nullptr;
  if (!has_q && a[10] != Py_None) return refuse("out without q"), nullptr;
  const double eps = PyFloat_AsDouble(a[8]);
  const int inter = PyObject_IsTrue(a[9]);
  if ((eps == -1.0 && PyErr_Occurred()) || inter < 0) return nullptr;
  if (!batch_of(a[4], dev, b) || (a[5] != Py_None && !rope_of(a[5], inter, dev, rope)))
    return nullptr;
  const float *gq, *gk;
  if (!gamma_of(a[6], "gamma_q", k.t.shape[2], dev, gq) ||
      !gamma_of(a[7], "gamma_k", k.t.shape[2], dev, gk))
    return nullptr;
  Ref y;
  if (has_q) {
    y.p = output(a[10], a[0], "out", q, oq);
    if (!y.p) return nullptr;
  } else {
    y.p = Py_NewRef(Py_None);
  }
  mnb_stream_t s;
  if (!stream_of(dev, s)) return nullptr;
  if (!status_ok(mnb_cache_append(has_q ? &q.h : nullptr, &k.h, &v.h, k.t.shape[0], gq, gk,
                                  static_cast<float>(eps), a[5] == Py_None ? nullptr : &rope,
                                  &c.c, &b, has_q ? &oq.h : nullptr, s),
                 "mnb_cache_append"))
    return nullptr;
  return y.take();
}

// q, cache, batch, scale (None: 1 / sqrt(head_dim)), window, out
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 6) return PyErr_Format(PyExc_TypeError, "6 arguments, not %zd", n);
  Rows q, o;
  Cache c;
  mnb_kv_batch b;
  if (!rows_of(a[0], "q", -1, nullptr, q)) return nullptr;
  const long dev = q.t.device;
  MNB_CURRENT_OR_RETURN(dev);
  if (!cache_of(a[1], dev, c)) return nullptr;
  if (q.t.dtype != c.k.dtype || q.t.shape[2] != c.k.shape[3])
    return refuse("q must have the head size and dtype of the cache"), nullptr;
  if (!batch_of(a[2], dev, b)) return nullptr;
  double scale = 1.0 / __builtin_sqrt(static_cast<double>(q.t.shape[2]));
  if (a[3] != Py_None) {
    scale = PyFloat_AsDouble(a[3]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  }
  const long long window = PyLong_AsLongLong(a[4]);
  if (window == -1 && PyErr_Occurred()) return nullptr;
  Ref y(output(a[5], a[0], "out", q, o));
  if (!y.p) return nullptr;
  // The workspace is freed on return to torch's allocator, which hands the
  // memory out again on the same stream only, after the call's kernels.
  const size_t need =
      mnb_paged_attention_workspace_size(q.t.shape[0], q.h.heads, &c.c, &b);
  Ref ws;
  int64_t at = 0;
  if (need) {
    Ref size(PyLong_FromSize_t(need));
    Ref fn(PyObject_GetAttr(a[0], s_new_empty));
    if (!size.p || !fn.p) return nullptr;
    PyObject *args[] = {size.p, t_u8};
    ws.p = PyObject_Vectorcall(fn.p, args, 1, kw_u8);
    if (!ws.p || !call_long(ws.p, s_data_ptr, at)) return nullptr;
  }
  mnb_stream_t s;
  if (!stream_of(dev, s)) return nullptr;
  if (!status_ok(mnb_paged_attention(&q.h, q.t.shape[0], &c.c, &b, static_cast<float>(scale),
                                     window, &o.h, reinterpret_cast<void *>(at), need, s),
                 "mnb_paged_attention"))
    return nullptr;
  return y.take();
}

// setup(torch, check): torch's module, and the binding's function that raises
// for a status.
PyObject *setup(PyObject *, PyObject *args) {
  PyObject *torch, *check;
  if (!PyArg_ParseTuple(args, "OO", &torch, &check)) return nullptr;
  struct {
    PyObject **to;
    const char *name;
  } const dtypes[] = {{&t_f32, "float32"}, {&t_bf16, "bfloat16"}, {&t_i32, "int32"},
                      {&t_u8, "uint8"}};
  for (const auto &d : dtypes)
    if (!(*d.to = PyObject_GetAttrString(torch, d.name))) return nullptr;
  Ref c(PyObject_GetAttrString(torch, "_C"));
  if (!c.p || !(raw_stream = PyObject_GetAttrString(c.p, "_cuda_getCurrentRawStream")) ||
      !(current_device = PyObject_GetAttrString(c.p, "_cuda_getDevice")))
    return nullptr;
  check_status = Py_NewRef(check);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(qk_norm_rope), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(cache_append), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(paged_attention), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mnb_py", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mnb_py() {
  struct {
    PyObject **to;
    const char *name;
  } const names[] = {{&s_data_ptr, "data_ptr"}, {&s_stride, "stride"},   {&s_shape, "shape"},
                     {&s_dtype, "dtype"},       {&s_get_device, "get_device"},
                     {&s_new_empty, "new_empty"}, {&s_cos, "cos"},       {&s_sin, "sin"},
                     {&s_k, "k"},               {&s_v, "v"},             {&s_starts, "starts"},
                     {&s_lengths, "lengths"},   {&s_table, "table"}};
  for (const auto &s : names)
    if (!(*s.to = PyUnicode_InternFromString(s.name))) return nullptr;
  if (!(kw_u8 = Py_BuildValue("(s)", "dtype"))) return nullptr;
  return PyModule_Create(&module);
}
