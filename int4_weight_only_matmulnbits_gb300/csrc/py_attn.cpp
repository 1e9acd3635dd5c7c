// Argument marshalling of the attention block's calls for the Python binding:
// tensors are read through torch's C++ interface, checked, and handed to the C
// ABI; outputs and workspaces are torch's. These calls run a few microseconds
// on the GPU in a decode step: through ctypes they took 20 to 30 on the host,
// and much of that was a dozen small Python calls into torch for each.
//
// Every function works on the current device and its current stream, and
// returns NotImplemented for tensors of another device; the Python functions
// around them (binding.py) then change over, and hold the documentation.
// Arguments are read with the interpreter held; allocations and launches, which
// may wait for the GPU or the driver, run without it, so that the process's other
// Python threads go on.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>

#include "../../include/mnb.h"

namespace {

PyObject *s_cos, *s_sin, *s_k, *s_v, *s_starts, *s_lengths, *s_table;  // interned names
PyObject *check_status;

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

struct Released {  // the interpreter, for the scope's length
  PyThreadState *state = PyEval_SaveThread();
  Released() = default;
  Released(const Released &) = delete;
  Released &operator=(const Released &) = delete;
  ~Released() { PyEval_RestoreThread(state); }
};

bool refuse(const char *format, ...) {
  va_list ap;
  va_start(ap, format);
  PyErr_FormatV(PyExc_ValueError, format, ap);
  va_end(ap);
  return false;
}

struct Tensor {
  at::Tensor keep;  // the memory stays while the interpreter is released
  uint64_t ptr = 0;
  long device = -1;
  int dims = 0;
  int64_t shape[4] = {}, stride[4] = {};
  at::ScalarType dtype = at::kByte;
};

bool describe(PyObject *o, const char *name, Tensor &t) {
  if (!THPVariable_Check(o)) return refuse("%s must be a tensor", name);
  const at::Tensor &x = THPVariable_Unpack(o);
  if (!x.defined() || x.layout() != at::kStrided) return refuse("%s must be a dense tensor", name);
  t.keep = x;
  t.dims = static_cast<int>(x.dim());
  for (int i = 0; i < t.dims && i < 4; ++i) {
    t.shape[i] = x.size(i);
    t.stride[i] = x.stride(i);
  }
  t.ptr = reinterpret_cast<uint64_t>(x.const_data_ptr());
  t.device = x.is_cuda() ? x.get_device() : -1;
  t.dtype = x.scalar_type();
  return true;
}

int dtype_code(at::ScalarType d) {
  if (d == at::kFloat) return MNB_F32;
  if (d == at::kBFloat16) return MNB_BF16;
  PyErr_Format(PyExc_TypeError, "unsupported dtype %s: fp32 or bf16", c10::toString(d));
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

// An output: the caller's tensor, or (made) a new one of the input's shape.
bool output_of(PyObject *given, const char *name, const Rows &in, Rows &r) {
  return given == Py_None || rows_of(given, name, in.t.device, &in, r);
}
void make_output(PyObject *given, const Rows &in, Rows &r) {
  if (given != Py_None) return;
  r.t.keep = at::empty({in.t.shape[0], in.t.shape[1], in.t.shape[2]},
                       at::TensorOptions().dtype(in.t.dtype).device(at::kCUDA, in.t.device));
  r.h = mnb_heads{r.t.keep.mutable_data_ptr(), in.t.shape[1] * in.t.shape[2], in.t.shape[2],
                  in.h.heads, 0};
}
PyObject *result(PyObject *given, const Rows &r) {
  return given != Py_None ? Py_NewRef(given) : THPVariable_Wrap(r.t.keep);
}

struct Gamma {
  Tensor t;
  const float *p = nullptr;
};
bool gamma_of(PyObject *o, const char *name, int64_t D, long device, Gamma &out) {
  if (o == Py_None) return true;
  Tensor &t = out.t;
  if (!describe(o, name, t) || !on_device(t, name, device)) return false;
  if (t.dtype != at::kFloat || t.dims != 1 || t.shape[0] != D || !contiguous(t))
    return refuse("%s must be a contiguous fp32 [%lld] tensor", name, (long long)D);
  out.p = reinterpret_cast<const float *>(t.ptr);
  return true;
}

struct Rope {
  Tensor cos, sin;
  mnb_rope r;
};
bool rope_of(PyObject *o, int interleaved, long device, Rope &out) {
  Ref c(PyObject_GetAttr(o, s_cos)), s(PyObject_GetAttr(o, s_sin));
  if (!c.p || !s.p) return false;
  Tensor &tc = out.cos, &ts = out.sin;
  if (!describe(c.p, "cos", tc) || !describe(s.p, "sin", ts) || !on_device(tc, "cos", device) ||
      !on_device(ts, "sin", device))
    return false;
  if (tc.dims != 2 || ts.dims != 2 || tc.shape[0] != ts.shape[0] || tc.shape[1] != ts.shape[1] ||
      tc.dtype != at::kFloat || ts.dtype != at::kFloat || !contiguous(tc) || !contiguous(ts))
    return refuse("cos and sin must be contiguous fp32 [positions, rot_dim / 2] tensors");
  if (tc.shape[1] > (1 << 20)) return refuse("cos and sin are too wide");
  out.r = mnb_rope{reinterpret_cast<const float *>(tc.ptr),
                   reinterpret_cast<const float *>(ts.ptr), tc.shape[0],
                   static_cast<int32_t>(2 * tc.shape[1]), interleaved ? 1 : 0};
  return true;
}

struct Cache {
  Tensor k, v;
  mnb_kv_cache c;
};
bool cache_of(PyObject *o, long device, Cache &out) {
  Ref k(PyObject_GetAttr(o, s_k)), v(PyObject_GetAttr(o, s_v));
  if (!k.p || !v.p) return false;
  Tensor &tk = out.k, &tv = out.v;
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

struct Batch {
  Tensor starts, lengths, table;
  mnb_kv_batch b;
};
bool batch_of(PyObject *o, long device, Batch &out) {
  Ref s(PyObject_GetAttr(o, s_starts)), l(PyObject_GetAttr(o, s_lengths)),
      t(PyObject_GetAttr(o, s_table));
  if (!s.p || !l.p || !t.p) return false;
  Tensor &ts = out.starts, &tl = out.lengths, &tt = out.table;
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
    if (all[i]->dtype != at::kInt) return refuse("%s must be int32", names[i]);
    const int last = all[i]->dims - 1;
    if (all[i]->stride[last] != 1 && all[i]->shape[last] > 1)
      return refuse("%s must be contiguous", names[i]);
  }
  out.b = mnb_kv_batch{reinterpret_cast<const int32_t *>(ts.ptr),
                       reinterpret_cast<const int32_t *>(tl.ptr),
                       reinterpret_cast<const int32_t *>(tt.ptr),
                       tl.shape[0],
                       tt.shape[1],
                       tl.shape[0] > 1 ? tt.stride[0] : tt.shape[1]};
  return true;
}

bool is_current(long device) { return c10::cuda::current_device() == device; }
mnb_stream_t stream_of(long device) {
  return reinterpret_cast<mnb_stream_t>(
      c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
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
  if (!is_current(dev)) return Py_NewRef(Py_NotImplemented);
  const bool has_k = a[1] != Py_None;
  if (has_k && !rows_of(a[1], "k", dev, &q, k)) return nullptr;
  Rope rope;
  const double eps = PyFloat_AsDouble(a[6]);
  const int inter = PyObject_IsTrue(a[7]);
  if ((eps == -1.0 && PyErr_Occurred()) || inter < 0) return nullptr;
  if (a[2] != Py_None && !rope_of(a[2], inter, dev, rope)) return nullptr;
  Tensor t;
  const int32_t *pos = nullptr;
  if (a[3] != Py_None) {
    if (!describe(a[3], "positions", t) || !on_device(t, "positions", dev)) return nullptr;
    if (t.dtype != at::kInt || t.dims != 1 || t.shape[0] != q.t.shape[0] || !contiguous(t))
      return refuse("positions must be a contiguous int32 [T] tensor"), nullptr;
    pos = reinterpret_cast<const int32_t *>(t.ptr);
  }
  if (!has_k && a[9] != Py_None) return refuse("out_k without k"), nullptr;
  Gamma gq, gk;
  if (!gamma_of(a[4], "gamma_q", q.t.shape[2], dev, gq) ||
      !gamma_of(a[5], "gamma_k", q.t.shape[2], dev, gk))
    return nullptr;
  const int code = dtype_code(q.t.dtype);
  if (code < 0) return nullptr;
  if (q.t.shape[2] > INT32_MAX) return refuse("q's heads are too long"), nullptr;
  if (!output_of(a[8], "out_q", q, oq) || (has_k && !output_of(a[9], "out_k", k, ok)))
    return nullptr;
  mnb_status st;
  {
    const Released released;
    make_output(a[8], q, oq);
    if (has_k) make_output(a[9], k, ok);
    st = mnb_qk_norm_rope(&q.h, has_k ? &k.h : nullptr, q.t.shape[0],
                          static_cast<int>(q.t.shape[2]), static_cast<mnb_dtype>(code), gq.p, gk.p,
                          static_cast<float>(eps), a[2] == Py_None ? nullptr : &rope.r, pos, &oq.h,
                          has_k ? &ok.h : nullptr, stream_of(dev));
  }
  if (!status_ok(st, "mnb_qk_norm_rope")) return nullptr;
  Ref yq(result(a[8], oq)), yk(has_k ? result(a[9], ok) : Py_NewRef(Py_None));
  return yq.p && yk.p ? PyTuple_Pack(2, yq.p, yk.p) : nullptr;
}

// q, k, v, cache, batch, rope, gamma_q, gamma_k, eps, interleaved, out
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 11) return PyErr_Format(PyExc_TypeError, "11 arguments, not %zd", n);
  Rows q, k, v, oq;
  Cache c;
  Batch b;
  Rope rope;
  if (!rows_of(a[1], "k", -1, nullptr, k)) return nullptr;
  const long dev = k.t.device;
  if (!is_current(dev)) return Py_NewRef(Py_NotImplemented);
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
  Gamma gq, gk;
  if (!gamma_of(a[6], "gamma_q", k.t.shape[2], dev, gq) ||
      !gamma_of(a[7], "gamma_k", k.t.shape[2], dev, gk) ||
      (has_q && !output_of(a[10], "out", q, oq)))
    return nullptr;
  mnb_status st;
  {
    const Released released;
    if (has_q) make_output(a[10], q, oq);
    st = mnb_cache_append(has_q ? &q.h : nullptr, &k.h, &v.h, k.t.shape[0], gq.p, gk.p,
                          static_cast<float>(eps), a[5] == Py_None ? nullptr : &rope.r, &c.c, &b.b,
                          has_q ? &oq.h : nullptr, stream_of(dev));
  }
  if (!status_ok(st, "mnb_cache_append")) return nullptr;
  return has_q ? result(a[10], oq) : Py_NewRef(Py_None);
}

// q, cache, batch, scale (None: 1 / sqrt(head_dim)), window, out
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 6) return PyErr_Format(PyExc_TypeError, "6 arguments, not %zd", n);
  Rows q, o;
  Cache c;
  Batch b;
  if (!rows_of(a[0], "q", -1, nullptr, q)) return nullptr;
  const long dev = q.t.device;
  if (!is_current(dev)) return Py_NewRef(Py_NotImplemented);
  if (!cache_of(a[1], dev, c)) return nullptr;
  if (q.t.dtype != c.k.dtype || q.t.shape[2] != c.k.shape[3])
    return refuse("q must have the head size and dtype of the cache"), nullptr;
  if (!batch_of(a[2], dev, b)) return nullptr;
  double scale = 1.0 / std::sqrt(static_cast<double>(q.t.shape[2]));
  if (a[3] != Py_None) {
    scale = PyFloat_AsDouble(a[3]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  }
  const long long window = PyLong_AsLongLong(a[4]);
  if (window == -1 && PyErr_Occurred()) return nullptr;
  if (!output_of(a[5], "out", q, o)) return nullptr;
  mnb_status st;
  {
    const Released released;
    make_output(a[5], q, o);
    // The workspace is freed to torch's allocator after the call, which hands the
    // memory out again on the same stream only, after the call's kernels.
    const size_t need =
        mnb_paged_attention_workspace_size(q.t.shape[0], q.h.heads, &c.c, &b.b);
    at::Tensor ws;
    if (need)
      ws = at::empty({static_cast<int64_t>(need)},
                     at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev));
    st = mnb_paged_attention(&q.h, q.t.shape[0], &c.c, &b.b, static_cast<float>(scale), window,
                             &o.h, need ? ws.mutable_data_ptr() : nullptr, need, stream_of(dev));
  }
  if (!status_ok(st, "mnb_paged_attention")) return nullptr;
  return result(a[5], o);
}

// frequencies, n, first, magnitude, device (-1: the current one)
PyObject *rope_table(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 5) return PyErr_Format(PyExc_TypeError, "5 arguments, not %zd", n);
  Tensor f;
  if (!describe(a[0], "frequencies", f)) return nullptr;
  if (f.device >= 0 || f.dtype != at::kDouble || f.dims != 1 || !contiguous(f) ||
      !THPVariable_Unpack(a[0]).is_cpu())
    return refuse("frequencies must be a contiguous float64 vector on the CPU"), nullptr;
  const long long rows = PyLong_AsLongLong(a[1]), first = PyLong_AsLongLong(a[2]);
  const double magnitude = PyFloat_AsDouble(a[3]);
  long dev = PyLong_AsLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  if (dev < 0) dev = c10::cuda::current_device();
  if (!is_current(dev)) return Py_NewRef(Py_NotImplemented);
  const int64_t pairs = f.shape[0];
  if (rows < 0 || pairs > (1 << 20)) return refuse("n must not be negative"), nullptr;
  at::Tensor c, s;
  mnb_status st;
  {
    const Released released;
    const auto options = at::TensorOptions().dtype(at::kFloat).device(at::kCUDA, dev);
    c = at::empty({rows, pairs}, options);
    s = at::empty({rows, pairs}, options);
    st = mnb_rope_table(reinterpret_cast<const double *>(f.ptr), static_cast<int>(2 * pairs), first,
                        rows, magnitude, static_cast<float *>(c.mutable_data_ptr()),
                        static_cast<float *>(s.mutable_data_ptr()), stream_of(dev));
  }
  if (!status_ok(st, "mnb_rope_table")) return nullptr;
  Ref pc(THPVariable_Wrap(c)), ps(THPVariable_Wrap(s));
  if (!pc.p || !ps.p) return nullptr;
  return PyTuple_Pack(2, pc.p, ps.p);
}

// Torch's exceptions (out of memory, a device's error) as Python's.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return F(self, a, n);
  END_HANDLE_TH_ERRORS
}

// setup(check): the binding's function that raises for a status.
PyObject *setup(PyObject *, PyObject *check) {
  Py_XSETREF(check_status, Py_NewRef(check));
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(guarded<F>), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {{"setup", setup, METH_O, nullptr},
                         method<rope_table>("rope_table"),
                         method<qk_norm_rope>("qk_norm_rope"),
                         method<cache_append>("cache_append"),
                         method<paged_attention>("paged_attention"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mnb_py", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mnb_py() {
  struct {
    PyObject **to;
    const char *name;
  } const names[] = {{&s_cos, "cos"},       {&s_sin, "sin"},         {&s_k, "k"},
                     {&s_v, "v"},           {&s_starts, "starts"},   {&s_lengths, "lengths"},
                     {&s_table, "table"}};
  for (const auto &s : names)
    if (!(*s.to = PyUnicode_InternFromString(s.name))) return nullptr;
  return PyModule_Create(&module);
}
