// The calls of the operators around the attention from Python, without ctypes:
// small calls cost the host more than the GPU, and most of that in marshalling
// one argument after another.  Each function makes the checks that the Python
// form makes, allocates the outputs, and calls the C ABI; where a check fails, or
// the call needs more than the plain path (another device than the current one),
// it returns None and the Python form runs, which says what is wrong.  (A decode
// step's norms: 22 us a call through ctypes, 5 here.)  Copies of pages, which
// are rare beside the steps, are not among them (13 us a call of 6 pages).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "dash.h"

namespace {

PyObject *g_check = nullptr;  // raises what a status says

// A call's tensors: all on one CUDA device, the current one.
struct Call {
  c10::Device device{c10::kCPU};
  bool ok = true;

  const at::Tensor *get(PyObject *o) {
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (device.is_cpu()) {
      device = t.device();
      ok = ok && device.is_cuda() && device.index() == c10::cuda::current_device();
    }
    ok = ok && t.device() == device && t.layout() == c10::kStrided;
    return &t;
  }
  // [rows, heads, D] bf16, contiguous in D; a negative extent may be any
  const at::Tensor *rows(PyObject *o, int64_t rows, int64_t heads, int64_t dim) {
    const at::Tensor *t = get(o);
    ok = ok && t->scalar_type() == at::kBFloat16 && t->dim() == 3 && t->stride(2) == 1 &&
         (rows < 0 || t->size(0) == rows) && (heads < 0 || t->size(1) == heads) && (dim < 0 || t->size(2) == dim);
    return t;
  }
  // contiguous, of one or two dimensions
  const at::Tensor *plain(PyObject *o, at::ScalarType type, int64_t a, int64_t dims = 1) {
    const at::Tensor *t = get(o);
    ok = ok && t->scalar_type() == type && t->dim() == dims && t->is_contiguous() && (a < 0 || t->size(0) == a);
    return t;
  }
  const at::Tensor *table(PyObject *o, int64_t seqs) {
    const at::Tensor *t = get(o);
    ok = ok && t->scalar_type() == at::kInt && t->dim() == 2 && t->size(0) == seqs &&
         (t->size(1) <= 1 || t->stride(1) == 1);
    return t;
  }
  const at::Tensor *pages(PyObject *o, at::ScalarType type, const at::Tensor *like) {
    const at::Tensor *t = get(o);
    ok = ok && t->scalar_type() == type && t->dim() == 4 && t->stride(3) == 1 && (!like || t->sizes() == like->sizes());
    return t;
  }
  const at::Tensor *scales(PyObject *o, const at::Tensor *like) {
    const at::Tensor *t = get(o);
    ok = ok && t->scalar_type() == at::kFloat && t->dim() == 3 && t->sizes() == like->sizes().slice(0, 3);
    return t;
  }
  at::Tensor empty(c10::IntArrayRef size, at::ScalarType type) const {
    return at::empty(size, at::TensorOptions().dtype(type).device(device));
  }
  dash_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
};

struct Strides {
  int64_t v[20];
  int n = 0;
  void add(const at::Tensor &t, int dims) {
    for (int i = 0; i < dims; ++i) v[n++] = t.stride(i);
  }
};

template <class T = void>
T *ptr(const at::Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}

bool number(PyObject *o, double *out) {
  *out = PyFloat_AsDouble(o);
  if (*out == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}
bool whole(PyObject *o, int64_t *out) {
  *out = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return PyLong_Check(o);
}
bool decode_scale(PyObject *o, int64_t dim, double *out) {
  if (o != Py_None) return number(o, out);
  *out = 1.0 / std::sqrt((double)dim);
  return true;
}

PyObject *failed(int status) { return PyObject_CallFunction(g_check, "i", status); }
template <class... T>
PyObject *tensors(const T &...t) {
  PyObject *out = PyTuple_New(sizeof...(t));
  Py_ssize_t i = 0;
  if (out) ((void)PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t)), ...);
  return out;
}
bool fits(int64_t a) { return a >= 0 && a <= INT32_MAX; }

struct Norm {
  const at::Tensor *q, *k, *wq, *wk, *rope, *positions;
  double eps;
  int pairs;
  bool of(Call &c, PyObject *const *a, PyObject *const *w) {
    q = c.rows(a[0], -1, -1, -1);
    if (!c.ok) return false;
    k = c.rows(a[1], q->size(0), -1, q->size(2));
    const at::Tensor *first = c.get(w[0]);
    if (!c.ok || (first->scalar_type() != at::kBFloat16 && first->scalar_type() != at::kFloat)) return false;
    wq = c.plain(w[0], first->scalar_type(), q->size(2));
    wk = c.plain(w[1], first->scalar_type(), q->size(2));
    rope = c.plain(w[2], at::kFloat, -1, 2);
    positions = c.plain(w[3], at::kInt, q->size(0));
    pairs = PyObject_IsTrue(w[5]);
    if (pairs < 0) PyErr_Clear();  // the Python form says it again
    return c.ok && number(w[4], &eps) && pairs >= 0 && fits(q->size(1)) && fits(k->size(1)) && fits(rope->size(0));
  }
};

// (q, k, q_weight, k_weight, rope, positions, eps, pairs)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Call c;
  Norm x;
  if (n != 8 || !x.of(c, a, a + 2)) Py_RETURN_NONE;
  const at::Tensor zq = c.empty(x.q->sizes(), at::kBFloat16), zk = c.empty(x.k->sizes(), at::kBFloat16);
  Strides s;
  for (const at::Tensor *t : {x.q, x.k, &zq, &zk}) s.add(*t, 2);
  const int st = dash_qk_norm_rope(ptr(*x.q), ptr(*x.k), ptr(zq), ptr(zk), ptr(*x.wq), ptr(*x.wk),
                                   x.wq->scalar_type() == at::kFloat, ptr<float>(*x.rope), ptr<int32_t>(*x.positions),
                                   x.q->size(0), (int)x.q->size(1), (int)x.k->size(1), (int)x.q->size(2),
                                   (int)x.rope->size(1), (int)x.rope->size(0), x.pairs, (float)x.eps, s.v, c.stream());
  return st ? failed(st) : tensors(zq, zk);
}

// (q, k, dq_out, dk_out, q_weight, k_weight, rope, positions, eps, pairs)
PyObject *qk_norm_rope_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Call c;
  Norm x;
  if (n != 10 || !x.of(c, a, a + 4)) Py_RETURN_NONE;
  const int64_t dim = x.q->size(2);
  const at::Tensor *gq = c.rows(a[2], x.q->size(0), x.q->size(1), dim),
                   *gk = c.rows(a[3], x.q->size(0), x.k->size(1), dim);
  const int64_t need = dash_norm_rope_workspace(x.q->size(0), (int)x.q->size(1), (int)x.k->size(1), (int)dim);
  if (!c.ok || need < 0) Py_RETURN_NONE;
  const at::Tensor dq = c.empty(x.q->sizes(), at::kBFloat16), dk = c.empty(x.k->sizes(), at::kBFloat16);
  const at::Tensor wq = c.empty({dim}, at::kFloat), wk = c.empty({dim}, at::kFloat);
  at::Tensor ws;
  if (need > 0) ws = c.empty({need}, at::kByte);
  Strides s;
  for (const at::Tensor *t : {x.q, x.k, gq, gk, &dq, &dk}) s.add(*t, 2);
  const int st = dash_qk_norm_rope_bwd(
      ptr(*x.q), ptr(*x.k), ptr(*gq), ptr(*gk), ptr(dq), ptr(dk), ptr(*x.wq), ptr(*x.wk),
      x.wq->scalar_type() == at::kFloat, ptr<float>(wq), ptr<float>(wk), ptr<float>(*x.rope),
      ptr<int32_t>(*x.positions), x.q->size(0), (int)x.q->size(1), (int)x.k->size(1), (int)dim, (int)x.rope->size(1),
      (int)x.rope->size(0), x.pairs, (float)x.eps, s.v, need > 0 ? ptr(ws) : nullptr, need, c.stream());
  return st ? failed(st) : tensors(dq, dk, wq, wk);
}

struct Cache8 {
  const at::Tensor *kp, *vp, *ks, *vs;
  bool of(Call &c, PyObject *const *a) {
    kp = c.pages(a[0], at::kFloat8_e4m3fn, nullptr);
    if (!c.ok) return false;
    vp = c.pages(a[1], at::kFloat8_e4m3fn, kp);
    ks = c.scales(a[2], kp);
    vs = c.scales(a[3], kp);
    return c.ok && fits(kp->size(0)) && fits(kp->size(1)) && fits(kp->size(2)) && fits(kp->size(3));
  }
  void strides(Strides &s) const {
    for (const at::Tensor *t : {kp, vp, ks, vs}) s.add(*t, 3);
  }
};

// `rest`: page_table, starts, cu
int rows8(bool write, Call &c, const Cache8 &x, const at::Tensor &k, const at::Tensor &v, const at::Tensor &table,
          const at::Tensor &starts, const at::Tensor &cu) {
  Strides s;
  s.add(k, 2);
  s.add(v, 2);
  x.strides(s);
  s.v[s.n++] = table.stride(0);
  const int B = (int)starts.size(0), heads = (int)x.kp->size(2), D = (int)x.kp->size(3), n = (int)x.kp->size(0),
            page = (int)x.kp->size(1), most = (int)table.size(1);
  return write ? dash_cache_write_fp8(ptr(k), ptr(v), ptr(*x.kp), ptr(*x.vp), ptr<float>(*x.ks), ptr<float>(*x.vs),
                                      ptr<int32_t>(table), ptr<int32_t>(starts), ptr<int32_t>(cu), k.size(0), B, heads,
                                      D, n, page, most, s.v, c.stream())
               : dash_cache_read_fp8(ptr(k), ptr(v), ptr(*x.kp), ptr(*x.vp), ptr<float>(*x.ks), ptr<float>(*x.vs),
                                     ptr<int32_t>(table), ptr<int32_t>(starts), ptr<int32_t>(cu), k.size(0), B, heads,
                                     D, n, page, most, s.v, c.stream());
}

// (k, v, k_pages, v_pages, k_scales, v_scales, page_table, starts, cu)
PyObject *cache_write_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Call c;
  Cache8 x;
  if (n != 9 || !x.of(c, a + 2)) Py_RETURN_NONE;
  const at::Tensor *k = c.rows(a[0], -1, x.kp->size(2), x.kp->size(3));
  if (!c.ok) Py_RETURN_NONE;
  const at::Tensor *v = c.rows(a[1], k->size(0), x.kp->size(2), x.kp->size(3)), *starts = c.plain(a[7], at::kInt, -1);
  if (!c.ok) Py_RETURN_NONE;
  const at::Tensor *cu = c.plain(a[8], at::kInt, starts->size(0) + 1), *table = c.table(a[6], starts->size(0));
  if (!c.ok || !fits(table->size(1)) || !fits(starts->size(0))) Py_RETURN_NONE;
  const int st = rows8(true, c, x, *k, *v, *table, *starts, *cu);
  if (st) return failed(st);
  Py_RETURN_TRUE;
}

// (k_pages, v_pages, k_scales, v_scales, page_table, starts, cu, rows)
PyObject *cache_read_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Call c;
  Cache8 x;
  int64_t rows;
  if (n != 8 || !x.of(c, a) || !whole(a[7], &rows) || rows < 0) Py_RETURN_NONE;
  const at::Tensor *starts = c.plain(a[5], at::kInt, -1);
  if (!c.ok) Py_RETURN_NONE;
  const at::Tensor *cu = c.plain(a[6], at::kInt, starts->size(0) + 1), *table = c.table(a[4], starts->size(0));
  if (!c.ok || !fits(table->size(1)) || !fits(starts->size(0))) Py_RETURN_NONE;
  const at::Tensor k = c.empty({rows, x.kp->size(2), x.kp->size(3)}, at::kBFloat16),
                   v = c.empty({rows, x.kp->size(2), x.kp->size(3)}, at::kBFloat16);
  const int st = rows8(false, c, x, k, v, *table, *starts, *cu);
  return st ? failed(st) : tensors(k, v);
}

// (q, k_pages, v_pages, k_scales, v_scales, page_table, lengths, scale)
PyObject *attn_decode_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Call c;
  Cache8 x;
  double scale;
  if (n != 8 || !x.of(c, a + 1)) Py_RETURN_NONE;
  const at::Tensor *q = c.rows(a[0], -1, -1, x.kp->size(3));
  if (!c.ok || !decode_scale(a[7], q->size(2), &scale)) Py_RETURN_NONE;
  const at::Tensor *table = c.table(a[5], q->size(0)), *lengths = c.plain(a[6], at::kInt, q->size(0));
  if (!c.ok || !fits(table->size(1)) || !fits(q->size(0)) || !fits(q->size(1))) Py_RETURN_NONE;
  const int B = (int)q->size(0), heads = (int)q->size(1), hkv = (int)x.kp->size(2), D = (int)x.kp->size(3),
            pages = (int)x.kp->size(0), page = (int)x.kp->size(1), most = (int)table->size(1);
  const at::Tensor o = c.empty(q->sizes(), at::kBFloat16), lse = c.empty({B, heads}, at::kFloat);
  const long long need = dash_decode_workspace(B, heads, D, page, most);
  at::Tensor ws;
  if (need > 0) ws = c.empty({need}, at::kByte);
  Strides s;
  s.add(*q, 2);
  s.add(o, 2);
  x.strides(s);
  s.v[s.n++] = table->stride(0);
  const int st = dash_attn_decode_fp8(ptr(*q), ptr(*x.kp), ptr(*x.vp), ptr<float>(*x.ks), ptr<float>(*x.vs),
                                      ptr<int32_t>(*table), ptr<int32_t>(*lengths), ptr(o), ptr<float>(lse), B, heads,
                                      hkv, D, pages, page, most, s.v, (float)scale, need > 0 ? ptr(ws) : nullptr,
                                      need > 0 ? need : 0, c.stream());
  return st ? failed(st) : tensors(o, lse);
}

// (q, k_pages, v_pages, page_table, lengths, prefix, scale)
PyObject *attn_decode_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Call c;
  double scale;
  int64_t prefix;
  if (n != 7 || !whole(a[5], &prefix) || !fits(prefix)) Py_RETURN_NONE;
  const at::Tensor *kp = c.pages(a[1], at::kBFloat16, nullptr);
  if (!c.ok) Py_RETURN_NONE;
  const at::Tensor *vp = c.pages(a[2], at::kBFloat16, kp), *q = c.rows(a[0], -1, -1, kp->size(3));
  if (!c.ok || !decode_scale(a[6], q->size(2), &scale)) Py_RETURN_NONE;
  const at::Tensor *table = c.table(a[3], q->size(0)), *lengths = c.plain(a[4], at::kInt, q->size(0));
  if (!c.ok || !fits(table->size(1)) || !fits(q->size(0)) || !fits(q->size(1))) Py_RETURN_NONE;
  for (int i = 0; i < 4; ++i)
    if (!fits(kp->size(i))) Py_RETURN_NONE;
  const int B = (int)q->size(0), heads = (int)q->size(1), hkv = (int)kp->size(2), D = (int)kp->size(3),
            pages = (int)kp->size(0), page = (int)kp->size(1), most = (int)table->size(1);
  const at::Tensor o = c.empty(q->sizes(), at::kBFloat16), lse = c.empty({B, heads}, at::kFloat);
  const long long need = dash_decode_shared_workspace(B, heads, hkv, D, page, most, (int)prefix);
  at::Tensor ws;
  if (need > 0) ws = c.empty({need}, at::kByte);
  Strides s;
  s.add(*q, 2);
  s.add(o, 2);
  s.add(*kp, 3);
  s.add(*vp, 3);
  s.v[s.n++] = table->stride(0);
  const int st = dash_attn_decode_shared(ptr(*q), ptr(*kp), ptr(*vp), ptr<int32_t>(*table), ptr<int32_t>(*lengths),
                                         (int)prefix, ptr(o), ptr<float>(lse), B, heads, hkv, D, pages, page, most,
                                         s.v, (float)scale, need > 0 ? ptr(ws) : nullptr, need > 0 ? need : 0,
                                         c.stream());
  return st ? failed(st) : tensors(o, lse);
}

// C++ exceptions (an allocation that fails, say) become Python's.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return F(self, a, n);
  END_HANDLE_TH_ERRORS
}

PyObject *setup(PyObject *, PyObject *check) {
  Py_INCREF(check);
  Py_XDECREF(g_check);
  g_check = check;
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef fast(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {{"setup", setup, METH_O, nullptr},
                           fast<qk_norm_rope>("qk_norm_rope"),
                           fast<qk_norm_rope_bwd>("qk_norm_rope_bwd"),
                           fast<cache_write_fp8>("cache_write_fp8"),
                           fast<cache_read_fp8>("cache_read_fp8"),
                           fast<attn_decode_fp8>("attn_decode_fp8"),
                           fast<attn_decode_shared>("attn_decode_shared"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
