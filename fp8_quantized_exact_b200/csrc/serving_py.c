/* Argument marshalling of the serving calls, as a CPython module: the checks
 * that serving.py documents, then one call through the C ABI.
 *
 * A decode step makes three of these calls per layer and each runs a few
 * microseconds on the GPU.  Read from Python with ctypes, the attributes of the
 * six to ten tensors and the twenty-odd arguments took 8 to 10 us of host time
 * per call, more than the kernels.  The library stays what ctypes loaded:
 * bind() takes the addresses of its functions.  They run without the interpreter
 * lock, as through ctypes: a launch can block, and another thread may have to
 * free it. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "sage_b200.h"

static PyObject *s_dtype, *s_shape, *s_stride, *s_get_device, *s_data_ptr, *s_element_size;
static PyObject *t_bf16, *t_i32, *t_f32, *t_f64, *t_i8, *t_e4m3;
static PyObject *f_get_device, *f_raw_stream, *c_error;

static int (*p_rope)(sage_view_bf16, int, void*, int64_t, int64_t, int64_t, sage_view_bf16, int, void*, int64_t, int64_t,
                     int64_t, const int32_t*, int64_t, const double*, float, int, int, int, int, int, int, void*);
static int (*p_append)(const sage_cache*, sage_view_bf16, sage_view_bf16, const int32_t*, int, const int32_t*,
                       const int32_t*, int, int, void*, size_t, void*);
static int (*p_read)(const sage_cache*, const int32_t*, int, const int32_t*, const int32_t*, void*, int64_t, int64_t,
                     int64_t, void*, int64_t, int64_t, int64_t, int, int, void*, size_t, void*);
static int (*p_attn)(sage_view_bf16, const sage_cache*, const int32_t*, int, const int32_t*, const int32_t*,
                     const uint32_t*, void*, int64_t, int64_t, int64_t, float*, int, int, int, float, void*, size_t,
                     void*);

#define MAX_DIMS 4
typedef struct {
  void* ptr;
  PyObject* dtype; /* borrowed: torch keeps its dtypes for good */
  int nd;
  int64_t shape[MAX_DIMS], stride[MAX_DIMS];
} tensor;

typedef struct {
  const char* what;
  long device; /* the current one; -1 before the first tensor */
} call;

static int ints(PyObject* tuple, int64_t* to, int n) {
  int i;
  for (i = 0; i < n; ++i) {
    to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (to[i] == -1 && PyErr_Occurred()) return -1;
  }
  return 0;
}

static long as_long(PyObject* o) { /* steals o */
  long v;
  if (!o) return -2;
  v = PyLong_AsLong(o);
  Py_DECREF(o);
  return v == -1 && PyErr_Occurred() ? -2 : v;
}

/* A tensor's attributes; it has to be on the current CUDA device. */
static int get(call* c, PyObject* o, tensor* t, const char* name) {
  PyObject* x;
  long dev;
  Py_ssize_t n;
  if (!(x = PyObject_GetAttr(o, s_dtype))) {
    if (PyErr_ExceptionMatches(PyExc_AttributeError))
      PyErr_Format(PyExc_ValueError, "%s: %s must be a tensor, not %s", c->what, name, Py_TYPE(o)->tp_name);
    return -1;
  }
  t->dtype = x;
  Py_DECREF(x);
  dev = as_long(PyObject_CallMethodNoArgs(o, s_get_device));
  if (dev == -2) return -1;
  if (dev >= 0 && c->device < 0 && (c->device = as_long(PyObject_CallNoArgs(f_get_device))) < 0) return -1;
  if (dev < 0 || dev != c->device) {
    PyErr_Format(PyExc_ValueError, "%s: %s must be on the current CUDA device", c->what, name);
    return -1;
  }
  if (!(x = PyObject_GetAttr(o, s_shape))) return -1;
  n = PyTuple_Check(x) ? PyTuple_GET_SIZE(x) : -1;
  if (n < 0 || n > MAX_DIMS) {
    Py_DECREF(x);
    PyErr_Format(PyExc_ValueError, "%s: %s must be a tensor of at most 4 dimensions", c->what, name);
    return -1;
  }
  t->nd = (int)n;
  if (ints(x, t->shape, t->nd)) { Py_DECREF(x); return -1; }
  Py_DECREF(x);
  if (!(x = PyObject_CallMethodNoArgs(o, s_stride))) return -1;
  if (!PyTuple_Check(x) || PyTuple_GET_SIZE(x) != n || ints(x, t->stride, t->nd)) {
    Py_DECREF(x);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s: %s has no strides", c->what, name);
    return -1;
  }
  Py_DECREF(x);
  if (!(x = PyObject_CallMethodNoArgs(o, s_data_ptr))) return -1;
  t->ptr = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return t->ptr == NULL && PyErr_Occurred() ? -1 : 0;
}

static int bad(call* c, const char* name, const char* must) {
  PyErr_Format(PyExc_ValueError, "%s: %s must be %s", c->what, name, must);
  return -1;
}

static int contiguous(const tensor* t) {
  int64_t run = 1;
  int i;
  for (i = 0; i < t->nd; ++i)
    if (t->shape[i] == 0) return 1;
  for (i = t->nd - 1; i >= 0; --i) {
    if (t->shape[i] != 1 && t->stride[i] != run) return 0;
    run *= t->shape[i];
  }
  return 1;
}

/* A contiguous tensor of a type and shape (-1: any extent), or None. */
static int plain(call* c, PyObject* o, tensor* t, const char* name, PyObject* dtype, int nd, const int64_t* shape,
                 const char* must, int optional) {
  int i, ok;
  if (o == Py_None) {
    t->ptr = NULL;
    return optional ? 0 : bad(c, name, must);
  }
  if (get(c, o, t, name)) return -1;
  ok = t->dtype == dtype && t->nd == nd && contiguous(t);
  for (i = 0; ok && i < nd; ++i) ok = shape[i] < 0 || t->shape[i] == shape[i];
  return ok ? 0 : bad(c, name, must);
}

/* A BF16 [B, N, H, D] view (shape entries -1: any). */
static int view(call* c, PyObject* o, tensor* t, const char* name, const int64_t* shape) {
  int i, ok;
  if (get(c, o, t, name)) return -1;
  ok = t->dtype == t_bf16 && t->nd == 4 && t->stride[3] == 1;
  for (i = 0; ok && i < 4; ++i) ok = shape[i] < 0 || t->shape[i] == shape[i];
  return ok ? 0 : bad(c, name, "a bfloat16 [B, N, H, D] view of the call's sizes with unit stride over D");
}
static sage_view_bf16 as_view(const tensor* t) {
  sage_view_bf16 v;
  v.data = t->ptr;
  v.stride_b = t->stride[0];
  v.stride_n = t->stride[1];
  v.stride_h = t->stride[2];
  return v;
}

static int cache(call* c, PyObject* o, sage_cache* k) {
  static const char* must = "four contiguous CUDA tensors: codes int8 or float8_e4m3fn [pages, H, page_size, D], scales "
                            "float32 [pages, H, page_size]";
  tensor t[4];
  int i, f[2];
  PyObject* seq = PySequence_Fast(o, "");
  if (!seq) {
    if (!PyErr_ExceptionMatches(PyExc_TypeError)) return -1;
    PyErr_Clear();
    return bad(c, "the cache", must);
  }
  if (PySequence_Fast_GET_SIZE(seq) != 4) {
    Py_DECREF(seq);
    return bad(c, "the cache", must);
  }
  for (i = 0; i < 4; ++i)
    if (get(c, PySequence_Fast_GET_ITEM(seq, i), &t[i], "the cache")) {
      Py_DECREF(seq);
      return -1;
    }
  Py_DECREF(seq);
  for (i = 0; i < 2; ++i) {
    const tensor *codes = &t[2 * i], *scale = &t[2 * i + 1];
    f[i] = codes->dtype == t_i8 ? SAGE_CACHE_INT8 : codes->dtype == t_e4m3 ? SAGE_CACHE_E4M3 : -1;
    if (f[i] < 0 || codes->nd != 4 || scale->nd != 3 || scale->dtype != t_f32 || !contiguous(codes) ||
        !contiguous(scale) || codes->shape[0] != t[0].shape[0] || codes->shape[1] != t[0].shape[1] ||
        codes->shape[2] != t[0].shape[2] || codes->shape[3] != t[0].shape[3] || scale->shape[0] != t[0].shape[0] ||
        scale->shape[1] != t[0].shape[1] || scale->shape[2] != t[0].shape[2])
      return bad(c, "the cache", must);
  }
  for (i = 0; i < 4; ++i)
    if (t[0].shape[i] > INT32_MAX) return bad(c, "the cache", must);
  k->k_codes = t[0].ptr;
  k->k_scale = (float*)t[1].ptr;
  k->v_codes = t[2].ptr;
  k->v_scale = (float*)t[3].ptr;
  k->k_format = f[0];
  k->v_format = f[1];
  k->pages = (int)t[0].shape[0];
  k->H = (int)t[0].shape[1];
  k->page_size = (int)t[0].shape[2];
  k->D = (int)t[0].shape[3];
  return 0;
}

static int table(call* c, PyObject* o, tensor* t, int64_t B) {
  const int64_t shape[2] = {B, -1};
  if (plain(c, o, t, "page_table", t_i32, 2, shape, "a contiguous int32 [B, pages of a sequence] tensor", 0)) return -1;
  return t->shape[1] > INT32_MAX ? bad(c, "page_table", "at most 2^31 - 1 pages wide") : 0;
}

static int lengths(call* c, PyObject* o, tensor* t, const char* name, int64_t B, int optional) {
  return plain(c, o, t, name, t_i32, 1, &B, "a contiguous int32 [B] tensor", optional);
}

static int workspace(call* c, PyObject* o, tensor* t, size_t* bytes) {
  int64_t n = 1;
  long size;
  int i;
  if (get(c, o, t, "workspace")) return -1;
  if (!contiguous(t)) return bad(c, "workspace", "contiguous");
  for (i = 0; i < t->nd; ++i) n *= t->shape[i];
  size = as_long(PyObject_CallMethodNoArgs(o, s_element_size));
  if (size < 0) return -1;
  *bytes = (size_t)n * (size_t)size;
  return 0;
}

/* The current stream, or the handle that the caller took from a stream. */
static int stream_of(call* c, PyObject* o, void** s) {
  PyObject *dev, *x;
  if (o != Py_None) {
    *s = PyLong_AsVoidPtr(o);
    return *s == NULL && PyErr_Occurred() ? -1 : 0;
  }
  if (!(dev = PyLong_FromLong(c->device))) return -1;
  x = PyObject_CallOneArg(f_raw_stream, dev);
  Py_DECREF(dev);
  if (!x) return -1;
  *s = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return *s == NULL && PyErr_Occurred() ? -1 : 0;
}

static int sizes(call* c, const tensor* t) {
  int i;
  for (i = 0; i < t->nd; ++i)
    if (t->shape[i] > INT32_MAX) return bad(c, "every size", "below 2^31");
  return 0;
}

static PyObject* done(const call* c, int rc) {
  PyObject* e;
  if (rc == SAGE_OK) Py_RETURN_NONE;
  e = PyObject_CallFunction(c_error, "is", rc, c->what);
  if (e) {
    PyErr_SetObject(c_error, e);
    Py_DECREF(e);
  }
  return NULL;
}

static int count_args(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return 0;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return -1;
}

/* rope(q, k, q_out, k_out, positions, inv_freq, mscale, layout, rot_dim, inverse, stream) */
static PyObject* rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  call c = {"sage_rope", -1};
  tensor q, k, qo, ko, pos, f;
  const int64_t any[4] = {-1, -1, -1, -1};
  int64_t half[1] = {-1}, kshape[4];
  sage_view_bf16 vk = {NULL, 0, 0, 0};
  long layout, rot;
  int inverse, has_pos, has_k;
  double mscale;
  void* s;
  int rc;
  (void)self;
  if (count_args(n, 11)) return NULL;
  has_k = a[1] != Py_None;
  has_pos = a[4] != Py_None;
  if (view(&c, a[0], &q, "q", any) || sizes(&c, &q) || view(&c, a[2], &qo, "q_out", q.shape)) return NULL;
  memset(&ko, 0, sizeof ko);
  memset(&k, 0, sizeof k);
  if (has_k) {
    kshape[0] = q.shape[0]; kshape[1] = q.shape[1]; kshape[2] = -1; kshape[3] = q.shape[3];
    if (view(&c, a[1], &k, "k", kshape) || sizes(&c, &k) || view(&c, a[3], &ko, "k_out", k.shape)) return NULL;
    vk = as_view(&k);
  }
  if (plain(&c, a[5], &f, "inv_freq", t_f64, 1, half, "a contiguous float64 [rot_dim / 2] tensor", 0)) return NULL;
  rot = a[8] == Py_None ? 2 * (long)f.shape[0] : PyLong_AsLong(a[8]);
  if (rot == -1 && PyErr_Occurred()) return NULL;
  if (2 * f.shape[0] != rot || rot > INT32_MAX) {
    bad(&c, "inv_freq", "float64 [rot_dim / 2]");
    return NULL;
  }
  memset(&pos, 0, sizeof pos);
  if (has_pos) {
    if (get(&c, a[4], &pos, "positions")) return NULL;
    if (pos.dtype != t_i32 || (pos.nd != 1 && pos.nd != 2) || pos.shape[pos.nd - 1] != q.shape[1] ||
        (pos.nd == 2 && pos.shape[0] != q.shape[0]) || (q.shape[1] > 1 && pos.stride[pos.nd - 1] != 1)) {
      bad(&c, "positions", "int32 [B, N] or [N] with unit stride over N");
      return NULL;
    }
  }
  mscale = PyFloat_AsDouble(a[6]);
  layout = PyLong_AsLong(a[7]);
  inverse = PyObject_IsTrue(a[9]);
  if (PyErr_Occurred() || stream_of(&c, a[10], &s)) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = p_rope(as_view(&q), (int)q.shape[2], qo.ptr, qo.stride[0], qo.stride[1], qo.stride[2], vk,
              has_k ? (int)k.shape[2] : 0, ko.ptr, ko.stride[0], ko.stride[1], ko.stride[2],
              (const int32_t*)pos.ptr, pos.nd == 2 ? pos.stride[0] : 0, (const double*)f.ptr, (float)mscale,
              (int)layout, (int)rot, inverse, (int)q.shape[0], (int)q.shape[1], (int)q.shape[3], s);
  Py_END_ALLOW_THREADS
  return done(&c, rc);
}

/* append(cache, k, v, page_table, start, count, workspace, stream) */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  call c = {"sage_cache_append", -1};
  sage_cache kv;
  tensor k, v, tb, first, count, ws;
  int64_t shape[4] = {-1, -1, 0, 0};
  size_t bytes;
  void* s;
  int rc;
  (void)self;
  if (count_args(n, 8) || cache(&c, a[0], &kv)) return NULL;
  shape[2] = kv.H;
  shape[3] = kv.D;
  if (view(&c, a[1], &k, "k", shape) || sizes(&c, &k) || view(&c, a[2], &v, "v", k.shape) ||
      table(&c, a[3], &tb, k.shape[0]) || lengths(&c, a[4], &first, "start", k.shape[0], 1) ||
      lengths(&c, a[5], &count, "count", k.shape[0], 1) || workspace(&c, a[6], &ws, &bytes) || stream_of(&c, a[7], &s))
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = p_append(&kv, as_view(&k), as_view(&v), (const int32_t*)tb.ptr, (int)tb.shape[1],
                (const int32_t*)first.ptr, (const int32_t*)count.ptr, (int)k.shape[0], (int)k.shape[1],
                ws.ptr, bytes, s);
  Py_END_ALLOW_THREADS
  return done(&c, rc);
}

/* read(cache, page_table, start, count, k_out, v_out, workspace, stream) */
static PyObject* read_back(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  call c = {"sage_cache_read", -1};
  sage_cache kv;
  tensor k, v, tb, first, count, ws;
  const tensor* like;
  int64_t shape[4] = {-1, -1, 0, 0};
  size_t bytes;
  void* s;
  int rc;
  (void)self;
  if (count_args(n, 8) || cache(&c, a[0], &kv)) return NULL;
  shape[2] = kv.H;
  shape[3] = kv.D;
  memset(&k, 0, sizeof k);
  memset(&v, 0, sizeof v);
  if (a[4] == Py_None && a[5] == Py_None) {
    bad(&c, "k_out or v_out", "given");
    return NULL;
  }
  if (a[4] != Py_None && (view(&c, a[4], &k, "k_out", shape) || sizes(&c, &k))) return NULL;
  if (a[5] != Py_None && (view(&c, a[5], &v, "v_out", a[4] != Py_None ? k.shape : shape) || sizes(&c, &v))) return NULL;
  like = a[4] != Py_None ? &k : &v;
  if (table(&c, a[1], &tb, like->shape[0]) || lengths(&c, a[2], &first, "start", like->shape[0], 1) ||
      lengths(&c, a[3], &count, "count", like->shape[0], 1) || workspace(&c, a[6], &ws, &bytes) || stream_of(&c, a[7], &s))
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = p_read(&kv, (const int32_t*)tb.ptr, (int)tb.shape[1], (const int32_t*)first.ptr,
              (const int32_t*)count.ptr, k.ptr, k.stride[0], k.stride[1], k.stride[2], v.ptr, v.stride[0],
              v.stride[1], v.stride[2], (int)like->shape[0], (int)like->shape[1], ws.ptr, bytes, s);
  Py_END_ALLOW_THREADS
  return done(&c, rc);
}

/* attn(q, cache, page_table, context, count, mask, out, lse, sm_scale, workspace, stream) */
static PyObject* attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  call c = {"sage_cache_attn", -1};
  sage_cache kv;
  tensor q, out, tb, ctx, count, mask, lse, ws;
  int64_t shape[4] = {-1, -1, -1, 0}, words[3], rows[3];
  double scale;
  size_t bytes;
  void* s;
  int rc;
  (void)self;
  if (count_args(n, 11) || cache(&c, a[1], &kv)) return NULL;
  shape[3] = kv.D;
  if (view(&c, a[0], &q, "q", shape) || sizes(&c, &q)) return NULL;
  if (kv.H == 0 || q.shape[2] % kv.H) {
    bad(&c, "q's heads", "a multiple of the cache's");
    return NULL;
  }
  words[0] = rows[0] = q.shape[0];
  words[1] = rows[1] = q.shape[1];
  words[2] = (q.shape[1] + 31) / 32;
  rows[2] = q.shape[2];
  if (view(&c, a[6], &out, "out", q.shape) || table(&c, a[2], &tb, q.shape[0]) ||
      lengths(&c, a[3], &ctx, "context", q.shape[0], 0) || lengths(&c, a[4], &count, "count", q.shape[0], 1) ||
      plain(&c, a[5], &mask, "mask", t_i32, 3, words, "a contiguous int32 [B, T, ceil(T / 32)] tensor", 1) ||
      plain(&c, a[7], &lse, "lse", t_f32, 3, rows, "a contiguous float32 [B, T, Hq] tensor", 1) ||
      workspace(&c, a[9], &ws, &bytes))
    return NULL;
  scale = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred() || stream_of(&c, a[10], &s)) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = p_attn(as_view(&q), &kv, (const int32_t*)tb.ptr, (int)tb.shape[1], (const int32_t*)ctx.ptr,
              (const int32_t*)count.ptr, (const uint32_t*)mask.ptr, out.ptr, out.stride[0], out.stride[1],
              out.stride[2], (float*)lse.ptr, (int)q.shape[0], (int)q.shape[1], (int)q.shape[2],
              (float)scale, ws.ptr, bytes, s);
  Py_END_ALLOW_THREADS
  return done(&c, rc);
}

/* bind(rope, append, read, attn: function addresses; SageError) */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  void* p[4];
  int i;
  (void)self;
  if (count_args(n, 5)) return NULL;
  for (i = 0; i < 4; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function address");
      return NULL;
    }
  memcpy(&p_rope, &p[0], sizeof p_rope);
  memcpy(&p_append, &p[1], sizeof p_append);
  memcpy(&p_read, &p[2], sizeof p_read);
  memcpy(&p_attn, &p[3], sizeof p_attn);
  Py_INCREF(a[4]);
  Py_XSETREF(c_error, a[4]);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
                                {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, NULL},
                                {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
                                {"read", (PyCFunction)(void (*)(void))read_back, METH_FASTCALL, NULL},
                                {"attn", (PyCFunction)(void (*)(void))attn, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sage_serving", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__sage_serving(void) {
  PyObject *m = NULL, *torch = NULL, *tc = NULL;
  if (!(s_dtype = PyUnicode_InternFromString("dtype")) || !(s_shape = PyUnicode_InternFromString("shape")) ||
      !(s_stride = PyUnicode_InternFromString("stride")) || !(s_get_device = PyUnicode_InternFromString("get_device")) ||
      !(s_data_ptr = PyUnicode_InternFromString("data_ptr")) ||
      !(s_element_size = PyUnicode_InternFromString("element_size")))
    return NULL;
  if (!(torch = PyImport_ImportModule("torch")) || !(tc = PyImport_ImportModule("torch._C"))) goto out;
  if (!(t_bf16 = PyObject_GetAttrString(torch, "bfloat16")) || !(t_i32 = PyObject_GetAttrString(torch, "int32")) ||
      !(t_f32 = PyObject_GetAttrString(torch, "float32")) || !(t_f64 = PyObject_GetAttrString(torch, "float64")) ||
      !(t_i8 = PyObject_GetAttrString(torch, "int8")) || !(t_e4m3 = PyObject_GetAttrString(torch, "float8_e4m3fn")) ||
      !(f_get_device = PyObject_GetAttrString(tc, "_cuda_getDevice")) ||
      !(f_raw_stream = PyObject_GetAttrString(tc, "_cuda_getCurrentRawStream")))
    goto out;
  m = PyModule_Create(&module);
out:
  Py_XDECREF(torch);
  Py_XDECREF(tc);
  return m;
}
