/*
 * The paged operators' Python binding (module _paged): reads the tensors'
 * attributes, checks them and calls the C ABI. A call of the operators on a
 * few rows takes the GPU 3 to 6 us; the same marshalling over ctypes took the
 * host 9 to 14 us, here half of that.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "sf.h"

static PyObject *s_dtype, *s_shape, *s_device, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_stride;
static PyObject *t_f32, *t_bf16, *t_f16, *t_i32, *t_i64, *t_u8;

/* ValueError naming what a tensor should have been and what it is. */
static int wrong(const char* name, const char* want, PyObject* t) {
  PyObject *d = PyObject_GetAttr(t, s_dtype), *s = d ? PyObject_GetAttr(t, s_shape) : NULL,
           *v = s ? PyObject_GetAttr(t, s_device) : NULL;
  if (v) PyErr_Format(PyExc_ValueError, "%s: expected %s, got %S %S on %S", name, want, d, s, v);
  Py_XDECREF(d);
  Py_XDECREF(s);
  Py_XDECREF(v);
  return -1;
}

/* An attribute that is one of torch's dtype singletons (borrowed use only). */
static PyObject* dtype_of(PyObject* t) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  Py_XDECREF(d);
  return d;
}

static int long_method(PyObject* t, PyObject* name, long long* out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return -1;
  *out = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int pointer(PyObject* t, void** out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!r) return -1;
  *out = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !*out && PyErr_Occurred() ? -1 : 0;
}

/* A tuple of integers (shape or strides); returns their number or -1. */
static int tuple_of(PyObject* seq, long long* out, int max) {
  if (!seq) return -1;
  int n = -1;
  if (PyTuple_Check(seq) && PyTuple_GET_SIZE(seq) <= max) {
    n = (int)PyTuple_GET_SIZE(seq);
    for (int i = 0; i < n; ++i) {
      out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(seq, i));
      if (out[i] == -1 && PyErr_Occurred()) n = -1;
    }
  }
  Py_DECREF(seq);
  return n;
}
static int shape_of(PyObject* t, long long* out, int max) {
  const int n = tuple_of(PyObject_GetAttr(t, s_shape), out, max);
  if (n < 0) PyErr_Clear();
  return n;
}

static int on_device(PyObject* t, int dev) {
  long long d;
  if (long_method(t, s_get_device, &d)) {
    PyErr_Clear();
    return 0;
  }
  return d == dev;
}

/* The address of a contiguous tensor of this type and shape on device dev (NULL for None). */
static int flat(PyObject* t, const char* name, PyObject* dtype, int nd, long long n0, long long n1, long long n2, int dev,
                void** out) {
  *out = NULL;
  if (t == Py_None) return 0;
  const long long want[3] = {n0, n1, n2};
  long long got[4];
  PyObject* d = dtype_of(t);
  if (!d) return -1;
  int ok = d == dtype && shape_of(t, got, 4) == nd && on_device(t, dev);
  for (int i = 0; ok && i < nd; ++i) ok = got[i] == want[i];
  if (ok) {
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!c) return -1;
    ok = c == Py_True;
    Py_DECREF(c);
  }
  if (!ok) {
    char buf[160];
    if (nd == 1) snprintf(buf, sizeof(buf), "a contiguous tensor [%lld] on cuda:%d of the documented type", n0, dev);
    else if (nd == 2)
      snprintf(buf, sizeof(buf), "a contiguous tensor [%lld, %lld] on cuda:%d of the documented type", n0, n1, dev);
    else
      snprintf(buf, sizeof(buf), "a contiguous tensor [%lld, %lld, %lld] on cuda:%d of the documented type", n0, n1, n2,
               dev);
    return wrong(name, buf, t);
  }
  return pointer(t, out);
}

static int sf_type(PyObject* d) {
  return d == t_f32 ? SF_DT_F32 : d == t_bf16 ? SF_DT_BF16 : d == t_f16 ? SF_DT_F16 : -1;
}

/* Rows [n, heads, hd], the last dimension contiguous. */
static int rows_of(PyObject* t, const char* name, long long n, long long hd, int dev, sf_rows* r) {
  long long s[4], st[4];
  PyObject* d = dtype_of(t);
  if (!d) return -1;
  const int dt = sf_type(d);
  if (dt < 0 || shape_of(t, s, 4) != 3 || s[0] != n || s[2] != hd || s[1] > INT32_MAX || !on_device(t, dev) ||
      tuple_of(PyObject_CallMethodNoArgs(t, s_stride), st, 4) != 3 || st[2] != 1) {
    PyErr_Clear();
    char buf[160];
    snprintf(buf, sizeof(buf), "rows [%lld, heads, %lld] on cuda:%d (fp32, bf16 or fp16, last dimension contiguous)", n,
             hd, dev);
    return wrong(name, buf, t);
  }
  r->dtype = dt;
  r->n_heads = (int32_t)s[1];
  r->row = st[0];
  r->head = st[1];
  return pointer(t, &r->data);
}

static int cache_of(PyObject* k, PyObject* v, int dev, sf_paged_cache* c) {
  long long s[4], sv[4], st[4], sw[4];
  PyObject *dk = dtype_of(k), *dv = dk ? dtype_of(v) : NULL;
  if (!dv) return -1;
  const int dt = sf_type(dk);
  int ok = dk == dv && dt >= 0 && shape_of(k, s, 4) == 4 && shape_of(v, sv, 4) == 4 && on_device(k, dev) &&
           on_device(v, dev) && tuple_of(PyObject_CallMethodNoArgs(k, s_stride), st, 4) == 4 &&
           tuple_of(PyObject_CallMethodNoArgs(v, s_stride), sw, 4) == 4 && st[3] == 1 && sw[3] == 1;
  for (int i = 0; ok && i < 4; ++i) ok = s[i] == sv[i] && s[i] <= INT32_MAX;
  if (!ok) {
    PyErr_Clear();
    char buf[200];
    snprintf(buf, sizeof(buf), "k and v [pages, kv_heads, page, head_dim] of one shape and type on cuda:%d, the last "
             "dimension contiguous", dev);
    return wrong("caches", buf, k);
  }
  c->dtype = dt;
  c->n_pages = (int32_t)s[0];
  c->n_kv_heads = (int32_t)s[1];
  c->page = (int32_t)s[2];
  c->head_dim = (int32_t)s[3];
  c->reserved = 0;
  c->k_page = st[0], c->k_head = st[1], c->k_slot = st[2];
  c->v_page = sw[0], c->v_head = sw[1], c->v_slot = sw[2];
  if (pointer(k, &c->k)) return -1;
  return pointer(v, &c->v);
}

static int ints(PyObject* const* args, int n, long long* out) {
  for (int i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(args[i]);
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return 0;
}

static int count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return -1;
}

/* (dev, stream, page, n_rows, lens, starts, tables, held, free, n_free, slots, positions, held_out, n_free_out, status) */
static PyObject* page_plan(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long c[4], tab[4], cap[4];
  if (count(n, 15) || ints(a, 4, c)) return NULL;
  const int dev = (int)c[0];
  if (shape_of(a[6], tab, 4) != 2 || shape_of(a[8], cap, 4) != 1 || tab[0] > INT32_MAX - 1 || tab[1] > INT32_MAX ||
      cap[0] > INT32_MAX || c[2] < INT32_MIN || c[2] > INT32_MAX || c[3] < 0 || c[3] > INT32_MAX)
    return PyErr_Format(PyExc_ValueError, "tables must be [B, W], free [capacity], n_rows not negative"), NULL;
  const long long B = tab[0];
  void *lens, *starts, *tables, *held, *fr, *nf, *slots, *pos, *ho, *nfo, *status;
  if (flat(a[4], "lens", t_i32, 1, B, 0, 0, dev, &lens) || flat(a[5], "starts", t_i32, 1, B + 1, 0, 0, dev, &starts) ||
      flat(a[6], "tables", t_i32, 2, B, tab[1], 0, dev, &tables) || flat(a[7], "held", t_i32, 1, B, 0, 0, dev, &held) ||
      flat(a[8], "free", t_i32, 1, cap[0], 0, 0, dev, &fr) || flat(a[9], "n_free", t_i32, 1, 1, 0, 0, dev, &nf) ||
      flat(a[10], "slots", t_i32, 1, c[3], 0, 0, dev, &slots) ||
      flat(a[11], "positions", t_i32, 1, c[3], 0, 0, dev, &pos) ||
      flat(a[12], "held_out", t_i32, 1, B, 0, 0, dev, &ho) || flat(a[13], "n_free_out", t_i32, 1, 1, 0, 0, dev, &nfo) ||
      flat(a[14], "status", t_i32, 1, B, 0, 0, dev, &status))
    return NULL;
  return PyLong_FromLong(sf_page_plan(lens, starts, (int32_t)B, (int32_t)c[2], tables, (int32_t)tab[1], held, fr,
                                      (int32_t)cap[0], nf, (int32_t)c[3], slots, pos, ho, nfo, status, (void*)c[1]));
}

/* (dev, stream, k, v, slots, k_cache, v_cache, q, q_out, positions, rope) */
static PyObject* kv_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long c[2], s[4], rs[4] = {0};
  if (count(n, 11) || ints(a, 2, c)) return NULL;
  const int dev = (int)c[0];
  sf_paged_cache cache;
  sf_rows k, v, q, qo;
  void *slots, *pos = NULL, *rope = NULL;
  if (cache_of(a[5], a[6], dev, &cache)) return NULL;
  if (shape_of(a[2], s, 4) != 3 || s[0] > INT32_MAX) return wrong("k", "rows [n, kv_heads, head_dim]", a[2]), NULL;
  const int has_q = a[7] != Py_None, has_rope = a[10] != Py_None;
  if (rows_of(a[2], "k", s[0], cache.head_dim, dev, &k) || rows_of(a[3], "v", s[0], cache.head_dim, dev, &v) ||
      flat(a[4], "slots", t_i32, 1, s[0], 0, 0, dev, &slots) ||
      (has_q && (rows_of(a[7], "q", s[0], cache.head_dim, dev, &q) ||
                 rows_of(a[8], "q_out", s[0], cache.head_dim, dev, &qo))))
    return NULL;
  if (has_rope) {
    if (shape_of(a[10], rs, 4) != 3 || rs[0] > INT32_MAX)
      return wrong("rope", "a table [n_pos, head_dim / 2, 2]", a[10]), NULL;
    if (flat(a[9], "positions", t_i32, 1, s[0], 0, 0, dev, &pos) ||
        flat(a[10], "rope", t_f32, 3, rs[0], cache.head_dim / 2, 2, dev, &rope))
      return NULL;
  }
  return PyLong_FromLong(sf_kv_append(&cache, (int32_t)s[0], &k, &v, slots, has_q ? &q : NULL, has_q ? &qo : NULL, pos,
                                      rope, (int32_t)rs[0], (void*)c[1]));
}

/* (dev, stream, max_rows, scale or None, q, k_cache, v_cache, tables, lens, starts, mask, out, lse, workspace) */
static PyObject* paged_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long c[3], s[4], tab[4], wb[4];
  if (count(n, 14) || ints(a, 3, c)) return NULL;
  const int dev = (int)c[0];
  sf_paged_cache cache;
  sf_rows q, out;
  void *tables, *lens, *starts, *mask, *lse, *ws;
  if (cache_of(a[5], a[6], dev, &cache)) return NULL;
  if (shape_of(a[4], s, 4) != 3 || s[0] > INT32_MAX) return wrong("q", "rows [n, heads, head_dim]", a[4]), NULL;
  if (shape_of(a[7], tab, 4) != 2 || tab[0] > INT32_MAX - 1 || tab[1] > INT32_MAX)
    return wrong("tables", "block tables [B, W]", a[7]), NULL;
  if (c[2] < 0 || c[2] > INT32_MAX) return PyErr_Format(PyExc_ValueError, "max_rows out of range"), NULL;
  float scale = 0.f;
  if (a[3] == Py_None) {
    scale = cache.head_dim == 64 ? 0.125f : 0.08838834764831845f;   /* 1 / sqrt(head_dim), which is 64 or 128 */
  } else {
    const double x = PyFloat_AsDouble(a[3]);
    if (x == -1.0 && PyErr_Occurred()) return NULL;
    scale = (float)x;
  }
  if (rows_of(a[4], "q", s[0], cache.head_dim, dev, &q) || rows_of(a[11], "out", s[0], cache.head_dim, dev, &out) ||
      flat(a[7], "tables", t_i32, 2, tab[0], tab[1], 0, dev, &tables) ||
      flat(a[8], "lens", t_i32, 1, tab[0], 0, 0, dev, &lens) ||
      flat(a[9], "starts", t_i32, 1, tab[0] + 1, 0, 0, dev, &starts) ||
      flat(a[10], "mask", t_i64, 1, s[0], 0, 0, dev, &mask) || flat(a[12], "lse", t_f32, 2, s[0], s[1], 0, dev, &lse))
    return NULL;
  const size_t need =
      sf_paged_attention_workspace_bytes((int32_t)s[1], cache.n_kv_heads, cache.head_dim, (int32_t)c[2]);
  if (shape_of(a[13], wb, 4) != 1 || (size_t)wb[0] < need) {
    char buf[80];
    snprintf(buf, sizeof(buf), "at least %zu contiguous bytes on cuda:%d", need, dev);
    return wrong("workspace", buf, a[13]), NULL;
  }
  if (flat(a[13], "workspace", t_u8, 1, wb[0], 0, 0, dev, &ws)) return NULL;
  return PyLong_FromLong(sf_paged_attention(&cache, &q, &out, (int32_t)s[0], tables, (int32_t)tab[1], lens, starts,
                                            (int32_t)tab[0], (int32_t)c[2], mask, scale, lse, ws, (void*)c[1]));
}

static PyMethodDef methods[] = {
    {"page_plan", (PyCFunction)(void*)page_plan, METH_FASTCALL, NULL},
    {"kv_append", (PyCFunction)(void*)kv_append, METH_FASTCALL, NULL},
    {"paged_attention", (PyCFunction)(void*)paged_attention, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__paged(void) {
  PyObject* torch = PyImport_ImportModule("torch");
  if (!torch) return NULL;
  struct {
    PyObject** to;
    const char* name;
  } types[] = {{&t_f32, "float32"}, {&t_bf16, "bfloat16"}, {&t_f16, "float16"}, {&t_i32, "int32"}, {&t_i64, "int64"},
               {&t_u8, "uint8"}},
    names[] = {{&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_device, "device"}, {&s_get_device, "get_device"},
               {&s_is_contiguous, "is_contiguous"}, {&s_data_ptr, "data_ptr"}, {&s_stride, "stride"}};
  for (size_t i = 0; i < sizeof(types) / sizeof(types[0]); ++i)
    if (!(*types[i].to = PyObject_GetAttrString(torch, types[i].name))) return NULL;
  Py_DECREF(torch);
  for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
  return PyModule_Create(&module);
}
