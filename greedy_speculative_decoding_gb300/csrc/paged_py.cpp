/*
 * The paged operators' and token_logprobs' Python binding (module _paged): checks the tensors and
 * calls the C ABI. A call of the operators on a few rows takes the GPU 3 to 6
 * us; marshalling it over ctypes took the host 9 to 14 us, reading the
 * tensors' Python attributes from C 6 to 8, the tensors themselves (here) 3 to
 * 5, launches included.
 */
#define PY_SSIZE_T_CLEAN
#include <ATen/core/grad_mode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <string>

#include "sf.h"

namespace {

/* What a check says; becomes a ValueError. */
struct Refused {
  char text[320];
};

[[noreturn]] __attribute__((format(printf, 1, 2))) void refuse(const char* fmt, ...) {
  Refused r;
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(r.text, sizeof(r.text), fmt, ap);
  va_end(ap);
  throw r;
}

const char* type_name(at::ScalarType t) {
  return t == at::kFloat ? "float32" : t == at::kBFloat16 ? "bfloat16" : t == at::kHalf ? "float16"
       : t == at::kInt ? "int32" : t == at::kLong ? "int64" : t == at::kByte ? "uint8" : "another type";
}

/* Refuses a tensor, naming what it should have been and what it is. */
[[noreturn]] void wrong(const char* name, const char* want, const at::Tensor& t) {
  char shape[120] = "";
  int at = 0;
  for (const int64_t n : t.sizes())
    if (at < 90) at += snprintf(shape + at, sizeof(shape) - at, "%s%lld", at ? ", " : "", (long long)n);
  refuse("%s: expected %s, got %s [%s] on %s", name, want, type_name(t.scalar_type()), shape,
         t.is_cuda() ? ("cuda:" + std::to_string(t.get_device())).c_str() : "another device");
}

/* The calls have no gradients: a tensor that wants one is refused while gradients are on. */
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s: expected a tensor, got %.60s", name, Py_TYPE(o)->tp_name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.requires_grad() && at::GradMode::is_enabled())
    refuse("%s requires grad, and this call has no gradient (detach it, or call under torch.no_grad())", name);
  return t;
}

bool on_device(const at::Tensor& t, int dev) { return t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev; }

/* The address of a contiguous tensor of this type and shape (null for None). */
void* flat(PyObject* o, const char* name, at::ScalarType type, int dev, std::initializer_list<int64_t> want) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || !on_device(t, dev) || t.sizes() != at::IntArrayRef(want) || !t.is_contiguous()) {
    char shape[100], text[200];
    int at = 0;
    for (const int64_t n : want) at += snprintf(shape + at, sizeof(shape) - at, "%s%lld", at ? ", " : "", (long long)n);
    snprintf(text, sizeof(text), "a contiguous %s tensor [%s] on cuda:%d", type_name(type), shape, dev);
    wrong(name, text, t);
  }
  return t.data_ptr();
}

int sf_type(at::ScalarType t) {
  return t == at::kFloat ? SF_DT_F32 : t == at::kBFloat16 ? SF_DT_BF16 : t == at::kHalf ? SF_DT_F16 : -1;
}

/* Rows [n, heads, hd], the last dimension contiguous. */
sf_rows rows_of(PyObject* o, const char* name, int64_t n, int64_t hd, int dev) {
  const at::Tensor& t = tensor(o, name);
  const int dt = sf_type(t.scalar_type());
  if (dt < 0 || t.dim() != 3 || !on_device(t, dev) || t.size(0) != n || t.size(2) != hd || t.size(1) > INT32_MAX ||
      t.stride(2) != 1) {
    char text[160];
    snprintf(text, sizeof(text), "rows [%lld, heads, %lld] on cuda:%d (fp32, bf16 or fp16, last dimension contiguous)",
             (long long)n, (long long)hd, dev);
    wrong(name, text, t);
  }
  sf_rows r{};
  r.data = t.data_ptr();
  r.dtype = dt;
  r.n_heads = (int32_t)t.size(1);
  r.row = t.stride(0);
  r.head = t.stride(1);
  return r;
}

/* The cache, or its first layer where the tensors have `layers` (0 or 1) dimensions in front. */
sf_paged_cache layer_of(const at::Tensor& k, const at::Tensor& v, int dev, int layers = 0) {
  const int dt = sf_type(k.scalar_type());
  bool good = dt >= 0 && k.scalar_type() == v.scalar_type() && k.dim() == 4 + layers && k.sizes() == v.sizes() &&
              on_device(k, dev) && on_device(v, dev) && k.stride(3 + layers) == 1 && v.stride(3 + layers) == 1;
  for (int i = 0; good && i < 4 + layers; ++i) good = k.size(i) <= INT32_MAX;
  if (!good) {
    char text[160];
    snprintf(text, sizeof(text), "k and v [pages, kv_heads, page, head_dim] of one shape and type on cuda:%d, the last "
             "dimension contiguous", dev);
    wrong("caches", text, k);
  }
  sf_paged_cache c{};
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.dtype = dt;
  c.n_pages = (int32_t)k.size(layers);
  c.n_kv_heads = (int32_t)k.size(layers + 1);
  c.page = (int32_t)k.size(layers + 2);
  c.head_dim = (int32_t)k.size(layers + 3);
  c.k_page = k.stride(layers), c.k_head = k.stride(layers + 1), c.k_slot = k.stride(layers + 2);
  c.v_page = v.stride(layers), c.v_head = v.stride(layers + 1), c.v_slot = v.stride(layers + 2);
  return c;
}

sf_paged_cache cache_of(PyObject* ok, PyObject* ov, int dev) {
  return layer_of(tensor(ok, "k_cache"), tensor(ov, "v_cache"), dev);
}

/* A tensor's size along its first dimensions, each within 32 bits. */
const at::Tensor& shaped(PyObject* o, const char* name, int dims, const char* want) {
  const at::Tensor& t = tensor(o, name);
  bool good = t.dim() == dims;
  for (int i = 0; good && i < dims; ++i) good = t.size(i) < INT32_MAX;
  if (!good) wrong(name, want, t);
  return t;
}

int64_t integer(PyObject* o, const char* name, int64_t lo, int64_t hi) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw std::exception();   // (the Python error stands)
  if (x < lo || x > hi) refuse("%s out of range: %lld", name, x);
  return x;
}
void* stream_of(PyObject* o) { return reinterpret_cast<void*>(integer(o, "stream", INT64_MIN, INT64_MAX)); }

/* Tells autograd that tensors (or None) have been written in place: one that a
 * graph has saved is then noticed. */
sf_status written(sf_status s, PyObject* const* a, std::initializer_list<int> which) {
  if (s != SF_OK) return s;
  for (const int i : which) {
    if (a[i] == Py_None) continue;
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
  return s;
}

/* A call: C++ exceptions become Python's. */
template <int N, sf_status (*F)(PyObject* const*)>
PyObject* method(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
  try {
    return PyLong_FromLong(F(a));
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.text);
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

/* dev, stream, page, n_rows, lens, starts, tables, held, free, n_free, slots, positions, held_out, n_free_out, status */
sf_status page_plan(PyObject* const* a) {
  const int dev = (int)integer(a[0], "device", 0, INT32_MAX);
  const int page = (int)integer(a[2], "page", INT32_MIN, INT32_MAX), n = (int)integer(a[3], "n_rows", 0, INT32_MAX);
  const at::Tensor &tab = shaped(a[6], "tables", 2, "block tables [B, W]"),
                   &stack = shaped(a[8], "free", 1, "a stack of pages [capacity]");
  const int64_t B = tab.size(0), W = tab.size(1), cap = stack.size(0);
  auto i32 = [&](int i, const char* name, int64_t size) {
    return static_cast<int32_t*>(flat(a[i], name, at::kInt, dev, {size}));
  };
  const sf_status s = sf_page_plan(
      i32(4, "lens", B), i32(5, "starts", B + 1), (int32_t)B, page,
      static_cast<int32_t*>(flat(a[6], "tables", at::kInt, dev, {B, W})), (int32_t)W, i32(7, "held", B),
      i32(8, "free", cap), (int32_t)cap, i32(9, "n_free", 1), n, i32(10, "slots", n), i32(11, "positions", n),
      i32(12, "held_out", B), i32(13, "n_free_out", 1), i32(14, "status", B), stream_of(a[1]));
  return written(s, a, {6, 8, 10, 11, 12, 13, 14});
}

/* dev, stream, k, v, slots, k_cache, v_cache, q, q_out, positions, rope */
sf_status kv_append(PyObject* const* a) {
  const int dev = (int)integer(a[0], "device", 0, INT32_MAX);
  const sf_paged_cache cache = cache_of(a[5], a[6], dev);
  const int64_t n = shaped(a[2], "k", 3, "rows [n, kv_heads, head_dim]").size(0);
  const sf_rows k = rows_of(a[2], "k", n, cache.head_dim, dev), v = rows_of(a[3], "v", n, cache.head_dim, dev);
  const bool has_q = a[7] != Py_None;
  sf_rows q{}, q_out{};
  if (has_q) {
    q = rows_of(a[7], "q", n, cache.head_dim, dev);
    q_out = rows_of(a[8], "q_out", n, cache.head_dim, dev);
  }
  void *positions = nullptr, *rope = nullptr;
  int64_t n_pos = 0;
  if (a[10] != Py_None) {
    n_pos = shaped(a[10], "rope", 3, "a table [n_pos, head_dim / 2, 2]").size(0);
    positions = flat(a[9], "positions", at::kInt, dev, {n});
    rope = flat(a[10], "rope", at::kFloat, dev, {n_pos, cache.head_dim / 2, 2});
  }
  auto* slots = static_cast<int32_t*>(flat(a[4], "slots", at::kInt, dev, {n}));
  const sf_status s =
      sf_kv_append(&cache, (int32_t)n, &k, &v, slots, has_q ? &q : nullptr, has_q ? &q_out : nullptr,
                   static_cast<int32_t*>(positions), static_cast<float*>(rope), (int32_t)n_pos, stream_of(a[1]));
  return written(s, a, {5, 6, 8});
}

/* Both attentions. dev, stream, max_rows, scale or None, q, k_cache, v_cache, tables, lens, starts, mask, out, lse,
 * workspace */
template <bool CHUNK>
sf_status attention(PyObject* const* a) {
  const int dev = (int)integer(a[0], "device", 0, INT32_MAX), max_rows = (int)integer(a[2], "max_rows", 0, INT32_MAX);
  const sf_paged_cache cache = cache_of(a[5], a[6], dev);
  const int64_t n = shaped(a[4], "q", 3, "rows [n, heads, head_dim]").size(0);
  const at::Tensor& tab = shaped(a[7], "tables", 2, "block tables [B, W]");
  const int64_t B = tab.size(0), W = tab.size(1);
  float scale = cache.head_dim == 64 ? 0.125f : 0.08838834764831845f;   /* 1 / sqrt(head_dim), which is 64 or 128 */
  if (a[3] != Py_None) {
    const double x = PyFloat_AsDouble(a[3]);
    if (x == -1.0 && PyErr_Occurred()) throw std::exception();
    scale = (float)x;
  }
  const sf_rows q = rows_of(a[4], "q", n, cache.head_dim, dev), out = rows_of(a[11], "out", n, cache.head_dim, dev);
  auto i32 = [&](int i, const char* name, std::initializer_list<int64_t> shape) {
    return static_cast<int32_t*>(flat(a[i], name, at::kInt, dev, shape));
  };
  const int32_t *tables = i32(7, "tables", {B, W}), *lens = i32(8, "lens", {B}), *starts = i32(9, "starts", {B + 1});
  void *mask = flat(a[10], "mask", at::kLong, dev, {n}), *lse = flat(a[12], "lse", at::kFloat, dev, {n, q.n_heads});
  const size_t need = (CHUNK ? sf_chunk_attention_workspace_bytes : sf_paged_attention_workspace_bytes)(
      q.n_heads, cache.n_kv_heads, cache.head_dim, max_rows);
  const at::Tensor& ws = tensor(a[13], "workspace");
  if (ws.dim() != 1 || (size_t)ws.size(0) < need) {
    char text[80];
    snprintf(text, sizeof(text), "at least %zu contiguous bytes on cuda:%d", need, dev);
    wrong("workspace", text, ws);
  }
  void* scratch = flat(a[13], "workspace", at::kByte, dev, {ws.size(0)});
  const sf_status s =
      CHUNK ? sf_chunk_attention(&cache, &q, &out, (int32_t)n, tables, (int32_t)W, lens, starts, (int32_t)B, max_rows,
                                 scale, static_cast<float*>(lse), scratch, stream_of(a[1]))
            : sf_paged_attention(&cache, &q, &out, (int32_t)n, tables, (int32_t)W, lens, starts, (int32_t)B, max_rows,
                                 static_cast<uint64_t*>(mask), scale, static_cast<float*>(lse), scratch, stream_of(a[1]));
  return written(s, a, {11, 12, 13});
}

/* The address of a contiguous int32 tensor [size]. */
int32_t* ints(PyObject* o, const char* name, int dev, int64_t size) {
  return static_cast<int32_t*>(flat(o, name, at::kInt, dev, {size}));
}
int64_t size_of(PyObject* o, const char* name) { return shaped(o, name, 1, "int32 [n]").size(0); }

/* dev, stream, page, requests, keep, tables, held, shares, free, n_free, status */
sf_status page_free(PyObject* const* a) {
  const int dev = (int)integer(a[0], "device", 0, INT32_MAX), page = (int)integer(a[2], "page", INT32_MIN, INT32_MAX);
  const at::Tensor& tab = shaped(a[5], "tables", 2, "block tables [B, W]");
  const int64_t B = tab.size(0), W = tab.size(1), n = size_of(a[3], "requests"), P = size_of(a[7], "shares"),
                cap = size_of(a[8], "free");
  const sf_status s =
      sf_page_free(ints(a[3], "requests", dev, n), ints(a[4], "keep", dev, n), (int32_t)n, (int32_t)B, page,
                   static_cast<int32_t*>(flat(a[5], "tables", at::kInt, dev, {B, W})), (int32_t)W,
                   ints(a[6], "held", dev, B), ints(a[7], "shares", dev, P), (int32_t)P, ints(a[8], "free", dev, cap),
                   (int32_t)cap, ints(a[9], "n_free", dev, 1), ints(a[10], "status", dev, n), stream_of(a[1]));
  return written(s, a, {6, 7, 8, 9, 10});
}

/* dev, stream, page, src, dst, lens, tables, held, shares, free, n_free, source, target, slots, status */
sf_status page_fork(PyObject* const* a) {
  const int dev = (int)integer(a[0], "device", 0, INT32_MAX), page = (int)integer(a[2], "page", INT32_MIN, INT32_MAX);
  const at::Tensor& tab = shaped(a[6], "tables", 2, "block tables [B, W]");
  const int64_t B = tab.size(0), W = tab.size(1), n = size_of(a[3], "src"), P = size_of(a[8], "shares"),
                cap = size_of(a[9], "free");
  const sf_status s = sf_page_fork(
      ints(a[3], "src", dev, n), ints(a[4], "dst", dev, n), (int32_t)n, ints(a[5], "lens", dev, B), (int32_t)B, page,
      static_cast<int32_t*>(flat(a[6], "tables", at::kInt, dev, {B, W})), (int32_t)W, ints(a[7], "held", dev, B),
      ints(a[8], "shares", dev, P), (int32_t)P, ints(a[9], "free", dev, cap), (int32_t)cap,
      ints(a[10], "n_free", dev, 1), ints(a[11], "source", dev, n), ints(a[12], "target", dev, n),
      ints(a[13], "slots", dev, n), ints(a[14], "status", dev, n), stream_of(a[1]));
  return written(s, a, {6, 7, 8, 10, 11, 12, 13, 14});
}

/* dev, stream, tables, held, shares, tables_out, shares_out, free, n_free, source, target, count */
sf_status page_compact(PyObject* const* a) {
  const int dev = (int)integer(a[0], "device", 0, INT32_MAX);
  const at::Tensor& tab = shaped(a[2], "tables", 2, "block tables [B, W]");
  const int64_t B = tab.size(0), W = tab.size(1), P = size_of(a[4], "shares"), cap = size_of(a[7], "free"),
                moves = size_of(a[9], "source");
  const sf_status s = sf_page_compact(
      static_cast<int32_t*>(flat(a[2], "tables", at::kInt, dev, {B, W})), (int32_t)B, (int32_t)W,
      ints(a[3], "held", dev, B), ints(a[4], "shares", dev, P), (int32_t)P,
      static_cast<int32_t*>(flat(a[5], "tables_out", at::kInt, dev, {B, W})), ints(a[6], "shares_out", dev, P),
      ints(a[7], "free", dev, cap), (int32_t)cap, ints(a[8], "n_free", dev, 1), ints(a[9], "source", dev, moves),
      ints(a[10], "target", dev, moves), (int32_t)moves, ints(a[11], "count", dev, 1), stream_of(a[1]));
  return written(s, a, {5, 6, 7, 8, 9, 10, 11});
}

/* dev, stream, source, target, k_cache, v_cache, slots, count */
sf_status page_copy(PyObject* const* a) {
  const int dev = (int)integer(a[0], "device", 0, INT32_MAX);
  const at::Tensor &k = tensor(a[4], "k_cache"), &v = tensor(a[5], "v_cache");
  const bool deep = k.dim() == 5;   // [layers, ...]
  const sf_paged_cache cache = layer_of(k, v, dev, deep);
  const int64_t layers = deep ? k.size(0) : 1;
  const int64_t n = size_of(a[2], "source");
  const sf_status s = sf_page_copy(&cache, (int32_t)layers, deep ? k.stride(0) : 0, deep ? v.stride(0) : 0,
                                   ints(a[2], "source", dev, n), ints(a[3], "target", dev, n),
                                   ints(a[6], "slots", dev, n), (int32_t)n, ints(a[7], "count", dev, 1), stream_of(a[1]));
  return written(s, a, {4, 5});
}

/* dev, stream, top, logits, tokens, logprob, entropy, rank, top_ids, top_logprobs */
sf_status token_logprobs(PyObject* const* a) {
  const int dev = (int)integer(a[0], "device", 0, INT32_MAX), top = (int)integer(a[2], "top", INT32_MIN, INT32_MAX);
  const at::Tensor& x = shaped(a[3], "logits", 2, "rows of logits [n, vocab]");
  const int64_t n = x.size(0), vocab = x.size(1);
  if (sf_type(x.scalar_type()) < 0 || !on_device(x, dev) || (vocab > 1 && x.stride(1) != 1))
    wrong("logits", "rows [n, vocab] (fp32, bf16 or fp16, last dimension contiguous) on the current device", x);
  auto f32 = [&](int i, const char* name, std::initializer_list<int64_t> shape) {
    return static_cast<float*>(flat(a[i], name, at::kFloat, dev, shape));
  };
  const sf_status s = sf_token_logprobs(
      x.data_ptr(), sf_type(x.scalar_type()), n > 1 ? x.stride(0) : 0, (int32_t)n, (int32_t)vocab,
      ints(a[4], "tokens", dev, n), top, f32(5, "logprob", {n}), f32(6, "entropy", {n}), ints(a[7], "rank", dev, n),
      static_cast<int32_t*>(flat(a[8], "top_ids", at::kInt, dev, {n, top})), f32(9, "top_logprobs", {n, top}),
      stream_of(a[1]));
  return written(s, a, {5, 6, 7, 8, 9});
}

template <int N, sf_status (*F)(PyObject* const*)>
constexpr PyMethodDef entry(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(method<N, F>)), METH_FASTCALL, nullptr};
}

}  // namespace

PyMODINIT_FUNC PyInit__paged(void) {
  static PyMethodDef methods[] = {entry<15, page_plan>("page_plan"), entry<11, kv_append>("kv_append"),
                                  entry<14, attention<false>>("paged_attention"),
                                  entry<14, attention<true>>("chunk_attention"), entry<11, page_free>("page_free"),
                                  entry<15, page_fork>("page_fork"), entry<12, page_compact>("page_compact"),
                                  entry<8, page_copy>("page_copy"), entry<10, token_logprobs>("token_logprobs"),
                                  {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&module);
}
