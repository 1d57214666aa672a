// The binding's native calls: the entry points that a program makes once per
// layer and audio frame, whose argument checks and marshalling cost more in
// Python than their kernels take (host time of a call through ctypes and from
// here: sf_attention_packed 11.0 and 5.1 us, sf_kv_append 9.8 and 3.2,
// sf_attention_cached 8.8 and 3.5, of which the launch is 2.5).  Same names,
// arguments, checks and errors as every other call of binding.py, which hands
// this module its error class, engine table and the library's functions in
// setup().
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>

#include "sf.h"

namespace {

struct {
  decltype(&sf_attention_packed) packed;
  decltype(&sf_kv_append) append;
  decltype(&sf_attention_cached) cached;
  decltype(&sf_attention_cached_workspace) workspace;
  PyObject *error, *engines, *check, *raw_stream, *scratch, *params, *desc, *device, *value;
} g;

struct Failed {};   // a Python error is set

[[noreturn]] void fail(const char* format, ...) {
  va_list va;
  va_start(va, format);
  PyErr_FormatV(g.error, format, va);
  va_end(va);
  throw Failed();
}

// positional and keyword arguments in the order of names (nullptr-terminated);
// the first `required` must be there
void take(const char* fn, const char* const* names, int required, PyObject* const* args, Py_ssize_t n, PyObject* kw, PyObject** out) {
  int count = 0;
  while (names[count]) out[count++] = nullptr;
  if (n > count) {
    PyErr_Format(PyExc_TypeError, "%s() takes %d arguments, got %zd", fn, count, n);
    throw Failed();
  }
  for (Py_ssize_t i = 0; i < n; ++i) out[i] = args[i];
  for (Py_ssize_t k = 0, m = kw ? PyTuple_GET_SIZE(kw) : 0; k < m; ++k) {
    PyObject* key = PyTuple_GET_ITEM(kw, k);
    int i = 0;
    while (names[i] && PyUnicode_CompareWithASCIIString(key, names[i]) != 0) ++i;
    if (!names[i] || out[i]) {
      PyErr_Format(PyExc_TypeError, names[i] ? "%s() got %U twice" : "%s() got an unexpected argument %U", fn, key);
      throw Failed();
    }
    out[i] = args[n + k];
  }
  for (int i = 0; i < count; ++i) {
    if (i < required && !out[i]) {
      PyErr_Format(PyExc_TypeError, "%s() needs %s", fn, names[i]);
      throw Failed();
    }
    if (out[i] == Py_None) out[i] = nullptr;
  }
  for (int i = 0; i < required; ++i)
    if (!out[i]) fail("SF_EINVAL: %s is None", names[i]);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail("SF_EINVAL: %s must be a torch tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
int64_t length(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() < 1) fail("SF_EINVAL: %s has no dimension", name);
  return t.size(0);
}

struct Ref {   // owned
  PyObject* o;
  explicit Ref(PyObject* x) : o(x) {}
  Ref(const Ref&) = delete;
  ~Ref() { Py_XDECREF(o); }
};

struct Engine {
  Ref key;   // the handle as an int
  sf_engine* e;
  at::ScalarType act;
  int device;

  // eng: an int, or the ctypes pointer that holds it
  explicit Engine(PyObject* eng) : key(PyLong_Check(eng) ? Py_NewRef(eng) : PyObject_GetAttr(eng, g.value)) {
    PyObject* known = key.o ? PyDict_GetItemWithError(g.engines, key.o) : nullptr;
    if (!known) {
      if (PyErr_Occurred()) PyErr_Clear();
      fail("SF_EINVAL: not an engine of sf_create");
    }
    e = static_cast<sf_engine*>(PyLong_AsVoidPtr(key.o));
    act = PyObject_IsTrue(PyTuple_GET_ITEM(known, 0)) ? at::kBFloat16 : at::kFloat;
    device = (int)PyLong_AsLong(PyTuple_GET_ITEM(known, 1));
    if (PyErr_Occurred()) throw Failed();
  }
  // pointer and row stride of an act tensor [T, heads, dim] whose rows may be strided
  void* rows(PyObject* o, int64_t T, int64_t heads, int64_t dim, const char* name, int64_t& ld) const {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != act || !t.is_cuda() || t.get_device() != device || t.dim() != 3 || t.size(0) != T ||
        t.size(1) != heads || t.size(2) != dim) {
      PyObject *dt = PyObject_GetAttrString(o, "dtype"), *sh = PyObject_GetAttrString(o, "shape"), *dv = PyObject_GetAttrString(o, "device");
      if (dt && sh && dv)
        PyErr_Format(g.error, "SF_EINVAL: %s must be %s (%lld, %lld, %lld) on the engine's device (cuda:%d), got %S %S on %S", name,
                     act == at::kBFloat16 ? "torch.bfloat16" : "torch.float32", (long long)T, (long long)heads, (long long)dim,
                     device, dt, sh, dv);
      Py_XDECREF(dt);
      Py_XDECREF(sh);
      Py_XDECREF(dv);
      throw Failed();
    }
    if (T && (t.stride(2) != 1 || (t.stride(1) != dim && heads != 1))) fail("SF_EINVAL: the heads and dims of %s must be dense", name);
    ld = T > 1 ? t.stride(0) : heads * dim;
    return t.data_ptr();
  }
  // pointer of a dense device array [n] or [n, cols]; none stays none
  void* array(PyObject* o, at::ScalarType type, int64_t n, int64_t cols, const char* name) const {
    if (!o) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != device || t.dim() != (cols < 0 ? 1 : 2) || t.size(0) != n ||
        (cols >= 0 && t.size(1) != cols) || !t.is_contiguous()) {
      const char* ty = type == at::kInt ? "torch.int32" : "torch.float32";
      if (cols < 0) fail("SF_EINVAL: %s must be a contiguous %s (%lld,) on the engine's device (cuda:%d)", name, ty, (long long)n, device);
      fail("SF_EINVAL: %s must be a contiguous %s (%lld, %lld) on the engine's device (cuda:%d)", name, ty, (long long)n,
           (long long)cols, device);
    }
    return t.data_ptr();
  }
  // the stream given, or torch's current one on the engine's device
  void* stream(PyObject* s) const {
    PyObject* at = s ? Py_NewRef(s) : PyObject_CallFunction(g.raw_stream, "i", device);
    if (!at) throw Failed();
    void* st = PyLong_AsVoidPtr(at);
    Py_DECREF(at);
    if (!st && PyErr_Occurred()) throw Failed();
    return st;
  }
  void done(sf_status rc) const {
    if (rc == SF_OK) return;
    PyObject* r = PyObject_CallFunction(g.check, "iO", (int)rc, key.o);
    Py_XDECREF(r);
    throw Failed();
  }
};

// a copy of a ctypes structure's contents
template <typename S>
S contents(PyObject* o, const char* name) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Failed();
  if (b.len != (Py_ssize_t)sizeof(S)) {
    PyBuffer_Release(&b);
    fail("SF_EINVAL: %s has another size", name);
  }
  S s;
  memcpy(&s, b.buf, sizeof(S));
  PyBuffer_Release(&b);
  return s;
}
sf_attn_params view_of(PyObject* o) {
  if (!PyObject_TypeCheck(o, (PyTypeObject*)g.params)) fail("SF_EINVAL: params must come from attn_params");
  return contents<sf_attn_params>(o, "params");
}
sf_kv_cache cache_of(PyObject* o, const Engine& en) {
  PyObject *dev = PyObject_GetAttr(o, g.device), *desc = dev ? PyObject_GetAttr(o, g.desc) : nullptr;
  const long d = dev ? PyLong_AsLong(dev) : -1;
  Py_XDECREF(dev);
  if (!desc) throw Failed();
  sf_kv_cache c;
  try {
    c = contents<sf_kv_cache>(desc, "cache");
  } catch (...) {
    Py_DECREF(desc);
    throw;
  }
  Py_DECREF(desc);
  if (PyErr_Occurred()) throw Failed();
  if (d != en.device) fail("SF_EINVAL: the cache is on another device");
  return c;
}
int as_int(int64_t v, const char* name) {
  if (v < INT_MIN || v > INT_MAX) fail("SF_ESHAPE: %s is beyond 32 bits", name);
  return (int)v;
}

// runs a call's body; its failures become Python errors
template <typename F>
PyObject* guarded(F body) {
  try {
    body();
    Py_RETURN_NONE;
  } catch (const Failed&) {
  } catch (const std::exception& x) {
    PyErr_SetString(g.error, x.what());
  }
  return nullptr;
}

PyObject* packed(PyObject*, PyObject* const* args, Py_ssize_t n_args, PyObject* kw) {
  return guarded([&] {
    static const char* const names[] = {"eng", "q", "k", "v", "cu", "out", "params", "slopes", "prefix", "stream", nullptr};
    PyObject* a[10];
    take("sf_attention_packed", names, 7, args, n_args, kw, a);
    const Engine en(a[0]);
    const sf_attn_params p = view_of(a[6]);
    const int64_t T = length(a[1], "q"), n = length(a[4], "cu") - 1;
    int64_t ldq, ldk, ldv, ldo;
    void *q = en.rows(a[1], T, p.n_heads, p.head_dim, "q", ldq), *k = en.rows(a[2], T, p.n_kv_heads, p.head_dim, "k", ldk);
    void *v = en.rows(a[3], T, p.n_kv_heads, p.head_dim, "v", ldv), *out = en.rows(a[5], T, p.n_heads, p.head_dim, "out", ldo);
    const int* cu = (const int*)en.array(a[4], at::kInt, n + 1, -1, "cu");
    const float* slopes = (const float*)en.array(a[7], at::kFloat, p.n_heads, -1, "slopes");
    const int* prefix = (const int*)en.array(a[8], at::kInt, n, -1, "prefix");
    void* st = en.stream(a[9]);
    const int ni = as_int(n, "n");
    sf_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g.packed(en.e, q, ldq, k, ldk, v, ldv, T, cu, ni, &p, slopes, prefix, out, ldo, st);
    Py_END_ALLOW_THREADS
    en.done(rc);
  });
}

PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n_args, PyObject* kw) {
  return guarded([&] {
    static const char* const names[] = {"eng", "k", "v", "cu", "held", "table", "cache", "stream", nullptr};
    PyObject* a[8];
    take("sf_kv_append", names, 7, args, n_args, kw, a);
    const Engine en(a[0]);
    const sf_kv_cache c = cache_of(a[6], en);
    const int64_t T = length(a[1], "k"), n = length(a[4], "held"), cols = tensor(a[5], "table").dim() == 2 ? tensor(a[5], "table").size(1) : 0;
    int64_t ldk, ldv;
    void *k = en.rows(a[1], T, c.n_kv_heads, c.head_dim, "k", ldk), *v = en.rows(a[2], T, c.n_kv_heads, c.head_dim, "v", ldv);
    const int* cu = (const int*)en.array(a[3], at::kInt, n + 1, -1, "cu");
    const int* held = (const int*)en.array(a[4], at::kInt, n, -1, "held");
    const int* table = (const int*)en.array(a[5], at::kInt, n, cols, "table");
    void* st = en.stream(a[7]);
    const int ni = as_int(n, "n"), ci = as_int(cols, "table");
    sf_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g.append(en.e, k, ldk, v, ldv, T, cu, ni, held, table, ci, &c, st);
    Py_END_ALLOW_THREADS
    en.done(rc);
  });
}

PyObject* cached(PyObject*, PyObject* const* args, Py_ssize_t n_args, PyObject* kw) {
  return guarded([&] {
    static const char* const names[] = {"eng", "q", "cu", "held", "table", "cache", "out", "params", "slopes", "prefix", "max_len", "stream", nullptr};
    PyObject* a[12];
    take("sf_attention_cached", names, 8, args, n_args, kw, a);
    const Engine en(a[0]);
    const sf_kv_cache c = cache_of(a[5], en);
    const sf_attn_params p = view_of(a[7]);
    const int64_t T = length(a[1], "q"), n = length(a[3], "held"), cols = tensor(a[4], "table").dim() == 2 ? tensor(a[4], "table").size(1) : 0;
    int64_t ldq, ldo, longest = a[10] ? PyLong_AsLongLong(a[10]) : 0;
    if (PyErr_Occurred()) throw Failed();
    void *q = en.rows(a[1], T, p.n_heads, p.head_dim, "q", ldq), *out = en.rows(a[6], T, p.n_heads, p.head_dim, "out", ldo);
    const int* cu = (const int*)en.array(a[2], at::kInt, n + 1, -1, "cu");
    const int* held = (const int*)en.array(a[3], at::kInt, n, -1, "held");
    const int* table = (const int*)en.array(a[4], at::kInt, n, cols, "table");
    const float* slopes = (const float*)en.array(a[8], at::kFloat, p.n_heads, -1, "slopes");
    const int* prefix = (const int*)en.array(a[9], at::kInt, n, -1, "prefix");
    void* st = en.stream(a[11]);
    const int ni = as_int(n, "n"), ci = as_int(cols, "table");
    const int most = as_int(longest ? longest : std::min<int64_t>(cols * c.page, INT_MAX), "max_len");
    uint64_t size = 0;
    PyObject* scratch = nullptr;
    void* ws = nullptr;
    if (T) {
      en.done(g.workspace(en.e, T, ni, most, &p, &size));
      if (size) {   // few, long sequences
        scratch = PyObject_CallFunction(g.scratch, "KOO", (unsigned long long)size, a[1], a[11] ? a[11] : Py_None);
        if (!scratch) throw Failed();
        ws = THPVariable_Unpack(scratch).data_ptr();
      }
    }
    sf_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g.cached(en.e, q, ldq, T, cu, ni, held, table, ci, most, &c, &p, slopes, prefix, out, ldo, ws, size, st);
    Py_END_ALLOW_THREADS
    Py_XDECREF(scratch);
    en.done(rc);
  });
}

// setup(error, engines, check, raw_stream, scratch, params type, (addresses of the four functions))
PyObject* setup(PyObject*, PyObject* args) {
  unsigned long long f[4];
  if (!PyArg_ParseTuple(args, "OOOOOO(KKKK)", &g.error, &g.engines, &g.check, &g.raw_stream, &g.scratch, &g.params, f, f + 1, f + 2, f + 3))
    return nullptr;
  for (PyObject* o : {g.error, g.engines, g.check, g.raw_stream, g.scratch, g.params}) Py_INCREF(o);
  g.packed = reinterpret_cast<decltype(g.packed)>(f[0]);
  g.append = reinterpret_cast<decltype(g.append)>(f[1]);
  g.cached = reinterpret_cast<decltype(g.cached)>(f[2]);
  g.workspace = reinterpret_cast<decltype(g.workspace)>(f[3]);
  g.desc = PyUnicode_InternFromString("desc");
  g.device = PyUnicode_InternFromString("device");
  g.value = PyUnicode_InternFromString("value");
  Py_RETURN_NONE;
}

#define CALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL | METH_KEYWORDS
PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, nullptr},
    {"sf_attention_packed", CALL(packed),
     "sf_attention_packed(eng, q, k, v, cu, out, params, slopes=None, prefix=None, stream=None)\n--\n\n"
     "q, out: act [T, n_heads, head_dim]; k, v: act [T, n_kv_heads, head_dim] (rows may be strided);\n"
     "cu: i32 [n + 1]; slopes: f32 [n_heads]; prefix: i32 [n]; all on the device."},
    {"sf_kv_append", CALL(append),
     "sf_kv_append(eng, k, v, cu, held, table, cache, stream=None)\n--\n\n"
     "k, v: act [T, n_kv_heads, head_dim] new rows; cu: i32 [n + 1], held: i32 [n] (lengths with the new rows),\n"
     "table: i32 [n, table_cols]; cache: kv_cache(...)."},
    {"sf_attention_cached", CALL(cached),
     "sf_attention_cached(eng, q, cu, held, table, cache, out, params, slopes=None, prefix=None, max_len=0, stream=None)\n--\n\n"
     "q, out: act [T, n_heads, head_dim], the sequences' newest rows; cu, held, table, cache as for sf_kv_append.\n"
     "Few, long sequences take a workspace from torch's allocator, on the call's stream (captured by torch.cuda.graph,\n"
     "whose pool keeps it)."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
