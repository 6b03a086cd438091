// Python binding of the paged attention's calls (moe_attn_*): checks torch
// tensors and passes their pointers and strides to the C ABI.
//
// A decode step's calls run for a few microseconds on the GPU; reading types,
// shapes, strides and pointers of their tensors attribute by attribute from
// Python and through ctypes took 7 to 8 us of host time each, this takes about
// 2, most of it the launch.  The functions take the context as (handle,
// n_heads, n_kv_heads, head_dim, rope_dim, device index) and a cache as
// (descriptor's address, n_kv_heads, head_dim, device index), tuples that
// attention.py makes once.  They raise ValueError for a tensor that does not
// fit, and return the C ABI's code.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "fp8moe.h"

namespace {

struct Context {
  moe_attn *handle;
  int64_t n_heads, n_kv, d, rope_dim, index;
};

// Thrown once a Python error is set.
struct Raised {};

template <class... A>
[[noreturn]] void raise(const char *format, A... a) {
  PyErr_Format(PyExc_ValueError, format, a...);
  throw Raised();
}

int64_t to_int(PyObject *o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
float to_float(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return (float)v;
}
void *to_ptr(PyObject *o) {
  if (o == Py_None) return nullptr;
  void *p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw Raised();
  return p;
}

Context context_of(PyObject *t) {
  if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 6) raise("the context is closed");
  const auto at = [&](int i) { return to_int(PyTuple_GET_ITEM(t, i)); };
  return Context{static_cast<moe_attn *>(to_ptr(PyTuple_GET_ITEM(t, 0))), at(1), at(2), at(3), at(4), at(5)};
}

const moe_paged_kv *cache_of(const Context &c, PyObject *t) {
  if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 4) raise("expected a PagedKVCache");
  const auto at = [&](int i) { return to_int(PyTuple_GET_ITEM(t, i)); };
  if (at(1) != c.n_kv || at(2) != c.d || at(3) != c.index)
    raise("the cache holds %lld heads of %lld on cuda:%lld; the context has %lld of %lld on cuda:%lld",
          (long long)at(1), (long long)at(2), (long long)at(3), (long long)c.n_kv, (long long)c.d,
          (long long)c.index);
  return static_cast<const moe_paged_kv *>(to_ptr(PyTuple_GET_ITEM(t, 0)));
}

const at::Tensor &tensor_of(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) raise("%s must be a tensor, got %.100s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

bool on(const at::Tensor &t, const Context &c) { return t.is_cuda() && t.get_device() == c.index; }

[[noreturn]] void misfit(const Context &c, PyObject *o, const char *name, const std::string &want) {
  PyObject *dtype = PyObject_GetAttrString(o, "dtype"), *shape = PyObject_GetAttrString(o, "shape"),
           *device = PyObject_GetAttrString(o, "device"), *stride = PyObject_CallMethod(o, "stride", nullptr);
  if (dtype && shape && device && stride)
    PyErr_Format(PyExc_ValueError, "%s must be %s on cuda:%lld, got %S %S with strides %S on %S", name,
                 want.c_str(), (long long)c.index, dtype, shape, stride, device);
  Py_XDECREF(dtype);
  Py_XDECREF(shape);
  Py_XDECREF(device);
  Py_XDECREF(stride);
  throw Raised();
}
std::string dims(std::initializer_list<int64_t> sizes) {
  std::string s;
  for (int64_t n : sizes) s += (s.empty() ? "[" : ", ") + std::to_string(n);
  return s + "]";
}

struct Rows {
  void *p;
  int64_t stride;  // of a token
};

// bf16 head rows [T, heads, d], the heads of a token next to each other.
Rows rows_of(const Context &c, PyObject *o, int64_t T, int64_t heads, const char *name) {
  const at::Tensor &t = tensor_of(o, name);
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.size(0) != T || t.size(1) != heads ||
      t.size(2) != c.d || !on(t, c) || t.stride(2) != 1 || (t.stride(1) != c.d && heads > 1))
    misfit(c, o, name, "bf16 " + dims({T, heads, c.d}) + " with a token's heads next to each other");
  return Rows{t.data_ptr(), T > 1 ? t.stride(0) : heads * c.d};
}

// A contiguous vector [n], or nullptr for None.
template <class V>
V *vec_of(const Context &c, PyObject *o, at::ScalarType type, const char *what, int64_t n, const char *name) {
  if (o == Py_None) return nullptr;
  const at::Tensor &t = tensor_of(o, name);
  if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n || !on(t, c) || !t.is_contiguous())
    misfit(c, o, name, what + (" " + dims({n})));
  return static_cast<V *>(t.data_ptr());
}
const int32_t *ints(const Context &c, PyObject *o, int64_t n, const char *name) {
  return vec_of<int32_t>(c, o, at::kInt, "contiguous int32", n, name);
}
const float *floats(const Context &c, PyObject *o, int64_t n, const char *name) {
  return vec_of<float>(c, o, at::kFloat, "contiguous f32", n, name);
}
const int64_t *slots_of(const Context &c, PyObject *o, int64_t n) {
  if (o == Py_None) raise("slots are needed");
  return vec_of<int64_t>(c, o, at::kLong, "contiguous int64", n, "slots");
}
const int32_t *positions_of(const Context &c, PyObject *o, int64_t n) {
  if (o == Py_None && c.rope_dim > 0) raise("positions are needed to rotate");
  return ints(c, o, n, "positions");
}

int64_t tokens_of(PyObject *o, const char *name) {
  const at::Tensor &t = tensor_of(o, name);
  if (t.dim() < 1) raise("%s has no dimensions", name);
  return t.size(0);
}

// Wraps f(args), which returns a code, for Python: nothing throws past it.
template <int N, class F>
PyObject *call(PyObject *const *args, Py_ssize_t n, F f) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f(args));
  } catch (const Raised &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (context, q, k, positions, q_weight, k_weight, eps, q_out, k_out, stream)
PyObject *norm_rope(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return call<10>(args, n, [](PyObject *const *p) {
    const Context c = context_of(p[0]);
    const int64_t T = tokens_of(p[1], "q");
    const Rows q = rows_of(c, p[1], T, c.n_heads, "q"), k = rows_of(c, p[2], T, c.n_kv, "k");
    const Rows qo = rows_of(c, p[7], T, c.n_heads, "q_out"), ko = rows_of(c, p[8], T, c.n_kv, "k_out");
    return moe_attn_norm_rope(c.handle, q.p, q.stride, k.p, k.stride, positions_of(c, p[3], T), T,
                              floats(c, p[4], c.d, "q_weight"), floats(c, p[5], c.d, "k_weight"),
                              to_float(p[6]), qo.p, qo.stride, ko.p, ko.stride, to_ptr(p[9]));
  });
}

// (context, cache, q, k, v, positions, slots, q_weight, k_weight, eps, q_out, stream)
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return call<12>(args, n, [](PyObject *const *p) {
    const Context c = context_of(p[0]);
    const int64_t T = tokens_of(p[2], "q");
    const Rows q = rows_of(c, p[2], T, c.n_heads, "q"), k = rows_of(c, p[3], T, c.n_kv, "k"),
               v = rows_of(c, p[4], T, c.n_kv, "v"), qo = rows_of(c, p[10], T, c.n_heads, "q_out");
    return moe_attn_append(c.handle, cache_of(c, p[1]), q.p, q.stride, k.p, k.stride, v.p, v.stride,
                           positions_of(c, p[5], T), slots_of(c, p[6], T), T, floats(c, p[7], c.d, "q_weight"),
                           floats(c, p[8], c.d, "k_weight"), to_float(p[9]), qo.p, qo.stride, to_ptr(p[11]));
  });
}

// (context, cache, k, v, slots, stream)
PyObject *write(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return call<6>(args, n, [](PyObject *const *p) {
    const Context c = context_of(p[0]);
    const int64_t T = tokens_of(p[2], "k");
    const Rows k = rows_of(c, p[2], T, c.n_kv, "k"), v = rows_of(c, p[3], T, c.n_kv, "v");
    return moe_attn_write(c.handle, cache_of(c, p[1]), k.p, k.stride, v.p, v.stride, slots_of(c, p[4], T), T,
                          to_ptr(p[5]));
  });
}

// (context, cache, slots, k_out, v_out, stream)
PyObject *read(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return call<6>(args, n, [](PyObject *const *p) {
    const Context c = context_of(p[0]);
    const int64_t T = tokens_of(p[2], "slots");
    const Rows k = rows_of(c, p[3], T, c.n_kv, "k_out"), v = rows_of(c, p[4], T, c.n_kv, "v_out");
    return moe_attn_read(c.handle, cache_of(c, p[1]), slots_of(c, p[2], T), T, k.p, k.stride, v.p, v.stride,
                         to_ptr(p[5]));
  });
}

// (context, cache, q, page_table, seq_lens, starts, scale, softcap, slopes, window, out, lse, stream)
PyObject *decode(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return call<13>(args, n, [](PyObject *const *p) {
    const Context c = context_of(p[0]);
    const int64_t B = tokens_of(p[2], "q");
    const Rows q = rows_of(c, p[2], B, c.n_heads, "q");
    const at::Tensor &table = tensor_of(p[3], "page_table");
    if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != B || !on(table, c) ||
        (table.size(1) > 1 && table.stride(1) != 1))
      raise("page_table must be int32 [%lld, max_pages] on cuda:%lld with contiguous rows", (long long)B,
            (long long)c.index);
    if (p[4] == Py_None) raise("seq_lens are needed");
    const Rows out = rows_of(c, p[10], B, c.n_heads, "out");
    if (out.stride != c.n_heads * c.d) raise("out must be contiguous");
    float *lse = nullptr;
    if (p[11] != Py_None) {
      const at::Tensor &t = tensor_of(p[11], "lse");
      if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != B || t.size(1) != c.n_heads ||
          !on(t, c) || !t.is_contiguous())
        misfit(c, p[11], "lse", "contiguous f32 " + dims({B, c.n_heads}));
      lse = static_cast<float *>(t.data_ptr());
    }
    const int64_t window = to_int(p[9]);
    if (window < 0 || window > INT32_MAX) raise("window must be 0 or a positive int32");
    return moe_attn_decode(c.handle, cache_of(c, p[1]), q.p, q.stride,
                           static_cast<const int32_t *>(table.data_ptr()), table.stride(0), table.size(1),
                           ints(c, p[4], B, "seq_lens"), ints(c, p[5], B, "starts"), B, to_float(p[6]),
                           to_float(p[7]), floats(c, p[8], c.n_heads, "slopes"), (int32_t)window, out.p,
                           lse, to_ptr(p[12]));
  });
}

#define FASTCALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FASTCALL(norm_rope), FASTCALL(append), FASTCALL(write),
                         FASTCALL(read),      FASTCALL(decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&module); }
