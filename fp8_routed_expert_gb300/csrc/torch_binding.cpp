// Python binding of the attention's and the projections' calls (moe_attn_*,
// moe_proj_*): checks torch tensors and passes their pointers and strides to the C
// ABI.
//
// A decode step's calls run for a few microseconds on the GPU; reading types,
// shapes, strides and pointers of their tensors attribute by attribute from
// Python and through ctypes took 7 to 8 us of host time each, this takes about
// 2, most of it the launch.  The functions take the context as (handle,
// n_heads, n_kv_heads, head_dim, rope_dim, device index) and a cache as
// (descriptor's address, n_kv_heads, head_dim, device index), tuples that
// attention.py makes once; the projections take (handle, device index).  They raise ValueError for a tensor that does not
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

// (context, q, k, v, q_starts, k_starts, causal, scale, softcap, slopes, window, out, lse, stream)
PyObject *prefill(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return call<14>(args, n, [](PyObject *const *p) {
    const Context c = context_of(p[0]);
    const int64_t Tq = tokens_of(p[1], "q"), Tk = tokens_of(p[2], "k"), starts = tokens_of(p[4], "q_starts");
    if (starts < 1) raise("q_starts must hold one more start than there are sequences");
    const Rows q = rows_of(c, p[1], Tq, c.n_heads, "q"), k = rows_of(c, p[2], Tk, c.n_kv, "k"),
               v = rows_of(c, p[3], Tk, c.n_kv, "v"), out = rows_of(c, p[11], Tq, c.n_heads, "out");
    const int32_t *qs = ints(c, p[4], starts, "q_starts");
    const int32_t *ks = p[5] == Py_None ? nullptr : ints(c, p[5], starts, "k_starts");
    if (ks == nullptr) raise("k_starts are needed");
    float *lse = nullptr;
    if (p[12] != Py_None) {
      const at::Tensor &t = tensor_of(p[12], "lse");
      if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != Tq || t.size(1) != c.n_heads || !on(t, c) ||
          !t.is_contiguous())
        misfit(c, p[12], "lse", "contiguous f32 " + dims({Tq, c.n_heads}));
      lse = static_cast<float *>(t.data_ptr());
    }
    const int64_t window = to_int(p[10]);
    if (window < 0 || window > INT32_MAX) raise("window must be 0 or a positive int32");
    const int causal = PyObject_IsTrue(p[6]);
    if (causal < 0) throw Raised();
    return moe_attn_prefill(c.handle, q.p, q.stride, Tq, k.p, k.stride, v.p, v.stride, Tk, qs, ks, starts - 1, causal,
                            to_float(p[7]), to_float(p[8]), floats(c, p[9], c.n_heads, "slopes"), (int32_t)window, out.p,
                            out.stride, lse, to_ptr(p[13]));
  });
}

struct Proj {
  moe_proj *handle;
  Context on;  // for the checks of tensors
};
Proj proj_of(PyObject *t) {
  if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 2) raise("the context is closed");
  return Proj{static_cast<moe_proj *>(to_ptr(PyTuple_GET_ITEM(t, 0))), Context{nullptr, 0, 0, 0, 0, to_int(PyTuple_GET_ITEM(t, 1))}};
}

// A matrix [rows, columns] whose rows are contiguous, or a null pointer for None.
Rows matrix_of(const Context &c, PyObject *o, at::ScalarType type, const char *what, int64_t rows, int64_t columns, const char *name) {
  if (o == Py_None) return Rows{nullptr, 0};
  const at::Tensor &t = tensor_of(o, name);
  if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != rows || t.size(1) != columns || !on(t, c) ||
      (t.stride(1) != 1 && columns > 1))
    misfit(c, o, name, what + (" " + dims({rows, columns})) + " with contiguous rows");
  // a single row has no stride of its own: any one that fits the alignment
  return Rows{t.data_ptr(), rows > 1 ? t.stride(0) : (columns + 15) / 16 * 16};
}
struct Scales {
  float *p;
  int64_t row, block;
};
Scales scales_of(const Context &c, PyObject *o, int64_t rows, int64_t blocks, const char *name) {
  if (o == Py_None) return Scales{nullptr, 0, 0};
  const at::Tensor &t = tensor_of(o, name);
  if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != rows || t.size(1) != blocks || !on(t, c))
    misfit(c, o, name, "f32 " + dims({rows, blocks}));
  return Scales{static_cast<float *>(t.data_ptr()), rows > 1 ? t.stride(0) : 1, blocks > 1 ? t.stride(1) : 1};
}
// [rows, columns] of a tensor.
void sizes_of(PyObject *o, const char *name, int64_t *rows, int64_t *columns) {
  const at::Tensor &t = tensor_of(o, name);
  if (t.dim() != 2) raise("%s must have two dimensions", name);
  *rows = t.size(0), *columns = t.size(1);
}

// (context, x, residual, weight, eps, residual_out, out, codes, scales, stream)
PyObject *norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return call<10>(args, n, [](PyObject *const *p) {
    const Proj pr = proj_of(p[0]);
    const Context &c = pr.on;
    int64_t T, H;
    sizes_of(p[1], "x", &T, &H);
    const Rows x = matrix_of(c, p[1], at::kBFloat16, "bf16", T, H, "x"),
               r = matrix_of(c, p[2], at::kBFloat16, "bf16", T, H, "residual"),
               ro = matrix_of(c, p[5], at::kBFloat16, "bf16", T, H, "residual_out"),
               o = matrix_of(c, p[6], at::kBFloat16, "bf16", T, H, "out"),
               codes = matrix_of(c, p[7], at::kByte, "uint8", T, H, "codes");
    const Scales sc = scales_of(c, p[8], T, (H + 127) / 128, "scales");
    return moe_proj_norm(pr.handle, x.p, x.stride, r.p, r.stride, T, H, floats(c, p[3], H, "weight"), to_float(p[4]), ro.p,
                         ro.stride, o.p, o.stride, static_cast<uint8_t *>(codes.p), codes.stride, sc.p, sc.row, sc.block,
                         to_ptr(p[9]));
  });
}

// (context, codes, scales, w, w_scale, out, stream)
PyObject *matmul(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return call<7>(args, n, [](PyObject *const *p) {
    const Proj pr = proj_of(p[0]);
    const Context &c = pr.on;
    int64_t M, N, K, k;
    sizes_of(p[1], "codes", &M, &K);
    sizes_of(p[3], "w", &N, &k);
    const Rows a = matrix_of(c, p[1], at::kByte, "uint8", M, K, "codes"), w = matrix_of(c, p[3], at::kByte, "uint8", N, K, "w"),
               o = matrix_of(c, p[5], at::kBFloat16, "bf16", M, N, "out");
    const int64_t blocks = (K + 127) / 128;
    if (p[2] == Py_None || p[4] == Py_None || p[5] == Py_None) raise("scales, w_scale and out are needed");
    const Scales sa = scales_of(c, p[2], M, blocks, "scales"), sw = scales_of(c, p[4], (N + 127) / 128, blocks, "w_scale");
    if (!tensor_of(p[4], "w_scale").is_contiguous()) raise("w_scale must be contiguous");
    return moe_proj_matmul(pr.handle, static_cast<const uint8_t *>(a.p), a.stride, sa.p, sa.row, sa.block, M,
                           static_cast<const uint8_t *>(w.p), w.stride, sw.p, N, K, o.p, o.stride, to_ptr(p[6]));
  });
}

#define FASTCALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FASTCALL(norm_rope), FASTCALL(append), FASTCALL(write),
                         FASTCALL(read),      FASTCALL(decode), FASTCALL(prefill),
                         FASTCALL(norm),      FASTCALL(matmul), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&module); }
