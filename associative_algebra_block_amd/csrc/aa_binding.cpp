// The Python binding of the operators around the row-typed FFN (LayerNorm,
// paged decode attention, the mixture-of-experts layer), as an extension
// module: torch tensors in, checked, passed to the C entry points of libaa.so
// as device pointers.
//
// These are calls of a few microseconds, and a dozen checks of tensors in
// Python cost as much as the launch behind them: one LayerNorm of one token
// took 6.8 us a call with its arguments marshalled in Python.  Nothing is
// computed here.  The module is told the addresses of the entry points
// (bind) and links neither libaa.so nor the HIP runtime.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/ScalarType.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <string>

namespace {

typedef int status_t;
constexpr int kBf16 = 0, kF32 = 1;   // aa_dtype_t

// ------------------------------------------------------- entry points ---

struct Entries {
  status_t (*layernorm_fwd)(const void*, const void*, const float*, const float*, void*, void*, float*, float*,
                            int64_t, int64_t, float, int, int, int, void*);
  status_t (*layernorm_bwd)(const void*, const void*, const float*, const float*, const float*, const void*, void*,
                            float*, float*, int64_t, int64_t, int, int, void*, size_t, void*);
  status_t (*kv_append)(const void*, const void*, int64_t, int64_t, int, void*, void*, int64_t, int32_t, int32_t,
                        int32_t, const int32_t*, int64_t, int64_t, const int32_t*, const int32_t*, int64_t, void*);
  status_t (*attn_decode)(const void*, int64_t, int, const void*, const void*, int64_t, int32_t, int32_t, int32_t,
                          int32_t, const int32_t*, int64_t, int64_t, const int32_t*, float, void*, int, void*, size_t,
                          void*);
  status_t (*moe_ffn_fwd)(void*, void*, const void*, const void*, int32_t, int32_t, int32_t, const void*, const void*,
                          const void*, void*, int32_t*, float*, int64_t, int64_t, const int32_t*, void*, size_t,
                          void*);
} entry;
PyObject* current_device;   // () -> index of the current device
PyObject* current_stream;   // index -> the current stream's handle there
PyObject* given_stream;     // (stream, index) -> its handle; raises if it is another device's

// -------------------------------------------------------------- checks ---

// A failed check has set the Python error.
struct Failed {};

[[noreturn]] void fail(PyObject* type, const char* name, const std::string& what) {
  PyErr_SetString(type, (std::string(name) + ": " + what).c_str());
  throw Failed();
}

std::string text(at::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

enum Types { kBFloat = 1, kFloat = 2, kFloats = 3, kInt = 4 };

int type_bit(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return kBFloat;
    case at::kFloat: return kFloat;
    case at::kInt: return kInt;
    default: return 0;
  }
}
int code(const at::Tensor& t) { return t.scalar_type() == at::kFloat ? kF32 : kBf16; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, name, "expected a tensor");
  return THPVariable_Unpack(o);
}

void check_type(const at::Tensor& t, const char* name, int types) {
  if (type_bit(t) & types) return;
  static const char* const names[] = {"", "bfloat16", "float32", "bfloat16 or float32", "int32"};
  fail(PyExc_TypeError, name, std::string("dtype ") + c10::toString(t.scalar_type()) + ", expected " + names[types]);
}

void check_device(const at::Tensor& t, const char* name, int device) {
  if (t.is_cuda() && t.device().index() == device) return;
  fail(PyExc_ValueError, name, "on " + t.device().str() + ", expected cuda:" + std::to_string(device));
}

// Device pointer of a dense tensor of one of the types, the given shape and
// device; of None, none.
void* dense(PyObject* o, const char* name, std::initializer_list<int64_t> shape, int types, int device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  check_type(t, name, types);
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want) fail(PyExc_ValueError, name, "shape " + text(t.sizes()) + ", expected " + text(want));
  check_device(t, name, device);
  if (!t.is_contiguous()) fail(PyExc_ValueError, name, "must be contiguous");
  return t.data_ptr();
}
template <typename T>
T* dense_as(PyObject* o, const char* name, std::initializer_list<int64_t> shape, int types, int device) {
  return static_cast<T*>(dense(o, name, shape, types, device));
}

// n rows of heads x dim values, [n, heads * dim] or [n, heads, dim]: a row is
// dense, the rows may lie further apart.
void* token_rows(const at::Tensor& t, const char* name, int64_t n, int64_t heads, int64_t dim, int types, int device,
                 int64_t* ld) {
  check_type(t, name, types);
  check_device(t, name, device);
  const at::IntArrayRef s = t.sizes(), st = t.strides();
  const bool flat = s.size() == 2 && s[0] == n && s[1] == heads * dim;
  if (!flat && !(s.size() == 3 && s[0] == n && s[1] == heads && s[2] == dim))
    fail(PyExc_ValueError, name, "shape " + text(s) + ", expected " + text({n, heads * dim}) + " or " +
                                     text({n, heads, dim}));
  if (n && ((st.back() != 1 && s.back() > 1) || (!flat && heads > 1 && st[1] != dim)))
    fail(PyExc_ValueError, name, "the values of a token must be contiguous");
  *ld = n > 1 ? st[0] : heads * dim;
  return t.data_ptr();
}

struct Space {
  void* p;
  size_t bytes;
};
Space workspace(PyObject* o, int device) {
  if (o == Py_None) return {nullptr, 0};
  const at::Tensor& t = tensor(o, "workspace");
  check_device(t, "workspace", device);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "workspace", "must be contiguous");
  return {t.data_ptr(), t.nbytes()};
}

// The device of a call's first operand, which must be the current one: the
// launch goes to a stream of the current device.
int call_device(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) fail(PyExc_ValueError, name, "must be a device tensor");
  PyObject* r = PyObject_CallNoArgs(current_device);
  if (!r) throw Failed();
  const long now = PyLong_AsLong(r);
  Py_DECREF(r);
  if (t.device().index() != now)
    fail(PyExc_ValueError, name, "on " + t.device().str() + ", but the current device is " + std::to_string(now));
  return int(now);
}

void* stream_of(PyObject* o, int device) {
  PyObject* index = PyLong_FromLong(device);
  PyObject* r = o == Py_None ? PyObject_CallOneArg(current_stream, index)
                             : PyObject_CallFunctionObjArgs(given_stream, o, index, nullptr);
  Py_DECREF(index);
  if (!r) throw Failed();
  void* s = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  if (PyErr_Occurred()) throw Failed();
  return s;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed();
  return v;
}
int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v != int32_t(v)) fail(PyExc_ValueError, name, "out of range");
  return int32_t(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed();
  return float(v);
}

// Sizes travel to the entry points as int32 where they have that type.
int32_t size32(int64_t v, const char* name) {
  if (v > INT32_MAX) fail(PyExc_ValueError, name, "too large");
  return int32_t(v);
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Failed&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <typename F>
status_t unlocked(F f) {
  status_t st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return st;
}

// --------------------------------------------------------------- calls ---

struct Shape2 {
  int64_t rows, cols;
};
Shape2 two_dims(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) fail(PyExc_ValueError, name, "expected two dimensions");
  return {t.size(0), t.size(1)};
}

// X, gamma, beta, Y, delta, S, mean, rstd, eps, stream
PyObject* layernorm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const at::Tensor& x = tensor(a[0], "X");
    const int dev = call_device(x, "X");
    const auto [M, d] = two_dims(x, "X");
    const void* X = dense(a[0], "X", {M, d}, kFloats, dev);
    const void* delta = dense(a[4], "delta", {M, d}, kFloats, dev);
    const float* gamma = dense_as<float>(a[1], "gamma", {d}, kFloat, dev);
    const float* beta = dense_as<float>(a[2], "beta", {d}, kFloat, dev);
    void* S = dense(a[5], "S", {M, d}, type_bit(x), dev);
    const at::Tensor& y = tensor(a[3], "Y");
    void* Y = dense(a[3], "Y", {M, d}, kFloats, dev);
    float* mean = dense_as<float>(a[6], "mean", {M}, kFloat, dev);
    float* rstd = dense_as<float>(a[7], "rstd", {M}, kFloat, dev);
    const int dt = delta ? code(THPVariable_Unpack(a[4])) : kF32;
    const float eps = real(a[8]);
    void* s = stream_of(a[9], dev);
    return unlocked([&, M = M, d = d] {
      return entry.layernorm_fwd(X, delta, gamma, beta, S, Y, mean, rstd, M, d, eps, code(x), dt, code(y), s);
    });
  });
}

// X, dY, gamma, mean, rstd, dX, dgamma, dbeta, dS, workspace, stream
PyObject* layernorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const at::Tensor& x = tensor(a[0], "X");
    const int dev = call_device(x, "X");
    const auto [M, d] = two_dims(x, "X");
    const void* X = dense(a[0], "X", {M, d}, kFloats, dev);
    const at::Tensor& dy = tensor(a[1], "dY");
    const void* dY = dense(a[1], "dY", {M, d}, kFloats, dev);
    const float* gamma = dense_as<float>(a[2], "gamma", {d}, kFloat, dev);
    const float* mean = dense_as<float>(a[3], "mean", {M}, kFloat, dev);
    const float* rstd = dense_as<float>(a[4], "rstd", {M}, kFloat, dev);
    const void* dS = dense(a[8], "dS", {M, d}, type_bit(x), dev);
    void* dX = dense(a[5], "dX", {M, d}, type_bit(x), dev);
    float* dgamma = dense_as<float>(a[6], "dgamma", {d}, kFloat, dev);
    float* dbeta = dense_as<float>(a[7], "dbeta", {d}, kFloat, dev);
    const Space ws = workspace(a[9], dev);
    void* s = stream_of(a[10], dev);
    return unlocked([&, M = M, d = d] {
      return entry.layernorm_bwd(X, dY, gamma, mean, rstd, dS, dX, dgamma, dbeta, M, d, code(x), code(dy), ws.p,
                                 ws.bytes, s);
    });
  });
}

struct Cache {
  const at::Tensor &k, &table;
  int dev;
  int64_t n_pages, hkv, page, dim, n_seqs, max_pages;
  void *kp, *vp;
  const int32_t* ids;
};
Cache cache(PyObject* k, PyObject* v, PyObject* table) {
  const at::Tensor &kt = tensor(k, "k_pages"), &tt = tensor(table, "page_table");
  Cache c{kt, tt, call_device(kt, "k_pages"), 0, 0, 0, 0, 0, 0, nullptr, nullptr, nullptr};
  if (kt.dim() != 4) fail(PyExc_ValueError, "k_pages", "expected four dimensions");
  c.n_pages = kt.size(0);
  c.hkv = kt.size(1);
  c.page = kt.size(2);
  c.dim = kt.size(3);
  const Shape2 t = two_dims(tt, "page_table");
  c.n_seqs = t.rows;
  c.max_pages = t.cols;
  c.kp = dense(k, "k_pages", {c.n_pages, c.hkv, c.page, c.dim}, kBFloat, c.dev);
  tensor(v, "v_pages");
  c.vp = dense(v, "v_pages", {c.n_pages, c.hkv, c.dim, c.page}, kBFloat, c.dev);
  c.ids = dense_as<int32_t>(table, "page_table", {c.n_seqs, c.max_pages}, kInt, c.dev);
  return c;
}

// K, V, k_pages, v_pages, page_table, pos, seq, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 8, [&] {
    const Cache c = cache(a[2], a[3], a[4]);
    const at::Tensor &k = tensor(a[0], "K"), &v = tensor(a[1], "V"), &pos = tensor(a[5], "pos");
    if (pos.dim() != 1) fail(PyExc_ValueError, "pos", "expected one dimension");
    const int64_t n = pos.size(0);
    int64_t ldk, ldv;
    const void* K = token_rows(k, "K", n, c.hkv, c.dim, kFloats, c.dev, &ldk);
    const void* V = token_rows(v, "V", n, c.hkv, c.dim, type_bit(k), c.dev, &ldv);
    const int32_t* seq = dense_as<int32_t>(a[6], "seq", {n}, kInt, c.dev);
    const int32_t* where = dense_as<int32_t>(a[5], "pos", {n}, kInt, c.dev);
    const int32_t page = size32(c.page, "k_pages"), hkv = size32(c.hkv, "k_pages"), dim = size32(c.dim, "k_pages");
    void* s = stream_of(a[7], c.dev);
    return unlocked([&] {
      return entry.kv_append(K, V, ldk, ldv, code(k), c.kp, c.vp, c.n_pages, page, hkv, dim, c.ids, c.n_seqs,
                             c.max_pages, seq, where, n, s);
    });
  });
}

// Q, k_pages, v_pages, page_table, lengths, O, scale, workspace, stream
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 9, [&] {
    const Cache c = cache(a[1], a[2], a[3]);
    const at::Tensor &q = tensor(a[0], "Q"), &o = tensor(a[5], "O");
    tensor(a[4], "lengths");
    if (o.dim() != 3) fail(PyExc_ValueError, "O", "expected three dimensions");
    const int64_t heads = o.size(1);
    int64_t ldq;
    const void* Q = token_rows(q, "Q", c.n_seqs, heads, c.dim, kFloats, c.dev, &ldq);
    const int32_t* lengths = dense_as<int32_t>(a[4], "lengths", {c.n_seqs}, kInt, c.dev);
    void* O = dense(a[5], "O", {c.n_seqs, heads, c.dim}, kFloats, c.dev);
    const float scale = real(a[6]);
    const Space ws = workspace(a[7], c.dev);
    const int32_t page = size32(c.page, "k_pages"), hkv = size32(c.hkv, "k_pages"), dim = size32(c.dim, "k_pages"),
                  h = size32(heads, "O");
    void* s = stream_of(a[8], c.dev);
    return unlocked([&] {
      return entry.attn_decode(Q, ldq, code(q), c.kp, c.vp, c.n_pages, page, h, hkv, dim, c.ids, c.n_seqs,
                               c.max_pages, lengths, scale, O, code(o), ws.p, ws.bytes, s);
    });
  });
}

// up, down (handles), D, F, out dtype, X, Wr, Wg, Wu, Wd, Y, top_k, normalize, experts, weights, workspace, pos_offset,
// row_types, stream
PyObject* moe_ffn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 19, [&] {
    void* plan[2];
    for (int i = 0; i < 2; ++i) {
      plan[i] = a[i] == Py_None ? nullptr : PyLong_AsVoidPtr(a[i]);
      if (PyErr_Occurred()) throw Failed();
    }
    const int64_t D = integer(a[2]), nw = D * integer(a[3]);
    const at::Tensor &x = tensor(a[5], "X"), &r = tensor(a[6], "Wr");
    const int dev = call_device(x, "X");
    const int64_t M = two_dims(x, "X").rows, E = two_dims(r, "Wr").rows;
    const int32_t top_k = integer32(a[11], "top_k");
    const void* X = dense(a[5], "X", {M, D}, kBFloat, dev);
    const void* Wr = dense(a[6], "Wr", {E, D}, kBFloat, dev);
    const void* Wg = dense(a[7], "Wg_packed", {E, nw}, kBFloat, dev);
    const void* Wu = dense(a[8], "Wu_packed", {E, nw}, kBFloat, dev);
    const void* Wd = dense(a[9], "Wd_packed", {E, nw}, kBFloat, dev);
    void* Y = dense(a[10], "Y", {M, D}, integer(a[4]) == kF32 ? kFloat : kBFloat, dev);
    int32_t* experts = dense_as<int32_t>(a[13], "experts", {M, top_k}, kInt, dev);
    float* weights = dense_as<float>(a[14], "weights", {M, top_k}, kFloat, dev);
    const Space ws = workspace(a[15], dev);
    const int32_t* types = dense_as<int32_t>(a[17], "row_types", {M}, kInt, dev);
    const int normalize = PyObject_IsTrue(a[12]);
    if (normalize < 0) throw Failed();
    const int64_t pos = integer(a[16]);
    const int32_t experts_n = size32(E, "Wr");
    void* s = stream_of(a[18], dev);
    return unlocked([&] {
      return entry.moe_ffn_fwd(plan[0], plan[1], X, Wr, experts_n, top_k, normalize, Wg, Wu, Wd, Y, experts, weights, M,
                               pos, types, ws.p, ws.bytes, s);
    });
  });
}

// bind(addresses of the five entry points in the order of Entries, current
// device, current stream, given stream)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind: expected 8 arguments");
    return nullptr;
  }
  void* f[5];
  for (int i = 0; i < 5; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  entry = {reinterpret_cast<decltype(entry.layernorm_fwd)>(f[0]), reinterpret_cast<decltype(entry.layernorm_bwd)>(f[1]),
           reinterpret_cast<decltype(entry.kv_append)>(f[2]), reinterpret_cast<decltype(entry.attn_decode)>(f[3]),
           reinterpret_cast<decltype(entry.moe_ffn_fwd)>(f[4])};
  for (int i = 5; i < 8; ++i) Py_INCREF(a[i]);
  current_device = a[5];
  current_stream = a[6];
  given_stream = a[7];
  Py_RETURN_NONE;
}

#define AA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {AA_METHOD(bind),      AA_METHOD(layernorm_fwd), AA_METHOD(layernorm_bwd),
                         AA_METHOD(kv_append), AA_METHOD(attn_decode),   AA_METHOD(moe_ffn_fwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_aa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__aa_binding() { return PyModule_Create(&module); }
