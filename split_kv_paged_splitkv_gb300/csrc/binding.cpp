// The cache operators' arguments, from Python objects to the C ABI.
//
// A decode step makes several of these calls, each with up to 24 arguments of
// which a dozen are tensors.  Checking those and converting the call through
// ctypes costs 8 to 13 us of the interpreter's time, more than the kernels of a
// small step take; here it is under 2.  Every function takes its arguments by
// position (the package's functions name and document them) and returns the
// library's status; a wrong argument raises.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstring>
#include <initializer_list>

#include "splitkv.h"

namespace {

using at::ScalarType;

// Products of counts, at most INT64_MAX.
int64_t times(std::initializer_list<int64_t> factors) {
  int64_t n = 1;
  for (int64_t f : factors)
    if (__builtin_mul_overflow(n, f, &n)) return INT64_MAX;
  return n;
}

bool wrong(PyObject* kind, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(kind, format, args);
  va_end(args);
  return false;
}

// The shape of an array, as the kernels index it.
struct Shape {
  int64_t dim[4];
  int n;
  Shape(std::initializer_list<int64_t> dims) : dim{}, n(0) {
    for (int64_t x : dims) dim[n++] = x;
  }
  int64_t numel() const { return n ? times({dim[0], row()}) : 1; }
  int64_t row() const {  // elements of an entry of the first dimension
    int64_t r = 1;
    for (int i = 1; i < n; ++i) r = times({r, dim[i]});
    return r;
  }
  // Whether a contiguous tensor has these elements where they are looked for: it
  // has no others, or its others are at the end, so that what lies apart by its
  // first dimension's stride are rows of the array.  (A buffer with room for more
  // in another dimension has rows of another length.)  `by_row`: without others,
  // too, it has the array's rows or is flat.
  bool lies_in(const at::Tensor& t, bool by_row) const {
    int64_t first = 0, has = 1, want = 1;
    while (first < t.dim() - 1 && t.size(first) == 1) ++first;
    for (int64_t k = t.dim() - 1; k > first; --k) has = times({has, t.size(k)});
    if (t.numel() == numel() && (!by_row || has == 1)) return true;
    int outer = 0;
    while (outer < n - 1 && dim[outer] == 1) ++outer;
    for (int k = n - 1; k > outer; --k)
      if ((want = times({want, dim[k]})) == has) return true;
    return outer == n - 1;  // a single row
  }
};

// The shapes of a call's arrays.
struct Sizes {
  splitkv_desc_t d{};
  Shape k_pool{}, v_pool{}, table{}, state{};
  ScalarType pool{};
};

bool sizes(PyObject* desc, Sizes& z) {
  Py_buffer b;
  if (PyObject_GetBuffer(desc, &b, PyBUF_SIMPLE) != 0) return false;
  const bool fits = b.len == Py_ssize_t(sizeof(z.d));
  if (fits) memcpy(&z.d, b.buf, sizeof(z.d));
  PyBuffer_Release(&b);
  if (!fits) return wrong(PyExc_TypeError, "desc must be a splitkv_desc_t");
  const splitkv_desc_t& d = z.d;
  const bool nhd = d.kv_layout == SPLITKV_LAYOUT_NHD;
  const int64_t outer = nhd ? d.page_size : d.num_kv_heads, inner = nhd ? d.num_kv_heads : d.page_size;
  z.k_pool = {d.num_pages_total, outer, inner, d.qk_dim};
  z.v_pool = {d.num_pages_total, outer, inner, d.v_dim};
  z.table = {d.batch, d.max_pages_per_seq};
  z.state = {d.batch, d.num_kv_heads, times({d.max_pages_per_seq, d.page_size})};
  z.pool = d.kv_dtype == SPLITKV_FP8_E4M3 ? ScalarType::Byte : ScalarType::BFloat16;
  return true;
}

// One call's arguments in order.  The first that is wrong raises; what follows
// it is not looked at.
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a), ok_(n == want) {
    if (!ok_) wrong(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
  }
  bool ok() const { return ok_; }

  Sizes desc() {
    Sizes z;
    if (PyObject* x = next()) ok_ = sizes(x, z);
    return z;
  }
  int64_t integer() {
    PyObject* x = next();
    if (!x) return 0;
    const long long v = PyLong_AsLongLong(x);
    ok_ = !(v == -1 && PyErr_Occurred());
    return v;
  }
  int32_t int32(const char* name) {
    const int64_t v = integer();
    if (ok_ && v != int32_t(v)) ok_ = wrong(PyExc_OverflowError, "%s does not fit 32 bits", name);
    return int32_t(v);
  }
  float real() {
    PyObject* x = next();
    if (!x) return 0.f;
    const double v = PyFloat_AsDouble(x);
    ok_ = !(v == -1.0 && PyErr_Occurred());
    return float(v);
  }
  // An address, as an integer or None.
  void* address() {
    PyObject* x = next();
    return x ? raw(x) : nullptr;
  }
  // A contiguous tensor that holds an array of `type` and `shape`, on the call's
  // device; addresses and None pass unchecked.
  template <class T>
  T* tensor(const char* name, ScalarType type, const Shape& shape, int64_t device, bool by_row = false) {
    PyObject* x = next();
    if (!x) return nullptr;
    if (x == Py_None || PyLong_Check(x)) return static_cast<T*>(raw(x));
    const at::Tensor* t = typed(name, x, type);
    if (!t) return nullptr;
    if (t->numel() < shape.numel())
      ok_ = wrong(PyExc_ValueError, "%s has %lld elements, the call needs %lld", name, (long long)t->numel(),
                  (long long)shape.numel());
    else if (!shape.lies_in(*t, by_row))
      ok_ = wrong(PyExc_ValueError, "%s has %lld elements, but does not begin with %lld rows of %lld", name,
                  (long long)t->numel(), (long long)shape.dim[0], (long long)shape.row());
    else if (on(name, *t, device))
      return static_cast<T*>(t->data_ptr());
    return nullptr;
  }
  // Two arguments: a workspace and its bytes.  None for the bytes means all of the
  // tensor's; a number is at most those (the kernels write as many).
  void* workspace(int64_t device, size_t* bytes) {
    PyObject* x = next();
    const int64_t given = ok_ && a_[i_] == Py_None ? (next(), -1) : count("workspace_bytes");
    if (!ok_) return nullptr;
    *bytes = given < 0 ? 0 : size_t(given);
    if (x == Py_None || PyLong_Check(x)) return raw(x);
    const at::Tensor* t = typed("workspace", x, ScalarType::Byte);
    if (!t) return nullptr;
    if (given > t->numel()) {
      ok_ = wrong(PyExc_ValueError, "workspace_bytes is %lld, workspace has %lld", (long long)given, (long long)t->numel());
    } else if (on("workspace", *t, device)) {
      if (given < 0) *bytes = size_t(t->numel());
      return t->data_ptr();
    }
    return nullptr;
  }
  // The tokens of a bf16 tensor (`per_token` elements each), or of an argument
  // that says so where it is an address.  Looks ahead: nothing is taken.
  int64_t tokens(int tensor_at, int64_t per_token) {
    PyObject* n = next();
    if (!n) return 0;
    if (n != Py_None) {
      const long long v = PyLong_AsLongLong(n);
      ok_ = !(v == -1 && PyErr_Occurred());
      if (ok_ && v != int32_t(v)) ok_ = wrong(PyExc_OverflowError, "n_tokens does not fit 32 bits");
      return v;
    }
    PyObject* x = a_[tensor_at];
    if (x == Py_None) return 0;
    if (PyLong_Check(x)) {
      ok_ = wrong(PyExc_TypeError, "n_tokens is needed where the tokens are an address");
      return 0;
    }
    if (!is_tensor("the tokens", x)) return 0;
    const int64_t count = THPVariable_Unpack(x).numel() / (per_token > 0 ? per_token : 1);
    if (count != int32_t(count)) ok_ = wrong(PyExc_OverflowError, "n_tokens does not fit 32 bits");
    return count;
  }
  // A bf16 tensor [tokens][heads][dim] (or contiguous [..][..][heads][dim])
  // whose tokens may be strided.
  void* rows(const char* name, int64_t tokens, int64_t heads, int64_t dim, int64_t device, int64_t* stride) {
    *stride = times({heads, dim});
    PyObject* x = next();
    if (!x) return nullptr;
    if (x == Py_None || PyLong_Check(x)) return raw(x);
    if (!is_tensor(name, x)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(x);
    const int64_t nd = t.dim();
    const bool flat = nd == 4 && t.is_contiguous();
    if (t.scalar_type() != ScalarType::BFloat16 || !(nd == 3 || flat) || t.size(nd - 1) != dim || t.size(nd - 2) != heads ||
        times({t.size(0), flat ? t.size(1) : 1}) != tokens) {
      ok_ = wrong(PyExc_ValueError, "%s must be a bfloat16 tensor [%lld][%lld][%lld]", name, (long long)tokens,
                  (long long)heads, (long long)dim);
    } else if (!flat && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != dim))) {
      ok_ = wrong(PyExc_ValueError, "the heads of a token of %s must be adjacent", name);
    } else if (on(name, t, device)) {
      if (!flat && tokens > 1) *stride = t.stride(0);
      return t.data_ptr();
    }
    return nullptr;
  }

 private:
  PyObject* next() { return ok_ ? a_[i_++] : nullptr; }
  void* raw(PyObject* x) {
    if (x == Py_None) return nullptr;
    void* p = PyLong_AsVoidPtr(x);
    ok_ = !(!p && PyErr_Occurred());
    return p;
  }
  // A non-negative integer.
  int64_t count(const char* name) {
    const int64_t v = integer();
    if (ok_ && v < 0) ok_ = wrong(PyExc_ValueError, "%s must be >= 0, got %lld", name, (long long)v);
    return v;
  }
  const at::Tensor* typed(const char* name, PyObject* x, ScalarType type) {
    if (!is_tensor(name, x)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(x);
    if (t.scalar_type() == type && t.is_contiguous()) return &t;
    ok_ = wrong(PyExc_ValueError, "%s must be a contiguous %s tensor, got %s", name, c10::toString(type),
                c10::toString(t.scalar_type()));
    return nullptr;
  }
  bool is_tensor(const char* name, PyObject* x) {
    if (!THPVariable_Check(x))
      ok_ = wrong(PyExc_TypeError, "%s must be a tensor, an address or None, got %s", name, Py_TYPE(x)->tp_name);
    return ok_;
  }
  bool on(const char* name, const at::Tensor& t, int64_t device) {
    if (!t.is_cuda() || t.get_device() != device)
      ok_ = wrong(PyExc_ValueError, "%s is not on the current CUDA device", name);
    return ok_;
  }

  PyObject* const* a_;
  Py_ssize_t i_ = 0;
  bool ok_;
};

// Runs `body` (which returns a status, or anything once its arguments are
// wrong); nothing that torch throws leaves.
template <class F>
PyObject* guarded(Args& in, F&& body) {
  try {
    const int status = in.ok() ? body() : 0;
    return in.ok() ? PyLong_FromLong(status) : nullptr;
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// The library call, with the interpreter free meanwhile.
template <class F>
int call(F&& f) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  return status;
}

constexpr ScalarType kInt = ScalarType::Int, kFloat = ScalarType::Float;

PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  Args in(a, n_args, 22);
  return guarded(in, [&]() -> int {
    const int64_t dev = in.integer();
    const Sizes z = in.desc();
    const splitkv_desc_t& d = z.d;
    const auto* rope = static_cast<const splitkv_rope_t*>(in.address());
    const int64_t axes = in.integer();
    const int64_t n = in.tokens(7, times({d.num_kv_heads, d.qk_dim}));
    // ([n][axes], easily given instead, has as many elements)
    auto* positions = in.tensor<int32_t>("positions", kInt, {axes, n}, dev, true);
    int64_t qs, ks, vs, os;
    void* q = in.rows("q", n, d.num_q_heads, d.qk_dim, dev, &qs);
    void* k = in.rows("k", n, d.num_kv_heads, d.qk_dim, dev, &ks);
    void* v = in.rows("v", n, d.num_kv_heads, d.v_dim, dev, &vs);
    auto* table = in.tensor<int32_t>("block_table", kInt, z.table, dev);
    auto* lens = in.tensor<int32_t>("seq_lens", kInt, {d.batch}, dev);
    void* q_out = in.rows("q_out", n, d.num_q_heads, d.qk_dim, dev, &os);
    void* k_pages = in.tensor<void>("k_pages", z.pool, z.k_pool, dev);
    void* v_pages = in.tensor<void>("v_pages", z.pool, z.v_pool, dev);
    auto* cu = in.tensor<int32_t>("cu_tokens", kInt, {int64_t(d.batch) + 1}, dev);
    const float kv_scale = in.real();
    auto* k_scale = in.tensor<float>("k_scale", kFloat, {d.num_kv_heads}, dev);
    auto* v_scale = in.tensor<float>("v_scale", kFloat, {d.num_kv_heads}, dev);
    auto* weights = in.tensor<float>("key_weights", kFloat, z.state, dev);
    auto* key_positions = in.tensor<int32_t>("key_positions", kInt, z.state, dev);
    auto* status = in.tensor<int32_t>("status", kInt, {1}, dev);
    void* stream = in.address();
    if (!in.ok()) return 0;
    return call([&] {
      return splitkv_append(&d, rope, int32_t(n), cu, positions, q, qs, k, ks, v, vs, table, lens, kv_scale, k_scale,
                            v_scale, q_out, os, k_pages, v_pages, weights, key_positions, status, stream);
    });
  });
}

PyObject* key_weights(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  Args in(a, n_args, 15);
  return guarded(in, [&]() -> int {
    const int64_t dev = in.integer();
    const Sizes z = in.desc();
    const splitkv_desc_t& d = z.d;
    void* q = in.tensor<void>("q", ScalarType::BFloat16, {d.batch, d.q_tokens, d.num_q_heads, d.qk_dim}, dev);
    void* k_pages = in.tensor<void>("k_pages", z.pool, z.k_pool, dev);
    auto* table = in.tensor<int32_t>("block_table", kInt, z.table, dev);
    auto* lens = in.tensor<int32_t>("seq_lens", kInt, {d.batch}, dev);
    auto* lse = in.tensor<float>("lse", kFloat, {d.batch, d.q_tokens, d.num_q_heads}, dev);
    const float scale = in.real(), kv_scale = in.real(), decay = in.real();
    auto* w_in = in.tensor<float>("weights_in", kFloat, z.state, dev);
    auto* w_out = in.tensor<float>("weights_out", kFloat, z.state, dev);
    auto* k_scale = in.tensor<float>("k_scale", kFloat, {d.num_kv_heads}, dev);
    auto* status = in.tensor<int32_t>("status", kInt, {1}, dev);
    void* stream = in.address();
    if (!in.ok()) return 0;
    return call([&] {
      return splitkv_key_weights(&d, q, k_pages, table, lens, lse, scale, kv_scale, k_scale, decay, w_in, w_out, status,
                                 stream);
    });
  });
}

PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  Args in(a, n_args, 18);
  return guarded(in, [&]() -> int {
    const int64_t dev = in.integer();
    const Sizes z = in.desc();
    const splitkv_desc_t& d = z.d;
    const int32_t budget = in.int32("budget"), sink = in.int32("sink"), recent = in.int32("recent");
    void* k_pages = in.tensor<void>("k_pages", z.pool, z.k_pool, dev);
    void* v_pages = in.tensor<void>("v_pages", z.pool, z.v_pool, dev);
    auto* table = in.tensor<int32_t>("block_table", kInt, z.table, dev);
    auto* lens = in.tensor<int32_t>("seq_lens", kInt, {d.batch}, dev);
    auto* w_in = in.tensor<float>("weights_in", kFloat, z.state, dev);
    auto* p_in = in.tensor<int32_t>("positions_in", kInt, z.state, dev);
    auto* w_out = in.tensor<float>("weights_out", kFloat, z.state, dev);
    auto* p_out = in.tensor<int32_t>("positions_out", kInt, z.state, dev);
    auto* lens_out = in.tensor<int32_t>("seq_lens_out", kInt, {d.batch}, dev);
    size_t bytes = 0;
    void* workspace = in.workspace(dev, &bytes);
    auto* status = in.tensor<int32_t>("status", kInt, {1}, dev);
    void* stream = in.address();
    if (!in.ok()) return 0;
    return call([&] {
      return splitkv_evict(&d, budget, sink, recent, k_pages, v_pages, table, lens, w_in, p_in, w_out, p_out, lens_out,
                           workspace, bytes, status, stream);
    });
  });
}

PyObject* cross_attend(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  Args in(a, n_args, 16);
  return guarded(in, [&]() -> int {
    const int64_t dev = in.integer();
    const Sizes z = in.desc();
    const splitkv_desc_t& d = z.d;
    const int64_t n = in.tokens(4, times({d.num_q_heads, d.qk_dim}));
    auto* cu = in.tensor<int32_t>("cu_tokens", kInt, {int64_t(d.batch) + 1}, dev);
    int64_t qs;
    void* q = in.rows("q", n, d.num_q_heads, d.qk_dim, dev, &qs);
    void* k_pages = in.tensor<void>("k_pages", z.pool, z.k_pool, dev);
    void* v_pages = in.tensor<void>("v_pages", z.pool, z.v_pool, dev);
    auto* table = in.tensor<int32_t>("block_table", kInt, z.table, dev);
    auto* lens = in.tensor<int32_t>("seq_lens", kInt, {d.batch}, dev);
    const float scale = in.real();
    void* out = in.tensor<void>("out", ScalarType::BFloat16, {n, d.num_q_heads, d.v_dim}, dev);
    auto* lse = in.tensor<float>("lse", kFloat, {n, d.num_q_heads}, dev);
    size_t bytes = 0;
    void* workspace = in.workspace(dev, &bytes);
    auto* status = in.tensor<int32_t>("status", kInt, {1}, dev);
    void* stream = in.address();
    if (!in.ok()) return 0;
    return call([&] {
      return splitkv_cross_attend(&d, int32_t(n), cu, q, qs, k_pages, v_pages, table, lens, scale, out, lse, workspace,
                                  bytes, status, stream);
    });
  });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST(append), FAST(key_weights), FAST(evict), FAST(cross_attend), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
