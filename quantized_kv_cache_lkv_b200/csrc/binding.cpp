// binding.cpp -- the CPython module `_native`: argument checks and calls of
// the serving-step entry points of include/lkv.h from torch tensors.
//
// A decode step makes a few of these calls for every layer, so what the host
// spends on one counts: type, size, contiguity and device of a dozen tensors
// cost about 8 microseconds checked from Python and a tenth of that here.
// Module functions take the arguments of the C calls by position or name, the
// stream last (None: torch's current one).  A nonzero lkv_status raises
// LkvError, and so does a tensor that does not fit (LKV_ERR_INVALID_ARG).
// Integer arguments in a tensor's place are device addresses and go through
// unchecked.
// The entry points' addresses come from the loaded liblkv.so (connect()).
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstring>
#include <exception>
#include <string>

#include "../../include/lkv.h"

namespace {

PyObject* g_error = nullptr;  // lkv.LkvError

struct Entries {
  decltype(&lkv_page_plan) page_plan;
  decltype(&lkv_rope_table) rope_table;
  decltype(&lkv_rope_append_kv) rope_append;
  decltype(&lkv_decode_attention_multi) multi;
  decltype(&lkv_decode_attention_multi_paged) multi_paged;
} g_entry;

struct Failed {};  // a Python error is set

void raise(int status, const char* what) {
  PyObject* e = PyObject_CallFunction(g_error, "is", status, what);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
}

// Product of sizes that no tensor has when it passes 64 bits.
template <typename... Sizes>
int64_t product(int64_t first, Sizes... more) {
  int64_t p = first;
  if ((__builtin_mul_overflow(p, (int64_t)more, &p) || ...)) return INT64_MAX;
  return p;
}

// An entry point's argument names, in order; the last `optional` may be left out (None).
struct Names {
  const char* call;
  int count, optional;
  const char* const* names;
};
constexpr int kMostArgs = 30;

// The arguments of one call, taken in order.
class Args {
 public:
  Args(const Names& n, PyObject* const* a, Py_ssize_t given, PyObject* kwnames) : name_(n.call) {
    if (given > n.count) {
      PyErr_Format(PyExc_TypeError, "%s: %zd arguments given, %d wanted", name_, given, n.count);
      throw Failed{};
    }
    for (int i = 0; i < n.count; ++i) a_[i] = i < given ? a[i] : nullptr;
    const Py_ssize_t named = kwnames == nullptr ? 0 : PyTuple_GET_SIZE(kwnames);
    for (Py_ssize_t k = 0; k < named; ++k) {
      PyObject* key = PyTuple_GET_ITEM(kwnames, k);
      int i = 0;
      while (i < n.count && PyUnicode_CompareWithASCIIString(key, n.names[i]) != 0) ++i;
      if (i == n.count || a_[i] != nullptr) {
        PyErr_Format(PyExc_TypeError, i == n.count ? "%s: no argument %U" : "%s: argument %U given twice", name_, key);
        throw Failed{};
      }
      a_[i] = a[given + k];
    }
    for (int i = 0; i < n.count; ++i)
      if (a_[i] == nullptr) {
        if (i < n.count - n.optional) {
          PyErr_Format(PyExc_TypeError, "%s: argument %s is missing", name_, n.names[i]);
          throw Failed{};
        }
        a_[i] = Py_None;
      }
  }

  int64_t i64() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw Failed{};
    return v;
  }
  int i32() { return number32(next()); }
  float f32() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw Failed{};
    return (float)v;
  }
  PyObject* object() { return next(); }
  PyObject* at(int i) { return a_[i]; }
  bool flag() {
    PyObject* o = next();
    if (o == Py_None) return false;
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Failed{};
    if (v != 0 && v != 1) bad_flag_ = true;
    return v != 0;
  }
  bool bad_flag() const { return bad_flag_; }
  [[noreturn]] void refuse_arg(const char* what) {
    raise(LKV_ERR_INVALID_ARG, (std::string(name_) + ": " + what).c_str());
    throw Failed{};
  }

  // A quantizer spec: an lkv_qspec or (k_bits, v_bits, group).
  lkv_qspec spec() {
    PyObject* o = next();
    lkv_qspec q;
    if ((PyTuple_Check(o) || PyList_Check(o)) && PySequence_Fast_GET_SIZE(o) == 3) {
      q.k_bits = number32(PySequence_Fast_GET_ITEM(o, 0));
      q.v_bits = number32(PySequence_Fast_GET_ITEM(o, 1));
      q.group = number32(PySequence_Fast_GET_ITEM(o, 2));
    } else {
      read(o, &q, sizeof q);
    }
    return q;
  }

  // A ctypes structure, by value.
  template <typename T>
  T structure() {
    T v;
    read(next(), &v, sizeof v);
    return v;
  }

  // Address of a contiguous tensor of this type and at least numel values on the current device.
  template <typename T = void>
  T* ptr(at::ScalarType type, int64_t numel) { return static_cast<T*>(address(next(), type, numel)); }

  // No tensor has room for a negative number of values.
  void* address(PyObject* o, at::ScalarType type, int64_t numel) {
    if (o == Py_None) return nullptr;
    if (PyLong_Check(o)) return number(o);
    const at::Tensor& t = tensor(o);
    if (numel >= 0 && t.scalar_type() == type && t.numel() >= numel && t.is_contiguous() && on_device(t)) return t.data_ptr();
    refuse(t, std::to_string(numel) + " or more contiguous " + c10::toString(type));
  }

  // bf16 [n][heads][D] rows whose heads lie side by side; stride: elements from token to token.
  void* rows(PyObject* s, int64_t n, int64_t heads, int64_t D, int64_t& stride) {
    PyObject* o = next();
    stride = heads * D;
    if (o == Py_None || PyLong_Check(o)) {
      if (s != Py_None) {
        stride = PyLong_AsLongLong(s);
        if (stride == -1 && PyErr_Occurred()) throw Failed{};
      }
      return o == Py_None ? nullptr : number(o);
    }
    const at::Tensor& t = tensor(o);
    // torch gives a dimension of one row or one head any stride
    if (t.scalar_type() == at::kBFloat16 && t.dim() == 3 && t.size(0) >= n && t.size(1) == heads && t.size(2) == D &&
        t.stride(2) == 1 && (t.stride(1) == D || heads == 1) && on_device(t)) {
      if (t.size(0) > 1) stride = t.stride(0);
      return t.data_ptr();
    }
    refuse(t, "BFloat16 [" + std::to_string(n) + "][" + std::to_string(heads) + "][" + std::to_string(D) +
                  "] with the heads of a token side by side");
  }

  // The four cache tensors of `rows` rows; a 16-bit tensor has no pairs.
  struct Cache {
    void* kc;
    float* ksz;
    void* vc;
    float* vsz;
  };
  Cache cache(lkv_qspec spec, int64_t rows, int64_t D) {
    const auto bytes = [&](int bits) {
      const int64_t all = product(rows, D, bits);
      return all == INT64_MAX ? all : all / 8;
    };
    const int64_t pairs = spec.group > 0 ? product(rows, D / spec.group, 2) : 0;
    Cache c{};
    c.kc = ptr(at::kByte, bytes(spec.k_bits));
    c.ksz = spec.k_bits == 16 ? (next(), nullptr) : ptr<float>(at::kFloat, pairs);
    c.vc = ptr(at::kByte, bytes(spec.v_bits));
    c.vsz = spec.v_bits == 16 ? (next(), nullptr) : ptr<float>(at::kFloat, pairs);
    return c;
  }

  // A score rule and the tensors that it names.
  lkv_score_rule rule(int64_t Hq, int64_t B) {
    PyObject* o = next();
    lkv_score_rule r;
    read(o, &r, sizeof r);
    PyObject* t = PyObject_GetAttrString(o, "tensors");
    if (t == nullptr) throw Failed{};
    const bool ok = PyTuple_Check(t) && PyTuple_GET_SIZE(t) == 3;
    try {
      if (ok) {
        address(PyTuple_GET_ITEM(t, 0), at::kFloat, Hq);
        address(PyTuple_GET_ITEM(t, 1), at::kInt, B);
        address(PyTuple_GET_ITEM(t, 2), at::kInt, B);
      }
    } catch (...) {
      Py_DECREF(t);
      throw;
    }
    Py_DECREF(t);
    if (!ok) {
      PyErr_Format(PyExc_TypeError, "%s: an lkv_score_rule wanted", name_);
      throw Failed{};
    }
    return r;
  }

  void* stream() {
    PyObject* o = next();
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    if (PyLong_Check(o)) return number(o);
    PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
    if (s == nullptr) throw Failed{};
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (p == nullptr && PyErr_Occurred()) throw Failed{};
    return p;
  }

 private:
  int number32(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Failed{};
    if (v != (int)v) {
      PyErr_Format(PyExc_OverflowError, "%s: %lld does not fit an int", name_, v);
      throw Failed{};
    }
    return (int)v;
  }

  static void* number(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw Failed{};
    return p;
  }

  PyObject* next() { return a_[i_++]; }

  void read(PyObject* o, void* to, size_t bytes) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Failed{};
    const bool ok = (size_t)b.len == bytes;
    if (ok) std::memcpy(to, b.buf, bytes);
    PyBuffer_Release(&b);
    if (!ok) {
      PyErr_Format(PyExc_TypeError, "%s: a structure of %zu bytes wanted", name_, bytes);
      throw Failed{};
    }
  }

  const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s: a tensor, an address or None wanted, not %s", name_, Py_TYPE(o)->tp_name);
      throw Failed{};
    }
    return THPVariable_Unpack(o);
  }

  bool on_device(const at::Tensor& t) {
    if (!t.is_cuda()) return false;
    if (dev_ < 0) dev_ = c10::cuda::current_device();
    return t.get_device() == dev_;
  }

  [[noreturn]] void refuse(const at::Tensor& t, const std::string& wanted) {
    std::string s = std::string(name_) + ": " + wanted + " on the current device wanted, not " + c10::toString(t.scalar_type()) + " [";
    for (int64_t d = 0; d < t.dim(); ++d) s += (d ? ", " : "") + std::to_string(t.size(d));
    s += "] with strides [";
    for (int64_t d = 0; d < t.dim(); ++d) s += (d ? ", " : "") + std::to_string(t.stride(d));
    s += "] on " + t.device().str();
    raise(LKV_ERR_INVALID_ARG, s.c_str());
    throw Failed{};
  }

  const char* name_;
  PyObject* a_[kMostArgs];  // borrowed for the call
  int i_ = 0, dev_ = -1;
  bool bad_flag_ = false;
};

// Runs f, which returns an lkv_status; no C++ exception leaves.
template <typename F>
PyObject* guarded(const Names& n, PyObject* const* args, Py_ssize_t given, PyObject* kwnames, F f) {
  try {
    if (g_error == nullptr) {
      PyErr_SetString(PyExc_RuntimeError, "_native is not connected to liblkv.so");
      return nullptr;
    }
    Args a(n, args, given, kwnames);
    const int status = f(a);
    if (status == LKV_OK) Py_RETURN_NONE;
    raise(status, n.call);
  } catch (const Failed&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <size_t N>
constexpr Names named(const char* call, int optional, const char* const (&names)[N]) {
  static_assert(N <= kMostArgs, "room for the arguments");
  return Names{call, (int)N, optional, names};
}

constexpr const char* kPlanArgs[] = {"B", "pages_per_seq", "num_pages", "n_cap", "seq_lens", "n_new", "free_pages", "free_cap",
                                     "free_count", "block_table", "new_lens", "cu_new", "positions", "token_seq", "slots",
                                     "free_left", "status", "stream"};
PyObject* page_plan(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded(named("lkv_page_plan", 1, kPlanArgs), args, n, kw, [](Args& a) {
    const int B = a.i32(), pps = a.i32(), pages = a.i32(), cap = a.i32();
    auto* lens = a.ptr<int32_t>(at::kInt, B);
    auto* add = a.ptr<int32_t>(at::kInt, B);
    PyObject* free_pages = a.object();
    const int free_cap = a.i32();
    auto* free = static_cast<int32_t*>(a.address(free_pages, at::kInt, free_cap));
    auto* count = a.ptr<int32_t>(at::kInt, 1);
    auto* table = a.ptr<int32_t>(at::kInt, (int64_t)B * pps);
    auto* new_lens = a.ptr<int32_t>(at::kInt, B);
    auto* cu = a.ptr<int32_t>(at::kInt, (int64_t)B + 1);
    auto* pos = a.ptr<int32_t>(at::kInt, cap);
    auto* seq = a.ptr<int32_t>(at::kInt, cap);
    auto* slots = a.ptr<int64_t>(at::kLong, cap);
    auto* left = a.ptr<int32_t>(at::kInt, 1);
    auto* status = a.ptr<int32_t>(at::kInt, 1);
    return g_entry.page_plan(B, pps, pages, cap, lens, add, free, free_cap, count, table, new_lens, cu, pos, seq, slots,
                             left, status, a.stream());
  });
}

constexpr const char* kTableArgs[] = {"spec", "rows", "table", "stream"};
PyObject* rope_table(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded(named("lkv_rope_table", 1, kTableArgs), args, n, kw, [](Args& a) {
    const auto spec = a.structure<lkv_rope_spec>();
    const int rows = a.i32();
    auto* table = a.ptr<float>(at::kFloat, (int64_t)rows * spec.rot_dim);
    return g_entry.rope_table(spec, rows, table, a.stream());
  });
}

constexpr const char* kAppendArgs[] = {
    "spec", "n_cap", "Hq", "Hkv", "num_pages", "page_tokens", "D", "n_tokens", "positions", "slots", "q", "k", "v", "q_weight",
    "k_weight", "eps", "rot_dim", "interleaved", "table", "table_rows", "q_out", "k_codes", "k_sz", "v_codes", "v_sz",
    "q_stride", "k_stride", "v_stride", "reciprocal", "stream"};
PyObject* rope_append(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded(named("lkv_rope_append_kv", 5, kAppendArgs), args, n, kw, [](Args& a) {
    const lkv_qspec spec = a.spec();
    const int cap = a.i32(), Hq = a.i32(), Hkv = a.i32(), pages = a.i32(), page_tokens = a.i32(), D = a.i32();
    auto* n_tokens = a.ptr<int32_t>(at::kInt, 1);
    auto* positions = a.ptr<int32_t>(at::kInt, cap);
    auto* slots = a.ptr<int64_t>(at::kLong, cap);
    int64_t qs, ks, vs;
    void* q = a.rows(a.at(25), cap, Hq, D, qs);
    void* k = a.rows(a.at(26), cap, Hkv, D, ks);
    void* v = a.rows(a.at(27), cap, Hkv, D, vs);
    void* wq = a.ptr(at::kBFloat16, D);
    void* wk = a.ptr(at::kBFloat16, D);
    const float eps = a.f32();
    const int rot = a.i32(), inter = a.i32();
    PyObject* table_o = a.object();
    const int rows = a.i32();
    auto* table = static_cast<float*>(a.address(table_o, at::kFloat, (int64_t)rows * rot));
    void* q_out = a.ptr(at::kBFloat16, product(cap, Hq, D));
    const auto c = a.cache(spec, product(pages, Hkv, page_tokens), D);
    for (int i = 0; i < 3; ++i) a.object();  // the strides
    const bool reciprocal = a.flag();
    return g_entry.rope_append(spec, cap, Hq, Hkv, pages, page_tokens, D, n_tokens, positions, slots, q, qs, k, ks, v, vs,
                               wq, wk, eps, rot, inter, table, rows, q_out, c.kc, c.ksz, c.vc, c.vsz,
                               a.bad_flag() ? 2 : reciprocal, a.stream());
  });
}

// What both forms of the attention take behind the cache.
struct Tail {
  lkv_score_rule rule;
  float *out, *lse;
  void* ws;
  int64_t bytes;
  void* stream;
};
Tail tail(Args& a, int64_t Hq, int64_t B, int64_t rows, int64_t D) {
  Tail t;
  t.rule = a.rule(Hq, B);
  t.out = a.ptr<float>(at::kFloat, product(rows, Hq, D));
  t.lse = a.ptr<float>(at::kFloat, rows * Hq);
  PyObject* ws = a.object();
  t.bytes = a.i64();
  if (t.bytes < 0) a.refuse_arg("ws_bytes is negative");  // a size_t of it would pass for all the room there is
  t.ws = a.address(ws, at::kByte, t.bytes);
  t.stream = a.stream();
  return t;
}

constexpr const char* kMultiArgs[] = {"spec", "B", "Hq", "Hkv", "T_cap", "D", "max_q", "n_rows", "seq_lens", "cu_q", "q",
                                      "k_codes", "k_sz", "v_codes", "v_sz", "rule", "out", "lse", "workspace", "ws_bytes", "stream"};
PyObject* multi(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded(named("lkv_decode_attention_multi", 1, kMultiArgs), args, n, kw, [](Args& a) {
    const lkv_qspec spec = a.spec();
    const int B = a.i32(), Hq = a.i32(), Hkv = a.i32(), T = a.i32(), D = a.i32(), max_q = a.i32(), rows = a.i32();
    auto* lens = a.ptr<int32_t>(at::kInt, B);
    auto* cu = a.ptr<int32_t>(at::kInt, (int64_t)B + 1);
    void* q = a.ptr(at::kBFloat16, product(rows, Hq, D));
    const auto c = a.cache(spec, product(B, Hkv, T), D);
    const Tail t = tail(a, Hq, B, rows, D);
    return g_entry.multi(spec, B, Hq, Hkv, T, D, max_q, rows, lens, cu, q, c.kc, c.ksz, c.vc, c.vsz, t.rule, t.out, t.lse, t.ws,
                         (size_t)t.bytes, t.stream);
  });
}

constexpr const char* kPagedArgs[] = {"spec", "B", "Hq", "Hkv", "pages_per_seq", "num_pages", "D", "max_q", "n_rows", "seq_lens",
                                      "cu_q", "q", "block_table", "k_pool", "k_sz_pool", "v_pool", "v_sz_pool", "rule", "out",
                                      "lse", "workspace", "ws_bytes", "stream"};
PyObject* multi_paged(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded(named("lkv_decode_attention_multi_paged", 1, kPagedArgs), args, n, kw, [](Args& a) {
    const lkv_qspec spec = a.spec();
    const int B = a.i32(), Hq = a.i32(), Hkv = a.i32(), pps = a.i32(), pages = a.i32(), D = a.i32(), max_q = a.i32(), rows = a.i32();
    auto* lens = a.ptr<int32_t>(at::kInt, B);
    auto* cu = a.ptr<int32_t>(at::kInt, (int64_t)B + 1);
    void* q = a.ptr(at::kBFloat16, product(rows, Hq, D));
    auto* table = a.ptr<int32_t>(at::kInt, (int64_t)B * pps);
    const auto c = a.cache(spec, product(pages, Hkv, LKV_PAGE_TOKENS), D);
    const Tail t = tail(a, Hq, B, rows, D);
    return g_entry.multi_paged(spec, B, Hq, Hkv, pps, pages, D, max_q, rows, lens, cu, q, table, c.kc, c.ksz, c.vc, c.vsz,
                               t.rule, t.out, t.lse, t.ws, (size_t)t.bytes, t.stream);
  });
}

// connect(LkvError, addresses of the five entry points in the order of Entries)
PyObject* connect(PyObject*, PyObject* args) {
  PyObject* error;
  unsigned long long p[5];
  if (!PyArg_ParseTuple(args, "OKKKKK", &error, &p[0], &p[1], &p[2], &p[3], &p[4])) return nullptr;
  static_assert(sizeof(Entries) == sizeof p, "five addresses");
  std::memcpy(&g_entry, p, sizeof p);
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS
PyMethodDef g_methods[] = {
    {"connect", connect, METH_VARARGS, "connect(LkvError, addresses of the entry points)"},
    {"lkv_page_plan", FAST(page_plan),
     "lkv_page_plan(B, pages_per_seq, num_pages, n_cap, seq_lens, n_new, free_pages, free_cap, free_count, block_table, new_lens, "
     "cu_new, positions, token_seq, slots, free_left, status, stream=None)\n--\n\nThe call of include/lkv.h."},
    {"lkv_rope_table", FAST(rope_table), "lkv_rope_table(spec, rows, table, stream=None)\n--\n\nThe call of include/lkv.h."},
    {"lkv_rope_append_kv", FAST(rope_append),
     "lkv_rope_append_kv(spec, n_cap, Hq, Hkv, num_pages, page_tokens, D, n_tokens, positions, slots, q, k, v, q_weight, k_weight, "
     "eps, rot_dim, interleaved, table, table_rows, q_out, k_codes, k_sz, v_codes, v_sz, q_stride=None, k_stride=None, "
     "v_stride=None, reciprocal=None, stream=None)\n--\n\nThe call of include/lkv.h.  q, k, v: bf16 [n_cap][heads][D], views of a fused "
     "projection among them (the strides are for integer addresses only)."},
    {"lkv_decode_attention_multi", FAST(multi),
     "lkv_decode_attention_multi(spec, B, Hq, Hkv, T_cap, D, max_q, n_rows, seq_lens, cu_q, q, k_codes, k_sz, v_codes, v_sz, rule, "
     "out, lse, workspace, ws_bytes, stream=None)\n--\n\nThe call of include/lkv.h."},
    {"lkv_decode_attention_multi_paged", FAST(multi_paged),
     "lkv_decode_attention_multi_paged(spec, B, Hq, Hkv, pages_per_seq, num_pages, D, max_q, n_rows, seq_lens, cu_q, q, block_table, "
     "k_pool, k_sz_pool, v_pool, v_sz_pool, rule, out, lse, workspace, ws_bytes, stream=None)\n--\n\nThe call of include/lkv.h."},
    {nullptr, nullptr, 0, nullptr},
};
#ifdef LKV_NATIVE_KEY
// What the module was built against: the build looks for it in the file.
__attribute__((used)) const char g_key[] = LKV_NATIVE_KEY;
#endif
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
