// binding.cpp -- the CPython module `_native`: argument checks and calls of
// the serving-step entry points of include/lkv.h from torch tensors.
//
// A decode step makes a few of these calls for every layer, so what the host
// spends on one counts: type, size, contiguity and device of a dozen tensors
// cost about 8 microseconds checked from Python and a tenth of that here.
// Module functions take the arguments of the C calls in their order, the
// stream last (None: torch's current one), and return the lkv_status; a
// tensor that does not fit raises LkvError with LKV_ERR_INVALID_ARG.  Integer
// arguments in a tensor's place are device addresses and go through unchecked.
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

// The arguments of one call, taken in order.
class Args {
 public:
  Args(const char* name, PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : name_(name), a_(a) {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%s: %zd arguments given, %zd wanted", name, n, want);
      throw Failed{};
    }
  }

  int64_t i64() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw Failed{};
    return v;
  }
  int i32() {
    const int64_t v = i64();
    if (v != (int)v) {
      PyErr_Format(PyExc_OverflowError, "%s: %lld does not fit an int", name_, (long long)v);
      throw Failed{};
    }
    return (int)v;
  }
  float f32() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw Failed{};
    return (float)v;
  }
  PyObject* object() { return next(); }

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

  void* address(PyObject* o, at::ScalarType type, int64_t numel) {
    if (o == Py_None) return nullptr;
    if (PyLong_Check(o)) return number(o);
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() == type && t.numel() >= numel && t.is_contiguous() && on_device(t)) return t.data_ptr();
    refuse(t, std::to_string(numel) + " or more contiguous " + c10::toString(type));
  }

  // bf16 [n][heads][D] rows whose heads lie side by side; stride: elements from token to token.
  void* rows(int64_t n, int64_t heads, int64_t D, int64_t& stride) {
    PyObject *o = next(), *s = next();
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
    const int64_t pairs = spec.group > 0 ? rows * (D / spec.group) * 2 : 0;
    Cache c{};
    c.kc = ptr(at::kByte, rows * D * spec.k_bits / 8);
    c.ksz = spec.k_bits == 16 ? (next(), nullptr) : ptr<float>(at::kFloat, pairs);
    c.vc = ptr(at::kByte, rows * D * spec.v_bits / 8);
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
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)LKV_ERR_INVALID_ARG, s.c_str());
    if (e != nullptr) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    throw Failed{};
  }

  const char* name_;
  PyObject* const* a_;
  Py_ssize_t i_ = 0;
  int dev_ = -1;
};

// Runs f, which returns an lkv_status; no C++ exception leaves.
template <typename F>
PyObject* guarded(F f) {
  try {
    if (g_error == nullptr) {
      PyErr_SetString(PyExc_RuntimeError, "_native is not connected to liblkv.so");
      return nullptr;
    }
    return PyLong_FromLong(f());
  } catch (const Failed&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* page_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a("lkv_page_plan", args, n, 18);
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

PyObject* rope_table(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a("lkv_rope_table", args, n, 4);
    const auto spec = a.structure<lkv_rope_spec>();
    const int rows = a.i32();
    auto* table = a.ptr<float>(at::kFloat, (int64_t)rows * spec.rot_dim);
    return g_entry.rope_table(spec, rows, table, a.stream());
  });
}

PyObject* rope_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a("lkv_rope_append_kv", args, n, 30);
    const auto spec = a.structure<lkv_qspec>();
    const int cap = a.i32(), Hq = a.i32(), Hkv = a.i32(), pages = a.i32(), page_tokens = a.i32(), D = a.i32();
    auto* n_tokens = a.ptr<int32_t>(at::kInt, 1);
    auto* positions = a.ptr<int32_t>(at::kInt, cap);
    auto* slots = a.ptr<int64_t>(at::kLong, cap);
    int64_t qs, ks, vs;
    void* q = a.rows(cap, Hq, D, qs);
    void* k = a.rows(cap, Hkv, D, ks);
    void* v = a.rows(cap, Hkv, D, vs);
    void* wq = a.ptr(at::kBFloat16, D);
    void* wk = a.ptr(at::kBFloat16, D);
    const float eps = a.f32();
    const int rot = a.i32(), inter = a.i32();
    PyObject* table_o = a.object();
    const int rows = a.i32();
    auto* table = static_cast<float*>(a.address(table_o, at::kFloat, (int64_t)rows * rot));
    void* q_out = a.ptr(at::kBFloat16, (int64_t)cap * Hq * D);
    const auto c = a.cache(spec, (int64_t)pages * Hkv * page_tokens, D);
    const int reciprocal = a.i32();
    return g_entry.rope_append(spec, cap, Hq, Hkv, pages, page_tokens, D, n_tokens, positions, slots, q, qs, k, ks, v, vs,
                               wq, wk, eps, rot, inter, table, rows, q_out, c.kc, c.ksz, c.vc, c.vsz, reciprocal, a.stream());
  });
}

PyObject* multi(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a("lkv_decode_attention_multi", args, n, 21);
    const auto spec = a.structure<lkv_qspec>();
    const int B = a.i32(), Hq = a.i32(), Hkv = a.i32(), T = a.i32(), D = a.i32(), max_q = a.i32(), rows = a.i32();
    auto* lens = a.ptr<int32_t>(at::kInt, B);
    auto* cu = a.ptr<int32_t>(at::kInt, (int64_t)B + 1);
    void* q = a.ptr(at::kBFloat16, (int64_t)rows * Hq * D);
    const auto c = a.cache(spec, (int64_t)B * Hkv * T, D);
    const auto rule = a.rule(Hq, B);
    auto* out = a.ptr<float>(at::kFloat, (int64_t)rows * Hq * D);
    auto* lse = a.ptr<float>(at::kFloat, (int64_t)rows * Hq);
    PyObject* ws_o = a.object();
    const int64_t bytes = a.i64();
    void* ws = a.address(ws_o, at::kByte, bytes);
    return g_entry.multi(spec, B, Hq, Hkv, T, D, max_q, rows, lens, cu, q, c.kc, c.ksz, c.vc, c.vsz, rule, out, lse, ws,
                         (size_t)bytes, a.stream());
  });
}

PyObject* multi_paged(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a("lkv_decode_attention_multi_paged", args, n, 23);
    const auto spec = a.structure<lkv_qspec>();
    const int B = a.i32(), Hq = a.i32(), Hkv = a.i32(), pps = a.i32(), pages = a.i32(), D = a.i32(), max_q = a.i32(), rows = a.i32();
    auto* lens = a.ptr<int32_t>(at::kInt, B);
    auto* cu = a.ptr<int32_t>(at::kInt, (int64_t)B + 1);
    void* q = a.ptr(at::kBFloat16, (int64_t)rows * Hq * D);
    auto* table = a.ptr<int32_t>(at::kInt, (int64_t)B * pps);
    const auto c = a.cache(spec, (int64_t)pages * Hkv * LKV_PAGE_TOKENS, D);
    const auto rule = a.rule(Hq, B);
    auto* out = a.ptr<float>(at::kFloat, (int64_t)rows * Hq * D);
    auto* lse = a.ptr<float>(at::kFloat, (int64_t)rows * Hq);
    PyObject* ws_o = a.object();
    const int64_t bytes = a.i64();
    void* ws = a.address(ws_o, at::kByte, bytes);
    return g_entry.multi_paged(spec, B, Hq, Hkv, pps, pages, D, max_q, rows, lens, cu, q, table, c.kc, c.ksz, c.vc, c.vsz,
                               rule, out, lse, ws, (size_t)bytes, a.stream());
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

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {
    {"connect", connect, METH_VARARGS, "connect(LkvError, addresses of the entry points)"},
    {"lkv_page_plan", FAST(page_plan), nullptr},
    {"lkv_rope_table", FAST(rope_table), nullptr},
    {"lkv_rope_append_kv", FAST(rope_append), nullptr},
    {"lkv_decode_attention_multi", FAST(multi), nullptr},
    {"lkv_decode_attention_multi_paged", FAST(multi_paged), nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
