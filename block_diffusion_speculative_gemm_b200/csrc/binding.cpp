// Calls of the target-side attention operators from Python (module _calls): the
// checks of the tensors and the call itself.  These operators run in 2 to 5 us at
// the smallest sizes, once or more per layer of a decode step; the same checks in
// Python with a ctypes call took 18 us.  dflash.py hands over the addresses of
// the library's functions (bind), so that this module is built without linking to
// libdflash.so, and any build of it can be loaded.
//
// Every function takes its arguments by position and returns the status code.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "dflash.h"

namespace {

decltype(&dflash_qk_norm_rope) g_qk = nullptr;
decltype(&dflash_kv_append_paged) g_append = nullptr;
decltype(&dflash_attention_paged) g_attn = nullptr;

// A refused argument: the Python exception's type and text.
struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void bad_type(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void bad_value(const std::string& s) { throw Refused{PyExc_ValueError, s}; }
struct Raised {};  // a Python exception is set already

std::string type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    default: return std::string("torch.") + c10::toString(t);
  }
}
std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

int dtype_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return DFLASH_F32;
    case at::kBFloat16: return DFLASH_BF16;
    case at::kHalf: return DFLASH_F16;
    default: bad_type(std::string(name) + ": unsupported type " + type_name(t.scalar_type()));
  }
}

struct Call {
  c10::DeviceIndex dev = -1;  // asked for once a CUDA tensor is seen

  const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) bad_value(std::string(name) + " must be a CUDA tensor");
    if (dev < 0) dev = c10::cuda::current_device();
    if (t.get_device() != dev)
      bad_value(std::string(name) + " must be on the current CUDA device " + std::to_string(dev) +
                ", is on cuda:" + std::to_string(t.get_device()));
    return t;
  }
  void of_type(const at::Tensor& t, const char* name, at::ScalarType want) {
    if (t.scalar_type() != want)
      bad_type(std::string(name) + " must be " + type_name(want) + ", got " +
               type_name(t.scalar_type()));
  }
  void of_shape(const at::Tensor& t, const char* name, at::IntArrayRef want) {
    if (t.sizes() != want)
      bad_value(std::string(name) + " must have shape " + shape_text(want) + ", got " +
                shape_text(t.sizes()));
  }
  // A contiguous operand.
  const at::Tensor& whole(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
    return t;
  }
  const at::Tensor& whole(PyObject* o, const char* name, at::ScalarType type) {
    const at::Tensor& t = whole(o, name);
    of_type(t, name, type);
    return t;
  }
  const int32_t* ints(PyObject* o, const char* name, int64_t n) {
    const at::Tensor& t = whole(o, name, at::kInt);
    of_shape(t, name, {n});
    return static_cast<const int32_t*>(t.const_data_ptr());
  }
  // [n_rows, heads, head_dim] with contiguous heads; the row stride in elements.
  const at::Tensor& rows(PyObject* o, const char* name, int64_t& stride) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 3) bad_value(std::string(name) + " must be [n_rows, heads, head_dim]");
    const int64_t n = t.size(0), h = t.size(1), hd = t.size(2);
    if ((t.stride(2) != 1 && hd > 1) || (t.stride(1) != hd && h > 1))
      bad_value(std::string(name) + "'s heads must be contiguous");
    stride = n > 1 ? t.stride(0) : std::max(t.stride(0), h * hd);
    return t;
  }
  const at::Tensor& rows_like(PyObject* o, const char* name, const at::Tensor& like,
                              int64_t& stride) {
    const at::Tensor& t = tensor(o, name);
    of_type(t, name, like.scalar_type());
    of_shape(t, name, like.sizes());
    return rows(o, name, stride);
  }
  const void* gain(PyObject* o, const char* name, const at::Tensor& like) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = whole(o, name, like.scalar_type());
    of_shape(t, name, {like.size(2)});
    return t.const_data_ptr();
  }
  const float* rope(PyObject* o, int64_t hd, int& max_pos) {
    max_pos = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor& t = whole(o, "rope", at::kFloat);
    if (t.dim() != 3 || t.size(0) != 2 || t.size(2) * 2 != hd)
      bad_value("rope must be [2, max_pos, head_dim / 2]");
    // without positions it has no address, which would stand for no rotation
    if (t.size(1) < 1) bad_value("rope has no positions");
    max_pos = count(t.size(1), "rope");
    return static_cast<const float*>(t.const_data_ptr());
  }
  static int count(int64_t n, const char* name) {
    if (n > 0x7fffffff) bad_value(std::string(name) + " is too large");
    return (int)n;
  }
  struct Pool {
    void *k, *v;
    int dtype, n_kv, n_pages, page, max_pages;
    const int32_t* table;
  };
  Pool pool(PyObject* ko, PyObject* vo, PyObject* to, int64_t hd, int64_t n_kv, int64_t batch) {
    const at::Tensor& k = whole(ko, "k_pool");
    Pool p;
    p.dtype = dtype_of(k, "k_pool");
    const at::Tensor& v = whole(vo, "v_pool", k.scalar_type());
    of_shape(v, "v_pool", k.sizes());
    if (k.dim() != 4 || (n_kv >= 0 && k.size(1) != n_kv) || k.size(3) != hd)
      bad_value("k_pool must be [n_pages, n_kv, page_size, head_dim]");
    const at::Tensor& t = whole(to, "page_table", at::kInt);
    if (t.dim() != 2 || t.size(0) != batch) bad_value("page_table must be [batch, max_pages]");
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    p.n_kv = count(k.size(1), "k_pool");
    p.n_pages = count(k.size(0), "k_pool");
    p.page = count(k.size(2), "k_pool");
    p.max_pages = count(t.size(1), "page_table");
    p.table = static_cast<const int32_t*>(t.const_data_ptr());
    return p;
  }
  void* stream(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Raised{};
    void* s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!s && PyErr_Occurred()) throw Raised{};
    return s;
  }
  // The request count that the tensor `start_pos` stands for.
  int batch_of(PyObject* o) {
    const at::Tensor& t = whole(o, "start_pos", at::kInt);
    if (t.dim() != 1) bad_value("start_pos must be [batch]");
    return count(t.size(0), "start_pos");
  }
};

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
int integer(PyObject* o, const char* name) {
  int over = 0;
  const long v = PyLong_AsLongAndOverflow(o, &over);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (over || v > 0x7fffffffL || v < -0x80000000L) bad_value(std::string(name) + " is out of range");
  return (int)v;
}

// Gives up the interpreter lock while it lives: a launch can wait for room in its
// stream's queue, and the work in front of it for a host function in Python.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// Runs f, turning what it throws into a Python exception.
template <typename F>
PyObject* guarded(const char* name, Py_ssize_t have, Py_ssize_t want, F f) {
  try {
    if (have != want)
      bad_type(std::string(name) + " takes " + std::to_string(want) + " arguments");
    return PyLong_FromLong(f());
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

void need_bound(const void* f) {
  if (!f) throw std::runtime_error("bind was not called");
}

// q, k, g_q, g_k, rope, cu_rows, start_pos, q_out, k_out, ws, eps, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qk_norm_rope", n, 12, [&]() -> int {
    const bool has_q = a[0] != Py_None, has_k = a[1] != Py_None;
    if (!has_q && !has_k) bad_value("q and k are both None");
    Call c;
    int64_t qs = 0, qos = 0, ks = 0, kos = 0;
    const at::Tensor *q = nullptr, *k = nullptr, *qo = nullptr, *ko = nullptr;
    if (has_q) {
      q = &c.rows(a[0], "q", qs);
      qo = &c.rows_like(a[7], "q_out", *q, qos);
    }
    if (has_k) {
      k = &c.rows(a[1], "k", ks);
      if (has_q) {
        c.of_type(*k, "k", q->scalar_type());
        c.of_shape(*k, "k", {q->size(0), k->size(1), q->size(2)});
      }
      ko = &c.rows_like(a[8], "k_out", *k, kos);
    }
    const at::Tensor& t = has_q ? *q : *k;
    const int dt = dtype_of(t, "q"), batch = c.batch_of(a[6]);
    const void *gq = c.gain(a[2], "g_q", t), *gk = c.gain(a[3], "g_k", t);
    int max_pos;
    const float* rope = c.rope(a[4], t.size(2), max_pos);
    const int32_t* cu = c.ints(a[5], "cu_rows", (int64_t)batch + 1);
    const int32_t* st = c.ints(a[6], "start_pos", batch);
    const at::Tensor& ws = c.whole(a[9], "ws", at::kByte);
    const float eps = (float)number(a[10]);
    const int nq = has_q ? c.count(q->size(1), "q") : 0, nkv = has_k ? c.count(k->size(1), "k") : 0;
    const int hd = c.count(t.size(2), "q"), n_rows = c.count(t.size(0), "q");
    void* const stream = c.stream(a[11]);
    need_bound((const void*)g_qk);
    const Unlocked unlocked;
    return g_qk(nq ? q->const_data_ptr() : nullptr, qs, nkv ? k->const_data_ptr() : nullptr, ks,
                dt, gq, gk, eps, rope, max_pos, cu, st, batch, n_rows, nq, nkv, hd,
                nq ? qo->data_ptr() : nullptr, qos, nkv ? ko->data_ptr() : nullptr, kos,
                ws.data_ptr(), (size_t)ws.numel(), stream);
  });
}

// k, v, g_k, rope, cu_rows, start_pos, k_pool, v_pool, page_table, ws, eps, stream
PyObject* kv_append_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("kv_append_paged", n, 12, [&]() -> int {
    Call c;
    int64_t ks, vs;
    const at::Tensor& k = c.rows(a[0], "k", ks);
    const at::Tensor& v = c.rows_like(a[1], "v", k, vs);
    const int dt = dtype_of(k, "k"), batch = c.batch_of(a[5]);
    const void* gk = c.gain(a[2], "g_k", k);
    int max_pos;
    const float* rope = c.rope(a[3], k.size(2), max_pos);
    const int32_t* cu = c.ints(a[4], "cu_rows", (int64_t)batch + 1);
    const int32_t* st = c.ints(a[5], "start_pos", batch);
    const Call::Pool p = c.pool(a[6], a[7], a[8], k.size(2), k.size(1), batch);
    const at::Tensor& ws = c.whole(a[9], "ws", at::kByte);
    const float eps = (float)number(a[10]);
    const int hd = c.count(k.size(2), "k"), n_rows = c.count(k.size(0), "k");
    void* const stream = c.stream(a[11]);
    need_bound((const void*)g_append);
    const Unlocked unlocked;
    return g_append(k.const_data_ptr(), ks, v.const_data_ptr(), vs, dt, gk, eps, rope, max_pos, cu,
                    st, batch, n_rows, p.n_kv, hd, p.k, p.v, p.dtype, p.n_pages, p.page, p.table,
                    p.max_pages, ws.data_ptr(), (size_t)ws.numel(), stream);
  });
}

// q, cu_rows, start_pos, kv_len, k_pool, v_pool, page_table, out, ws, scale, causal,
// window, lse, stream
PyObject* attention_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("attention_paged", n, 14, [&]() -> int {
    Call c;
    int64_t qs, os;
    const at::Tensor& q = c.rows(a[0], "q", qs);
    const at::Tensor& out = c.rows_like(a[7], "out", q, os);
    const int dt = dtype_of(q, "q"), batch = c.batch_of(a[2]);
    const int32_t* cu = c.ints(a[1], "cu_rows", (int64_t)batch + 1);
    const int32_t* st = c.ints(a[2], "start_pos", batch);
    const int32_t* len = a[3] == Py_None ? nullptr : c.ints(a[3], "kv_len", batch);
    c.of_type(c.tensor(a[4], "k_pool"), "k_pool", q.scalar_type());
    const Call::Pool p = c.pool(a[4], a[5], a[6], q.size(2), -1, batch);
    float* lse = nullptr;
    if (a[12] != Py_None) {
      const at::Tensor& t = c.whole(a[12], "lse", at::kFloat);
      c.of_shape(t, "lse", {q.size(0), q.size(1)});
      lse = static_cast<float*>(t.data_ptr());
    }
    const at::Tensor& ws = c.whole(a[8], "ws", at::kByte);
    const int hd = c.count(q.size(2), "q");
    const float scale = (float)(a[9] == Py_None ? 1.0 / std::sqrt((double)hd) : number(a[9]));
    const int causal = PyObject_IsTrue(a[10]);
    if (causal < 0) throw Raised{};
    const int window = integer(a[11], "window");
    const int n_rows = c.count(q.size(0), "q"), nq = c.count(q.size(1), "q");
    void* const stream = c.stream(a[13]);
    need_bound((const void*)g_attn);
    const Unlocked unlocked;
    return g_attn(q.const_data_ptr(), qs, dt, cu, st, len, batch, n_rows, nq, p.n_kv, hd, p.k, p.v,
                  p.n_pages, p.page, p.table, p.max_pages, scale, causal, window, out.data_ptr(),
                  os, lse, ws.data_ptr(), (size_t)ws.numel(), stream);
  });
}

// Addresses of dflash_qk_norm_rope, dflash_kv_append_paged, dflash_attention_paged.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("bind", n, 3, [&]() -> int {
    void* f[3];
    for (int i = 0; i < 3; ++i) {
      f[i] = PyLong_AsVoidPtr(a[i]);
      if (!f[i]) throw std::runtime_error("bind: no address");
    }
    g_qk = reinterpret_cast<decltype(g_qk)>(f[0]);
    g_append = reinterpret_cast<decltype(g_append)>(f[1]);
    g_attn = reinterpret_cast<decltype(g_attn)>(f[2]);
    return 0;
  });
}

PyMethodDef kMethods[] = {
    {"qk_norm_rope", (PyCFunction)(void*)qk_norm_rope, METH_FASTCALL, nullptr},
    {"kv_append_paged", (PyCFunction)(void*)kv_append_paged, METH_FASTCALL, nullptr},
    {"attention_paged", (PyCFunction)(void*)attention_paged, METH_FASTCALL, nullptr},
    {"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The Python and torch that this module's types are of: looked for in the file before it
// is loaded.
extern "C" __attribute__((visibility("default"), used)) const char kBuiltFor[] = DFLASH_BUILT_FOR;

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
