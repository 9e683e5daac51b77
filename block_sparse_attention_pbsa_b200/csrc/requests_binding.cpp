// Python arguments of the entry points for requests over a 4-bit cache: tensors checked and their pointers handed to
// libpbsa.so.  Those calls are made for every layer and step, and last 2 to 9 us on the GPU: the same checks in Python,
// with ctypes, took 7 to 12 us a call, here 2 to 4.  Nothing else is done here, and nothing is kept between calls.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits>
#include <stdexcept>
#include <string>

#include "pbsa.h"

namespace {

// libpbsa.so's entry points, as the loader found them
decltype(&pbsa_request_tables) f_tables;
decltype(&pbsa_append_q4) f_append;
decltype(&pbsa_expand_q4) f_expand;
decltype(&pbsa_attend_q4) f_attend;
decltype(&pbsa_q4_block_bytes) f_block_bytes;
decltype(&pbsa_attend_q4_workspace_bytes) f_ws_bytes;

struct Refused : std::runtime_error {   // a ValueError
  using std::runtime_error::runtime_error;
};
struct Raised {};                       // a Python error is set

std::string type_name(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    default: return c10::toString(t);
  }
}

// A call's device and stream.
struct Env {
  int index;
  void* stream;
  explicit Env(PyObject* s) : index(c10::cuda::current_device()) {
    if (s == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(index).stream();
      return;
    }
    // a launch on another device's stream fails, or runs there on this device's memory
    PyObject* d = PyObject_GetAttrString(s, "device_index");
    if (d != nullptr) {
      const long at = PyLong_AsLong(d);
      Py_DECREF(d);
      if (at == -1 && PyErr_Occurred()) throw Raised();
      if (at != index) throw Refused("stream must be one of the current CUDA device");
    } else if (PyErr_ExceptionMatches(PyExc_AttributeError)) {
      PyErr_Clear();   // a stream of another library, which does not tell
    } else {
      throw Raised();
    }
    PyObject* h = PyObject_GetAttrString(s, "cuda_stream");
    if (h == nullptr) throw Raised();
    stream = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Raised();
  }
};

int to_int(int64_t n, const char* name) {
  if (n < std::numeric_limits<int>::min() || n > std::numeric_limits<int>::max())
    throw Refused(std::string(name) + " does not fit 32 bits");
  return (int)n;
}
int number(PyObject* o, const char* name) {
  const long n = PyLong_AsLong(o);
  if (n == -1 && PyErr_Occurred()) throw Raised();
  return to_int(n, name);
}

const at::Tensor& tensor(PyObject* o, at::ScalarType type, const char* name, const Env& env) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != env.index)
    throw Refused(std::string(name) + " must be a tensor of the current CUDA device");
  if (t.scalar_type() != type)
    throw Refused(std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
  return t;
}
// ... contiguous, of `numel` elements (any number if negative)
const at::Tensor& dense(PyObject* o, at::ScalarType type, const char* name, int64_t numel, const Env& env) {
  const at::Tensor& t = tensor(o, type, name, env);
  if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
  if (numel >= 0 && t.numel() != numel)
    throw Refused(std::string(name) + " must have " + std::to_string(numel) + " elements, got " + std::to_string(t.numel()));
  return t;
}
template <typename T = int>
T* pointer(PyObject* o, at::ScalarType type, const char* name, int64_t numel, const Env& env) {
  return static_cast<T*>(dense(o, type, name, numel, env).data_ptr());
}
int* ints(PyObject* o, const char* name, int64_t numel, const Env& env) { return pointer<int>(o, at::kInt, name, numel, env); }

// [tokens, heads, d] whose tokens may lie apart
struct Tokens {
  void* p;
  long long ld;
  int n;
  Tokens(PyObject* o, at::ScalarType type, const char* name, int64_t heads, int64_t d, const Env& env) {
    const at::Tensor& t = tensor(o, type, name, env);
    if (t.dim() != 3 || t.size(1) != heads || t.size(2) != d)
      throw Refused(std::string(name) + " must be [tokens, " + std::to_string(heads) + ", " + std::to_string(d) + "]");
    n = to_int(t.size(0), name);
    if (n > 0 && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d)))
      throw Refused(std::string(name) + ": the heads of a token must be contiguous");
    p = t.data_ptr();
    ld = n > 1 ? t.stride(0) : heads * d;
  }
};

void* workspace(PyObject* o, size_t need, const Env& env) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refused("ws must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != env.index) throw Refused("ws must be a tensor of the current CUDA device");
  if (!t.is_contiguous() || (size_t)t.nbytes() < need)
    throw Refused("ws must be contiguous and hold " + std::to_string(need) + " bytes");
  return t.data_ptr();
}

struct Geometry {
  pbsa_req_geom g;
  at::ScalarType type;
  int64_t block;
  explicit Geometry(PyObject* o) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Raised();
    const bool ok = b.len == (Py_ssize_t)sizeof(g);
    if (ok) memcpy(&g, b.buf, sizeof(g));
    PyBuffer_Release(&b);
    if (!ok) throw Refused("g must be a ReqGeom");
    type = g.dtype == PBSA_BF16 ? at::kBFloat16 : at::kFloat;
    block = (int64_t)f_block_bytes(&g);
  }
};

void shape2(PyObject* o, const char* name, const Env& env, int* rows, int* ld) {
  const at::Tensor& t = dense(o, at::kInt, name, -1, env);
  if (t.dim() != 2) throw Refused(std::string(name) + " must be two-dimensional");
  *rows = to_int(t.size(0), name);
  *ld = to_int(t.size(1), name);
}

template <typename F>
PyObject* call(const char* name, Py_ssize_t want, Py_ssize_t got, F f) {
  if (want != got) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
    return nullptr;
  }
  if (f_tables == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "libpbsa.so is not loaded");
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}
// the call itself, without the interpreter's lock
template <typename F>
int unlocked(F f) {
  PyThreadState* s = PyEval_SaveThread();
  const int code = f();
  PyEval_RestoreThread(s);
  return code;
}

PyObject* request_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("request_tables", 13, n, [&] {
    const Env env(a[12]);
    int R, ld;
    shape2(a[2], "block_table", env, &R, &ld);
    const int T = to_int(dense(a[9], at::kInt, "slot_map", -1, env).numel(), "slot_map");
    const int S = to_int(dense(a[3], at::kInt, "free_slot", -1, env).numel(), "free_slot");
    const int *step = ints(a[0], "step_len", R, env), *seq = ints(a[1], "seq_len", R, env);
    int *table = ints(a[2], "block_table", -1, env), *stack = ints(a[3], "free_slot", -1, env);
    const int* cnt = ints(a[4], "free_cnt", 1, env);
    int *q_start = ints(a[5], "q_start", (int64_t)R + 1, env), *q_len = ints(a[6], "q_len", R, env);
    int *kv_len = ints(a[7], "kv_len", R, env), *cnt_out = ints(a[8], "free_cnt_out", 1, env);
    int* map = T > 0 ? ints(a[9], "slot_map", -1, env) : nullptr;
    int* position = a[10] == Py_None ? nullptr : ints(a[10], "position", T, env);
    void* ws = workspace(a[11], 256, env);
    return unlocked([&] {
      return f_tables(step, seq, R, table, ld, stack, cnt, S, T, q_start, q_len, kv_len, cnt_out, map, position, ws, env.stream);
    });
  });
}

PyObject* append_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("append_q4", 8, n, [&] {
    const Env env(a[7]);
    const Geometry geo(a[0]);
    const pbsa_req_geom& g = geo.g;
    const Tokens k(a[1], geo.type, "k", g.kv_heads, g.head_dim, env), v(a[2], geo.type, "v", g.kv_heads, g.head_dim, env);
    if (k.n != v.n) throw Refused("k and v must have the same number of tokens");
    const int* map = ints(a[3], "slot_map", k.n, env);
    const int slots = number(a[5], "pool_slots");
    void* pool = pointer<void>(a[4], at::kByte, "pool", geo.block * g.kv_heads * slots, env);
    void* ws = workspace(a[6], 256, env);
    return unlocked([&] { return f_append(&g, k.p, k.ld, v.p, v.ld, k.n, map, pool, slots, ws, env.stream); });
  });
}

PyObject* expand_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("expand_q4", 8, n, [&] {
    const Env env(a[7]);
    const Geometry geo(a[0]);
    const pbsa_req_geom& g = geo.g;
    const int slots = number(a[2], "pool_slots");
    const void* pool = pointer<void>(a[1], at::kByte, "pool", geo.block * g.kv_heads * slots, env);
    const at::Tensor& src = dense(a[3], at::kInt, "src_slot", -1, env);
    const int m = to_int(src.numel(), "src_slot");
    const int64_t size = (int64_t)g.kv_heads * m * 64 * g.head_dim;
    void *k = pointer<void>(a[4], geo.type, "k_pool", size, env), *v = pointer<void>(a[5], geo.type, "v_pool", size, env);
    void* ws = workspace(a[6], 256, env);
    const int* from = static_cast<const int*>(src.data_ptr());
    return unlocked([&] { return f_expand(&g, pool, slots, from, m, k, v, ws, env.stream); });
  });
}

PyObject* attend_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("attend_q4", 14, n, [&] {
    const Env env(a[13]);
    const Geometry geo(a[0]);
    const pbsa_req_geom& g = geo.g;
    const Tokens q(a[1], geo.type, "q", g.q_heads, g.head_dim, env), o(a[10], geo.type, "o", g.q_heads, g.head_dim, env);
    if (q.n != o.n) throw Refused("o must have q's tokens");
    int R, ld;
    shape2(a[8], "block_table", env, &R, &ld);
    const at::Tensor& start = dense(a[2], at::kInt, "q_start", -1, env);
    if (start.numel() != R && start.numel() != (int64_t)R + 1)
      throw Refused("q_start must have " + std::to_string(R) + " or " + std::to_string((int64_t)R + 1) + " elements, got " +
                    std::to_string(start.numel()));
    const int *q_len = ints(a[3], "q_len", R, env), *kv_len = ints(a[4], "kv_len", R, env);
    const int max_q = number(a[5], "max_q_len"), slots = number(a[7], "pool_slots");
    const void* pool = pointer<void>(a[6], at::kByte, "pool", geo.block * g.kv_heads * slots, env);
    const int* table = ints(a[8], "block_table", -1, env);
    const int causal = PyObject_IsTrue(a[9]);
    if (causal < 0) throw Raised();
    float* lse = a[11] == Py_None ? nullptr : pointer<float>(a[11], at::kFloat, "lse", (int64_t)g.q_heads * q.n, env);
    if (a[12] == Py_None) throw Refused("pbsa_attend_q4 needs a workspace");
    void* ws = workspace(a[12], f_ws_bytes(&g), env);
    const int* q_start = static_cast<const int*>(start.data_ptr());
    return unlocked([&] {
      return f_attend(&g, q.p, q.ld, q.n, q_start, q_len, kv_len, R, max_q, pool, slots, table, ld, causal ? PBSA_CAUSAL : 0, o.p,
                      o.ld, lse, ws, env.stream);
    });
  });
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* f[6];
  for (int i = 0; i < 6; ++i) {
    f[i] = n == 6 ? PyLong_AsVoidPtr(a[i]) : nullptr;
    if (f[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "bind takes the addresses of six functions");
      return nullptr;
    }
  }
  f_tables = reinterpret_cast<decltype(f_tables)>(f[0]);
  f_append = reinterpret_cast<decltype(f_append)>(f[1]);
  f_expand = reinterpret_cast<decltype(f_expand)>(f[2]);
  f_attend = reinterpret_cast<decltype(f_attend)>(f[3]);
  f_block_bytes = reinterpret_cast<decltype(f_block_bytes)>(f[4]);
  f_ws_bytes = reinterpret_cast<decltype(f_ws_bytes)>(f[5]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(request_tables), FAST(append_q4), FAST(expand_q4), FAST(attend_q4),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_requests", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__requests() { return PyModule_Create(&module); }
