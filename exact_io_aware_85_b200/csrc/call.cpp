// call.cpp — argument marshalling of the cache operators as a Python extension module.
//
// These calls run once per decoded token and layer, with up to fifteen tensors each; checked and
// marshalled in Python a call takes the host some 12 us, longer than its kernels take the GPU.
// Each function checks what the Python binding's slow path checks (CUDA tensors of the stated type
// and shape, contiguous, on the current device), calls the library and returns its status, or -1
// where an argument does not fit: the binding then explains which.  No computation happens here.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/fa.h"

namespace {

void* g_fn[6];  // addresses of the library's entry points, in the order of `bind`
enum { kKeyWeights, kEvictKeep, kEvictSlots, kAppend, kRead, kDecode };
// one of them, called by its prototype in fa.h
#define FA_ENTRY(i, f) Entry<decltype(&f)>{reinterpret_cast<decltype(&f)>(g_fn[i])}
// ... with the interpreter's lock let go: a launch blocks while the stream's queue is full, and what is queued
// before it may need a Python thread
template <typename F>
struct Entry {
  F f;
  template <typename... A>
  int operator()(A... a) const {
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = f(a...);
    Py_END_ALLOW_THREADS;
    return status;
  }
};

constexpr auto BF16 = at::ScalarType::BFloat16;
constexpr auto F32 = at::ScalarType::Float;
constexpr auto U8 = at::ScalarType::Byte;
constexpr auto I32 = at::ScalarType::Int;

// A checked tensor's memory, as whatever the entry point's prototype says.
struct Ptr {
  void* p = nullptr;
  template <typename T>
  operator T*() const {
    return static_cast<T*>(p);
  }
};

// One call's view of its arguments: `bad` once any of them does not fit.
struct Call {
  PyObject* const* args;
  int dev;
  bool bad = false;

  const at::Tensor* tensor(int i) {
    if (!THPVariable_Check(args[i])) return nullptr;
    return &THPVariable_Unpack(args[i]);
  }
  // a required tensor with this number of dimensions (its sizes are read before it is checked)
  const at::Tensor* shaped(int i, int64_t dims) {
    const at::Tensor* t = tensor(i);
    if (!t || t->dim() != dims) {
      bad = true;
      return nullptr;
    }
    return t;
  }
  Ptr get(int i, at::ScalarType type, std::initializer_list<int64_t> shape, bool required) {
    if (args[i] == Py_None) {
      bad = bad || required;
      return {};
    }
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != type || !t->is_cuda() || t->get_device() != dev || !t->is_contiguous() ||
        !t->sizes().equals(c10::IntArrayRef(shape))) {
      bad = true;
      return {};
    }
    return {t->data_ptr()};
  }
  double number(int i) {
    const double v = PyFloat_AsDouble(args[i]);
    if (PyErr_Occurred()) PyErr_Clear(), bad = true;
    return v;
  }
  int integer(int i) {
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(args[i], &overflow);
    if (PyErr_Occurred()) PyErr_Clear(), bad = true;
    if (overflow || v > INT32_MAX || v < INT32_MIN) bad = true;
    return static_cast<int>(v);
  }
  int truth(int i) {
    const int v = PyObject_IsTrue(args[i]);
    if (v < 0) PyErr_Clear(), bad = true;
    return v > 0;
  }
  // None: the current stream of the current device
  void* stream(int i) {
    if (args[i] == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    return PyLong_AsVoidPtr(args[i]);
  }
};

bool fits_int(std::initializer_list<int64_t> v) {
  for (int64_t x : v)
    if (x < 0 || x > INT32_MAX) return false;
  return true;
}

template <typename F>
PyObject* run(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, F body) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    const int dev = c10::cuda::device_count() > 0 ? static_cast<int>(c10::cuda::current_device()) : -1;
    Call c{args, dev};
    return PyLong_FromLong(body(c));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// q, k, lse, w, n_rows, workspace, causal, window or None, scale, stream
PyObject* key_weights(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 10, [](Call& c) -> int {
    const at::Tensor *q = c.shaped(0, 4), *k = c.shaped(1, 4), *w = c.shaped(3, 3), *ws = c.shaped(5, 1);
    if (c.bad) return -1;
    const int64_t B = q->size(0), H = q->size(1), N = q->size(2), d = q->size(3), Hkv = k->size(1), ldw = w->size(2);
    Ptr p[6] = {c.get(0, BF16, {B, H, N, d}, true), c.get(1, BF16, {B, Hkv, N, d}, true), c.get(2, F32, {B, H, N}, true),
                c.get(3, F32, {B, Hkv, ldw}, true), c.get(4, I32, {B}, false), c.get(5, U8, {ws->size(0)}, true)};
    const int causal = c.truth(6);
    const int window = c.args[7] == Py_None ? static_cast<int>(N) : c.integer(7);
    const float scale = static_cast<float>(c.number(8));
    if (c.bad || !fits_int({B, H, Hkv, N, ldw, d})) return -1;
    return FA_ENTRY(kKeyWeights, fa_key_weights)(p[0], p[1], p[2], p[3], p[4], B, H, Hkv, N, ldw, d, causal, window, scale,
                                                 p[5], ws->size(0), c.stream(9));
  });
}

// w, lens, idx, count, n_recent, n_sink, stream
PyObject* evict_keep(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 7, [](Call& c) -> int {
    const at::Tensor *w = c.shaped(0, 3), *idx = c.shaped(2, 3);
    if (c.bad) return -1;
    const int64_t B = w->size(0), Hkv = w->size(1), C = w->size(2), keep = idx->size(2);
    Ptr p[4] = {c.get(0, F32, {B, Hkv, C}, true), c.get(1, I32, {B, Hkv}, false), c.get(2, I32, {B, Hkv, keep}, true),
                c.get(3, I32, {B, Hkv}, true)};
    const int recent = c.integer(4), sink = c.integer(5);
    if (c.bad || !fits_int({B, Hkv, C, keep})) return -1;
    return FA_ENTRY(kEvictKeep, fa_evict_keep)(p[0], p[1], p[2], p[3], B, Hkv, C, keep, recent, sink, c.stream(6));
  });
}

// acc, pos, lens, seen, slots, budget, n_recent, n_sink, stream
PyObject* evict_slots(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 9, [](Call& c) -> int {
    const at::Tensor *acc = c.shaped(0, 3), *slots = c.shaped(4, 3);
    if (c.bad) return -1;
    const int64_t B = acc->size(0), Hkv = acc->size(1), C = acc->size(2), T = slots->size(2);
    Ptr p[5] = {c.get(0, F32, {B, Hkv, C}, true), c.get(1, I32, {B, Hkv, C}, true), c.get(2, I32, {B, Hkv}, true),
                c.get(3, I32, {B}, true), c.get(4, I32, {B, Hkv, T}, true)};
    const int budget = c.integer(5), recent = c.integer(6), sink = c.integer(7);
    if (c.bad || !fits_int({B, Hkv, C, T})) return -1;
    return FA_ENTRY(kEvictSlots, fa_evict_slots)(p[0], p[1], p[2], p[3], p[4], B, Hkv, C, budget, T, recent, sink,
                                                 c.stream(8));
  });
}

// k, v, signs, w, rows, slots, start, n_new, base, kc, ks, vc, vs, acc, pos, stream
PyObject* kv4_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 16, [](Call& c) -> int {
    const at::Tensor *k = c.shaped(0, 4), *kc = c.shaped(9, 4);
    if (c.bad) return -1;
    const int64_t B = kc->size(0), Hkv = kc->size(1), C = kc->size(2), half = kc->size(3), d = 2 * half, N = k->size(2);
    int64_t T = N, ldw = 0;
    if (c.args[4] != Py_None) {
      const at::Tensor* t = c.shaped(4, 3);
      if (t) T = t->size(2);
    } else if (c.args[5] != Py_None) {
      const at::Tensor* t = c.shaped(5, 3);
      if (t) T = t->size(2);
    }
    if (c.args[3] != Py_None) {
      const at::Tensor* t = c.shaped(3, 3);
      if (t) ldw = t->size(2);
    }
    if (c.bad) return -1;
    Ptr p[15] = {c.get(0, BF16, {B, Hkv, N, d}, true), c.get(1, BF16, {B, Hkv, N, d}, true),
                 c.get(2, F32, {d}, false),            c.get(3, F32, {B, Hkv, ldw}, false),
                 c.get(4, I32, {B, Hkv, T}, false),    c.get(5, I32, {B, Hkv, T}, false),
                 c.get(6, I32, {B, Hkv}, false),       c.get(7, I32, {B, Hkv}, false),
                 c.get(8, I32, {B}, false),            c.get(9, U8, {B, Hkv, C, half}, true),
                 c.get(10, BF16, {B, Hkv, C}, true),   c.get(11, U8, {B, Hkv, C, half}, true),
                 c.get(12, BF16, {B, Hkv, C}, true),   c.get(13, F32, {B, Hkv, C}, false),
                 c.get(14, I32, {B, Hkv, C}, false)};
    if (c.bad || !fits_int({B, Hkv, N, T, C, ldw, d})) return -1;
    return FA_ENTRY(kAppend, fa_kv4_append)(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11], p[12],
                                            p[13], p[14], B, Hkv, N, T, C, ldw, d, c.stream(15));
  });
}

// kc, ks, vc, vs, signs, slots, lens, k, v, first, stream
PyObject* kv4_read(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 11, [](Call& c) -> int {
    const at::Tensor *kc = c.shaped(0, 4), *k = c.shaped(7, 4);
    if (c.bad) return -1;
    const int64_t B = kc->size(0), Hkv = kc->size(1), C = kc->size(2), half = kc->size(3), d = 2 * half, T = k->size(2);
    Ptr p[9] = {c.get(0, U8, {B, Hkv, C, half}, true), c.get(1, BF16, {B, Hkv, C}, true),
                c.get(2, U8, {B, Hkv, C, half}, true), c.get(3, BF16, {B, Hkv, C}, true),
                c.get(4, F32, {d}, false),             c.get(5, I32, {B, Hkv, T}, false),
                c.get(6, I32, {B, Hkv}, false),        c.get(7, BF16, {B, Hkv, T, d}, true),
                c.get(8, BF16, {B, Hkv, T, d}, true)};
    const int first = c.integer(9);
    if (c.bad || !fits_int({B, Hkv, T, C, d})) return -1;
    return FA_ENTRY(kRead, fa_kv4_read)(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], B, Hkv, T, C, first, d,
                                        c.stream(10));
  });
}

// q, kc, ks, vc, vs, signs, lens, o, lse, acc, workspace, scale, stream
PyObject* decode_kv4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 13, [](Call& c) -> int {
    const at::Tensor *q = c.shaped(0, 3), *kc = c.shaped(1, 4), *ws = c.shaped(10, 1);
    if (c.bad) return -1;
    const int64_t B = kc->size(0), Hkv = kc->size(1), C = kc->size(2), half = kc->size(3), d = 2 * half, H = q->size(1);
    Ptr p[11] = {c.get(0, BF16, {B, H, d}, true),        c.get(1, U8, {B, Hkv, C, half}, true),
                 c.get(2, BF16, {B, Hkv, C}, true),      c.get(3, U8, {B, Hkv, C, half}, true),
                 c.get(4, BF16, {B, Hkv, C}, true),      c.get(5, F32, {d}, false),
                 c.get(6, I32, {B, Hkv}, true),          c.get(7, BF16, {B, H, d}, true),
                 c.get(8, F32, {B, H}, true),            c.get(9, F32, {B, Hkv, C}, false),
                 c.get(10, U8, {ws->size(0)}, true)};
    const float scale = static_cast<float>(c.number(11));
    if (c.bad || !fits_int({B, H, Hkv, C, d})) return -1;
    return FA_ENTRY(kDecode, fa_decode_kv4)(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], B, H, Hkv, C, d,
                                            scale, p[10], ws->size(0), c.stream(12));
  });
}

// the entry points' addresses: fa_key_weights, fa_evict_keep, fa_evict_slots, fa_kv4_append,
// fa_kv4_read, fa_decode_kv4
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "expected six addresses");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    g_fn[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
#define FA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
    FA_METHOD(bind),       FA_METHOD(key_weights), FA_METHOD(evict_keep), FA_METHOD(evict_slots),
    FA_METHOD(kv4_append), FA_METHOD(kv4_read),    FA_METHOD(decode_kv4), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fa_call", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_call() { return PyModule_Create(&kModule); }
