// bsa_torch.cpp -- the marshalling of the long-stream calls: checks of torch
// tensors, outputs allocated on the current stream, and the call into libbsa.so.
//
// These calls take a few microseconds on the device at a decode step's sizes, as
// long as the same checks take in Python (4 to 6 us a call beside the launch), so
// they are made here.  Nothing is computed: the module gets the library's functions
// by address from the binding, which keeps the signatures, defaults and docstrings.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <memory>
#include <stdexcept>
#include <string>

#include "bsa.h"

namespace {

struct Functions {
  decltype(&bsa_q4_write) q4_write;
  decltype(&bsa_q4_read) q4_read;
  decltype(&bsa_q4_decode) q4_decode;
  decltype(&bsa_q4_window_decode) q4_window_decode;
  decltype(&bsa_window_decode) window_decode;
  decltype(&bsa_window_forward) window_forward;
  decltype(&bsa_window_backward) window_backward;
  decltype(&bsa_window_backward_workspace_bytes) window_backward_workspace_bytes;
} lib = {};
PyObject* check = nullptr;  // check(code, name) raises the binding's exception

// An error to become a Python exception; Raised: one that is set already.
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Raised {};

[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v > INT_MAX || v < INT_MIN) refuse(std::string(name) + " is out of range");
  return static_cast<int>(v);
}

float scale_of(PyObject* o, int64_t d) {
  if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}

std::string text(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return t.get_device();
}

// A contiguous tensor of one shape and type on the call's device.
void* rows(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, int dev) {
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor " + text(shape) +
           " on cuda:" + std::to_string(dev));
  return t.data_ptr();
}

const int32_t* ints(PyObject* o, const char* name, int64_t n, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kInt || !t.is_contiguous() ||
      (n >= 0 && t.numel() != n))
    refuse(std::string(name) + " must be a contiguous int32 tensor" +
           (n >= 0 ? " of " + std::to_string(n) + " entries" : std::string()) + " on cuda:" + std::to_string(dev));
  return static_cast<const int32_t*>(t.data_ptr());
}

const int32_t* ints_or_none(PyObject* o, const char* name, int64_t n, int dev) {
  return o == Py_None ? nullptr : ints(o, name, n, dev);
}

// A bf16 tensor whose last dimension is contiguous; the stride of a dimension of one
// entry is never used.
bsa_view view(const at::Tensor& t, const char* name, at::IntArrayRef shape, int dev) {
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kBFloat16 || t.sizes() != shape)
    refuse(std::string(name) + " must be a bf16 tensor " + text(shape) + " on cuda:" + std::to_string(dev) + ", got " +
           text(t.sizes()));
  const auto s = t.strides();
  const bsa_view v = {t.data_ptr(), shape[0] == 1 ? 0 : s[0], shape[1] == 1 ? 0 : s[1], shape[2] == 1 ? 0 : s[2]};
  if (s[3] != 1 || ((v.stride_b | v.stride_h | v.stride_n) & 7) != 0)
    refuse(std::string(name) + " must have a contiguous last dimension and other strides that are multiples of 8");
  return v;
}

bsa_q4_cache cache_of(PyObject* o, int* dev) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) refuse("the cache must be a Q4Cache");
  const at::Tensor& kc = tensor(PyTuple_GET_ITEM(o, 0), "k_codes");
  const at::Tensor& kp = tensor(PyTuple_GET_ITEM(o, 1), "k_params");
  const at::Tensor& vc = tensor(PyTuple_GET_ITEM(o, 2), "v_codes");
  const at::Tensor& vp = tensor(PyTuple_GET_ITEM(o, 3), "v_params");
  if (kc.dim() != 4) refuse("k_codes must be [B, Hkv, L, d/2]");
  const auto s = kc.sizes();
  for (int i = 0; i < 4; ++i)
    if (s[i] > INT_MAX / 2) refuse("the cache's sizes are out of range");
  *dev = device_of(kc, "k_codes");
  const int64_t params[5] = {s[0], s[1], s[2], s[3] / 16, 2};
  return {rows(kc, "k_codes", s, at::kByte, *dev),
          rows(kp, "k_params", params, at::kHalf, *dev),
          rows(vc, "v_codes", s, at::kByte, *dev),
          rows(vp, "v_params", params, at::kHalf, *dev),
          static_cast<int32_t>(s[0]),
          static_cast<int32_t>(s[1]),
          static_cast<int32_t>(s[2]),
          static_cast<int32_t>(2 * s[3])};
}

// The call with its device current, on that device's current stream.
template <class F>
void call(int dev, const char* name, F f) {
  int rc;
  if (c10::cuda::current_device() == dev) {
    rc = f(static_cast<void*>(c10::cuda::getCurrentCUDAStream(dev).stream()));
  } else {
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    rc = f(static_cast<void*>(c10::cuda::getCurrentCUDAStream(dev).stream()));
  }
  if (rc != BSA_OK) {
    PyObject* r = PyObject_CallFunction(check, "is", rc, name);
    Py_XDECREF(r);
    throw Raised();
  }
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

PyObject* several(std::initializer_list<at::Tensor> list) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(list.size()));
  if (!r) throw Raised();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : list) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw Raised();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

at::Tensor out_rows(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like,
                    int dev) {
  if (o == Py_None) return at::empty(shape, like.options().dtype(type));
  const at::Tensor& t = tensor(o, name);
  rows(t, name, shape, type, dev);
  return t;
}

using Items = PyObject* const*;

struct Release {
  void operator()(PyObject* o) const { Py_DECREF(o); }
};
using Owned = std::unique_ptr<PyObject, Release>;

PyObject* q4_write(Items a) {  // cache, k, v, start, lens
  int dev;
  const bsa_q4_cache c = cache_of(a[0], &dev);
  const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  if (k.dim() != 4 || k.size(2) > INT_MAX) refuse("k, v must be [B, Hkv, T, d]");
  const int64_t shape[4] = {c.B, c.H, k.size(2), c.d};
  const bsa_view kv = view(k, "k", shape, dev), vv = view(v, "v", shape, dev);
  const int32_t *start = ints(a[3], "start", c.B, dev), *lens = ints_or_none(a[4], "lens", c.B, dev);
  call(dev, "bsa_q4_write",
       [&](void* s) { return lib.q4_write(&c, &kv, &vv, start, lens, static_cast<int>(shape[2]), s); });
  Py_RETURN_NONE;
}

PyObject* q4_read(Items a) {  // cache, start, T, lens, out
  int dev;
  const bsa_q4_cache c = cache_of(a[0], &dev);
  const int T = integer(a[2], "T");
  const int32_t *start = ints(a[1], "start", c.B, dev), *lens = ints_or_none(a[3], "lens", c.B, dev);
  if (T < 1) refuse("T must be 1 or more");
  const int64_t shape[4] = {c.B, c.H, T, c.d};
  Owned ko, vo;  // a sequence may make its items anew
  if (a[4] != Py_None) {
    const Py_ssize_t n = PySequence_Check(a[4]) ? PySequence_Size(a[4]) : 0;
    if (n < 0) throw Raised();
    if (n != 2) refuse("out must be a pair of tensors");
    ko.reset(PySequence_GetItem(a[4], 0));
    if (!ko) throw Raised();
    vo.reset(PySequence_GetItem(a[4], 1));
    if (!vo) throw Raised();
  }
  const at::Tensor& like = THPVariable_Unpack(PyTuple_GET_ITEM(a[0], 0));
  at::Tensor k = out_rows(ko ? ko.get() : Py_None, "out k", shape, at::kBFloat16, like, dev);
  at::Tensor v = out_rows(vo ? vo.get() : Py_None, "out v", shape, at::kBFloat16, like, dev);
  call(dev, "bsa_q4_read", [&](void* s) { return lib.q4_read(&c, start, lens, T, k.data_ptr(), v.data_ptr(), s); });
  return several({k, v});
}

// What every decode step shares: q, k_new, v_new, O and LSE.
struct Step {
  void *q, *k_new = nullptr, *v_new = nullptr;
  int H;
  float scale;
  at::Tensor out, lse;
};

Step step(PyObject* q_, int64_t B, int64_t Hkv, int64_t d, int dev, PyObject* scale, PyObject* kn, PyObject* vn,
          PyObject* out, PyObject* lse) {
  const at::Tensor& q = tensor(q_, "q");
  if (q.dim() != 3 || q.size(0) != B || q.size(2) != d || q.size(1) > INT_MAX || q.size(1) % (Hkv > 0 ? Hkv : 1) != 0)
    refuse("q must be [B, H, d] with the cache's B and d, and H a multiple of its heads");
  if ((kn == Py_None) != (vn == Py_None)) refuse("give both k_new and v_new, or neither");
  Step s;
  s.H = static_cast<int>(q.size(1));
  const int64_t shape[3] = {B, s.H, d}, fresh[3] = {B, Hkv, d}, heads[2] = {B, s.H};
  s.q = rows(q, "q", shape, at::kBFloat16, dev);
  if (kn != Py_None) {
    s.k_new = rows(tensor(kn, "k_new"), "k_new", fresh, at::kBFloat16, dev);
    s.v_new = rows(tensor(vn, "v_new"), "v_new", fresh, at::kBFloat16, dev);
  }
  s.scale = scale_of(scale, d);
  s.out = out_rows(out, "out", shape, at::kBFloat16, q, dev);
  s.lse = out_rows(lse, "lse", heads, at::kFloat, q, dev);
  return s;
}

PyObject* q4_decode(Items a) {  // q, cache, seq_len, row_ptr, col_idx, block_size, scale, k_new, v_new, out, lse
  int dev;
  const bsa_q4_cache c = cache_of(a[1], &dev);
  const int bs = integer(a[5], "block_size");
  if (bs < 1) refuse("block_size must be 1 or more");
  Step s = step(a[0], c.B, c.H, c.d, dev, a[6], a[7], a[8], a[9], a[10]);
  const int32_t* n = ints(a[2], "seq_len", c.B, dev);
  const int32_t* rp = ints(a[3], "row_ptr", static_cast<int64_t>(c.H) * (c.L / bs) + 1, dev);
  const int32_t* ci = ints(a[4], "col_idx", -1, dev);
  if (ci == nullptr) ci = rp;  // no entries
  call(dev, "bsa_q4_decode", [&](void* st) {
    return lib.q4_decode(s.q, s.k_new, s.v_new, &c, rp, ci, n, s.H, bs, s.scale, s.out.data_ptr(),
                         static_cast<float*>(s.lse.data_ptr()), st);
  });
  return several({s.out, s.lse});
}

PyObject* q4_window_decode(Items a) {  // q, cache, seq_len, window, sinks, scale, k_new, v_new, out, lse
  int dev;
  const bsa_q4_cache c = cache_of(a[1], &dev);
  const int window = integer(a[3], "window"), sinks = integer(a[4], "sinks");
  Step s = step(a[0], c.B, c.H, c.d, dev, a[5], a[6], a[7], a[8], a[9]);
  const int32_t* n = ints(a[2], "seq_len", c.B, dev);
  call(dev, "bsa_q4_window_decode", [&](void* st) {
    return lib.q4_window_decode(s.q, s.k_new, s.v_new, &c, n, s.H, window, sinks, s.scale, s.out.data_ptr(),
                                static_cast<float*>(s.lse.data_ptr()), st);
  });
  return several({s.out, s.lse});
}

PyObject* window_decode(Items a) {  // q, k_cache, v_cache, seq_len, window, sinks, scale, k_new, v_new, out, lse
  const at::Tensor &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache");
  if (k.dim() != 4) refuse("the caches must be [B, Hkv, L, d]");
  const auto z = k.sizes();
  for (int i = 0; i < 4; ++i)
    if (z[i] > INT_MAX) refuse("the caches' sizes are out of range");
  const int dev = device_of(k, "k_cache");
  void *kc = rows(k, "k_cache", z, at::kBFloat16, dev), *vc = rows(v, "v_cache", z, at::kBFloat16, dev);
  const int window = integer(a[4], "window"), sinks = integer(a[5], "sinks");
  Step s = step(a[0], z[0], z[1], z[3], dev, a[6], a[7], a[8], a[9], a[10]);
  const int32_t* n = ints(a[3], "seq_len", z[0], dev);
  call(dev, "bsa_window_decode", [&](void* st) {
    return lib.window_decode(s.q, s.k_new, s.v_new, kc, vc, n, static_cast<int>(z[0]), s.H, static_cast<int>(z[1]),
                             static_cast<int>(z[2]), static_cast<int>(z[3]), window, sinks, s.scale,
                             s.out.data_ptr(), static_cast<float*>(s.lse.data_ptr()), st);
  });
  return several({s.out, s.lse});
}

struct Heads {
  int B, H, Hkv, N, d, dev;
  int64_t qs[4], ks[4], ls[3];
};

Heads heads_of(const at::Tensor& q, const at::Tensor& k) {
  if (q.dim() != 4 || k.dim() != 4 || q.size(1) % (k.size(1) > 0 ? k.size(1) : 1) != 0)
    refuse("q must be [B, H, N, d] and k, v [B, Hkv, N, d], H a multiple of Hkv");
  for (int i = 0; i < 4; ++i)
    if (q.size(i) > INT_MAX || k.size(i) > INT_MAX) refuse("the sizes are out of range");
  Heads h;
  h.dev = device_of(q, "q");
  h.B = static_cast<int>(q.size(0));
  h.H = static_cast<int>(q.size(1));
  h.N = static_cast<int>(q.size(2));
  h.d = static_cast<int>(q.size(3));
  h.Hkv = static_cast<int>(k.size(1));
  for (int i = 0; i < 4; ++i) h.qs[i] = q.size(i);
  for (int i = 0; i < 4; ++i) h.ks[i] = i == 1 ? h.Hkv : h.qs[i];
  for (int i = 0; i < 3; ++i) h.ls[i] = h.qs[i];
  return h;
}

PyObject* window_forward(Items a) {  // q, k, v, window, sinks, scale, lens, out, lse
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const Heads h = heads_of(q, k);
  const bsa_view qv = view(q, "q", h.qs, h.dev), kv = view(k, "k", h.ks, h.dev), vv = view(v, "v", h.ks, h.dev);
  const int window = integer(a[3], "window"), sinks = integer(a[4], "sinks");
  const float scale = scale_of(a[5], h.d);
  const int32_t* lens = ints_or_none(a[6], "lens", h.B, h.dev);
  const at::Tensor out = a[7] == Py_None ? at::empty_like(q) : tensor(a[7], "out");
  const bsa_view ov = view(out, "out", h.qs, h.dev);
  const at::Tensor lse = out_rows(a[8], "lse", h.ls, at::kFloat, q, h.dev);
  call(h.dev, "bsa_window_forward", [&](void* s) {
    return lib.window_forward(&qv, &kv, &vv, lens, h.B, h.H, h.Hkv, h.N, h.d, window, sinks, scale, &ov,
                              static_cast<float*>(lse.data_ptr()), s);
  });
  return several({out, lse});
}

PyObject* window_backward(Items a) {  // q, k, v, o, do, lse, window, sinks, scale, lens, workspace
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const Heads h = heads_of(q, k);
  const bsa_view qv = view(q, "q", h.qs, h.dev), kv = view(k, "k", h.ks, h.dev), vv = view(v, "v", h.ks, h.dev);
  const bsa_view ov = view(tensor(a[3], "o"), "o", h.qs, h.dev), gv = view(tensor(a[4], "do"), "do", h.qs, h.dev);
  const at::Tensor lse = tensor(a[5], "lse").contiguous();
  const float* lp = static_cast<const float*>(rows(lse, "lse", h.ls, at::kFloat, h.dev));
  const int window = integer(a[6], "window"), sinks = integer(a[7], "sinks");
  const float scale = scale_of(a[8], h.d);
  const int32_t* lens = ints_or_none(a[9], "lens", h.B, h.dev);
  const size_t bytes = lib.window_backward_workspace_bytes(h.B, h.H, h.Hkv, h.N, h.d, window, sinks);
  at::Tensor ws;
  if (a[10] == Py_None) {
    ws = at::empty({static_cast<int64_t>(bytes > 16 ? bytes : 16)}, q.options().dtype(at::kByte));
  } else {
    ws = tensor(a[10], "workspace");
    if (!ws.is_cuda() || ws.get_device() != h.dev || !ws.is_contiguous())
      refuse("workspace must be a contiguous CUDA tensor on q's device");
  }
  const at::Tensor dq = at::empty_like(q), dk = at::empty_like(k), dv = at::empty_like(v);
  const bsa_view dqv = view(dq, "dq", h.qs, h.dev), dkv = view(dk, "dk", h.ks, h.dev), dvv = view(dv, "dv", h.ks, h.dev);
  call(h.dev, "bsa_window_backward", [&](void* s) {
    return lib.window_backward(&qv, &kv, &vv, &ov, &gv, lp, lens, h.B, h.H, h.Hkv, h.N, h.d, window, sinks, scale, &dqv,
                               &dkv, &dvv, ws.data_ptr(), static_cast<size_t>(ws.nbytes()), s);
  });
  return several({dq, dk, dv});
}

// A function of N positional arguments, with C++ exceptions turned into Python's.
template <PyObject* (*F)(Items), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {  // torch's own type, as its allocations raise it
    const Owned torch(PyImport_ImportModule("torch"));
    const Owned type(torch ? PyObject_GetAttrString(torch.get(), "OutOfMemoryError") : nullptr);
    if (type) PyErr_SetString(type.get(), e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// init(check, address of each function in the order of Functions)
PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr Py_ssize_t kCount = sizeof(Functions) / sizeof(void*);
  if (n != 1 + kCount) {
    PyErr_SetString(PyExc_TypeError, "init takes check and the library's functions");
    return nullptr;
  }
  void* at[kCount];
  for (Py_ssize_t i = 0; i < kCount; ++i) {
    at[i] = PyLong_AsVoidPtr(args[1 + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  static_assert(sizeof(lib) == sizeof(at), "one address each");
  memcpy(&lib, at, sizeof(lib));
  Py_INCREF(args[0]);
  Py_XSETREF(check, args[0]);
  Py_RETURN_NONE;
}

#define BSA_ENTRY(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<&name, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&init)), METH_FASTCALL, nullptr},
    BSA_ENTRY(q4_write, 5),
    BSA_ENTRY(q4_read, 5),
    BSA_ENTRY(q4_decode, 11),
    BSA_ENTRY(q4_window_decode, 10),
    BSA_ENTRY(window_decode, 11),
    BSA_ENTRY(window_forward, 9),
    BSA_ENTRY(window_backward, 11),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bsa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The torch and Python that this was built for, which the build gives.
PyMODINIT_FUNC PyInit__bsa_torch() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", BSA_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
