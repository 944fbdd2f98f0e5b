// Python's way into the calls around the layers (csa2.py wraps these functions): checks
// the tensors, fills the argument struct and issues the call on the tensors' device.
// In Python the same checks take 5 to 15 us a call on the host, several times the
// launches themselves and most of a decode-sized call (csa2_lora_linear with 12 tensors:
// 25 us a call, 4.2 of them in the library).
//
// A function returns the call's status; a tensor that cannot be passed raises
// TypeError or ValueError.  Nothing is kept between calls.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <limits.h>
#include <string.h>

#include <exception>
#include <optional>

#include "../../include/csa2.h"

namespace {

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kU8 = at::kByte;
constexpr auto kI32 = at::kInt;

struct Raised {};  // a Python error is set

[[noreturn]] void raise(PyObject* kind, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(kind, fmt, ap);
  va_end(ap);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: expected a torch tensor", name);
  return THPVariable_Unpack(o);
}

const char* dtype_name(at::ScalarType t) {
  return t == kBf16 ? "torch.bfloat16" : t == kF32 ? "torch.float32" : t == kU8 ? "torch.uint8" : t == kI32 ? "torch.int32" : c10::toString(t);
}

// Device of a call's first tensor.
int device_of(PyObject* o, const char* name) {
  const int dev = static_cast<int>(tensor(o, name).get_device());
  if (dev < 0) raise(PyExc_ValueError, "%s: CSA2 calls take CUDA tensors (no CPU path)", name);
  return dev;
}

const at::Tensor& checked(PyObject* o, const char* name, at::ScalarType kind, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != kind) raise(PyExc_TypeError, "%s: expected %s, got %s", name, dtype_name(kind), dtype_name(t.scalar_type()));
  const int at = static_cast<int>(t.get_device());
  if (at < 0) raise(PyExc_ValueError, "%s: CSA2 calls take CUDA tensors (no CPU path)", name);
  if (at != dev) raise(PyExc_ValueError, "%s: on cuda:%d, the call's first tensor on cuda:%d", name, at, dev);
  return t;
}

template <class T>
T* place(const at::Tensor& t) {
  void* p = t.data_ptr();
  // a given tensor without elements is not NULL; its length 0 goes along
  return static_cast<T*>(p ? p : reinterpret_cast<void*>(16));
}

int32_t size32(int64_t n, const char* name) {
  if (n > INT_MAX) raise(PyExc_ValueError, "%s: a size of %lld is too large", name, static_cast<long long>(n));
  return static_cast<int32_t>(n);
}

// Rows and columns of a 2-D tensor.
void two_d(const at::Tensor& t, const char* name, int64_t* rows, int64_t* cols) {
  if (t.dim() != 2) raise(PyExc_ValueError, "%s: expected a 2-D tensor, got %d dimensions", name, static_cast<int>(t.dim()));
  *rows = t.size(0);
  *cols = t.size(1);
}

// A 2-D tensor of the given shape whose rows are contiguous (and may be apart).
template <class T, class Ld>
void mat(PyObject* o, const char* name, at::ScalarType kind, int dev, int64_t rows, int64_t cols, T** at, Ld* ld) {
  const at::Tensor& t = checked(o, name, kind, dev);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols) {
    if (t.dim() != 2) raise(PyExc_ValueError, "%s: expected a 2-D tensor, got %d dimensions", name, static_cast<int>(t.dim()));
    raise(PyExc_ValueError, "%s: expected shape [%lld, %lld], got [%lld, %lld]", name, static_cast<long long>(rows),
          static_cast<long long>(cols), static_cast<long long>(t.size(0)), static_cast<long long>(t.size(1)));
  }
  *ld = cols;
  if (!t.is_contiguous()) {
    if ((t.stride(1) != 1 && cols > 1) || t.stride(0) < cols)
      raise(PyExc_ValueError, "%s: expected contiguous rows that do not overlap, got strides (%lld, %lld)", name,
            static_cast<long long>(t.stride(0)), static_cast<long long>(t.stride(1)));
    *ld = t.stride(0);
  }
  *at = place<T>(t);
}

// A contiguous 1-D tensor of n elements, or NULL for None.
template <class T>
T* vec(PyObject* o, const char* name, at::ScalarType kind, int dev, int64_t n) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = checked(o, name, kind, dev);
  if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    raise(PyExc_ValueError, "%s: expected %lld contiguous elements", name, static_cast<long long>(n));
  return place<T>(t);
}

int32_t int_of(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < INT_MIN || v > INT_MAX) raise(PyExc_OverflowError, "%ld does not fit 32 bits", v);
  return static_cast<int32_t>(v);
}
float float_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

// The call's device, made the current one, and its stream: that device's current
// stream, or a handle that the caller gives.
struct Place {
  std::optional<c10::cuda::CUDAGuard> guard;
  cudaStream_t stream;
  Place(int dev, PyObject* given) {
    if (dev != c10::cuda::current_device()) guard.emplace(static_cast<c10::DeviceIndex>(dev));
    if (given == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    } else {
      stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(given));
      if (!stream && PyErr_Occurred()) throw Raised{};
    }
  }
};

// A call's own scratch, from torch's allocator on the call's stream: it may be handed
// out again only behind the call's work (in a capture, within its graph).
struct Scratch {
  void* at;
  Scratch(size_t bytes, cudaStream_t st) : at(c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, st)) {}
  ~Scratch() { c10::cuda::CUDACachingAllocator::raw_delete(at); }
  Scratch(const Scratch&) = delete;
};

// No exception leaves a function that Python calls.
template <class F>
PyObject* guarded(F&& f) {
  try {
    return PyLong_FromLong(f());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}
void expect(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) raise(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
}

// (x, residual, residual_out, gamma, codes, scale, y, eps, stream)
PyObject* add_norm_fp8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    expect(n, 9);
    csa2_add_norm_fp8_args a = {};
    const int dev = device_of(v[0], "x");
    int64_t T, K;
    two_d(tensor(v[0], "x"), "x", &T, &K);
    a.T = size32(T, "x");
    a.K = size32(K, "x");
    mat(v[0], "x", kBf16, dev, T, K, &a.x, &a.ld_x);
    const at::ScalarType kind = tensor(v[1], "residual").scalar_type();
    if (kind != kBf16 && kind != kF32)
      raise(PyExc_TypeError, "residual: expected torch.bfloat16 or torch.float32, got %s", dtype_name(kind));
    a.residual_f32 = kind == kF32;
    mat(v[1], "residual", kind, dev, T, K, &a.residual, &a.ld_residual);
    mat(v[2], "residual_out", kind, dev, T, K, &a.residual_out, &a.ld_residual_out);
    if (v[3] == Py_None) raise(PyExc_TypeError, "gamma: expected a torch tensor");
    a.gamma = vec<float>(v[3], "gamma", kF32, dev, K);
    if (v[4] != Py_None) mat(v[4], "codes", kU8, dev, T, K, &a.codes, &a.ld_codes);
    if (v[5] != Py_None) mat(v[5], "scale", kF32, dev, T, (K + 127) / 128, &a.scale, &a.ld_scale);
    if (v[6] != Py_None) mat(v[6], "y", kBf16, dev, T, K, &a.y, &a.ld_y);
    a.eps = float_of(v[7]);
    const Place at(dev, v[8]);
    return csa2_add_norm_fp8(&a, at.stream);
  });
}

// (x, x_scale, w, w_scale, a, b, row_adapter, out, adapter_scale, out_scale, row_pos, rope_head, rope_theta, w_ready,
//  stream, ws)
PyObject* lora_linear(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    expect(n, 16);
    csa2_lora_linear_args a = {};
    csa2_fp8_linear_args& l = a.base;
    const int dev = device_of(v[0], "x");
    int64_t T, K, N, other;
    two_d(tensor(v[0], "x"), "x", &T, &K);
    two_d(tensor(v[2], "w"), "w", &N, &other);
    l.T = size32(T, "x");
    l.K = size32(K, "x");
    l.N = size32(N, "w");
    const int64_t nb = (K + 127) / 128;
    mat(v[0], "x", kU8, dev, T, K, &l.x, &l.ld_x);
    mat(v[2], "w", kU8, dev, N, K, &l.w, &l.ld_w);
    mat(v[1], "x_scale", kF32, dev, T, nb, &l.x_scale, &l.ld_x_scale);
    mat(v[3], "w_scale", kF32, dev, (N + 127) / 128, nb, &l.w_scale, &l.ld_w_scale);
    const at::ScalarType kind = tensor(v[7], "out").scalar_type();
    if (kind != kF32 && kind != kBf16 && kind != kU8)
      raise(PyExc_TypeError, "out: expected torch.float32, torch.bfloat16 or torch.uint8, got %s", dtype_name(kind));
    l.out_format = kind == kF32 ? CSA2_OUT_F32 : kind == kBf16 ? CSA2_OUT_BF16 : CSA2_OUT_FP8;
    mat(v[7], "out", kind, dev, T, N, &l.out, &l.ld_out);
    if (v[9] != Py_None) mat(v[9], "out_scale", kF32, dev, T, N / 128, &l.out_scale, &l.ld_out_scale);
    l.row_pos = vec<int32_t>(v[10], "row_pos", kI32, dev, T);
    l.rope_head = int_of(v[11]);
    l.rope_theta = float_of(v[12]);
    const int ready = PyObject_IsTrue(v[13]);
    if (ready < 0) throw Raised{};
    l.w_ready = ready;
    const at::Tensor& ta = checked(v[4], "a", kBf16, dev);
    const at::Tensor& tb = checked(v[5], "b", kBf16, dev);
    if (ta.dim() != 3 || !ta.is_contiguous()) raise(PyExc_ValueError, "a: expected a contiguous 3-D tensor");
    if (tb.dim() != 3 || !tb.is_contiguous()) raise(PyExc_ValueError, "b: expected a contiguous 3-D tensor");
    const int64_t count = ta.size(0), rank = ta.size(1);
    if (ta.size(2) != K || tb.size(0) != count || tb.size(1) != N || tb.size(2) != rank)
      raise(PyExc_ValueError, "a, b: expected [n, rank, %lld] and [n, %lld, rank], got [%lld, %lld, %lld] and [%lld, %lld, %lld]",
            static_cast<long long>(K), static_cast<long long>(N), static_cast<long long>(count), static_cast<long long>(rank),
            static_cast<long long>(ta.size(2)), static_cast<long long>(tb.size(0)), static_cast<long long>(tb.size(1)),
            static_cast<long long>(tb.size(2)));
    a.n_adapters = size32(count, "a");
    a.rank = size32(rank, "a");
    a.a = place<const uint16_t>(ta);
    a.b = place<const uint16_t>(tb);
    if (v[6] == Py_None) raise(PyExc_TypeError, "row_adapter: expected a torch tensor");
    a.row_adapter = vec<int32_t>(v[6], "row_adapter", kI32, dev, T);
    a.adapter_scale = vec<float>(v[8], "adapter_scale", kF32, dev, count);
    const Place at(dev, v[14]);
    if (v[15] != Py_None) {
      const at::Tensor& ws = checked(v[15], "ws", kU8, dev);
      if (!ws.is_contiguous()) raise(PyExc_ValueError, "ws: expected a contiguous tensor");
      return csa2_lora_linear(&a, place<void>(ws), static_cast<size_t>(ws.numel()), at.stream);
    }
    size_t bytes = 0;
    const int rc = csa2_workspace_size(CSA2_CALL_LORA_LINEAR, &a, &bytes);
    if (rc) return rc;
    const Scratch ws(bytes, at.stream);
    return csa2_lora_linear(&a, ws.at, bytes, at.stream);
  });
}

// (logits, token, logprob, entropy, lse, top_id, top_logprob, stream)
PyObject* logprobs(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    expect(n, 8);
    csa2_logprobs_args a = {};
    const int dev = device_of(v[0], "logits");
    int64_t T, V;
    two_d(tensor(v[0], "logits"), "logits", &T, &V);
    a.T = size32(T, "logits");
    a.V = size32(V, "logits");
    const at::ScalarType kind = tensor(v[0], "logits").scalar_type();
    if (kind != kF32 && kind != kBf16)
      raise(PyExc_TypeError, "logits: expected torch.float32 or torch.bfloat16, got %s", dtype_name(kind));
    a.logits_f32 = kind == kF32;
    mat(v[0], "logits", kind, dev, T, V, &a.logits, &a.ld_logits);
    a.token = vec<int32_t>(v[1], "token", kI32, dev, T);
    a.logprob = vec<float>(v[2], "logprob", kF32, dev, T);
    a.entropy = vec<float>(v[3], "entropy", kF32, dev, T);
    a.lse = vec<float>(v[4], "lse", kF32, dev, T);
    int64_t rows, top = 0, ld = 0;
    if (v[5] != Py_None) {
      two_d(tensor(v[5], "top_id"), "top_id", &rows, &top);
      mat(v[5], "top_id", kI32, dev, T, top, &a.top_id, &ld);
    }
    if (v[6] != Py_None) {
      if (v[5] == Py_None) two_d(tensor(v[6], "top_logprob"), "top_logprob", &rows, &top);
      int64_t ld_p;
      mat(v[6], "top_logprob", kF32, dev, T, top, &a.top_logprob, &ld_p);
      if (v[5] != Py_None && ld_p != ld) raise(PyExc_ValueError, "top_id, top_logprob: expected one row stride");
      ld = ld_p;
    }
    a.n_top = size32(top, "top_id");
    a.ld_top = ld;
    const Place at(dev, v[7]);
    return csa2_logprobs(&a, at.stream);
  });
}

PyMethodDef kMethods[] = {
    {"add_norm_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(add_norm_fp8)), METH_FASTCALL, nullptr},
    {"lora_linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(lora_linear)), METH_FASTCALL, nullptr},
    {"logprobs", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(logprobs)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_csa2_call", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__csa2_call(void) { return PyModule_Create(&kModule); }
