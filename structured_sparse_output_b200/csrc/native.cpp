// native.cpp -- argument marshalling of the scoring and softmax calls without the
// interpreter: the checks of haste.py (shape, dtype, device, contiguity of every
// tensor), then the C ABI call.  A call on a few samples takes 4 to 7 us on the GPU,
// and the same checks in Python 6 us more.
//
// Every function returns the call's status, or None when a check does not hold: the
// Python code then makes its own checks, which name what is wrong.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>

#include "../../include/haste.h"

namespace {

decltype(&haste_logprob) g_logprob = nullptr;
decltype(&haste_logprob_backward) g_logprob_backward = nullptr;
decltype(&haste_head_forward_i8) g_head_forward_i8 = nullptr;

constexpr auto kF32 = at::kFloat, kI32 = at::kInt, kI8 = at::kChar, kBF16 = at::kBFloat16;

// The tensor behind a Python object, if it is one on CUDA device dev.
const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

struct Args {
  int dev = -1;
  bool ok = true;

  // Address of a contiguous tensor of this shape and type on the call's device.
  template <typename P>
  P at(PyObject* o, c10::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(o);
    if (!t || !t->is_cuda() || t->get_device() != dev || t->scalar_type() != type || !t->is_contiguous() ||
        t->sizes() != at::IntArrayRef(shape)) {
      ok = false;
      return nullptr;
    }
    return static_cast<P>(t->data_ptr());
  }
  template <typename P>
  P maybe(PyObject* o, c10::ScalarType type, std::initializer_list<int64_t> shape) {
    return o == Py_None ? nullptr : at<P>(o, type, shape);
  }
  // A workspace of any type: address and bytes.
  void* workspace(PyObject* o, size_t* bytes) {
    *bytes = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor* t = tensor(o);
    if (!t || !t->is_cuda() || t->get_device() != dev || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    *bytes = t->nbytes();
    return t->data_ptr();
  }
  // The current stream, where the tensors are on the current device.
  void* stream() {
    if (dev < 0 || dev != c10::cuda::current_device()) {
      ok = false;
      return nullptr;
    }
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  }
};

// A CUDA matrix of a type that the library takes; sets the call's device.
const at::Tensor* matrix(PyObject* o, Args& a) {
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->dim() != 2 || (t->scalar_type() != kF32 && t->scalar_type() != kBF16) ||
      !t->is_contiguous())
    return nullptr;
  a.dev = t->get_device();
  return t;
}
haste_dtype_t code(const at::Tensor& t) { return t.scalar_type() == kBF16 ? HASTE_BF16 : HASTE_F32; }

// The given labels' lists and the values that go with them.
template <typename P>
haste_targets_t given(Args& a, PyObject* row_ptr, PyObject* ids, PyObject* per_id, int64_t B, int64_t* nnz, P* values) {
  *nnz = 0;
  *values = nullptr;
  if (row_ptr == Py_None) {
    if (ids != Py_None || per_id != Py_None) a.ok = false;
    return {nullptr, nullptr};
  }
  const at::Tensor* t = tensor(ids);
  if (!t || t->dim() != 1) {
    a.ok = false;
    return {nullptr, nullptr};
  }
  *nnz = t->size(0);
  *values = a.at<P>(per_id, kF32, {*nnz});
  return {a.at<const int32_t*>(row_ptr, kI32, {B + 1}), a.at<const int32_t*>(ids, kI32, {*nnz})};
}

// No C++ exception (a tensor without storage, say) leaves a function.
template <PyObject* (*kBody)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* v, Py_ssize_t n) {
  try {
    return kBody(v, n);
  } catch (...) {
    Py_RETURN_NONE;
  }
}

template <typename F>
PyObject* call(F f) {
  haste_status_t st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return PyLong_FromLong(st);
}

// logits, row_ptr, ids, logp, lse, entropy, top_logp, top_id, ws
PyObject* logprob(PyObject* const* v, Py_ssize_t n) {
  Args a;
  const at::Tensor* z = n == 9 ? matrix(v[0], a) : nullptr;
  if (!z) Py_RETURN_NONE;
  const int64_t B = z->size(0), N = z->size(1);
  int64_t nnz, k = 0;
  float* logp;
  const haste_targets_t g = given(a, v[1], v[2], v[3], B, &nnz, &logp);
  float* lse = a.maybe<float*>(v[4], kF32, {B});
  float* entropy = a.maybe<float*>(v[5], kF32, {B});
  if (v[7] != Py_None) {
    const at::Tensor* t = tensor(v[7]);
    if (!t || t->dim() != 2) Py_RETURN_NONE;
    k = t->size(1);
  } else if (v[6] != Py_None) {
    Py_RETURN_NONE;
  }
  float* top_logp = v[7] == Py_None ? nullptr : a.at<float*>(v[6], kF32, {B, k});
  int32_t* top_id = v[7] == Py_None ? nullptr : a.at<int32_t*>(v[7], kI32, {B, k});
  size_t bytes;
  void* ws = a.workspace(v[8], &bytes);
  void* st = a.stream();
  if (!a.ok || B > 0x7fffffff) Py_RETURN_NONE;
  const void* zp = z->data_ptr();
  const haste_dtype_t dt = code(*z);
  return call([&] {
    return g_logprob((int32_t)B, N, dt, zp, g, nnz, (int32_t)k, logp, lse, entropy, top_logp, top_id, ws, bytes, st);
  });
}

// logits, lse, entropy, row_ptr, ids, d_logp, d_entropy, d_logits
PyObject* logprob_backward(PyObject* const* v, Py_ssize_t n) {
  Args a;
  const at::Tensor* z = n == 8 ? matrix(v[0], a) : nullptr;
  if (!z) Py_RETURN_NONE;
  const int64_t B = z->size(0), N = z->size(1);
  const float* lse = a.at<const float*>(v[1], kF32, {B});
  const float* entropy = v[6] == Py_None ? a.maybe<const float*>(v[2], kF32, {B}) : a.at<const float*>(v[2], kF32, {B});
  int64_t nnz;
  const float* d_logp;
  const haste_targets_t g = given(a, v[3], v[4], v[5], B, &nnz, &d_logp);
  const float* d_entropy = a.maybe<const float*>(v[6], kF32, {B});
  void* dz = a.at<void*>(v[7], z->scalar_type(), {B, N});
  void* st = a.stream();
  if (!a.ok || B > 0x7fffffff) Py_RETURN_NONE;
  const void* zp = z->data_ptr();
  const haste_dtype_t dt = code(*z);
  return call([&] { return g_logprob_backward((int32_t)B, N, dt, zp, lse, entropy, g, nnz, d_logp, d_entropy, dz, st); });
}

// Xh, Wq, w_scale, logits, ws
PyObject* head_forward_i8(PyObject* const* v, Py_ssize_t n) {
  Args a;
  const at::Tensor* x = n == 5 ? matrix(v[0], a) : nullptr;
  const at::Tensor* w = n == 5 ? tensor(v[1]) : nullptr;
  const at::Tensor* z = n == 5 ? tensor(v[3]) : nullptr;
  if (!x || !w || w->dim() != 2 || !z || (z->scalar_type() != kF32 && z->scalar_type() != kBF16)) Py_RETURN_NONE;
  const int64_t B = x->size(0), d = x->size(1), H = w->size(0);
  const int8_t* wq = a.at<const int8_t*>(v[1], kI8, {H, (d + 15) / 16 * 16});
  const float* scale = a.at<const float*>(v[2], kF32, {H});
  void* out = a.at<void*>(v[3], z->scalar_type(), {B, H});
  size_t bytes;
  void* ws = a.workspace(v[4], &bytes);
  void* st = a.stream();
  if (!a.ok || B > 0x7fffffff || H > 0x7fffffff || d > 0x7fffffff) Py_RETURN_NONE;
  const void* xp = x->data_ptr();
  const haste_dtype_t dt = code(*x), odt = code(*z);
  return call([&] {
    return g_head_forward_i8((int32_t)B, (int32_t)H, (int32_t)d, dt, xp, wq, scale, odt, out, ws, bytes, st);
  });
}

// Addresses of the library's functions, in the order of their pointers above.
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "bind takes three addresses");
    return nullptr;
  }
  void* p[3];
  for (int i = 0; i < 3; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(v[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "NULL address");
      return nullptr;
    }
  g_logprob = reinterpret_cast<decltype(g_logprob)>(p[0]);
  g_logprob_backward = reinterpret_cast<decltype(g_logprob_backward)>(p[1]);
  g_head_forward_i8 = reinterpret_cast<decltype(g_head_forward_i8)>(p[2]);
  Py_RETURN_NONE;
}

#define FASTCALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", FASTCALL(bind)},
                         {"logprob", FASTCALL(guarded<logprob>)},
                         {"logprob_backward", FASTCALL(guarded<logprob_backward>)},
                         {"head_forward_i8", FASTCALL(guarded<head_forward_i8>)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
