// Shared by the native Python calls (kv4_py.cpp, cross_py.cpp): arguments as
// tensors, new tensors, the call itself.
#pragma once

#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sfa.h"

namespace {

using at::Tensor;

// A CUDA tensor on device `index` with memory of its own, or null.
const Tensor* tensor(PyObject* o, int index) {
  if (!THPVariable_Check(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && t.get_device() == index && !t.unsafeGetTensorImpl()->is_python_dispatch() ? &t : nullptr;
}

// The same, contiguous, of this type and shape.
const Tensor* dense(PyObject* o, int index, at::ScalarType type, at::IntArrayRef shape) {
  const Tensor* t = tensor(o, index);
  return t && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous() ? t : nullptr;
}

int32_t* ints(PyObject* o, int index, int64_t n) {
  const Tensor* t = dense(o, index, at::kInt, {n});
  return t ? static_cast<int32_t*>(t->data_ptr()) : nullptr;
}

// The current device, if o is a CUDA tensor; else -1, which no such tensor is on.
int current(PyObject* o) { return THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda() ? c10::cuda::current_device() : -1; }

bool fits(int64_t n) { return n >= 0 && n <= INT32_MAX; }

bool code(at::ScalarType type, int32_t* dtype) {
  *dtype = type == at::kBFloat16 ? SFA_BF16 : SFA_F32;
  return type == at::kBFloat16 || type == at::kFloat;
}

// t [N, heads, 64] with dense rows: the stride between them.
bool rows(const Tensor* t, int64_t* stride) {
  if (!t || t->dim() != 3 || t->size(2) != 64 || !fits(t->size(0)) || !fits(t->size(1))) return false;
  const int64_t n = t->size(0), h = t->size(1);
  *stride = 64 * h;
  if (t->is_contiguous()) return true;
  if (t->stride(2) != 1 || (t->stride(1) != 64 && h > 1)) return false;
  if (n <= 1) return true;
  *stride = t->stride(0);
  return *stride >= 64 * h && *stride * t->element_size() % 16 == 0;
}

Tensor empty(at::IntArrayRef shape, at::ScalarType type, int index) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)index), c10::nullopt);
}

// The call itself, without the interpreter's lock: a full queue waits in there.
template <typename F>
int enqueue(F&& f, int index) {
  void* const stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f(stream);
  Py_END_ALLOW_THREADS
  return rc;
}

#define SLOW Py_RETURN_NONE

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}

}  // namespace
