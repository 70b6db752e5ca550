// bind.hpp -- what the Python extensions of the operators around the GEMMs share
// (block_bind.cpp, model_bind.cpp): checks of tensor arguments and the way back.
// Host code only; compiled against torch's headers, one copy an extension.
#pragma once

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>

#include "gemm.h"

namespace {

using at::Tensor;
using Args = PyObject *const *;

// Set a Python error and leave: HANDLE_TH_ERRORS passes it on.
[[noreturn]] void fail(PyObject *type, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(type, fmt, ap);
    va_end(ap);
    throw python_error();
}

PyObject *g_check;   // the package's: raises what a failed status stands for

void check(gemm_status s) {
    if (s == GEMM_OK) return;
    PyObject *r = PyObject_CallFunction(g_check, "i", (int)s);
    Py_XDECREF(r);
    throw python_error();
}

std::string shape(const Tensor &t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + (t.dim() == 1 ? ",)" : ")");
}
const char *dtype_name(at::ScalarType t) { return c10::toString(t); }

// A tensor argument, undefined where it is None.
Tensor tensor(PyObject *o, const char *name) {
    if (o == Py_None) return Tensor();
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor, is %s", name, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}
Tensor needed(PyObject *o, const char *name) {
    Tensor t = tensor(o, name);
    if (!t.defined()) fail(PyExc_TypeError, "%s must be a tensor, is None", name);
    return t;
}
int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

gemm_dtype float_type(const Tensor &t, const char *name) {
    switch (t.scalar_type()) {
    case at::kFloat: return GEMM_F32;
    case at::kHalf: return GEMM_F16;
    case at::kBFloat16: return GEMM_BF16;
    default:
        fail(PyExc_TypeError, "%s has dtype %s, must be float32, float16 or bfloat16", name,
                               dtype_name(t.scalar_type()));
    }
}

// A tensor of the current device; its index.
int on_device(const Tensor &t, const char *name) {
    if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a device tensor", name);
    const int dev = t.get_device(), current = c10::hip::current_device();
    if (dev != current)
        fail(PyExc_ValueError, "%s is on device %d, the current device is %d", name, dev, current);
    return dev;
}

// What a layer holds, which its constructor has checked but for the device.
void held(const Tensor &t, const char *name, int dev) {
    if (!t.is_cuda() || t.get_device() != dev) on_device(t, name);
}

// A 2-D tensor of contiguous rows on device dev; its leading dimension.
int64_t rows(const Tensor &t, const char *name, int dev) {
    if (t.dim() != 2) fail(PyExc_ValueError, "%s must be 2-D, has shape %s", name, shape(t).c_str());
    if (!t.is_cuda() || t.get_device() != dev) on_device(t, name);
    const int64_t n = t.size(0), c = t.size(1), ld = t.stride(0);
    if (t.stride(1) != 1 && c > 1)
        fail(PyExc_ValueError, "%s must have contiguous rows, has strides (%lld, %lld)", name, (long long)ld,
                                (long long)t.stride(1));
    if (n <= 1 || c == 0) return c;
    if (ld < c)
        fail(PyExc_ValueError, "%s has overlapping rows, strides (%lld, %lld)", name, (long long)ld,
                                (long long)t.stride(1));
    return ld;
}
int64_t rows(const Tensor &t, const char *name, int dev, at::ScalarType dt) {
    const int64_t ld = rows(t, name, dev);
    if (t.scalar_type() != dt)
        fail(PyExc_TypeError, "%s has dtype %s, must be %s", name, dtype_name(t.scalar_type()), dtype_name(dt));
    return ld;
}
int64_t rows(const Tensor &t, const char *name, int dev, at::ScalarType dt, int64_t n, int64_t c) {
    const int64_t ld = rows(t, name, dev, dt);
    if (t.size(0) != n || t.size(1) != c)
        fail(PyExc_ValueError, "%s has shape %s, must be (%lld, %lld)", name, shape(t).c_str(), (long long)n,
                                (long long)c);
    return ld;
}

// n contiguous elements, or NULL for an undefined tensor.
const void *vector(const Tensor &t, const char *name, int dev, at::ScalarType dt, int64_t n) {
    if (!t.defined()) return nullptr;
    if (!t.is_cuda() || t.get_device() != dev) on_device(t, name);
    if (t.scalar_type() != dt)
        fail(PyExc_TypeError, "%s has dtype %s, must be %s", name, dtype_name(t.scalar_type()), dtype_name(dt));
    if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
        fail(PyExc_ValueError, "%s must be %lld contiguous elements, has shape %s", name, (long long)n,
                                shape(t).c_str());
    return t.data_ptr();
}

// New tensors are plain ones: nothing here takes part in autograd.
Tensor fresh(at::IntArrayRef size, at::ScalarType dt, const at::Device &device) {
    at::AutoDispatchBelowADInplaceOrView guard;
    return at::empty(size, at::TensorOptions().dtype(dt).device(device));
}
void *stream_of(int dev) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream(); }
void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
PyObject *wrap(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject *tuple(std::initializer_list<Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw python_error();
    Py_ssize_t i = 0;
    for (const Tensor &t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}
void count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) fail(PyExc_TypeError, "expected %lld arguments, got %lld", (long long)want, (long long)n);
}

// (function): what a failed status is given to
PyObject *set_check(PyObject *, PyObject *f) {
    Py_INCREF(f);
    Py_XSETREF(g_check, f);
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}

}  // namespace
