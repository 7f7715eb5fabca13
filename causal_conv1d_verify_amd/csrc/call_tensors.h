// Shared by the call modules: how a Python object becomes a tensor, a number or a pointer of the C
// ABI.  Each of these says no rather than raises.  Internal.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <exception>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "conv_verify.h"

namespace {

using at::Tensor;

// None: no tensor.  Anything else that is not a tensor: `ok` becomes false.
const Tensor *tensor(PyObject *o, bool &ok) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
        ok = false;
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}

int dtype_code(const Tensor &t) {
    return t.scalar_type() == at::kFloat ? CV_F32 : t.scalar_type() == at::kBFloat16 ? CV_BF16 : -1;
}

bool rows_in_order(const Tensor &t) { return t.size(-1) == 1 || t.stride(-1) == 1; }
int64_t stride(const Tensor &t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }

bool int32_vec(const Tensor *t, int64_t n) {
    return !t || (t->scalar_type() == at::kInt && t->dim() == 1 && t->size(0) == n && (n <= 1 || t->stride(0) == 1));
}

bool weights(const Tensor *t, int64_t dim) {
    return !t || (t->dim() == 1 && t->size(0) == dim && (dim == 1 || t->stride(0) == 1));
}

// All on one GPU, the current one.
bool one_gpu(std::initializer_list<const Tensor *> ts, c10::Device *dev) {
    bool first = true;
    for (const Tensor *t : ts) {
        if (!t) continue;
        if (first) *dev = t->device(), first = false;
        else if (t->device() != *dev) return false;
    }
    return !first && dev->is_cuda() && dev->index() == c10::hip::current_device();
}

void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

bool number(PyObject *o, double *x) {
    if (PyFloat_CheckExact(o)) *x = PyFloat_AS_DOUBLE(o);
    else if (PyLong_CheckExact(o)) *x = PyLong_AsDouble(o);
    else return false;
    return !PyErr_Occurred();
}

// No exception of torch's (out of memory, a tensor without storage) leaves through C: the long way
// meets it again and raises it.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n_args) {
    try {
        return F(self, args, n_args);
    } catch (const std::exception &) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<f>))
}  // namespace
