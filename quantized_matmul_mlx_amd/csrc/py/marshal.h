// What the CPython modules share: checks of tensor arguments, outputs from torch's allocator, the
// current stream, and errors as Python exceptions.
#pragma once

#include "qaff.h"

#include <ATen/ATen.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <Python.h>

#include <string>

namespace {

// A Python exception that is already set.
struct PyError {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
    PyErr_SetString(type, text.c_str());
    throw PyError();
}

std::string shape_of(const at::Tensor& t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}

// The status of a call as an exception: quantized_matmul_mlx_amd.QaffError(status, text).
void check(qaff_status st) {
    if (st == QAFF_OK) return;
    const std::string text = std::string(qaff_status_string(st)) + ": " + qaff_last_error();
    PyObject* mod = PyImport_ImportModule("quantized_matmul_mlx_amd._lib");
    PyObject* type = mod ? PyObject_GetAttrString(mod, "QaffError") : nullptr;
    PyObject* err = type ? PyObject_CallFunction(type, "is", (int)st, text.c_str()) : nullptr;
    if (err) PyErr_SetObject(type, err);
    Py_XDECREF(err);
    Py_XDECREF(type);
    Py_XDECREF(mod);
    throw PyError();
}

int64_t integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        PyObject* i = PyNumber_Index(o);
        if (!i) throw PyError();
        Py_DECREF(i);
        raise(PyExc_ValueError, std::string(name) + " does not fit 64 bits");
    }
    return v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PyError();
    return v != 0;
}

const char* type_name(at::ScalarType t) { return c10::toString(t); }

// A GPU tensor of one of the types (two that are equal: one type), on `device` where one is given.
const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType t0, at::ScalarType t1, const at::Tensor* like,
                         int64_t dim) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be on a GPU device, got " + t.device().str());
    if (like && t.device() != like->device())
        raise(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected " + like->device().str());
    if (t.scalar_type() != t0 && t.scalar_type() != t1)
        raise(PyExc_TypeError, std::string(name) + " has dtype " + type_name(t.scalar_type()) + ", expected " +
                                   type_name(t0) + (t1 != t0 ? std::string(" or ") + type_name(t1) : ""));
    if (dim >= 0 && t.dim() != dim)
        raise(PyExc_ValueError, std::string(name) + " must have " + std::to_string(dim) + " dimensions, got " +
                                    std::to_string(t.dim()));
    return t;
}

const at::Tensor& flat(PyObject* o, const char* name, at::ScalarType type, const at::Tensor* like, int64_t dim) {
    const at::Tensor& t = tensor(o, name, type, type, like, dim);
    if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t;
}

template <typename T> T* ptr(const at::Tensor& t) { return t.numel() ? static_cast<T*>(t.data_ptr()) : nullptr; }

qaff_dtype dtype_of(const at::Tensor& t) { return t.scalar_type() == at::kHalf ? QAFF_F16 : QAFF_BF16; }

// The device and the stream a call runs on.
struct Place {
    c10::DeviceGuard guard;
    hipStream_t stream;
    explicit Place(const at::Tensor& t)
        : guard(t.device()),
          stream(c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(t.device().index()).stream()) {}
};

at::Tensor empty(at::IntArrayRef sizes, const at::Tensor& like, at::ScalarType type) {
    return at::empty(sizes, like.options().dtype(type));
}

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw PyError();
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
    return r;
}

// No exception leaves a module function: C++ errors (torch's among them) become Python's.
template <typename F> PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const PyError&) {
        return nullptr;
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

}  // namespace
