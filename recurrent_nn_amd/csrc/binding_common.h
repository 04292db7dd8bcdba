// binding_common.h -- what the compiled calls of the torch binding share
// (binding.cpp says what they are for).
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <vector>

#include "../../include/recurrent_nn_amd.h"

namespace {

// What a check throws: this call is not one of the plain ones.
struct NotPlain {};

void need(bool ok)
{
    if (!ok)
        throw NotPlain{};
}

int32_t type_of(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return RNN_DTYPE_F32;
    case at::kBFloat16: return RNN_DTYPE_BF16;
    case at::kHalf: return RNN_DTYPE_F16;
    default: throw NotPlain{};
    }
}

using Sizes = std::initializer_list<int64_t>;

struct Call {
    int64_t device;
    void *stream;

    // A device tensor with memory of its own (a transform's wrapper has none), of
    // which no gradient is asked; null for None where that is allowed.
    const at::Tensor *tensor(PyObject *o, bool optional = false) const
    {
        if (optional && o == Py_None)
            return nullptr;
        need(THPVariable_Check(o));
        const at::Tensor &t = THPVariable_Unpack(o);
        need(t.is_cuda() && t.device().index() == device && t.has_storage());
        need(!(t.requires_grad() && at::GradMode::is_enabled()));
        return &t;
    }
    // A dense tensor of this type and shape.
    const at::Tensor *dense(PyObject *o, at::ScalarType type, Sizes sizes, bool optional = true) const
    {
        const at::Tensor *t = tensor(o, optional);
        if (t)
            need(t->scalar_type() == type && t->sizes() == at::IntArrayRef(sizes) && t->is_contiguous());
        return t;
    }
    // One whose last dimension is contiguous.
    const at::Tensor *rows(PyObject *o, at::ScalarType type, at::IntArrayRef sizes, bool optional) const
    {
        const at::Tensor *t = tensor(o, optional);
        if (t) {
            need(t->scalar_type() == type && t->sizes() == sizes);
            last_contiguous(*t);
        }
        return t;
    }
    static void last_contiguous(const at::Tensor &t) { need(t.size(-1) <= 1 || t.stride(-1) == 1); }
};

void *ptr(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

PyObject *results(int status, std::initializer_list<at::Tensor> outs)
{
    if (status != RNN_OK)
        return PyLong_FromLong(status);
    PyObject *tuple = PyTuple_New((Py_ssize_t)outs.size());
    if (!tuple)
        return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor &t : outs) {
        PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(tuple);
            return nullptr;
        }
        PyTuple_SET_ITEM(tuple, i++, o);
    }
    return tuple;
}

// A C entry point called without the interpreter lock.  What can throw (a
// tensor's pointer) is an argument, so it is over before the lock is given up;
// the entry points themselves let no exception out.
template <class F, class... A> int without_gil(F entry, A... args)
{
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = entry(args...);
    Py_END_ALLOW_THREADS
    return status;
}

// The last two arguments of every call: device index and stream handle.
template <class F> PyObject *plain_call(PyObject *const *args, Py_ssize_t n, Py_ssize_t expected, F &&body)
{
    HANDLE_TH_ERRORS
    if (n != expected) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    const Call call{PyLong_AsLongLong(args[n - 2]), PyLong_AsVoidPtr(args[n - 1])};
    if (PyErr_Occurred())
        return nullptr;
    try {
        return body(call);
    } catch (const NotPlain &) {
        Py_RETURN_NONE;
    }
    END_HANDLE_TH_ERRORS
}

at::Tensor bytes(const at::Tensor &like, size_t n)
{
    return n ? at::empty({(int64_t)n}, like.options().dtype(at::kByte)) : at::Tensor();
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw python_error();               // what it raised goes on
    return v;
}

// The addresses of a set of entry points, one for each of its members.
template <class Entries> PyObject *bind_entries(Entries &lib, PyObject *const *a, Py_ssize_t n)
{
    void *entries[sizeof(Entries) / sizeof(void *)];
    if (n != (Py_ssize_t)(sizeof(entries) / sizeof(void *))) {
        PyErr_SetString(PyExc_TypeError, "wrong number of entry points");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i)
        entries[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred())
        return nullptr;
    static_assert(sizeof(entries) == sizeof(lib), "an address for each");
    __builtin_memcpy((void *)&lib, entries, sizeof(lib));
    Py_RETURN_NONE;
}

}  // namespace

// The calls of binding_delta.cpp.
PyObject *bind_delta(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *delta_call(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *norm_call(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *beam_call(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *reorder_call(PyObject *, PyObject *const *a, Py_ssize_t n);
