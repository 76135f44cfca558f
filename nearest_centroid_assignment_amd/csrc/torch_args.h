// torch_args.h - what the modules that marshal torch tensors natively share
// (experts_torch.cpp, layers_torch.cpp).
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <array>
#include <vector>

#include "../../include/experts_mi355x.h"

namespace {

PyObject *check;  // check(status, name of the entry point) raises
extern const char *const module_name;  // the Python module of the operators

constexpr int64_t kBlock = 256;  // slack of a workspace; elements that share a scale

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

int code_of(at::ScalarType t) {
    return t == at::kFloat      ? EXPERTS_F32
           : t == at::kBFloat16 ? EXPERTS_BF16
           : t == at::kHalf     ? EXPERTS_F16
                                : -1;
}

// The device of the call, which is the current one, or -1.
int call_device(const at::Tensor &t) {
    if (!t.is_cuda()) return -1;
    const int dev = t.get_device();
    return dev == c10::hip::current_device() ? dev : -1;
}

struct Rows {
    void *p = nullptr;
    int64_t ld = 0;
};
// A non-empty rows x cols matrix of this type and device with dense rows.
bool rows_of(const at::Tensor *t, at::ScalarType type, int64_t rows, int64_t cols, int dev, Rows &r) {
    if (!t || t->scalar_type() != type || !t->is_cuda() || t->get_device() != dev || t->dim() != 2 ||
        t->size(0) != rows || t->size(1) != cols || rows < 1 || cols < 1)
        return false;
    if (t->stride(1) != 1 && cols != 1) return false;
    r.ld = rows == 1 ? cols : t->stride(0);
    if (r.ld < cols) return false;
    r.p = t->data_ptr();
    return true;
}
// A contiguous tensor of this type, device and shape: its pointer (never null).
void *dense(const at::Tensor *t, at::ScalarType type, at::IntArrayRef shape, int dev) {
    if (!t || t->scalar_type() != type || !t->is_cuda() || t->get_device() != dev ||
        t->sizes() != shape || !t->is_contiguous() || t->numel() == 0)
        return nullptr;
    return t->data_ptr();
}

// The truth of o; false where it has none (then Python says why).
bool truth(PyObject *o, bool &v) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) PyErr_Clear();
    v = t > 0;
    return t >= 0;
}

at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, int dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev));
}
void *queue(int dev) { return c10::hip::getCurrentHIPStream(dev).stream(); }

struct Scratch {
    at::Tensor t;
    void *p = nullptr;
    size_t n = 0;
    Scratch(size_t bytes, int dev) {
        if (bytes <= (size_t)kBlock) return;
        t = new_tensor({(int64_t)bytes}, at::kByte, dev);
        p = t.data_ptr();
        n = bytes;
    }
};

PyObject *wrap(const at::Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
PyObject *tuple_of(const at::Tensor &a, const at::Tensor &b) {
    PyObject *r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, wrap(a));
    PyTuple_SET_ITEM(r, 1, wrap(b));
    return r;
}
PyObject *tuple_of(const at::Tensor &a, const at::Tensor &b, const at::Tensor &c) {
    PyObject *r = PyTuple_New(3);
    PyTuple_SET_ITEM(r, 0, wrap(a));
    PyTuple_SET_ITEM(r, 1, wrap(b));
    PyTuple_SET_ITEM(r, 2, wrap(c));
    return r;
}

// Autograd is told that t was written in place, as it is by torch's own operators.
[[maybe_unused]] void written(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Warns where a graph is being recorded and one of these asks to be in it, or where one carries
// a forward-mode tangent: the operator is not, and its result has none. False if the warning
// has become an error.
bool say_unrecorded(const char *name, at::ArrayRef<const at::Tensor *> inputs) {
    const bool graph = c10::GradMode::is_enabled();
    const bool tangents = c10::AutogradState::get_tls_state().get_fw_grad_mode();
    if (!graph && !tangents) return true;
    for (const at::Tensor *t : inputs) {
        if (graph && t && t->requires_grad())
            return PyErr_WarnFormat(PyExc_UserWarning, 2,
                                    "%s.%s is not recorded for autograd: an input requires grad, but "
                                    "gradients are explicit calls (%s.%s_backward). Call it under "
                                    "torch.no_grad(), or with detached tensors",
                                    module_name, name, module_name, name) == 0;
        if (tangents && t && t->_fw_grad(0).defined())
            return PyErr_WarnFormat(PyExc_UserWarning, 2,
                                    "%s.%s is not recorded for autograd: an input has a forward-mode "
                                    "tangent, which the result does not. Call it with the primal",
                                    module_name, name) == 0;
    }
    return true;
}

// What a status of the C ABI other than KM_OK becomes.
PyObject *failed(int status, const char *name) {
    if (status == KM_ERR_HIP) {
        PyObject *r = PyObject_CallFunction(check, "is", status, name);
        Py_XDECREF(r);
        if (!r) return nullptr;
    }
    Py_RETURN_NONE;
}

#define NOT_HERE Py_RETURN_NONE
#define ARGS(n) \
    if (count != (n)) NOT_HERE

// (name of the operator, inputs...) -> None: the warning for a call that Python takes
PyObject *unrecorded(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    const char *name = count < 1 ? "" : PyUnicode_AsUTF8(a[0]);
    if (!name) return nullptr;
    std::vector<const at::Tensor *> inputs;
    for (Py_ssize_t i = 1; i < count; ++i) inputs.push_back(tensor(a[i]));
    if (!say_unrecorded(name, inputs)) return nullptr;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// bind({name: address of the C entry point}, check) for the entry points that `each` visits:
// all of them, or none (a module whose bind was refused stays as it was).
template <class F>
PyObject *bind_all(PyObject *const *a, Py_ssize_t count, F each) {
    if (count < 1 || !PyDict_Check(a[0])) {
        PyErr_SetString(PyExc_TypeError, "bind takes a dict of addresses");
        return nullptr;
    }
    bool whole = true;
    each([&](const char *name, auto &) {
        PyObject *v = PyDict_GetItemString(a[0], name);
        whole = whole && v && PyLong_AsVoidPtr(v);
    });
    if (!whole) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: an entry point is missing");
        return nullptr;
    }
    if (count != 2 || !PyCallable_Check(a[1])) {
        PyErr_SetString(PyExc_TypeError, "bind takes a dict of addresses and the check of a status");
        return nullptr;
    }
    each([&](const char *name, auto &f) {
        f = (std::remove_reference_t<decltype(f)>)PyLong_AsVoidPtr(PyDict_GetItemString(a[0], name));
    });
    Py_INCREF(a[1]);
    Py_XSETREF(check, a[1]);
    Py_RETURN_NONE;
}

#define KX_METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}

}  // namespace
