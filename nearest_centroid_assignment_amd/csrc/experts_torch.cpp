// experts_torch.cpp - the ordinary calls of experts.py, marshalled natively.
//
// The smallest operators take less time on the GPU than Python takes to check
// their arguments and hand them to the C ABI. Each function here takes the tensors
// of one call on the current stream with fresh outputs, and either makes that call
// of the C ABI and returns its outputs, or, when anything is out of the ordinary
// (a wrong type, shape or device, an empty or strange matrix, a refusal by the
// library's checks of arguments), returns None without having enqueued a kernel:
// experts.py then takes the call, and words the error if there is one. A HIP error
// may come after a launch, so it is raised here: a step in place must not be made
// again. The entry points are bound by address, so this module links against torch
// alone.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <array>
#include <vector>

#include "../../include/experts_mi355x.h"

namespace {

decltype(&experts_plan_workspace_bytes) plan_bytes;
decltype(&experts_plan) plan_call;
decltype(&experts_dispatch) dispatch_call;
decltype(&experts_dispatch_backward) dispatch_backward_call;
decltype(&experts_combine) combine_call;
decltype(&experts_combine_backward) combine_backward_call;
decltype(&experts_linear_workspace_bytes) linear_bytes;
decltype(&experts_linear) linear_call;
decltype(&experts_linear_backward) linear_backward_call;
decltype(&experts_adamw_state_elements) adamw_elements;
decltype(&experts_adamw_step) adamw_call;
PyObject *check;  // check(status, name of the entry point) raises

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

// order, place and offsets of a plan, on dev.
struct Plan {
    const int32_t *order = nullptr, *place = nullptr;
    int64_t tokens = 0, top = 0;
};
bool plan_of(PyObject *o, int dev, Plan &p) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) return false;
    const at::Tensor *order = tensor(PyTuple_GET_ITEM(o, 0)), *place = tensor(PyTuple_GET_ITEM(o, 1));
    if (!order || !place || place->dim() != 2) return false;
    p.tokens = place->size(0);
    p.top = place->size(1);
    p.order = (const int32_t *)dense(order, at::kInt, {p.tokens * p.top}, dev);
    p.place = (const int32_t *)dense(place, at::kInt, {p.tokens, p.top}, dev);
    return p.order && p.place;
}

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
void written(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Warns where a graph is being recorded and one of these asks to be in it: the operator
// is not. False if the warning has become an error.
bool say_unrecorded(const char *name, at::ArrayRef<const at::Tensor *> inputs) {
    if (!c10::GradMode::is_enabled()) return true;
    for (const at::Tensor *t : inputs)
        if (t && t->requires_grad())
            return PyErr_WarnFormat(PyExc_UserWarning, 2,
                                    "experts.%s is not recorded for autograd: an input requires grad, but "
                                    "gradients are explicit calls (experts.%s_backward). Call it under "
                                    "torch.no_grad(), or with detached tensors",
                                    name, name) == 0;
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

// (ids, experts) -> (order, place, offsets)
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(2);
    const at::Tensor *ids = tensor(a[0]);
    if (!ids || !PyLong_Check(a[1]) || ids->scalar_type() != at::kLong || !ids->is_contiguous() ||
        ids->dim() < 1 || ids->dim() > 2 || ids->numel() == 0)
        NOT_HERE;
    const int dev = call_device(*ids);
    const int64_t experts = PyLong_AsLongLong(a[1]);
    if (dev < 0 || experts < 1) {
        PyErr_Clear();
        NOT_HERE;
    }
    const int64_t tokens = ids->size(0), top = ids->dim() == 2 ? ids->size(1) : 1;
    const size_t bytes = plan_bytes(tokens, top, experts);
    if (bytes == 0) NOT_HERE;
    Scratch ws(bytes, dev);
    at::Tensor order = new_tensor({tokens * top}, at::kInt, dev);
    at::Tensor place = new_tensor({tokens, top}, at::kInt, dev);
    at::Tensor offsets = new_tensor({experts + 1}, at::kInt, dev);
    const int status = plan_call(
        (const int64_t *)ids->data_ptr(), tokens, top, experts, (int32_t *)order.data_ptr(),
        (int32_t *)place.data_ptr(), (int32_t *)offsets.data_ptr(), ws.p, ws.n, queue(dev));
    if (status != KM_OK) return failed(status, "experts_plan");
    return tuple_of(order, place, offsets);
    END_HANDLE_TH_ERRORS
}

// (x, plan) -> xs
PyObject *dispatch(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(2);
    const at::Tensor *x = tensor(a[0]);
    if (!x || x->dim() != 2) NOT_HERE;
    const int dev = call_device(*x), code = code_of(x->scalar_type());
    Plan p;
    Rows rx;
    if (dev < 0 || code < 0 || !plan_of(a[1], dev, p) ||
        !rows_of(x, x->scalar_type(), p.tokens, x->size(1), dev, rx))
        NOT_HERE;
    if (!say_unrecorded("dispatch", {x})) return nullptr;
    const int64_t width = x->size(1);
    at::Tensor xs = new_tensor({p.tokens * p.top, width}, x->scalar_type(), dev);
    const int status = dispatch_call(
        rx.p, rx.ld, code, p.tokens, p.top, width, p.order, p.place, xs.data_ptr(), width,
        queue(dev));
    if (status != KM_OK) return failed(status, "experts_dispatch");
    return wrap(xs);
    END_HANDLE_TH_ERRORS
}

// (dxs, plan) -> dx
PyObject *dispatch_backward(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(2);
    const at::Tensor *g = tensor(a[0]);
    if (!g || g->dim() != 2) NOT_HERE;
    const int dev = call_device(*g), code = code_of(g->scalar_type());
    Plan p;
    Rows rg;
    if (dev < 0 || code < 0 || !plan_of(a[1], dev, p) ||
        !rows_of(g, g->scalar_type(), p.tokens * p.top, g->size(1), dev, rg))
        NOT_HERE;
    const int64_t width = g->size(1);
    at::Tensor dx = new_tensor({p.tokens, width}, g->scalar_type(), dev);
    const int status = dispatch_backward_call(
        rg.p, rg.ld, code, p.tokens, p.top, width, p.place, dx.data_ptr(), width, queue(dev));
    if (status != KM_OK) return failed(status, "experts_dispatch_backward");
    return wrap(dx);
    END_HANDLE_TH_ERRORS
}

// (ys, weights, plan) -> y
PyObject *combine(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(3);
    const at::Tensor *ys = tensor(a[0]);
    if (!ys || ys->dim() != 2) NOT_HERE;
    const int dev = call_device(*ys), code = code_of(ys->scalar_type());
    Plan p;
    Rows ry;
    if (dev < 0 || code < 0 || !plan_of(a[2], dev, p) ||
        !rows_of(ys, ys->scalar_type(), p.tokens * p.top, ys->size(1), dev, ry))
        NOT_HERE;
    const float *w = (const float *)dense(tensor(a[1]), at::kFloat, {p.tokens, p.top}, dev);
    if (!w) NOT_HERE;
    if (!say_unrecorded("combine", {ys, tensor(a[1])})) return nullptr;
    const int64_t width = ys->size(1);
    at::Tensor y = new_tensor({p.tokens, width}, ys->scalar_type(), dev);
    const int status = combine_call(
        ry.p, ry.ld, w, code, p.tokens, p.top, width, p.place, y.data_ptr(), width, queue(dev));
    if (status != KM_OK) return failed(status, "experts_combine");
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

// (dy, ys, weights, plan) -> (dys, dweights)
PyObject *combine_backward(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(4);
    const at::Tensor *dy = tensor(a[0]);
    if (!dy || dy->dim() != 2) NOT_HERE;
    const int dev = call_device(*dy), code = code_of(dy->scalar_type());
    const int64_t width = dy->size(1);
    Plan p;
    Rows rg, ry;
    if (dev < 0 || code < 0 || !plan_of(a[3], dev, p) ||
        !rows_of(dy, dy->scalar_type(), p.tokens, width, dev, rg) ||
        !rows_of(tensor(a[1]), dy->scalar_type(), p.tokens * p.top, width, dev, ry))
        NOT_HERE;
    const float *w = (const float *)dense(tensor(a[2]), at::kFloat, {p.tokens, p.top}, dev);
    if (!w) NOT_HERE;
    at::Tensor dys = new_tensor({p.tokens * p.top, width}, dy->scalar_type(), dev);
    at::Tensor dw = new_tensor({p.tokens, p.top}, at::kFloat, dev);
    const int status = combine_backward_call(
        rg.p, rg.ld, ry.p, ry.ld, w, code, p.tokens, p.top, width, p.order, p.place,
        dys.data_ptr(), width, (float *)dw.data_ptr(), queue(dev));
    if (status != KM_OK) return failed(status, "experts_combine_backward");
    return tuple_of(dys, dw);
    END_HANDLE_TH_ERRORS
}

// w (and offsets, None for a dense layer) of a linear call.
struct Weights {
    void *w = nullptr;
    const int32_t *offsets = nullptr;
    int64_t outs = 0, ins = 0, experts = 1;
    at::IntArrayRef lead;  // the shape of a bias
};
bool weights_of(PyObject *ow, PyObject *oo, at::ScalarType type, int dev, Weights &r) {
    const at::Tensor *w = tensor(ow);
    const bool grouped = oo != Py_None;
    if (!w || w->dim() != (grouped ? 3 : 2)) return false;
    r.w = dense(w, type, w->sizes(), dev);
    r.outs = w->size(-2);
    r.ins = w->size(-1);
    r.lead = w->sizes().slice(0, w->dim() - 1);
    if (grouped) {
        r.experts = w->size(0);
        r.offsets = (const int32_t *)dense(tensor(oo), at::kInt, {r.experts + 1}, dev);
        if (!r.offsets) return false;
    }
    return r.w != nullptr;
}
int misplaced(const Rows &x, const Weights &w) {
    return (((uintptr_t)x.p | (uintptr_t)w.w) % 4 != 0) || ((x.ld | w.ins) % 2 != 0);
}

// (x, w, bias, residual, act code, offsets, save_pre) -> out or (out, pre)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(7);
    const at::Tensor *x = tensor(a[0]);
    if (!x || x->dim() != 2 || !PyLong_Check(a[4])) NOT_HERE;
    const int dev = call_device(*x), code = code_of(x->scalar_type());
    const at::ScalarType type = x->scalar_type();
    const int act = (int)PyLong_AsLong(a[4]);
    Weights w;
    Rows rx, rr;
    if (dev < 0 || code < 0 || act < 0 || !weights_of(a[1], a[5], type, dev, w) ||
        !rows_of(x, type, x->size(0), w.ins, dev, rx))
        NOT_HERE;
    const int64_t rows = x->size(0);
    const void *bias = nullptr;
    if (a[2] != Py_None && !(bias = dense(tensor(a[2]), type, w.lead, dev))) NOT_HERE;
    if (a[3] != Py_None && !rows_of(tensor(a[3]), type, rows, w.outs, dev, rr)) NOT_HERE;
    const size_t bytes =
        linear_bytes(rows, w.outs, w.ins, w.experts, code, 0, misplaced(rx, w));
    if (bytes == 0) NOT_HERE;
    if (!say_unrecorded("linear", {x, tensor(a[1]), tensor(a[2]), tensor(a[3])})) return nullptr;
    Scratch ws(bytes, dev);
    at::Tensor out = new_tensor({rows, w.outs}, type, dev), pre;
    const int save = PyObject_IsTrue(a[6]);
    if (save) pre = new_tensor({rows, w.outs}, type, dev);
    const int status = linear_call(
        rx.p, rx.ld, w.w, bias, rr.p, rr.ld, w.offsets, code, act, rows, w.outs, w.ins,
        w.experts, out.data_ptr(), w.outs, save ? pre.data_ptr() : nullptr, w.outs, ws.p, ws.n,
        queue(dev));
    if (status != KM_OK) return failed(status, "experts_linear");
    return save ? tuple_of(out, pre) : wrap(out);
    END_HANDLE_TH_ERRORS
}

// (dy, x, w, pre, act code, offsets, in_pre, in_act code, need_dx, need_dw,
// need_dbias) -> (dx, dw, dbias)
PyObject *linear_backward(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(11);
    const at::Tensor *dy = tensor(a[0]);
    if (!dy || dy->dim() != 2 || !PyLong_Check(a[4]) || !PyLong_Check(a[7])) NOT_HERE;
    const int dev = call_device(*dy), code = code_of(dy->scalar_type());
    const at::ScalarType type = dy->scalar_type();
    const int act = (int)PyLong_AsLong(a[4]), in_act = (int)PyLong_AsLong(a[7]);
    Weights w;
    Rows rg, rx, rp, ri;
    const int64_t rows = dy->size(0);
    if (dev < 0 || code < 0 || act < 0 || in_act < 0 || !weights_of(a[2], a[5], type, dev, w) ||
        !rows_of(dy, type, rows, w.outs, dev, rg) ||
        !rows_of(tensor(a[1]), type, rows, w.ins, dev, rx))
        NOT_HERE;
    if (act != EXPERTS_ACT_NONE && !rows_of(tensor(a[3]), type, rows, w.outs, dev, rp)) NOT_HERE;
    if (a[6] != Py_None && !rows_of(tensor(a[6]), type, rows, w.ins, dev, ri)) NOT_HERE;
    const bool need_dx = PyObject_IsTrue(a[8]), need_dw = PyObject_IsTrue(a[9]),
               need_db = PyObject_IsTrue(a[10]);
    if (!need_dx && !need_dw && !need_db) NOT_HERE;
    const size_t bytes =
        linear_bytes(rows, w.outs, w.ins, w.experts, code, 1, misplaced(rx, w));
    if (bytes == 0) NOT_HERE;
    Scratch ws(bytes, dev);
    at::Tensor dx, dw, db;
    if (need_dx) dx = new_tensor({rows, w.ins}, type, dev);
    if (need_dw) dw = new_tensor(THPVariable_Unpack(a[2]).sizes(), type, dev);
    if (need_db) db = new_tensor(w.lead, type, dev);
    const int status = linear_backward_call(
        rg.p, rg.ld, rx.p, rx.ld, w.w, rp.p, rp.ld, ri.p, ri.ld, w.offsets, code, act, in_act,
        rows, w.outs, w.ins, w.experts, need_dx ? dx.data_ptr() : nullptr, w.ins,
        need_dw ? dw.data_ptr() : nullptr, need_db ? db.data_ptr() : nullptr, ws.p, ws.n,
        queue(dev));
    if (status != KM_OK) return failed(status, "experts_linear_backward");
    return tuple_of(dx, dw, db);
    END_HANDLE_TH_ERRORS
}

// Pointers of a list of contiguous tensors of one type, as long as `like`'s.
bool pointers(PyObject *o, at::ScalarType type, int dev, const std::vector<const at::Tensor *> &like,
              std::vector<void *> &out) {
    if (!PyList_Check(o) || (size_t)PyList_GET_SIZE(o) != like.size()) return false;
    out.resize(like.size());
    for (size_t i = 0; i < like.size(); ++i) {
        const at::Tensor *t = tensor(PyList_GET_ITEM(o, (Py_ssize_t)i));
        if (!t || t->scalar_type() != type || !t->is_cuda() || t->get_device() != dev ||
            t->sizes() != like[i]->sizes() || !t->is_contiguous())
            return false;
        out[i] = t->data_ptr();
    }
    return true;
}

// (params, grads, m, v, lr, beta1, beta2, eps, weight_decay, step, m_scale, v_scale,
// copies, grad_scale) -> True
PyObject *adamw_step(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(14);
    if (!PyList_Check(a[0]) || !PyList_Check(a[1]) || PyList_GET_SIZE(a[0]) < 1 ||
        PyList_GET_SIZE(a[0]) != PyList_GET_SIZE(a[1]) || !PyLong_Check(a[9]))
        NOT_HERE;
    const Py_ssize_t n = PyList_GET_SIZE(a[0]);
    std::vector<const at::Tensor *> params((size_t)n);
    std::vector<int64_t> numels((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!(params[i] = tensor(PyList_GET_ITEM(a[0], i)))) NOT_HERE;
        numels[i] = params[i]->numel();
    }
    const at::Tensor *g0 = tensor(PyList_GET_ITEM(a[1], 0));
    const int dev = call_device(*params[0]);
    if (dev < 0 || !g0) NOT_HERE;
    const at::ScalarType pt = params[0]->scalar_type(), gt = g0->scalar_type();
    std::vector<void *> pp, pg, pk;
    if (code_of(pt) < 0 || code_of(gt) < 0 || !pointers(a[0], pt, dev, params, pp) ||
        !pointers(a[1], gt, dev, params, pg) ||
        (a[12] != Py_None && !pointers(a[12], at::kBFloat16, dev, params, pk)))
        NOT_HERE;
    const int64_t total = adamw_elements(numels.data(), n);
    const at::Tensor *m = tensor(a[2]);
    if (total < 1 || !m) NOT_HERE;
    const int bits = m->scalar_type() == at::kChar ? 8 : 32;
    void *pm = dense(m, bits == 8 ? at::kChar : at::kFloat, {total}, dev);
    void *pv = dense(tensor(a[3]), bits == 8 ? at::kByte : at::kFloat, {total}, dev);
    float *ms = nullptr, *vs = nullptr, *gs = nullptr;
    if (!pm || !pv || (bits == 8) != (a[10] != Py_None) || (bits == 8) != (a[11] != Py_None)) NOT_HERE;
    if (bits == 8) {
        ms = (float *)dense(tensor(a[10]), at::kFloat, {total / kBlock}, dev);
        vs = (float *)dense(tensor(a[11]), at::kFloat, {total / kBlock}, dev);
        if (!ms || !vs) NOT_HERE;
    }
    if (a[13] != Py_None && !(gs = (float *)dense(tensor(a[13]), at::kFloat, {1}, dev))) NOT_HERE;
    std::array<double, 5> h;
    for (int i = 0; i < 5; ++i) {
        h[i] = PyFloat_AsDouble(a[4 + i]);
        if (h[i] == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            NOT_HERE;
        }
    }
    const int64_t step = PyLong_AsLongLong(a[9]);
    if (step < 1) {
        PyErr_Clear();
        NOT_HERE;
    }
    const int status = adamw_call(
        pp.data(), pg.data(), a[12] == Py_None ? nullptr : pk.data(), numels.data(), n,
        code_of(pt), code_of(gt), pm, pv, ms, vs, bits, h[0], h[1], h[2], h[3], h[4], step, gs,
        queue(dev));
    if (status != KM_OK) return failed(status, "experts_adamw_step");
    for (PyObject *list : {a[0], a[12]})
        for (Py_ssize_t i = 0; list != Py_None && i < n; ++i)
            written(THPVariable_Unpack(PyList_GET_ITEM(list, i)));
    for (PyObject *o : {a[2], a[3], a[10], a[11]})
        if (o != Py_None) written(THPVariable_Unpack(o));
    Py_RETURN_TRUE;
    END_HANDLE_TH_ERRORS
}

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

// ({name: address of the C entry point}, check) -> None
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t count) {
    if (count < 1 || !PyDict_Check(a[0])) {
        PyErr_SetString(PyExc_TypeError, "bind takes a dict of addresses");
        return nullptr;
    }
    // All of them, or none: a module whose bind was refused stays as it was.
    auto each = [&](auto visit) {
        visit("experts_plan_workspace_bytes", plan_bytes);
        visit("experts_plan", plan_call);
        visit("experts_dispatch", dispatch_call);
        visit("experts_dispatch_backward", dispatch_backward_call);
        visit("experts_combine", combine_call);
        visit("experts_combine_backward", combine_backward_call);
        visit("experts_linear_workspace_bytes", linear_bytes);
        visit("experts_linear", linear_call);
        visit("experts_linear_backward", linear_backward_call);
        visit("experts_adamw_state_elements", adamw_elements);
        visit("experts_adamw_step", adamw_call);
    };
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
PyMethodDef methods[] = {KX_METHOD(bind),
                         KX_METHOD(plan),
                         KX_METHOD(dispatch),
                         KX_METHOD(dispatch_backward),
                         KX_METHOD(combine),
                         KX_METHOD(combine_backward),
                         KX_METHOD(linear),
                         KX_METHOD(linear_backward),
                         KX_METHOD(adamw_step),
                         KX_METHOD(unrecorded),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_experts_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__experts_torch() { return PyModule_Create(&module); }
