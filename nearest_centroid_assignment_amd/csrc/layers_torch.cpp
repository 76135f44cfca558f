// layers_torch.cpp - the ordinary calls of layers.py, marshalled natively: as
// experts_torch.cpp does for experts.py. Each function makes one call of the C ABI on the
// current stream with fresh outputs, or returns None without having enqueued a kernel.
#include "torch_args.h"

#include "../../include/layers_mi355x.h"

namespace {

decltype(&layers_embed) embed_call;
decltype(&layers_embed_backward_workspace_bytes) embed_bytes;
decltype(&layers_embed_backward) embed_backward_call;
decltype(&layers_norm) norm_call;
decltype(&layers_norm_backward_workspace_bytes) norm_bytes;
decltype(&layers_norm_backward) norm_backward_call;
decltype(&layers_route) route_call;
decltype(&layers_route_backward) route_backward_call;
decltype(&layers_cross_entropy_workspace_bytes) entropy_bytes;
decltype(&layers_cross_entropy) entropy_call;
decltype(&layers_cross_entropy_backward_workspace_bytes) entropy_backward_bytes;
decltype(&layers_cross_entropy_backward) entropy_backward_call;
const char *const module_name = "layers";

// The value of a float or an integer; false where it is neither.
bool number(PyObject *o, double &v) {
    v = PyFloat_AsDouble(o);
    if (v != -1.0 || !PyErr_Occurred()) return true;
    PyErr_Clear();
    return false;
}
bool integer(PyObject *o, int64_t &v) {
    if (!PyLong_Check(o)) return false;
    v = PyLong_AsLongLong(o);
    if (v != -1 || !PyErr_Occurred()) return true;
    PyErr_Clear();
    return false;
}
void *pointer(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// (ids, w, scale) -> out
PyObject *embed(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(3);
    const at::Tensor *ids = tensor(a[0]), *w = tensor(a[1]);
    double scale;
    if (!ids || ids->dim() != 1 || !w || w->dim() != 2 || !number(a[2], scale)) NOT_HERE;
    const int dev = call_device(*w), code = code_of(w->scalar_type());
    if (dev < 0 || code < 0) NOT_HERE;
    const int64_t tokens = ids->size(0), width = w->size(1);
    const void *pi = dense(ids, at::kLong, {tokens}, dev), *pw = dense(w, w->scalar_type(), w->sizes(), dev);
    if (!pi || !pw) NOT_HERE;
    if (!say_unrecorded("embed", {w})) return nullptr;
    at::Tensor out = new_tensor({tokens, width}, w->scalar_type(), dev);
    const int status = embed_call((const int64_t *)pi, tokens, pw, code, w->size(0), width, scale,
                                  out.data_ptr(), width, queue(dev));
    if (status != KM_OK) return failed(status, "layers_embed");
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// (dy, ids, classes, scale) -> dw
PyObject *embed_backward(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(4);
    const at::Tensor *dy = tensor(a[0]);
    int64_t classes;
    double scale;
    if (!dy || dy->dim() != 2 || !integer(a[2], classes) || !number(a[3], scale)) NOT_HERE;
    const int dev = call_device(*dy), code = code_of(dy->scalar_type());
    const int64_t tokens = dy->size(0), width = dy->size(1);
    Rows rg;
    if (dev < 0 || code < 0 || !rows_of(dy, dy->scalar_type(), tokens, width, dev, rg)) NOT_HERE;
    const void *pi = dense(tensor(a[1]), at::kLong, {tokens}, dev);
    const size_t bytes = embed_bytes(tokens, classes, width, code);
    if (!pi || bytes == 0) NOT_HERE;
    Scratch ws(bytes, dev);
    at::Tensor dw = new_tensor({classes, width}, dy->scalar_type(), dev);
    const int status = embed_backward_call(rg.p, rg.ld, (const int64_t *)pi, tokens, code, classes, width,
                                           scale, dw.data_ptr(), ws.p, ws.n, queue(dev));
    if (status != KM_OK) return failed(status, "layers_embed_backward");
    return wrap(dw);
    END_HANDLE_TH_ERRORS
}

// (x, weight, bias, eps, save_stats) -> out or (out, mean, rstd)
PyObject *layer_norm(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(5);
    const at::Tensor *x = tensor(a[0]);
    double eps;
    if (!x || x->dim() != 2 || !number(a[3], eps)) NOT_HERE;
    const int dev = call_device(*x), code = code_of(x->scalar_type());
    const int64_t rows = x->size(0), width = x->size(1);
    Rows rx;
    if (dev < 0 || code < 0 || !rows_of(x, x->scalar_type(), rows, width, dev, rx)) NOT_HERE;
    const at::Tensor *weight = tensor(a[1]), *bias = tensor(a[2]);
    const at::ScalarType kind = weight ? weight->scalar_type() : bias ? bias->scalar_type() : x->scalar_type();
    const void *pw = nullptr, *pb = nullptr;
    if (code_of(kind) < 0 || (a[1] != Py_None && !(pw = dense(weight, kind, {width}, dev))) ||
        (a[2] != Py_None && !(pb = dense(bias, kind, {width}, dev))))
        NOT_HERE;
    bool save;
    if (!truth(a[4], save)) NOT_HERE;
    if (!say_unrecorded("layer_norm", {x, weight, bias})) return nullptr;
    at::Tensor out = new_tensor({rows, width}, x->scalar_type(), dev), mean, rstd;
    if (save) {
        mean = new_tensor({rows}, at::kFloat, dev);
        rstd = new_tensor({rows}, at::kFloat, dev);
    }
    const int status = norm_call(rx.p, rx.ld, pw, pb, code, code_of(kind), rows, width, eps, out.data_ptr(),
                                 width, (float *)pointer(mean), (float *)pointer(rstd), queue(dev));
    if (status != KM_OK) return failed(status, "layers_norm");
    return save ? tuple_of(out, mean, rstd) : wrap(out);
    END_HANDLE_TH_ERRORS
}

// (dy, x, weight, mean, rstd, need_dx, need_dweight, need_dbias) -> (dx, dweight, dbias)
PyObject *layer_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(8);
    const at::Tensor *dy = tensor(a[0]);
    if (!dy || dy->dim() != 2) NOT_HERE;
    const int dev = call_device(*dy), code = code_of(dy->scalar_type());
    const at::ScalarType type = dy->scalar_type();
    const int64_t rows = dy->size(0), width = dy->size(1);
    Rows rg, rx;
    if (dev < 0 || code < 0 || !rows_of(dy, type, rows, width, dev, rg) ||
        !rows_of(tensor(a[1]), type, rows, width, dev, rx))
        NOT_HERE;
    const at::Tensor *weight = tensor(a[2]);
    const at::ScalarType kind = weight ? weight->scalar_type() : type;
    const void *pw = nullptr;
    if (code_of(kind) < 0 || (a[2] != Py_None && !(pw = dense(weight, kind, {width}, dev)))) NOT_HERE;
    const float *pm = (const float *)dense(tensor(a[3]), at::kFloat, {rows}, dev);
    const float *ps = (const float *)dense(tensor(a[4]), at::kFloat, {rows}, dev);
    bool need_dx, need_dw, need_db;
    if (!truth(a[5], need_dx) || !truth(a[6], need_dw) || !truth(a[7], need_db)) NOT_HERE;
    if (!pm || !ps || (!need_dx && !need_dw && !need_db)) NOT_HERE;
    const size_t bytes = need_dw || need_db ? norm_bytes(rows, width, code) : 1;
    if (bytes == 0) NOT_HERE;
    Scratch ws(bytes, dev);
    at::Tensor dx, dw, db;
    if (need_dx) dx = new_tensor({rows, width}, type, dev);
    if (need_dw) dw = new_tensor({width}, kind, dev);
    if (need_db) db = new_tensor({width}, kind, dev);
    const int status = norm_backward_call(rg.p, rg.ld, rx.p, rx.ld, pw, pm, ps, code, code_of(kind), rows,
                                          width, pointer(dx), width, pointer(dw), pointer(db), ws.p, ws.n,
                                          queue(dev));
    if (status != KM_OK) return failed(status, "layers_norm_backward");
    return tuple_of(dx, dw, db);
    END_HANDLE_TH_ERRORS
}

// (logits, top, score code, bias, groups, top_groups, group_best, renormalize, scale)
// -> (ids, weights)
PyObject *route(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(9);
    const at::Tensor *z = tensor(a[0]);
    int64_t top, score, groups, kept, best;
    double scale;
    if (!z || z->dim() != 2 || !integer(a[1], top) || !integer(a[2], score) || !integer(a[4], groups) ||
        !integer(a[5], kept) || !integer(a[6], best) || !number(a[8], scale) || top < 1)
        NOT_HERE;
    const int dev = call_device(*z), code = code_of(z->scalar_type());
    const int64_t tokens = z->size(0), experts = z->size(1);
    Rows rz;
    if (dev < 0 || code < 0 || !rows_of(z, z->scalar_type(), tokens, experts, dev, rz)) NOT_HERE;
    const float *pb = nullptr;
    if (a[3] != Py_None && !(pb = (const float *)dense(tensor(a[3]), at::kFloat, {experts}, dev))) NOT_HERE;
    bool renormalize;
    if (top > experts || !truth(a[7], renormalize)) NOT_HERE;
    if (!say_unrecorded("route", {z})) return nullptr;
    at::Tensor ids = new_tensor({tokens, top}, at::kLong, dev), w = new_tensor({tokens, top}, at::kFloat, dev);
    const int status = route_call(rz.p, rz.ld, code, tokens, experts, top, (int)score, pb, groups, kept, best,
                                  renormalize, scale, (int64_t *)ids.data_ptr(),
                                  (float *)w.data_ptr(), queue(dev));
    if (status != KM_OK) return failed(status, "layers_route");
    return tuple_of(ids, w);
    END_HANDLE_TH_ERRORS
}

// (dweights, logits, ids, score code, renormalize, scale) -> dlogits
PyObject *route_backward(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(6);
    const at::Tensor *z = tensor(a[1]), *ids = tensor(a[2]);
    int64_t score;
    double scale;
    if (!z || z->dim() != 2 || !ids || ids->dim() != 2 || !integer(a[3], score) || !number(a[5], scale)) NOT_HERE;
    const int dev = call_device(*z), code = code_of(z->scalar_type());
    const int64_t tokens = z->size(0), experts = z->size(1), top = ids->size(1);
    Rows rz;
    if (dev < 0 || code < 0 || !rows_of(z, z->scalar_type(), tokens, experts, dev, rz)) NOT_HERE;
    const int64_t *pi = (const int64_t *)dense(ids, at::kLong, {tokens, top}, dev);
    const float *pg = (const float *)dense(tensor(a[0]), at::kFloat, {tokens, top}, dev);
    bool renormalize;
    if (!pi || !pg || !truth(a[4], renormalize)) NOT_HERE;
    at::Tensor out = new_tensor({tokens, experts}, z->scalar_type(), dev);
    const int status = route_backward_call(pg, rz.p, rz.ld, pi, code, tokens, experts, top, (int)score,
                                           renormalize, scale, out.data_ptr(), experts, queue(dev));
    if (status != KM_OK) return failed(status, "layers_route_backward");
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// x, w and targets of a cross entropy.
struct Entropy {
    Rows x;
    const void *w = nullptr;
    const int64_t *targets = nullptr;
    int dev = -1, code = -1;
    int64_t rows = 0, classes = 0, width = 0;
    int misplaced() const {
        return (((uintptr_t)x.p | (uintptr_t)w) % 4 != 0) || ((x.ld | width) % 2 != 0);
    }
};
bool entropy_of(PyObject *ox, PyObject *ow, PyObject *ot, Entropy &e) {
    const at::Tensor *x = tensor(ox), *w = tensor(ow);
    if (!x || x->dim() != 2 || !w || w->dim() != 2) return false;
    e.dev = call_device(*x);
    e.code = code_of(x->scalar_type());
    e.rows = x->size(0);
    e.classes = w->size(0);
    e.width = w->size(1);
    if (e.dev < 0 || e.code < 0 || !rows_of(x, x->scalar_type(), e.rows, e.width, e.dev, e.x)) return false;
    e.w = dense(w, x->scalar_type(), w->sizes(), e.dev);
    e.targets = (const int64_t *)dense(tensor(ot), at::kLong, {e.rows}, e.dev);
    return e.w && e.targets;
}

// (x, w, targets) -> (loss, lse)
PyObject *cross_entropy(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(3);
    Entropy e;
    if (!entropy_of(a[0], a[1], a[2], e)) NOT_HERE;
    const size_t bytes = entropy_bytes(e.rows, e.classes, e.width, e.code, e.misplaced());
    if (bytes == 0) NOT_HERE;
    if (!say_unrecorded("cross_entropy", {tensor(a[0]), tensor(a[1])})) return nullptr;
    Scratch ws(bytes, e.dev);
    at::Tensor loss = new_tensor({e.rows}, at::kFloat, e.dev), lse = new_tensor({e.rows}, at::kFloat, e.dev);
    const int status = entropy_call(e.x.p, e.x.ld, e.w, e.targets, e.code, e.rows, e.classes, e.width,
                                    (float *)loss.data_ptr(), (float *)lse.data_ptr(), ws.p, ws.n,
                                    queue(e.dev));
    if (status != KM_OK) return failed(status, "layers_cross_entropy");
    return tuple_of(loss, lse);
    END_HANDLE_TH_ERRORS
}

// (dloss, x, w, targets, lse, dlse, need_dx, need_dw) -> (dx, dw)
PyObject *cross_entropy_backward(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    ARGS(8);
    Entropy e;
    if (!entropy_of(a[1], a[2], a[3], e)) NOT_HERE;
    const float *pg = (const float *)dense(tensor(a[0]), at::kFloat, {e.rows}, e.dev);
    const float *ps = (const float *)dense(tensor(a[4]), at::kFloat, {e.rows}, e.dev), *pd = nullptr;
    if (!pg || !ps) NOT_HERE;
    if (a[5] != Py_None && !(pd = (const float *)dense(tensor(a[5]), at::kFloat, {e.rows}, e.dev))) NOT_HERE;
    bool need_dx, need_dw;
    if (!truth(a[6], need_dx) || !truth(a[7], need_dw)) NOT_HERE;
    const size_t bytes = entropy_backward_bytes(e.rows, e.classes, e.width, e.code, e.misplaced());
    if (bytes == 0 || (!need_dx && !need_dw)) NOT_HERE;
    Scratch ws(bytes, e.dev);
    const at::ScalarType type = THPVariable_Unpack(a[1]).scalar_type();
    at::Tensor dx, dw;
    if (need_dx) dx = new_tensor({e.rows, e.width}, type, e.dev);
    if (need_dw) dw = new_tensor({e.classes, e.width}, type, e.dev);
    const int status = entropy_backward_call(pg, pd, e.x.p, e.x.ld, e.w, e.targets, ps, e.code, e.rows,
                                             e.classes, e.width, pointer(dx), e.width, pointer(dw), ws.p,
                                             ws.n, queue(e.dev));
    if (status != KM_OK) return failed(status, "layers_cross_entropy_backward");
    return tuple_of(dx, dw);
    END_HANDLE_TH_ERRORS
}

// ({name: address of the C entry point}, check) -> None
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t count) {
    return bind_all(a, count, [](auto visit) {
        visit("layers_embed", embed_call);
        visit("layers_embed_backward_workspace_bytes", embed_bytes);
        visit("layers_embed_backward", embed_backward_call);
        visit("layers_norm", norm_call);
        visit("layers_norm_backward_workspace_bytes", norm_bytes);
        visit("layers_norm_backward", norm_backward_call);
        visit("layers_route", route_call);
        visit("layers_route_backward", route_backward_call);
        visit("layers_cross_entropy_workspace_bytes", entropy_bytes);
        visit("layers_cross_entropy", entropy_call);
        visit("layers_cross_entropy_backward_workspace_bytes", entropy_backward_bytes);
        visit("layers_cross_entropy_backward", entropy_backward_call);
    });
}

PyMethodDef methods[] = {KX_METHOD(bind),
                         KX_METHOD(embed),
                         KX_METHOD(embed_backward),
                         KX_METHOD(layer_norm),
                         KX_METHOD(layer_norm_backward),
                         KX_METHOD(route),
                         KX_METHOD(route_backward),
                         KX_METHOD(cross_entropy),
                         KX_METHOD(cross_entropy_backward),
                         KX_METHOD(unrecorded),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers_torch() { return PyModule_Create(&module); }
