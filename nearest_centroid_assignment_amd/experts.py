"""Operators of a mixture of experts on an MI355X (declared in
include/experts_mi355x.h, in the same library as the k-means kernels).

    plan                tokens' expert numbers -> pairs sorted by expert
    dispatch            token rows in sorted order        (dispatch_backward)
    combine             weighted rows back to the tokens  (combine_backward)
    linear              act(x w^T + b) + residual, dense or per expert
                        (linear_backward)
    adamw_step          one AdamW step over many tensors, moments in 32 or 8 bits
                        (adamw_state, adamw_moments)

The labels of ``binding.assign`` are expert numbers as they are (one a token).
Tensors supply pointers, strides and the stream; every step of the computation
runs in the library's HIP kernels, and there is no CPU fallback. Matrices may
have any row stride, with the elements of a row next to each other. As in
``binding``, a call enqueues on ``stream`` (the current one by default) and
returns; gradients are explicit calls, given what the forward call returned.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from .binding import (KMeansError, _check, _record, _side_stream, _stream, _torch, _workspace,
                      lib as _kmeans_lib)

ACTS = {"none": 0, "relu": 1, "gelu_tanh": 2, "silu": 3}
BLOCK = 256  # elements of an 8-bit moment that share a scale

__all__ = ["KMeansError", "Plan", "plan", "dispatch", "dispatch_backward", "combine",
           "combine_backward", "linear", "linear_backward", "adamw_state", "adamw_step",
           "adamw_moments"]

_lib = None
_codes = None


def lib() -> ctypes.CDLL:
    """The HIP library with the experts' entry points declared."""
    global _lib, _codes
    if _lib is None:
        L = _kmeans_lib()
        i64, vp, sz, i32, f64 = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int,
                                 ctypes.c_double)
        for name, res, args in (
            ("experts_plan_workspace_bytes", sz, [i64] * 3),
            ("experts_plan", i32, [vp, i64, i64, i64, vp, vp, vp, vp, sz, vp]),
            ("experts_dispatch", i32, [vp, i64, i32, i64, i64, i64, vp, vp, vp, i64, vp]),
            ("experts_dispatch_backward", i32, [vp, i64, i32, i64, i64, i64, vp, vp, i64, vp]),
            ("experts_combine", i32, [vp, i64, vp, i32, i64, i64, i64, vp, vp, i64, vp]),
            ("experts_combine_backward", i32,
             [vp, i64, vp, i64, vp, i32, i64, i64, i64, vp, vp, vp, i64, vp, vp]),
            ("experts_linear_workspace_bytes", sz, [i64] * 4 + [i32] * 3),
            ("experts_linear", i32,
             [vp, i64, vp, vp, vp, i64, vp, i32, i32, i64, i64, i64, i64, vp, i64, vp, i64, vp, sz,
              vp]),
            ("experts_linear_backward", i32,
             [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i32, i32, i32, i64, i64, i64, i64, vp,
              i64, vp, vp, vp, sz, vp]),
            ("experts_adamw_state_elements", i64, [vp, i64]),
            ("experts_adamw_step", i32,
             [vp, vp, vp, vp, i64, i32, i32, vp, vp, vp, vp, i32] + [f64] * 5 + [i64, vp, vp]),
            ("experts_adamw_moments", i32, [vp, vp, vp, vp, i64, vp, vp, vp]),
        ):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        torch = _torch()
        _codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        _lib = L
    return _lib


# ------------------------------------------------------------- marshalling


def _code(dtype, name):
    lib()
    code = _codes.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return code


def _gpu(t, name):
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor, got {t.device}")


def _same(t, device, name):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _rows(t, dtype, shape, device, name):
    """(pointer, row stride) of a matrix whose rows are dense (None -> none)."""
    if t is None:
        return None, 0
    _gpu(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    _same(t, device, name)
    if not t.numel():
        return None, shape[1]
    ld, step = t.stride()
    if step != 1 and shape[1] != 1:
        raise ValueError(f"{name}'s rows must be dense (stride 1), got strides {t.stride()}")
    if shape[0] == 1:
        ld = shape[1]
    if ld < shape[1]:
        raise ValueError(f"{name}'s rows must not overlap, got strides {t.stride()}")
    return t.data_ptr(), ld


def _dense(t, dtype, shape, device, name):
    if t is None:
        return None
    _gpu(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    _same(t, device, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() if t.numel() else None


def _matrix(t, name):
    _gpu(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(t.shape)}")


class _On:
    """The device that a call's kernels go to, and outputs allocated on the stream they run on."""

    def __init__(self, device, stream):
        torch = _torch()
        self.device, self.stream = device, stream
        self.side = _side_stream(stream, device)
        self.change = device.index is not None and device.index != torch.cuda.current_device()

    def __enter__(self):
        torch = _torch()
        if self.change:
            self.before = torch.cuda.current_device()
            torch.cuda.set_device(self.device)
        return self

    def __exit__(self, *_):
        if self.change:
            _torch().cuda.set_device(self.before)

    def empty(self, shape, dtype):
        torch = _torch()
        if self.side is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.side):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def handle(self):
        return _stream(self.stream, self.device)

    def record(self, *tensors):
        if self.side is not None:
            _record(self.stream, self.device, *tensors)


# ------------------------------------------------------------------ tokens


class Plan(NamedTuple):
    """A batch's pairs sorted by expert: ``order`` (tokens * top,) int32, the
    pair at each place (-1: none); ``place`` (tokens, top) int32, its inverse
    (-1: dropped); ``offsets`` (experts + 1,) int32, the experts' places."""

    order: object
    place: object
    offsets: object


def plan(ids, experts, workspace=None, stream=None) -> Plan:
    """Sort the (tokens, top) or (tokens,) int64 expert numbers; numbers
    outside [0, experts) are dropped. Stable: an expert's pairs stay in order."""
    torch = _torch()
    _gpu(ids, "ids")
    if ids.dtype != torch.int64 or ids.dim() not in (1, 2) or not ids.is_contiguous():
        raise TypeError("ids must be a contiguous int64 tensor (tokens,) or (tokens, top)")
    tokens, top = ids.shape[0], ids.shape[1] if ids.dim() == 2 else 1
    L = lib()
    nbytes = L.experts_plan_workspace_bytes(tokens, top, experts)
    with _On(ids.device, stream) as on:
        workspace = _workspace(workspace, nbytes, ids.device, stream)
        # One allocation for the three outputs.
        pairs = tokens * top
        out = on.empty(2 * pairs + max(int(experts), 0) + 1, torch.int32)
        order, place, offsets = out[:pairs], out[pairs:2 * pairs].view(tokens, top), out[2 * pairs:]
        at = out.data_ptr()
        rc = L.experts_plan(ids.data_ptr() if pairs else None, tokens, top, experts, at,
                            at + 4 * pairs, at + 8 * pairs, workspace.data_ptr(),
                            workspace.numel(), on.handle())
        _check(rc, "experts_plan")
        on.record(ids, out, workspace)
    return Plan(order, place, offsets)


def _plan_sizes(p):
    tokens, top = p.place.shape
    return tokens, top, tokens * top


def _plan_ptrs(p, device):
    torch = _torch()
    tokens, top, pairs = _plan_sizes(p)
    return (_dense(p.order, torch.int32, (pairs,), device, "plan.order"),
            _dense(p.place, torch.int32, (tokens, top), device, "plan.place"))


def dispatch(x, plan, out=None, stream=None):
    """The rows of x (tokens, width) in sorted order: (tokens * top, width).
    Places without a pair get zero rows."""
    _matrix(x, "x")
    tokens, top, pairs = _plan_sizes(plan)
    width, dev, code = x.shape[1], x.device, _code(x.dtype, "x")
    px, ldx = _rows(x, x.dtype, (tokens, width), dev, "x")
    order, place = _plan_ptrs(plan, dev)
    with _On(dev, stream) as on:
        if out is None:
            out = on.empty((pairs, width), x.dtype)
        po, ldo = _rows(out, x.dtype, (pairs, width), dev, "out")
        _check(lib().experts_dispatch(px, ldx, code, tokens, top, width, order, place, po, ldo,
                                      on.handle()), "experts_dispatch")
        on.record(x, plan.order, plan.place, out)
    return out


def dispatch_backward(dxs, plan, out=None, stream=None):
    """Gradient of dispatch: each token's sum of its pairs' rows of dxs."""
    _matrix(dxs, "dxs")
    tokens, top, pairs = _plan_sizes(plan)
    width, dev, code = dxs.shape[1], dxs.device, _code(dxs.dtype, "dxs")
    pg, ldg = _rows(dxs, dxs.dtype, (pairs, width), dev, "dxs")
    _, place = _plan_ptrs(plan, dev)
    with _On(dev, stream) as on:
        if out is None:
            out = on.empty((tokens, width), dxs.dtype)
        po, ldo = _rows(out, dxs.dtype, (tokens, width), dev, "out")
        _check(lib().experts_dispatch_backward(pg, ldg, code, tokens, top, width, place, po, ldo,
                                               on.handle()), "experts_dispatch_backward")
        on.record(dxs, plan.place, out)
    return out


def combine(ys, weights, plan, out=None, stream=None):
    """Each token's weighted sum of its pairs' rows of ys (tokens * top, width);
    weights (tokens, top) float32."""
    torch = _torch()
    _matrix(ys, "ys")
    tokens, top, pairs = _plan_sizes(plan)
    width, dev, code = ys.shape[1], ys.device, _code(ys.dtype, "ys")
    py, ldy = _rows(ys, ys.dtype, (pairs, width), dev, "ys")
    pw = _dense(weights, torch.float32, (tokens, top), dev, "weights")
    _, place = _plan_ptrs(plan, dev)
    with _On(dev, stream) as on:
        if out is None:
            out = on.empty((tokens, width), ys.dtype)
        po, ldo = _rows(out, ys.dtype, (tokens, width), dev, "out")
        _check(lib().experts_combine(py, ldy, pw, code, tokens, top, width, place, po, ldo,
                                     on.handle()), "experts_combine")
        on.record(ys, weights, plan.place, out)
    return out


def combine_backward(dy, ys, weights, plan, need_dys=True, need_dweights=True, stream=None):
    """Gradients of combine: (dys, dweights), None for the one not needed."""
    torch = _torch()
    _matrix(dy, "dy")
    tokens, top, pairs = _plan_sizes(plan)
    width, dev, code = dy.shape[1], dy.device, _code(dy.dtype, "dy")
    pg, ldg = _rows(dy, dy.dtype, (tokens, width), dev, "dy")
    py, ldy = _rows(ys, dy.dtype, (pairs, width), dev, "ys") if need_dweights else (None, 0)
    pw = _dense(weights, torch.float32, (tokens, top), dev, "weights")
    order, place = _plan_ptrs(plan, dev)
    with _On(dev, stream) as on:
        dys = on.empty((pairs, width), dy.dtype) if need_dys else None
        dweights = on.empty((tokens, top), torch.float32) if need_dweights else None
        if tokens:
            _check(lib().experts_combine_backward(
                pg, ldg, py, ldy, pw, code, tokens, top, width, order, place,
                None if dys is None else dys.data_ptr(), width,
                None if dweights is None else dweights.data_ptr(), on.handle()),
                "experts_combine_backward")
        on.record(dy, ys, weights, plan.order, plan.place, dys, dweights)
    return dys, dweights


# ------------------------------------------------------------------ linear


def _act_code(act, name="act"):
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"{name} must be one of {', '.join(ACTS)}, got {act!r}")
    return code


def _weights(w, x, offsets):
    """(outs, ins, experts) of w, checked against x and offsets."""
    torch = _torch()
    _gpu(w, "w")
    if offsets is None:
        if w.dim() != 2:
            raise ValueError(f"w must be (outs, ins) without offsets, got shape {tuple(w.shape)}")
        experts = 1
    else:
        if w.dim() != 3:
            raise ValueError(f"w must be (experts, outs, ins) with offsets, got {tuple(w.shape)}")
        experts = w.shape[0]
        _dense(offsets, torch.int32, (experts + 1,), x.device, "offsets")
    return w.shape[-2], w.shape[-1], experts


def _misplaced(*pairs):
    """Whether any matrix (pointer, ld) misses the 16-byte boundaries."""
    return int(any(p is not None and (p % 16 or ld % 8) for p, ld in pairs))


def linear(x, w, bias=None, residual=None, act="none", offsets=None, save_pre=False, out=None,
           workspace=None, stream=None):
    """act(x w^T + bias) + residual for x (rows, ins).

    w (outs, ins) and bias (outs,) for all rows, or, with ``offsets`` (a plan's),
    w (experts, outs, ins) and bias (experts, outs): expert e has the rows
    offsets[e] to offsets[e + 1], and rows past the last expert's become zero.
    act: "none", "relu", "gelu_tanh", "silu". With ``save_pre`` returns (out,
    x w^T + bias), the latter for linear_backward."""
    _matrix(x, "x")
    dev, dtype = x.device, x.dtype
    code, act_code = _code(dtype, "x"), _act_code(act)
    outs, ins, experts = _weights(w, x, offsets)
    rows = x.shape[0]
    px, ldx = _rows(x, dtype, (rows, ins), dev, "x")
    pw = _dense(w, dtype, tuple(w.shape), dev, "w")
    pb = _dense(bias, dtype, tuple(w.shape[:-1]), dev, "bias")
    pr, ldr = _rows(residual, dtype, (rows, outs), dev, "residual")
    L = lib()
    with _On(dev, stream) as on:
        if out is None:
            out = on.empty((rows, outs), dtype)
        po, ldo = _rows(out, dtype, (rows, outs), dev, "out")
        pre = on.empty((rows, outs), dtype) if save_pre else None
        nbytes = L.experts_linear_workspace_bytes(rows, outs, ins, experts, code, 0,
                                                  _misplaced((px, ldx), (pw, ins)))
        workspace = _workspace(workspace, nbytes, dev, stream)
        _check(L.experts_linear(
            px, ldx, pw, pb, pr, ldr, None if offsets is None else offsets.data_ptr(), code,
            act_code, rows, outs, ins, experts, po, ldo,
            pre.data_ptr() if save_pre and rows else None, outs, workspace.data_ptr(),
            workspace.numel(), on.handle()), "experts_linear")
        on.record(x, w, bias, residual, offsets, out, pre, workspace)
    return (out, pre) if save_pre else out


def linear_backward(dy, x, w, pre=None, act="none", offsets=None, in_pre=None, in_act="none",
                    need_dx=True, need_dw=True, need_dbias=True, workspace=None, stream=None):
    """Gradients of linear: (dx, dw, dbias), None for those not needed; the
    residual's is dy itself. ``pre`` is what linear returned with save_pre (not
    needed without an activation). With ``in_pre`` (rows, ins), dx is multiplied by
    in_act'(in_pre): given the layer before's pre, dx is that layer's dz."""
    _matrix(dy, "dy")
    dev, dtype = dy.device, dy.dtype
    code, act_code, in_code = _code(dtype, "dy"), _act_code(act), _act_code(in_act, "in_act")
    outs, ins, experts = _weights(w, dy, offsets)
    rows = dy.shape[0]
    if act != "none" and pre is None:
        raise ValueError(f"pre is needed for the gradient of act={act!r}")
    pg, ldg = _rows(dy, dtype, (rows, outs), dev, "dy")
    px, ldx = _rows(x, dtype, (rows, ins), dev, "x")
    pw = _dense(w, dtype, tuple(w.shape), dev, "w")
    pp, ldp = _rows(pre if act != "none" else None, dtype, (rows, outs), dev, "pre")
    pi, ldi = _rows(in_pre, dtype, (rows, ins), dev, "in_pre")
    L = lib()
    with _On(dev, stream) as on:
        dx = on.empty((rows, ins), dtype) if need_dx else None
        dw = on.empty(tuple(w.shape), dtype) if need_dw else None
        dbias = on.empty(tuple(w.shape[:-1]), dtype) if need_dbias else None
        nbytes = L.experts_linear_workspace_bytes(rows, outs, ins, experts, code, 1,
                                                  _misplaced((px, ldx), (pw, ins)))
        workspace = _workspace(workspace, nbytes, dev, stream)
        if need_dw or need_dbias or (need_dx and rows):
            _check(L.experts_linear_backward(
                pg, ldg, px, ldx, pw, pp, ldp, pi, ldi,
                None if offsets is None else offsets.data_ptr(), code, act_code, in_code, rows,
                outs, ins, experts, dx.data_ptr() if need_dx and rows else None, ins,
                dw.data_ptr() if need_dw else None, dbias.data_ptr() if need_dbias else None,
                workspace.data_ptr(), workspace.numel(), on.handle()), "experts_linear_backward")
        on.record(dy, x, w, pre, in_pre, offsets, dx, dw, dbias, workspace)
    return dx, dw, dbias


# ------------------------------------------------------------------- adamw


def _numels(params):
    n = (ctypes.c_int64 * len(params))(*[p.numel() for p in params])
    total = lib().experts_adamw_state_elements(n, len(params))
    if total < 0:
        raise ValueError("the tensors' lengths are not supported")
    return n, total


def adamw_state(params, bits=32):
    """Zero moments for ``params`` as the keyword arguments of adamw_step: m and
    v, and with bits=8 m_scale and v_scale. One array for all tensors; a tensor's
    moments start on the next multiple of 256 elements."""
    torch = _torch()
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")
    total = _numels(params)[1]
    dev = params[0].device if params else "cuda"
    if bits == 32:
        return {"m": torch.zeros(total, device=dev), "v": torch.zeros(total, device=dev)}
    return {"m": torch.zeros(total, dtype=torch.int8, device=dev),
            "v": torch.zeros(total, dtype=torch.uint8, device=dev),
            "m_scale": torch.zeros(total // BLOCK, device=dev),
            "v_scale": torch.zeros(total // BLOCK, device=dev)}


def _pointers(tensors, dtype, params, device, name):
    """ctypes array of the tensors' pointers, each checked against its parameter."""
    if len(tensors) != len(params):
        raise ValueError(f"{name} must hold {len(params)} tensors, got {len(tensors)}")
    for t, p in zip(tensors, params):
        _gpu(t, name)
        if t.dtype != dtype:
            raise TypeError(f"{name} must all be {dtype}, got {t.dtype}")
        if t.shape != p.shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)} for a parameter of {tuple(p.shape)}")
        _same(t, device, name)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def adamw_step(params, grads, m, v, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, step=1,
               m_scale=None, v_scale=None, copies=None, grad_scale=None, stream=None):
    """One AdamW step, in place, over lists of tensors (one dtype for the
    parameters, one for the gradients). m, v (and the scales of 8-bit moments)
    as made by adamw_state. ``copies``: bfloat16 tensors that receive the new
    parameters. ``grad_scale``: a float32 GPU tensor of one element that
    multiplies the gradients (clipping, loss scaling). step counts from 1."""
    torch = _torch()
    params, grads = list(params), list(grads)
    if not params:
        return
    _gpu(params[0], "params")
    dev, pt, gt = params[0].device, params[0].dtype, grads[0].dtype if grads else None
    pc, gc = _code(pt, "params"), _code(gt, "grads")
    pp = _pointers(params, pt, params, dev, "params")
    pg = _pointers(grads, gt, params, dev, "grads")
    cs = None if copies is None else list(copies)
    pk = None if cs is None else _pointers(cs, torch.bfloat16, params, dev, "copies")
    n, total = _numels(params)
    bits = 8 if m.dtype == torch.int8 else 32
    ms = _dense(m, torch.int8 if bits == 8 else torch.float32, (total,), dev, "m")
    vs = _dense(v, torch.uint8 if bits == 8 else torch.float32, (total,), dev, "v")
    if (bits == 8) != (m_scale is not None) or (bits == 8) != (v_scale is not None):
        raise ValueError("m_scale and v_scale belong to 8-bit moments, and only to them")
    mk = _dense(m_scale, torch.float32, (total // BLOCK,), dev, "m_scale")
    vk = _dense(v_scale, torch.float32, (total // BLOCK,), dev, "v_scale")
    gk = _dense(grad_scale, torch.float32, (1,), dev, "grad_scale")
    with _On(dev, stream) as on:
        _check(lib().experts_adamw_step(pp, pg, pk, n, len(params), pc, gc, ms, vs, mk, vk, bits,
                                        lr, betas[0], betas[1], eps, weight_decay, step, gk,
                                        on.handle()), "experts_adamw_step")
        on.record(*params, *grads, *(cs or ()), m, v, m_scale, v_scale, grad_scale)


def adamw_moments(m, v, m_scale, v_scale, stream=None):
    """The float32 values of 8-bit moments: (m, v)."""
    torch = _torch()
    _gpu(m, "m")
    total, dev = m.numel(), m.device
    if total % BLOCK:
        raise ValueError(f"m must hold a multiple of {BLOCK} elements, got {total}")
    args = (_dense(m, torch.int8, (total,), dev, "m"), _dense(v, torch.uint8, (total,), dev, "v"),
            _dense(m_scale, torch.float32, (total // BLOCK,), dev, "m_scale"),
            _dense(v_scale, torch.float32, (total // BLOCK,), dev, "v_scale"))
    with _On(dev, stream) as on:
        mo, vo = on.empty(total, torch.float32), on.empty(total, torch.float32)
        _check(lib().experts_adamw_moments(*args, total, mo.data_ptr(), vo.data_ptr(),
                                           on.handle()), "experts_adamw_moments")
        on.record(m, v, m_scale, v_scale, mo, vo)
    return mo, vo
