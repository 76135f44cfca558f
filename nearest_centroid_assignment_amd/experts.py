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
have any row stride, with the elements of a row next to each other; the header
has the largest sizes. As in ``binding``, a call enqueues on ``stream`` (the current
one by default) and returns. Gradients are explicit calls, given what the forward call returned:
autograd records none of this, and a forward call with an input that requires grad
(not under ``torch.no_grad()``) or that has a forward-mode tangent warns of it.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
from typing import NamedTuple

import torch

from .binding import (HERE, KMeansError, _check, _check_workspace, _record, _side_stream, _stream,
                      lib as _kmeans_lib)

ACTS = {"none": 0, "relu": 1, "gelu_tanh": 2, "silu": 3}
TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
BLOCK = 256  # elements of an 8-bit moment that share a scale

__all__ = ["KMeansError", "Plan", "plan", "dispatch", "dispatch_backward", "combine",
           "combine_backward", "linear", "linear_backward", "adamw_state", "adamw_step",
           "adamw_moments"]

_lib = None
_native = None  # the torch module, once lib() has loaded it


def _load_native(L, names, name="_experts_torch"):
    """The module that takes the ordinary calls natively (csrc/experts_torch.cpp,
    csrc/layers_torch.cpp), bound to the library's entry points."""
    path = os.path.join(HERE, f"{name}.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m nearest_centroid_assignment_amd.build`")
    spec = importlib.util.spec_from_file_location(name, path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.bind({n: ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names}, _check)
    return module


def lib() -> ctypes.CDLL:
    """The HIP library with the experts' entry points declared."""
    global _lib, _native
    if _lib is None:
        L = _kmeans_lib()
        names = []
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
            names.append(name)
        _native = _load_native(L, names)
        _lib = L
    return _lib


def _module():
    lib()
    return _native


# ------------------------------------------------------------- marshalling
#
# The smallest calls cost more on the host than on the GPU. A call with fresh
# outputs on the current stream is therefore first offered to the native module,
# which takes it or, where anything about it is unusual, leaves it to the Python
# below (None): other streams, given outputs and workspaces, empty matrices, and
# everything that is to be refused. Both end in the same C entry point. An error of a
# launch is raised by whichever made it, and the call is not made again.


def _refuse(t, dtype, shape, dev, name):
    """Say what is wrong with t (something is)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    raise ValueError(f"{name}'s rows must be dense and must not overlap, got strides {t.stride()}")


def _first(t, name, dims):
    """(device index, dtype code) of the tensor that the others are held to."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor, got {t.device}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    code = TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return dev, code


def _rows(t, dtype, rows, cols, dev, name):
    """(pointer, row stride) of a matrix whose rows are dense."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.get_device() != dev \
            or t.shape != (rows, cols):
        _refuse(t, dtype, (rows, cols), dev, name)
    ld, step = t.stride()
    if rows <= 1:
        ld = cols
    if ld < cols or (step != 1 and cols > 1):
        if rows and cols:
            _refuse(t, dtype, (rows, cols), dev, name)
        ld = cols
    return t.data_ptr() or None, ld


def _dense(t, dtype, shape, dev, name):
    """Pointer of a contiguous tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.get_device() != dev \
            or t.shape != shape or not t.is_contiguous():
        _refuse(t, dtype, shape, dev, name)
    return t.data_ptr() or None


def _queue(stream, dev):
    """(raw stream, the torch stream if it is not the current one)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev), None
    device = torch.device("cuda", dev)
    return _stream(stream, device), _side_stream(stream, device)


def _new(like, side, shape, dtype=None):
    """A new tensor, allocated on the stream that the kernels run on."""
    if side is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(side):
        return like.new_empty(shape, dtype=dtype)


def _scratch(workspace, nbytes, like, side):
    """(workspace, pointer, bytes); nothing where the call needs nothing."""
    if workspace is None:
        if nbytes <= BLOCK:  # slack for alignment alone
            return None, None, 0
        workspace = _new(like, side, nbytes, torch.uint8)
    else:
        _check_workspace(workspace, like.device)
    return workspace, workspace.data_ptr(), workspace.numel()


def _mark(stream, dev, *tensors):
    _record(stream, torch.device("cuda", dev), *tensors)


def _written(*tensors):
    """Tell autograd that these were written in place (the native calls do too)."""
    torch.autograd.graph.increment_version(
        [t for t in tensors if t is not None and not t.is_inference()])


def _given(out, dtype, rows, cols, dev):
    """(pointer, row stride) of an output that the caller gives."""
    got = _rows(out, dtype, rows, cols, dev, "out")
    _written(out)
    return got


def _on_device(fn):
    """Run fn with its first tensor's device current: the library launches there."""

    @functools.wraps(fn)
    def call(t, *args, **kwargs):
        first = t
        if isinstance(first, (list, tuple)):
            first = first[0] if first else None
        dev = first.get_device() if isinstance(first, torch.Tensor) else -1
        if dev < 0 or dev == torch.cuda.current_device():
            return fn(t, *args, **kwargs)
        with torch.cuda.device(dev):
            return fn(t, *args, **kwargs)

    return call


# ------------------------------------------------------------------ tokens


class Plan(NamedTuple):
    """A batch's pairs sorted by expert: ``order`` (tokens * top,) int32, the
    pair at each place (-1: none); ``place`` (tokens, top) int32, its inverse
    (-1: dropped); ``offsets`` (experts + 1,) int32, the experts' places."""

    order: torch.Tensor
    place: torch.Tensor
    offsets: torch.Tensor


def plan(ids, experts, workspace=None, stream=None) -> Plan:
    """Sort the (tokens, top) or (tokens,) int64 expert numbers; numbers
    outside [0, experts) are dropped. Stable: an expert's pairs stay in order."""
    if workspace is None and stream is None:
        got = (_native or _module()).plan(ids, experts)
        if got is not None:
            return Plan(*got)
    return _plan(ids, experts, workspace, stream)


@_on_device
def _plan(ids, experts, workspace, stream):
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if not ids.is_cuda:
        raise ValueError(f"ids must be a GPU tensor, got {ids.device}")
    if ids.dtype != torch.int64 or ids.dim() not in (1, 2) or not ids.is_contiguous():
        raise TypeError("ids must be a contiguous int64 tensor (tokens,) or (tokens, top)")
    dev = ids.get_device()
    tokens, top = ids.shape if ids.dim() == 2 else (ids.shape[0], 1)
    pairs = tokens * top
    L = lib()
    queue, side = _queue(stream, dev)
    nbytes = L.experts_plan_workspace_bytes(tokens, top, experts)
    workspace, pw, nw = _scratch(workspace, nbytes, ids, side)
    # One allocation for the three outputs.
    out = _new(ids, side, 2 * pairs + max(int(experts), 0) + 1, torch.int32)
    at = out.data_ptr()
    _check(L.experts_plan(ids.data_ptr() or None, tokens, top, experts, at, at + 4 * pairs,
                          at + 8 * pairs, pw, nw, queue), "experts_plan")
    if side is not None:
        _mark(stream, dev, ids, out, workspace)
    order, place, offsets = out.split((pairs, pairs, experts + 1))
    return Plan(order, place.view(tokens, top), offsets)


def _sizes(plan):
    tokens, top = plan.place.shape
    return tokens, top, tokens * top


def dispatch(x, plan, out=None, stream=None):
    """The rows of x (tokens, width) in sorted order: (tokens * top, width).
    Places without a pair get zero rows."""
    if out is None and stream is None:
        got = (_native or _module()).dispatch(x, plan)
        if got is not None:
            return got
    _module().unrecorded("dispatch", x)
    return _dispatch(x, plan, out, stream)


@_on_device
def _dispatch(x, plan, out, stream):
    dev, code = _first(x, "x", 2)
    tokens, top, pairs = _sizes(plan)
    width, dtype = x.shape[1], x.dtype
    px, ldx = _rows(x, dtype, tokens, width, dev, "x")
    order = _dense(plan.order, torch.int32, (pairs,), dev, "plan.order")
    place = _dense(plan.place, torch.int32, (tokens, top), dev, "plan.place")
    queue, side = _queue(stream, dev)
    if out is None:
        out = _new(x, side, (pairs, width))
        po, ldo = out.data_ptr() or None, width
    else:
        po, ldo = _given(out, dtype, pairs, width, dev)
    _check(lib().experts_dispatch(px, ldx, code, tokens, top, width, order, place, po, ldo, queue),
           "experts_dispatch")
    if side is not None:
        _mark(stream, dev, x, plan.order, plan.place, out)
    return out


def dispatch_backward(dxs, plan, out=None, stream=None):
    """Gradient of dispatch: each token's sum of its pairs' rows of dxs."""
    if out is None and stream is None:
        got = (_native or _module()).dispatch_backward(dxs, plan)
        if got is not None:
            return got
    return _dispatch_backward(dxs, plan, out, stream)


@_on_device
def _dispatch_backward(dxs, plan, out, stream):
    dev, code = _first(dxs, "dxs", 2)
    tokens, top, pairs = _sizes(plan)
    width, dtype = dxs.shape[1], dxs.dtype
    pg, ldg = _rows(dxs, dtype, pairs, width, dev, "dxs")
    place = _dense(plan.place, torch.int32, (tokens, top), dev, "plan.place")
    queue, side = _queue(stream, dev)
    if out is None:
        out = _new(dxs, side, (tokens, width))
        po, ldo = out.data_ptr() or None, width
    else:
        po, ldo = _given(out, dtype, tokens, width, dev)
    _check(lib().experts_dispatch_backward(pg, ldg, code, tokens, top, width, place, po, ldo,
                                           queue), "experts_dispatch_backward")
    if side is not None:
        _mark(stream, dev, dxs, plan.place, out)
    return out


def combine(ys, weights, plan, out=None, stream=None):
    """Each token's weighted sum of its pairs' rows of ys (tokens * top, width);
    weights (tokens, top) float32."""
    if out is None and stream is None:
        got = (_native or _module()).combine(ys, weights, plan)
        if got is not None:
            return got
    _module().unrecorded("combine", ys, weights)
    return _combine(ys, weights, plan, out, stream)


@_on_device
def _combine(ys, weights, plan, out, stream):
    dev, code = _first(ys, "ys", 2)
    tokens, top, pairs = _sizes(plan)
    width, dtype = ys.shape[1], ys.dtype
    py, ldy = _rows(ys, dtype, pairs, width, dev, "ys")
    pw = _dense(weights, torch.float32, (tokens, top), dev, "weights")
    place = _dense(plan.place, torch.int32, (tokens, top), dev, "plan.place")
    queue, side = _queue(stream, dev)
    if out is None:
        out = _new(ys, side, (tokens, width))
        po, ldo = out.data_ptr() or None, width
    else:
        po, ldo = _given(out, dtype, tokens, width, dev)
    _check(lib().experts_combine(py, ldy, pw, code, tokens, top, width, place, po, ldo, queue),
           "experts_combine")
    if side is not None:
        _mark(stream, dev, ys, weights, plan.place, out)
    return out


def combine_backward(dy, ys, weights, plan, need_dys=True, need_dweights=True, stream=None):
    """Gradients of combine: (dys, dweights), None for the one not needed."""
    if need_dys and need_dweights and stream is None:
        got = (_native or _module()).combine_backward(dy, ys, weights, plan)
        if got is not None:
            return got
    return _combine_backward(dy, ys, weights, plan, need_dys, need_dweights, stream)


@_on_device
def _combine_backward(dy, ys, weights, plan, need_dys, need_dweights, stream):
    dev, code = _first(dy, "dy", 2)
    tokens, top, pairs = _sizes(plan)
    width, dtype = dy.shape[1], dy.dtype
    pg, ldg = _rows(dy, dtype, tokens, width, dev, "dy")
    py, ldy = _rows(ys, dtype, pairs, width, dev, "ys") if need_dweights else (None, 0)
    pw = _dense(weights, torch.float32, (tokens, top), dev, "weights")
    order = _dense(plan.order, torch.int32, (pairs,), dev, "plan.order")
    place = _dense(plan.place, torch.int32, (tokens, top), dev, "plan.place")
    queue, side = _queue(stream, dev)
    dys = _new(dy, side, (pairs, width)) if need_dys else None
    dweights = _new(dy, side, (tokens, top), torch.float32) if need_dweights else None
    if tokens and (need_dys or need_dweights):
        _check(lib().experts_combine_backward(
            pg, ldg, py, ldy, pw, code, tokens, top, width, order, place,
            dys.data_ptr() if need_dys else None, width,
            dweights.data_ptr() if need_dweights else None, queue), "experts_combine_backward")
    if side is not None:
        _mark(stream, dev, dy, ys, weights, plan.order, plan.place, dys, dweights)
    return dys, dweights


# ------------------------------------------------------------------ linear


def _act_code(act, name="act"):
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"{name} must be one of {', '.join(ACTS)}, got {act!r}")
    return code


def _weights(w, dtype, offsets, dev):
    """(pointer, outs, ins, experts, pointer of the offsets)."""
    if not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor")
    shape = w.shape
    if offsets is None:
        if len(shape) != 2:
            raise ValueError(f"w must be (outs, ins) without offsets, got shape {tuple(shape)}")
        return _dense(w, dtype, shape, dev, "w"), shape[0], shape[1], 1, None
    if len(shape) != 3:
        raise ValueError(f"w must be (experts, outs, ins) with offsets, got {tuple(shape)}")
    po = _dense(offsets, torch.int32, (shape[0] + 1,), dev, "offsets")
    return _dense(w, dtype, shape, dev, "w"), shape[1], shape[2], shape[0], po


def _misplaced(px, ldx, pw, ins):
    """Whether x or w misses the 4-byte boundaries that 16-bit rows are read on."""
    return ((px or 0) | (pw or 0)) % 4 != 0 or (ldx | ins) % 2 != 0


def linear(x, w, bias=None, residual=None, act="none", offsets=None, save_pre=False, out=None,
           workspace=None, stream=None):
    """act(x w^T + bias) + residual for x (rows, ins).

    w (outs, ins) and bias (outs,) for all rows, or, with ``offsets`` (a plan's),
    w (experts, outs, ins) and bias (experts, outs): expert e has the rows
    offsets[e] to offsets[e + 1], and rows past the last expert's become zero.
    act: "none", "relu", "gelu_tanh", "silu". With ``save_pre`` returns (out,
    x w^T + bias), the latter for linear_backward."""
    if out is None and workspace is None and stream is None:
        got = (_native or _module()).linear(x, w, bias, residual, ACTS.get(act, -1), offsets,
                                            save_pre)
        if got is not None:
            return got
    _module().unrecorded("linear", x, w, bias, residual)
    return _linear(x, w, bias, residual, act, offsets, save_pre, out, workspace, stream)


@_on_device
def _linear(x, w, bias, residual, act, offsets, save_pre, out, workspace, stream):
    dev, code = _first(x, "x", 2)
    dtype, act_code = x.dtype, _act_code(act)
    pw, outs, ins, experts, pf = _weights(w, dtype, offsets, dev)
    rows = x.shape[0]
    px, ldx = _rows(x, dtype, rows, ins, dev, "x")
    pb = None if bias is None else _dense(bias, dtype, w.shape[:-1], dev, "bias")
    pr, ldr = (None, 0) if residual is None else _rows(residual, dtype, rows, outs, dev, "residual")
    queue, side = _queue(stream, dev)
    if out is None:
        out = _new(x, side, (rows, outs))
        po, ldo = out.data_ptr() or None, outs
    else:
        po, ldo = _given(out, dtype, rows, outs, dev)
    pre = _new(x, side, (rows, outs)) if save_pre else None
    L = lib()
    nbytes = L.experts_linear_workspace_bytes(rows, outs, ins, experts, code, 0,
                                              _misplaced(px, ldx, pw, ins))
    workspace, ps, ns = _scratch(workspace, nbytes, x, side)
    _check(L.experts_linear(px, ldx, pw, pb, pr, ldr, pf, code, act_code, rows, outs, ins, experts,
                            po, ldo, (pre.data_ptr() or None) if save_pre else None, outs, ps, ns,
                            queue), "experts_linear")
    if side is not None:
        _mark(stream, dev, x, w, bias, residual, offsets, out, pre, workspace)
    return (out, pre) if save_pre else out


def linear_backward(dy, x, w, pre=None, act="none", offsets=None, in_pre=None, in_act="none",
                    need_dx=True, need_dw=True, need_dbias=True, workspace=None, stream=None):
    """Gradients of linear: (dx, dw, dbias), None for those not needed; the
    residual's is dy itself. ``pre`` is what linear returned with save_pre (not
    needed without an activation). With ``in_pre`` (rows, ins), dx is multiplied by
    in_act'(in_pre): given the layer before's pre, dx is that layer's dz."""
    if workspace is None and stream is None:
        got = (_native or _module()).linear_backward(
            dy, x, w, pre, ACTS.get(act, -1), offsets, in_pre, ACTS.get(in_act, -1), need_dx,
            need_dw, need_dbias)
        if got is not None:
            return got
    return _linear_backward(dy, x, w, pre, act, offsets, in_pre, in_act, need_dx, need_dw,
                            need_dbias, workspace, stream)


@_on_device
def _linear_backward(dy, x, w, pre, act, offsets, in_pre, in_act, need_dx, need_dw, need_dbias,
                     workspace, stream):
    dev, code = _first(dy, "dy", 2)
    dtype, act_code, in_code = dy.dtype, _act_code(act), _act_code(in_act, "in_act")
    pw, outs, ins, experts, pf = _weights(w, dtype, offsets, dev)
    rows = dy.shape[0]
    if act_code and pre is None:
        raise ValueError(f"pre is needed for the gradient of act={act!r}")
    pg, ldg = _rows(dy, dtype, rows, outs, dev, "dy")
    px, ldx = _rows(x, dtype, rows, ins, dev, "x")
    pp, ldp = _rows(pre, dtype, rows, outs, dev, "pre") if act_code else (None, 0)
    pi, ldi = (None, 0) if in_pre is None else _rows(in_pre, dtype, rows, ins, dev, "in_pre")
    queue, side = _queue(stream, dev)
    need_dx_now = need_dx and rows > 0
    dx = _new(dy, side, (rows, ins)) if need_dx else None
    dw = _new(w, side, w.shape) if need_dw else None
    dbias = _new(w, side, w.shape[:-1]) if need_dbias else None
    if need_dw or need_dbias or need_dx_now:
        L = lib()
        nbytes = L.experts_linear_workspace_bytes(rows, outs, ins, experts, code, 1,
                                                  _misplaced(px, ldx, pw, ins))
        workspace, ps, ns = _scratch(workspace, nbytes, dy, side)
        _check(L.experts_linear_backward(
            pg, ldg, px, ldx, pw, pp, ldp, pi, ldi, pf, code, act_code, in_code, rows, outs, ins,
            experts, dx.data_ptr() if need_dx_now else None, ins,
            dw.data_ptr() if need_dw else None, dbias.data_ptr() if need_dbias else None, ps, ns,
            queue), "experts_linear_backward")
    if side is not None:
        _mark(stream, dev, dy, x, w, pre, in_pre, offsets, dx, dw, dbias, workspace)
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
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")
    params = list(params)
    total = _numels(params)[1]
    dev = params[0].device if params else "cuda"
    f32 = dict(dtype=torch.float32, device=dev)
    if bits == 32:
        return {"m": torch.zeros(total, **f32), "v": torch.zeros(total, **f32)}
    return {"m": torch.zeros(total, dtype=torch.int8, device=dev),
            "v": torch.zeros(total, dtype=torch.uint8, device=dev),
            "m_scale": torch.zeros(total // BLOCK, **f32),
            "v_scale": torch.zeros(total // BLOCK, **f32)}


def _pointers(tensors, dtype, params, dev, name):
    """ctypes array of the tensors' pointers, each checked against its parameter."""
    if len(tensors) != len(params):
        raise ValueError(f"{name} must hold {len(params)} tensors, got {len(tensors)}")
    for t, p in zip(tensors, params):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.get_device() != dev \
                or t.shape != p.shape or not t.is_contiguous():
            _refuse(t, dtype, p.shape, dev, name)
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def adamw_step(params, grads, m, v, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, step=1,
               m_scale=None, v_scale=None, copies=None, grad_scale=None, stream=None):
    """One AdamW step, in place, over lists of tensors (one dtype for the
    parameters, one for the gradients; a tensor that is shared is given once). m, v (and the scales of 8-bit moments)
    as made by adamw_state. ``copies``: bfloat16 tensors that receive the new
    parameters. ``grad_scale``: a float32 GPU tensor of one element that
    multiplies the gradients (clipping, loss scaling); the step is taken whatever
    it holds, so an infinite or NaN gradient reaches the moments: with loss scaling,
    look at the gradients before the call. step counts from 1."""
    if stream is None and (_native or _module()).adamw_step(
            params, grads, m, v, lr, betas[0], betas[1], eps, weight_decay, step, m_scale, v_scale,
            copies, grad_scale):
        return
    _adamw_step(params, grads, m, v, lr, betas, eps, weight_decay, step, m_scale, v_scale, copies,
                grad_scale, stream)


@_on_device
def _adamw_step(params, grads, m, v, lr, betas, eps, weight_decay, step, m_scale, v_scale, copies,
                grad_scale, stream):
    if not params:
        return
    if len(grads) != len(params):
        raise ValueError(f"grads must hold {len(params)} tensors, got {len(grads)}")
    first, g0 = params[0], grads[0]
    dev, pc = _first(first, "params", first.dim() if isinstance(first, torch.Tensor) else 0)
    gc = _first(g0, "grads", g0.dim() if isinstance(g0, torch.Tensor) else 0)[1]
    pp = _pointers(params, first.dtype, params, dev, "params")
    pg = _pointers(grads, g0.dtype, params, dev, "grads")
    pk = None if copies is None else _pointers(copies, torch.bfloat16, params, dev, "copies")
    n, total = _numels(params)
    bits = 8 if m.dtype == torch.int8 else 32
    if (bits == 8) != (m_scale is not None) or (bits == 8) != (v_scale is not None):
        raise ValueError("m_scale and v_scale belong to 8-bit moments, and only to them")
    pm = _dense(m, torch.int8 if bits == 8 else torch.float32, (total,), dev, "m")
    pv = _dense(v, torch.uint8 if bits == 8 else torch.float32, (total,), dev, "v")
    ms = vs = gs = None
    if bits == 8:
        ms = _dense(m_scale, torch.float32, (total // BLOCK,), dev, "m_scale")
        vs = _dense(v_scale, torch.float32, (total // BLOCK,), dev, "v_scale")
    if grad_scale is not None:
        gs = _dense(grad_scale, torch.float32, (1,), dev, "grad_scale")
    queue, side = _queue(stream, dev)
    _check(lib().experts_adamw_step(pp, pg, pk, n, len(params), pc, gc, pm, pv, ms, vs, bits, lr,
                                    betas[0], betas[1], eps, weight_decay, step, gs, queue),
           "experts_adamw_step")
    _written(*params, *(copies or ()), m, v, m_scale, v_scale)
    if side is not None:
        _mark(stream, dev, *params, *grads, *(copies or ()), m, v, m_scale, v_scale, grad_scale)


def adamw_moments(m, v, m_scale, v_scale, stream=None):
    """The float32 values of 8-bit moments: (m, v)."""
    return _adamw_moments(m, v, m_scale, v_scale, stream)


@_on_device
def _adamw_moments(m, v, m_scale, v_scale, stream):
    if not isinstance(m, torch.Tensor) or not m.is_cuda:
        raise TypeError("m must be a GPU tensor")
    total, dev = m.numel(), m.get_device()
    if total % BLOCK:
        raise ValueError(f"m must hold a multiple of {BLOCK} elements, got {total}")
    blocks = (total // BLOCK,)
    pm = _dense(m, torch.int8, (total,), dev, "m")
    pv = _dense(v, torch.uint8, (total,), dev, "v")
    ms = _dense(m_scale, torch.float32, blocks, dev, "m_scale")
    vs = _dense(v_scale, torch.float32, blocks, dev, "v_scale")
    queue, side = _queue(stream, dev)
    mo, vo = _new(m_scale, side, total), _new(m_scale, side, total)
    _check(lib().experts_adamw_moments(pm, pv, ms, vs, total, mo.data_ptr() or None,
                                       vo.data_ptr() or None, queue), "experts_adamw_moments")
    if side is not None:
        _mark(stream, dev, m, v, m_scale, v_scale, mo, vo)
    return mo, vo
