"""Operators around a mixture of experts on an MI355X (declared in
include/layers_mi355x.h, in the same library as the k-means kernels).

    embed           rows of a table by number, scaled            (embed_backward)
    layer_norm      layer norm of rows                           (layer_norm_backward)
    route           scores of the experts to expert numbers and
                    weights, as ``experts.plan`` and
                    ``experts.combine`` take them                (route_backward)
    cross_entropy   softmax cross entropy of x w^T against one
                    class a row, the logits never kept           (cross_entropy_backward)

Numbers are the labels of ``binding.assign`` (codes of centroids) or any others. The
conventions are those of ``experts``: tensors supply pointers, strides and the stream; every
step of the computation runs in the library's HIP kernels, and there is no CPU fallback;
matrices may have any row stride, with the elements of a row next to each other; a call
enqueues on ``stream`` (the current one by default) and returns; gradients are explicit
calls, and a forward call with an input that requires grad or has a forward-mode tangent warns
of it.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import KMeansError, _check
from .experts import (_dense, _first, _given, _load_native, _mark, _new, _on_device, _queue, _rows,
                      _scratch, lib as _experts_lib)

SCORES = {"softmax": 0, "sigmoid": 1}

__all__ = ["KMeansError", "embed", "embed_backward", "layer_norm", "layer_norm_backward", "route",
           "route_backward", "cross_entropy", "cross_entropy_backward"]

_lib = None
_native = None  # the torch module (csrc/layers_torch.cpp), once lib() has loaded it


def lib() -> ctypes.CDLL:
    """The HIP library with the layers' entry points declared."""
    global _lib, _native
    if _lib is None:
        L = _experts_lib()
        names = []
        i64, vp, sz, i32, f64 = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int,
                                 ctypes.c_double)
        for name, res, args in (
            ("layers_embed", i32, [vp, i64, vp, i32, i64, i64, f64, vp, i64, vp]),
            ("layers_embed_backward_workspace_bytes", sz, [i64] * 3 + [i32]),
            ("layers_embed_backward", i32,
             [vp, i64, vp, i64, i32, i64, i64, f64, vp, vp, sz, vp]),
            ("layers_norm", i32,
             [vp, i64, vp, vp, i32, i32, i64, i64, f64, vp, i64, vp, vp, vp]),
            ("layers_norm_backward_workspace_bytes", sz, [i64] * 2 + [i32]),
            ("layers_norm_backward", i32,
             [vp, i64, vp, i64, vp, vp, vp, i32, i32, i64, i64, vp, i64, vp, vp, vp, sz, vp]),
            ("layers_route", i32,
             [vp, i64, i32, i64, i64, i64, i32, vp, i64, i64, i64, i32, f64, vp, vp, vp]),
            ("layers_route_backward", i32,
             [vp, vp, i64, vp, i32, i64, i64, i64, i32, i32, f64, vp, i64, vp]),
            ("layers_cross_entropy_workspace_bytes", sz, [i64] * 3 + [i32] * 2),
            ("layers_cross_entropy", i32, [vp, i64, vp, vp, i32, i64, i64, i64, vp, vp, vp, sz, vp]),
            ("layers_cross_entropy_backward_workspace_bytes", sz, [i64] * 3 + [i32] * 2),
            ("layers_cross_entropy_backward", i32,
             [vp, vp, vp, i64, vp, vp, vp, i32, i64, i64, i64, vp, i64, vp, vp, sz, vp]),
        ):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
            names.append(name)
        _native = _load_native(L, names, "_layers_torch")
        _lib = L
    return _lib


def _module():
    lib()
    return _native


# As in ``experts``, a call with fresh outputs on the current stream is first offered to the
# native module, which takes it or, where anything about it is unusual, leaves it to the
# Python below.


def _numbers(t, name, count, dev=None):
    """Pointer of a dense vector of int64 numbers (of `count` of them, and on dev)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor, got {t.device}")
    if t.dtype != torch.int64 or t.dim() != 1 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int64 vector, got {t.dtype} {tuple(t.shape)}")
    if count is not None and t.shape[0] != count:
        raise ValueError(f"{name} must have {count} numbers, got {t.shape[0]}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    return t.data_ptr() or None


def _table(w, dtype, dev):
    """(pointer, classes, width) of a dense table."""
    if not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor")
    if w.dim() != 2:
        raise ValueError(f"w must be (classes, width), got shape {tuple(w.shape)}")
    return _dense(w, dtype, w.shape, dev, "w"), w.shape[0], w.shape[1]


def _score_code(score):
    code = SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be one of {', '.join(SCORES)}, got {score!r}")
    return code


def _misplaced(px, ldx, pw, width):
    """Whether x or w misses the 4-byte boundaries that 16-bit rows are read on."""
    return ((px or 0) | (pw or 0)) % 4 != 0 or (ldx | width) % 2 != 0


# ------------------------------------------------------------------- embed


def embed(ids, w, scale=1.0, out=None, stream=None):
    """scale * w[ids] for int64 numbers ids (tokens,) and a table w (classes, width):
    (tokens, width). Numbers outside [0, classes) give zero rows."""
    if out is None and stream is None:
        got = (_native or _module()).embed(ids, w, scale)
        if got is not None:
            return got
    _module().unrecorded("embed", w)
    return _embed(ids, w, scale, out, stream)


@_on_device
def _embed(ids, w, scale, out, stream):
    pi = _numbers(ids, "ids", None)
    dev, code = _first(w, "w", 2)
    pw, classes, width = _table(w, w.dtype, dev)
    if ids.get_device() != dev:
        raise ValueError(f"ids must be on cuda:{dev}, got {ids.device}")
    tokens = ids.shape[0]
    queue, side = _queue(stream, dev)
    if out is None:
        out = _new(w, side, (tokens, width))
        po, ldo = out.data_ptr() or None, width
    else:
        po, ldo = _given(out, w.dtype, tokens, width, dev)
    _check(lib().layers_embed(pi, tokens, pw, code, classes, width, scale, po, ldo, queue),
           "layers_embed")
    if side is not None:
        _mark(stream, dev, ids, w, out)
    return out


def embed_backward(dy, ids, classes, scale=1.0, workspace=None, stream=None):
    """Gradient of embed's table (classes, width), in dy's type: scale times the sum of each
    number's rows of dy (tokens, width)."""
    if workspace is None and stream is None:
        got = (_native or _module()).embed_backward(dy, ids, classes, scale)
        if got is not None:
            return got
    return _embed_backward(dy, ids, classes, scale, workspace, stream)


@_on_device
def _embed_backward(dy, ids, classes, scale, workspace, stream):
    dev, code = _first(dy, "dy", 2)
    tokens, width = dy.shape
    pg, ldg = _rows(dy, dy.dtype, tokens, width, dev, "dy")
    pi = _numbers(ids, "ids", tokens, dev)
    queue, side = _queue(stream, dev)
    L = lib()
    nbytes = L.layers_embed_backward_workspace_bytes(tokens, classes, width, code)
    workspace, ps, ns = _scratch(workspace, nbytes, dy, side)
    dw = _new(dy, side, (classes, width)) if nbytes else None  # (a table that is supported)
    _check(L.layers_embed_backward(pg, ldg, pi, tokens, code, classes, width, scale,
                                   None if dw is None else dw.data_ptr() or None, ps, ns, queue),
           "layers_embed_backward")
    if side is not None:
        _mark(stream, dev, dy, ids, dw, workspace)
    return dw


# -------------------------------------------------------------- layer norm


def _norm_weights(dtype, weight, bias, width, dev):
    """(pointer of weight, of bias, their dtype and its code)."""
    kind = next((t.dtype for t in (weight, bias) if isinstance(t, torch.Tensor)), dtype)
    if kind not in (dtype, torch.float32):
        raise TypeError(f"weight and bias must be {dtype} or torch.float32, got {kind}")
    return (None if weight is None else _dense(weight, kind, (width,), dev, "weight"),
            None if bias is None else _dense(bias, kind, (width,), dev, "bias"), kind,
            {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[kind])


def layer_norm(x, weight=None, bias=None, eps=1e-5, save_stats=False, out=None, stream=None):
    """(x - mean) * rstd * weight + bias for the rows of x (rows, width), with
    rstd = 1 / sqrt(variance + eps); weight and bias (width,), of x's type or float32.
    With ``save_stats`` returns (out, mean, rstd), the latter (rows,) float32 for
    layer_norm_backward."""
    if out is None and stream is None:
        got = (_native or _module()).layer_norm(x, weight, bias, eps, save_stats)
        if got is not None:
            return got
    _module().unrecorded("layer_norm", x, weight, bias)
    return _layer_norm(x, weight, bias, eps, save_stats, out, stream)


@_on_device
def _layer_norm(x, weight, bias, eps, save_stats, out, stream):
    dev, code = _first(x, "x", 2)
    rows, width = x.shape
    px, ldx = _rows(x, x.dtype, rows, width, dev, "x")
    pw, pb, _, wcode = _norm_weights(x.dtype, weight, bias, width, dev)
    queue, side = _queue(stream, dev)
    if out is None:
        out = _new(x, side, (rows, width))
        po, ldo = out.data_ptr() or None, width
    else:
        po, ldo = _given(out, x.dtype, rows, width, dev)
    mean = rstd = pm = ps = None
    if save_stats:
        mean, rstd = (_new(x, side, rows, torch.float32) for _ in range(2))
        pm, ps = mean.data_ptr() or None, rstd.data_ptr() or None
    _check(lib().layers_norm(px, ldx, pw, pb, code, wcode, rows, width, eps, po, ldo, pm, ps, queue),
           "layers_norm")
    if side is not None:
        _mark(stream, dev, x, weight, bias, out, mean, rstd)
    return (out, mean, rstd) if save_stats else out


def layer_norm_backward(dy, x, weight, mean, rstd, need_dx=True, need_dweight=True, need_dbias=True,
                        workspace=None, stream=None):
    """Gradients of layer_norm: (dx, dweight, dbias), None for those not needed; dweight and
    dbias of weight's type (x's without a weight)."""
    if workspace is None and stream is None:
        got = (_native or _module()).layer_norm_backward(dy, x, weight, mean, rstd, need_dx, need_dweight,
                                                         need_dbias)
        if got is not None:
            return got
    return _layer_norm_backward(dy, x, weight, mean, rstd, need_dx, need_dweight, need_dbias, workspace,
                                stream)


@_on_device
def _layer_norm_backward(dy, x, weight, mean, rstd, need_dx, need_dweight, need_dbias, workspace, stream):
    dev, code = _first(dy, "dy", 2)
    rows, width = dy.shape
    pg, ldg = _rows(dy, dy.dtype, rows, width, dev, "dy")
    px, ldx = _rows(x, dy.dtype, rows, width, dev, "x")
    pw, _, kind, wcode = _norm_weights(dy.dtype, weight, None, width, dev)
    pm = _dense(mean, torch.float32, (rows,), dev, "mean")
    ps = _dense(rstd, torch.float32, (rows,), dev, "rstd")
    queue, side = _queue(stream, dev)
    dx = _new(dy, side, (rows, width)) if need_dx else None
    dweight = _new(dy, side, width, kind) if need_dweight else None
    dbias = _new(dy, side, width, kind) if need_dbias else None
    if need_dweight or need_dbias or (need_dx and rows > 0):
        L = lib()
        nbytes = L.layers_norm_backward_workspace_bytes(rows, width, code) \
            if need_dweight or need_dbias else 0
        workspace, pk, nk = _scratch(workspace, nbytes, dy, side)
        _check(L.layers_norm_backward(
            pg, ldg, px, ldx, pw, pm, ps, code, wcode, rows, width,
            (dx.data_ptr() or None) if need_dx else None, width,
            (dweight.data_ptr() or None) if need_dweight else None,
            (dbias.data_ptr() or None) if need_dbias else None, pk, nk, queue), "layers_norm_backward")
    if side is not None:
        _mark(stream, dev, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace)
    return dx, dweight, dbias


# ------------------------------------------------------------------- route


def route(logits, top, score="softmax", bias=None, groups=1, top_groups=None, group_best=1,
          renormalize=True, scale=1.0, stream=None):
    """The experts of each token and their weights: (ids (tokens, top) int64 for
    ``experts.plan``, weights (tokens, top) float32 for ``experts.combine``).

    logits (tokens, experts); a logit of -inf takes an expert out. The ``top`` experts with
    the largest score + bias are chosen, the largest first and ties to the lower number;
    score: "softmax" over the experts or "sigmoid"; bias (experts,) float32 counts in the
    choice alone. With ``groups`` equal runs of experts, only those of the
    ``top_groups`` groups with the largest sums of their ``group_best`` (1 or 2) largest
    score + bias. Weights are the scores, divided by their sum over the chosen with
    ``renormalize``, times ``scale``. Places for which no expert is left: id -1, weight 0 (all
    places of a softmax row with a NaN or +inf, where the choice needs more than the logits)."""
    if top_groups is None:
        top_groups = groups
    if stream is None:
        got = (_native or _module()).route(logits, top, SCORES.get(score, -1), bias, groups, top_groups,
                                           group_best, renormalize, scale)
        if got is not None:
            return got
    _module().unrecorded("route", logits)
    return _route(logits, top, score, bias, groups, top_groups, group_best, renormalize, scale, stream)


@_on_device
def _route(logits, top, score, bias, groups, top_groups, group_best, renormalize, scale, stream):
    dev, code = _first(logits, "logits", 2)
    tokens, experts = logits.shape
    pl, ld = _rows(logits, logits.dtype, tokens, experts, dev, "logits")
    pb = None if bias is None else _dense(bias, torch.float32, (experts,), dev, "bias")
    kind = _score_code(score)
    queue, side = _queue(stream, dev)
    shape = (tokens, top if 1 <= top <= experts else 0)  # (no other is taken)
    ids, weights = _new(logits, side, shape, torch.int64), _new(logits, side, shape, torch.float32)
    _check(lib().layers_route(pl, ld, code, tokens, experts, top, kind, pb, groups, top_groups, group_best,
                              bool(renormalize), scale, ids.data_ptr() or None,
                              weights.data_ptr() or None, queue), "layers_route")
    if side is not None:
        _mark(stream, dev, logits, bias, ids, weights)
    return ids, weights


def route_backward(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0, stream=None):
    """Gradient of route's weights with respect to the logits, the choice fixed:
    (tokens, experts) in the logits' type, for dweights (tokens, top) float32 and the ids
    that route gave."""
    if stream is None:
        got = (_native or _module()).route_backward(dweights, logits, ids, SCORES.get(score, -1), renormalize,
                                                    scale)
        if got is not None:
            return got
    return _route_backward(dweights, logits, ids, score, renormalize, scale, stream)


@_on_device
def _route_backward(dweights, logits, ids, score, renormalize, scale, stream):
    dev, code = _first(logits, "logits", 2)
    tokens, experts = logits.shape
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be (tokens, top)")
    top = ids.shape[1]
    pl, ld = _rows(logits, logits.dtype, tokens, experts, dev, "logits")
    pi = _dense(ids, torch.int64, (tokens, top), dev, "ids")
    pg = _dense(dweights, torch.float32, (tokens, top), dev, "dweights")
    kind = _score_code(score)
    queue, side = _queue(stream, dev)
    out = _new(logits, side, (tokens, experts))
    _check(lib().layers_route_backward(pg, pl, ld, pi, code, tokens, experts, top, kind,
                                       bool(renormalize), scale, out.data_ptr() or None, experts, queue),
           "layers_route_backward")
    if side is not None:
        _mark(stream, dev, dweights, logits, ids, out)
    return out


# ----------------------------------------------------------- cross entropy


def cross_entropy(x, w, targets, workspace=None, stream=None):
    """Softmax cross entropy of the logits x w^T, which are not kept: (loss, lse), both
    (rows,) float32, for x (rows, width), w (classes, width) and int64 targets (rows,).
    loss = lse - logit of the target, lse the log of the sum of e^logits. A target outside
    [0, classes) is ignored: its loss is 0."""
    if workspace is None and stream is None:
        got = (_native or _module()).cross_entropy(x, w, targets)
        if got is not None:
            return got
    _module().unrecorded("cross_entropy", x, w)
    return _cross_entropy(x, w, targets, workspace, stream)


@_on_device
def _cross_entropy(x, w, targets, workspace, stream):
    dev, code = _first(x, "x", 2)
    pw, classes, width = _table(w, x.dtype, dev)
    rows = x.shape[0]
    px, ldx = _rows(x, x.dtype, rows, width, dev, "x")
    pt = _numbers(targets, "targets", rows, dev)
    queue, side = _queue(stream, dev)
    L = lib()
    nbytes = L.layers_cross_entropy_workspace_bytes(rows, classes, width, code,
                                                    _misplaced(px, ldx, pw, width))
    workspace, ps, ns = _scratch(workspace, nbytes, x, side)
    loss, lse = (_new(x, side, rows, torch.float32) for _ in range(2))
    _check(L.layers_cross_entropy(px, ldx, pw, pt, code, rows, classes, width, loss.data_ptr() or None,
                                  lse.data_ptr() or None, ps, ns, queue), "layers_cross_entropy")
    if side is not None:
        _mark(stream, dev, x, w, targets, loss, lse, workspace)
    return loss, lse


def cross_entropy_backward(dloss, x, w, targets, lse, dlse=None, need_dx=True, need_dw=True,
                           workspace=None, stream=None):
    """Gradients of cross_entropy: (dx, dw), None for the one not needed, for dloss
    (rows,) float32 (1 / count for a mean) and, where lse is part of the loss too, dlse
    (rows,) float32. lse is what cross_entropy gave. The logits are computed again, in pieces of
    the classes."""
    if workspace is None and stream is None:
        got = (_native or _module()).cross_entropy_backward(dloss, x, w, targets, lse, dlse, need_dx, need_dw)
        if got is not None:
            return got
    return _cross_entropy_backward(dloss, x, w, targets, lse, dlse, need_dx, need_dw, workspace, stream)


@_on_device
def _cross_entropy_backward(dloss, x, w, targets, lse, dlse, need_dx, need_dw, workspace, stream):
    dev, code = _first(x, "x", 2)
    pw, classes, width = _table(w, x.dtype, dev)
    rows = x.shape[0]
    px, ldx = _rows(x, x.dtype, rows, width, dev, "x")
    pt = _numbers(targets, "targets", rows, dev)
    pg = _dense(dloss, torch.float32, (rows,), dev, "dloss")
    ps = _dense(lse, torch.float32, (rows,), dev, "lse")
    pd = None if dlse is None else _dense(dlse, torch.float32, (rows,), dev, "dlse")
    queue, side = _queue(stream, dev)
    dx = _new(x, side, (rows, width)) if need_dx else None
    dw = _new(w, side, (classes, width)) if need_dw else None
    if need_dw or (need_dx and rows > 0):
        L = lib()
        nbytes = L.layers_cross_entropy_backward_workspace_bytes(rows, classes, width, code,
                                                                 _misplaced(px, ldx, pw, width))
        workspace, pk, nk = _scratch(workspace, nbytes, x, side)
        _check(L.layers_cross_entropy_backward(
            pg, pd, px, ldx, pw, pt, ps, code, rows, classes, width,
            (dx.data_ptr() or None) if need_dx else None, width,
            (dw.data_ptr() or None) if need_dw else None, pk, nk, queue),
            "layers_cross_entropy_backward")
    if side is not None:
        _mark(stream, dev, dloss, dlse, x, w, targets, lse, dx, dw, workspace)
    return dx, dw
