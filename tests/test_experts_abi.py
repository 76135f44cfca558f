"""The experts' part of the C ABI: it exports what include/experts_mi355x.h
declares and rejects invalid arguments on the host (no GPU: every call here fails
validation before a kernel launch, or has nothing to launch)."""
import ctypes
import os
import re

import pytest

from nearest_centroid_assignment_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "experts_mi355x.h")

OK, NULL, SHAPE, ALIGN, WORKSPACE, ALIAS, HIP, OP = 0, -1, -2, -3, -4, -5, -6, -7
F32, BF16, F16 = 0, 1, 2

# Fake, far-apart device addresses: validation never dereferences them. Only where
# no GPU is present, so that a call let through could never reach a device.
no_gpu = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                            reason="fake-pointer validation tests run only without a GPU")
GIB = 1 << 30
A, B, C, D, E, F, G, H = (GIB * (16 << i) for i in range(8))


@pytest.fixture(scope="module")
def experts():
    pytest.importorskip("torch")
    from nearest_centroid_assignment_amd import experts as module

    return module


@pytest.fixture(scope="module")
def lib(experts):
    return experts.lib()


def test_exports_every_declared_symbol(lib):
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(experts_\w+)\s*\(", text))
    assert names == {
        "experts_plan_workspace_bytes", "experts_plan", "experts_dispatch", "experts_dispatch_backward",
        "experts_combine", "experts_combine_backward", "experts_linear_workspace_bytes", "experts_linear",
        "experts_linear_backward", "experts_adamw_state_elements", "experts_adamw_step",
        "experts_adamw_moments"}
    for name in names:
        assert hasattr(lib, name), name


def test_native_module(experts, lib):
    """The torch module is built beside the library and leaves what is not a GPU
    tensor to Python, which words the refusal."""
    import torch

    assert os.path.dirname(experts._native.__file__) == os.path.dirname(build.LIB_PATH)
    x = torch.zeros(4, 4)
    assert experts._native.linear(x, x, None, None, 0, None, False) is None
    assert experts._native.plan(x, 3) is None and experts._native.plan(7, 3) is None
    assert experts._native.dispatch(x, (1, 2)) is None
    assert experts._native.adamw_step([], [], x, x, 0.1, 0.9, 0.9, 0.0, 0.0, 1, None, None, None, None) is None
    for call in (lambda: experts.linear(x, x), lambda: experts.plan(torch.zeros(3, dtype=torch.int64), 3)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError):
        experts.linear([1.0], x)
    with pytest.raises(TypeError):
        experts._native.bind(3)
    with pytest.raises(ValueError):
        experts._native.bind({})


def test_workspace_bytes(lib):
    plan, linear = lib.experts_plan_workspace_bytes, lib.experts_linear_workspace_bytes
    assert plan(-1, 1, 4) == 0 and plan(4, 0, 4) == 0 and plan(4, 65, 4) == 0 and plan(4, 1, 0) == 0
    assert plan(4, 1, 65537) == 0 and plan(2**31, 1, 4) == 0 and plan(2**26, 64, 4) == 0
    assert plan(8, 2, 64) == 256 and plan(0, 1, 4) == 256
    for tokens, top, n in ((65536, 2, 1024), (100000, 1, 17), (5000, 1, 20000)):
        tiles = -(-tokens * top // 1024)
        assert 4 * tiles * n + 2 * tokens * top <= plan(tokens, top, n) <= 4 * (tiles + 1) * n + 2 * tokens * top + 2048
    assert linear(10, 0, 8, 1, F32, 0, 0) == 0 and linear(10, 8, 8, 0, F32, 0, 0) == 0
    assert linear(10, 8, 8, 1, 3, 0, 0) == 0 and linear(10, 8, 8, 1, F32, 2, 0) == 0
    assert linear(10, 8, 2**20 + 1, 1, F32, 0, 0) == 0 and linear(2**31, 8, 8, 1, F32, 0, 0) == 0
    # A large forward product needs none; padded copies only for odd 16-bit rows.
    assert linear(8192, 8192, 2048, 1, BF16, 0, 0) == 256
    odd = linear(8192, 8192, 2047, 1, BF16, 0, 0)
    assert 2 * 2048 * 16384 <= odd <= 2 * 2048 * 16384 + 1024
    assert linear(8192, 8192, 2047, 1, F32, 0, 0) == 256
    assert linear(8192, 8192, 2048, 1, BF16, 0, 1) == odd
    # The gradient keeps dz, and never more than dz, copies and partial sums.
    assert linear(8192, 8192, 2048, 1, BF16, 1, 0) >= 2 * 8192 * 8192
    # Many rows of wide layers are one launch.
    assert linear(1 << 20, 8192, 8192, 1, BF16, 0, 0) > 0 and linear(1 << 20, 8192, 8192, 64, F16, 1, 0) > 0


@no_gpu
def test_plan_validation(lib):
    def call(ids=A, tokens=5000, top=2, n=10, order=B, place=C, offsets=D, ws=E, wsb=1 << 24):
        return lib.experts_plan(ids, tokens, top, n, order, place, offsets, ws, wsb, None)

    assert call(ids=None) == NULL and call(order=None) == NULL and call(place=None) == NULL
    assert call(offsets=None) == NULL
    assert call(tokens=-1) == SHAPE and call(top=0) == SHAPE and call(top=65) == SHAPE
    assert call(n=0) == SHAPE and call(n=65537) == SHAPE and call(tokens=2**31) == SHAPE
    assert call(ids=A + 4) == ALIGN and call(order=B + 2) == ALIGN and call(offsets=D + 1) == ALIGN
    assert call(ws=None) == WORKSPACE and call(wsb=100) == WORKSPACE
    assert call(order=A) == ALIAS and call(place=B + 4) == ALIAS and call(offsets=C) == ALIAS
    assert call(ws=A + 8) == ALIAS


@no_gpu
def test_rows_validation(lib):
    def dispatch(x=A, ldx=16, dtype=BF16, tokens=10, top=2, width=16, order=B, place=C, xs=D, ldxs=16):
        return lib.experts_dispatch(x, ldx, dtype, tokens, top, width, order, place, xs, ldxs, None)

    assert dispatch(x=None) == NULL and dispatch(order=None) == NULL and dispatch(xs=None) == NULL
    assert dispatch(dtype=3) == OP and dispatch(dtype=-1) == OP
    assert dispatch(ldx=15) == SHAPE and dispatch(ldxs=15) == SHAPE and dispatch(width=0) == SHAPE
    assert dispatch(tokens=2**24, top=1) == SHAPE  # one block of 256 threads a token
    assert dispatch(x=A + 1) == ALIGN and dispatch(place=C + 2) == ALIGN
    assert dispatch(xs=A + 8) == ALIAS and dispatch(xs=B) == ALIAS
    assert dispatch(tokens=0, x=None, xs=None) == OK

    def combine(ys=A, ldys=16, w=B, dtype=F32, tokens=10, top=2, width=16, place=C, y=D, ldy=16):
        return lib.experts_combine(ys, ldys, w, dtype, tokens, top, width, place, y, ldy, None)

    assert combine(ys=None) == NULL and combine(w=None) == NULL and combine(place=None) == NULL
    assert combine(ldy=3) == SHAPE and combine(w=B + 2) == ALIGN and combine(dtype=9) == OP
    assert combine(y=A) == ALIAS and combine(y=B) == ALIAS

    def scatter(g=A, ldg=16, dtype=F16, tokens=10, top=2, width=16, place=B, dx=C, lddx=16):
        return lib.experts_dispatch_backward(g, ldg, dtype, tokens, top, width, place, dx, lddx, None)

    assert scatter(g=None) == NULL and scatter(place=None) == NULL and scatter(dx=None) == NULL
    assert scatter(lddx=8) == SHAPE and scatter(dx=A + 2) == ALIAS and scatter(dx=C + 1) == ALIGN

    def back(dy=A, lddy=16, ys=B, ldys=16, w=C, dtype=BF16, tokens=10, top=2, width=16, order=D, place=E, dys=F,
             lddys=16, dw=G):
        return lib.experts_combine_backward(dy, lddy, ys, ldys, w, dtype, tokens, top, width, order, place, dys,
                                            lddys, dw, None)

    assert back(dys=None, dw=None) == NULL and back(dy=None) == NULL and back(ys=None) == NULL
    assert back(w=None) == NULL and back(order=None) == NULL
    assert back(dw=G + 2) == ALIGN and back(lddys=15) == SHAPE and back(ldys=1) == SHAPE
    assert back(dys=B) == ALIAS and back(dw=F) == ALIAS and back(dtype=5) == OP


@no_gpu
def test_linear_validation(lib):
    def fwd(x=A, ldx=16, w=B, bias=C, res=D, ldr=24, off=None, dtype=BF16, act=1, rows=100, outs=24, ins=16, n=1,
            out=E, ldo=24, pre=F, ldpre=24, ws=G, wsb=1 << 24):
        return lib.experts_linear(x, ldx, w, bias, res, ldr, off, dtype, act, rows, outs, ins, n, out, ldo, pre,
                                  ldpre, ws, wsb, None)

    assert fwd(x=None) == NULL and fwd(w=None) == NULL and fwd(out=None) == NULL
    assert fwd(dtype=4) == OP and fwd(act=4) == OP and fwd(act=-1) == OP
    assert fwd(rows=-1) == SHAPE and fwd(outs=0) == SHAPE and fwd(ins=0) == SHAPE and fwd(n=2) == SHAPE
    assert fwd(ldx=15) == SHAPE and fwd(ldo=23) == SHAPE and fwd(ldr=1) == SHAPE and fwd(ldpre=1) == SHAPE
    assert fwd(ldx=2**20 + 2) == SHAPE
    assert fwd(x=A + 1) == ALIGN and fwd(bias=C + 1) == ALIGN and fwd(off=H + 2, n=3) == ALIGN
    assert fwd(out=A) == ALIAS and fwd(out=D) == ALIAS and fwd(pre=E) == ALIAS and fwd(ws=B) == ALIAS
    # Rows off 4 bytes need room for their padded copies.
    assert fwd(ldx=17, wsb=300) == WORKSPACE and fwd(ldx=17, ws=None, wsb=0) == WORKSPACE
    assert fwd(rows=0, x=None, out=None) == OK

    def back(dy=A, lddy=24, x=B, ldx=16, w=C, pre=D, ldpre=24, ip=None, ldin=16, off=None, dtype=BF16, act=1, ia=0,
             rows=100, outs=24, ins=16, n=1, dx=E, lddx=16, dw=F, db=G, ws=H, wsb=1 << 24):
        return lib.experts_linear_backward(dy, lddy, x, ldx, w, pre, ldpre, ip, ldin, off, dtype, act, ia, rows, outs,
                                           ins, n, dx, lddx, dw, db, ws, wsb, None)

    assert back(dx=None, dw=None, db=None) == NULL and back(dy=None) == NULL and back(pre=None) == NULL
    assert back(x=None) == NULL and back(w=None) == NULL
    assert back(ia=7) == OP and back(lddx=3) == SHAPE and back(lddy=3) == SHAPE and back(n=3) == SHAPE
    assert back(ip=A + 1) == ALIGN and back(dw=F + 1) == ALIGN
    assert back(wsb=1000) == WORKSPACE
    assert back(dx=A) == ALIAS and back(dw=B) == ALIAS and back(db=F) == ALIAS and back(dx=D) == ALIAS


@no_gpu
def test_adamw_validation(lib):
    def ptrs(*p):
        return (ctypes.c_void_p * len(p))(*p)

    lengths = (ctypes.c_int64 * 2)(1000, 24)
    assert lib.experts_adamw_state_elements(lengths, 2) == 1024 + 256
    assert lib.experts_adamw_state_elements((ctypes.c_int64 * 1)(-1), 1) == -1
    assert lib.experts_adamw_state_elements(None, 2) == -1 and lib.experts_adamw_state_elements(None, 0) == 0

    def step(p=(A, B), g=(C, D), c=None, n=lengths, count=2, pt=F32, gt=BF16, m=E, v=F, ms=None, vs=None, bits=32,
             lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, t=1, gs=None):
        return lib.experts_adamw_step(ptrs(*p), ptrs(*g), ptrs(*c) if c else None, n, count, pt, gt, m, v, ms, vs, bits,
                                      lr, b1, b2, eps, wd, t, gs, None)

    nan = float("nan")
    for bad in (dict(lr=-1.0), dict(lr=nan), dict(b1=1.0), dict(b2=-0.1), dict(b1=nan), dict(eps=-1.0), dict(wd=nan),
                dict(t=0), dict(bits=16), dict(pt=3), dict(gt=-1)):
        assert step(**bad) == OP, bad
    assert step(p=(A, None)) == NULL and step(g=(None, D)) == NULL and step(m=None) == NULL
    assert step(bits=8) == NULL and step(c=(G, None)) == NULL
    assert step(n=(ctypes.c_int64 * 2)(5, -3)) == SHAPE
    assert step(p=(A + 2, B)) == ALIGN and step(g=(C, D + 1)) == ALIGN and step(m=E + 2) == ALIGN
    assert step(gs=H + 1) == ALIGN
    assert step(g=(A, D)) == ALIAS and step(m=C + 4) == ALIAS and step(v=E + 1024) == ALIAS
    assert step(p=(E, B)) == ALIAS and step(c=(A, G)) == ALIAS
    assert step(count=0) == OK and step(n=(ctypes.c_int64 * 2)(0, 0), p=(None, None), g=(None, None)) == OK

    def moments(m=A, v=B, ms=C, vs=D, n=512, mo=E, vo=F):
        return lib.experts_adamw_moments(m, v, ms, vs, n, mo, vo, None)

    assert moments(n=100) == SHAPE and moments(n=-256) == SHAPE and moments(mo=None, vo=None) == NULL
    assert moments(m=None) == NULL and moments(vs=None) == NULL and moments(mo=E + 1) == ALIGN
    assert moments(vo=E) == ALIAS and moments(mo=A) == ALIAS and moments(n=0) == OK
