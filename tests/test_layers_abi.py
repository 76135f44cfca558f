"""The layers' part of the C ABI: it exports what include/layers_mi355x.h declares and
rejects invalid arguments on the host (no GPU: every call here fails validation before a
kernel launch, or has nothing to launch)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "layers_mi355x.h")

OK, NULL, SHAPE, ALIGN, WORKSPACE, ALIAS, HIP, OP = 0, -1, -2, -3, -4, -5, -6, -7
F32, BF16, F16 = 0, 1, 2

# Fake, far-apart device addresses: validation never dereferences them. Only where
# no GPU is present, so that a call let through could never reach a device.
no_gpu = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                            reason="fake-pointer validation tests run only without a GPU")
GIB = 1 << 30
A, B, C, D, E, F, G, H, I = (GIB * (16 << i) for i in range(9))


@pytest.fixture(scope="module")
def layers():
    pytest.importorskip("torch")
    from nearest_centroid_assignment_amd import layers as module

    return module


@pytest.fixture(scope="module")
def lib(layers):
    return layers.lib()


def test_exports_every_declared_symbol(lib):
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(layers_\w+)\s*\(", text))
    assert names == {
        "layers_embed", "layers_embed_backward_workspace_bytes", "layers_embed_backward", "layers_norm",
        "layers_norm_backward_workspace_bytes", "layers_norm_backward", "layers_route", "layers_route_backward",
        "layers_cross_entropy_workspace_bytes", "layers_cross_entropy",
        "layers_cross_entropy_backward_workspace_bytes", "layers_cross_entropy_backward"}
    for name in names:
        assert hasattr(lib, name), name


def test_python_refuses_without_a_gpu_tensor(layers):
    import torch

    x, ids = torch.zeros(4, 4), torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    for call in (lambda: layers.embed(ids, x), lambda: layers.embed_backward(x, ids, 4),
                 lambda: layers.layer_norm(x), lambda: layers.layer_norm_backward(x, x, None, f, f),
                 lambda: layers.route(x, 2), lambda: layers.route_backward(x, x, ids[:, None]),
                 lambda: layers.cross_entropy(x, x, ids), lambda: layers.cross_entropy_backward(f, x, x, ids, f)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError):
        layers.embed([1], x)
    with pytest.raises(TypeError):
        layers.layer_norm([1.0])


def test_workspace_bytes(lib):
    embed, norm = lib.layers_embed_backward_workspace_bytes, lib.layers_norm_backward_workspace_bytes
    fwd, bwd = lib.layers_cross_entropy_workspace_bytes, lib.layers_cross_entropy_backward_workspace_bytes
    assert embed(-1, 4, 4, F32) == 0 and embed(4, 0, 4, F32) == 0 and embed(4, 4, 0, F32) == 0
    assert embed(4, 4, 4, 3) == 0 and embed(4, 2 ** 20 + 1, 4, F32) == 0 and embed(2 ** 26, 4, 4, F32) == 0
    assert embed(2 ** 24, 50000, 2 ** 20, BF16) == 0  # more blocks than one dispatch has
    # Parts of 64 places or fewer: two float32 rows for each.
    for tokens, classes, width in ((65536, 50000, 2048), (300000, 1000, 64), (100, 5, 24)):
        assert embed(tokens, classes, width, BF16) <= (tokens // 16 + 1) * 8 * width + 24 * tokens + 8 * classes \
            + 4 * (tokens // 1024 + 1) * 2048 + 8192
    assert embed(0, 5, 8, F32) > 0
    assert norm(-1, 4, F32) == 0 and norm(4, 0, F32) == 0 and norm(2 ** 24, 4, F32) == 0 and norm(4, 4, 5) == 0
    assert 0 < norm(1 << 20, 2048, BF16) <= 512 * 2 * 2048 * 4 + 512 and norm(0, 4, F32) > 0
    for q in (fwd, bwd):
        assert q(-1, 4, 4, F32, 0) == 0 and q(4, 0, 4, F32, 0) == 0 and q(4, 4, 0, F32, 0) == 0
        assert q(4, 4, 4, 3, 0) == 0 and q(4, 2 ** 20 + 1, 4, F32, 0) == 0 and q(2 ** 31, 4, 4, F32, 0) == 0
        assert q(0, 4, 4, F32, 0) > 0
        # Padded copies of x and w, for odd 16-bit rows alone.
        even, odd = q(8192, 65536, 2048, BF16, 0), q(8192, 65536, 2048, BF16, 1)
        assert 2 * 2048 * (8192 + 65536) <= odd - even <= 2 * 2048 * (8192 + 65536) + 4096
        assert odd - 2 ** 16 <= q(8192, 65536, 2047, BF16, 0) <= odd and q(8192, 65536, 2047, F32, 0) == q(8192, 65536, 2047, F32, 1)
    # The logits would take 1 GiB in 16 bits; the forward call keeps 1/64 of that.
    assert fwd(8192, 65536, 2048, BF16, 0) <= 2 ** 24 + 2 ** 16
    # The gradient: half a GiB of dz, dx in float32 between pieces.
    assert bwd(8192, 65536, 2048, BF16, 0) <= 2 ** 29 + 4 * 8192 * 2048 + 4096
    assert bwd(1 << 20, 65536, 64, BF16, 0) <= 2 ** 29 + 4 * 64 * (1 << 20) * 9


@no_gpu
def test_embed_validation(lib):
    def fwd(ids=A, tokens=10, w=B, dtype=BF16, classes=7, width=16, scale=1.0, out=C, ldo=16):
        return lib.layers_embed(ids, tokens, w, dtype, classes, width, scale, out, ldo, None)

    assert fwd(ids=None) == NULL and fwd(w=None) == NULL and fwd(out=None) == NULL
    assert fwd(dtype=3) == OP and fwd(ldo=15) == SHAPE and fwd(classes=0) == SHAPE and fwd(width=0) == SHAPE
    assert fwd(tokens=-1) == SHAPE and fwd(tokens=2 ** 26) == SHAPE and fwd(classes=2 ** 20 + 1) == SHAPE
    assert fwd(ids=A + 4) == ALIGN and fwd(w=B + 1) == ALIGN and fwd(out=C + 1) == ALIGN
    assert fwd(out=A) == ALIAS and fwd(out=B + 200) == ALIAS
    assert fwd(tokens=0, ids=None, w=None, out=None) == OK

    def back(dy=A, lddy=16, ids=B, tokens=10, dtype=F16, classes=7, width=16, dw=C, ws=D, wsb=1 << 20):
        return lib.layers_embed_backward(dy, lddy, ids, tokens, dtype, classes, width, 1.0, dw, ws, wsb, None)

    assert back(dy=None) == NULL and back(ids=None) == NULL and back(dw=None) == NULL
    assert back(dtype=-1) == OP and back(lddy=15) == SHAPE and back(classes=0) == SHAPE
    assert back(ids=B + 4) == ALIGN and back(dw=C + 1) == ALIGN and back(dy=A + 1) == ALIGN
    assert back(ws=None) == WORKSPACE and back(wsb=300) == WORKSPACE
    assert back(dw=A + 32) == ALIAS and back(ws=B) == ALIAS and back(ws=C) == ALIAS


@no_gpu
def test_norm_validation(lib):
    def fwd(x=A, ldx=16, w=B, b=C, dtype=BF16, kind=BF16, rows=10, width=16, eps=1e-5, out=D, ldo=16, mean=E, rstd=F):
        return lib.layers_norm(x, ldx, w, b, dtype, kind, rows, width, eps, out, ldo, mean, rstd, None)

    assert fwd(x=None) == NULL and fwd(out=None) == NULL and fwd(mean=None) == NULL and fwd(rstd=None) == NULL
    assert fwd(dtype=3) == OP and fwd(kind=F16) == OP and fwd(dtype=F32, kind=BF16) == OP
    assert fwd(eps=-1e-9) == OP and fwd(eps=float("nan")) == OP
    assert fwd(ldx=15) == SHAPE and fwd(ldo=15) == SHAPE and fwd(width=0) == SHAPE and fwd(rows=-1) == SHAPE
    assert fwd(rows=2 ** 24) == SHAPE and fwd(width=2 ** 20 + 1, ldx=2 ** 21, ldo=2 ** 21) == SHAPE
    assert fwd(x=A + 1) == ALIGN and fwd(w=B + 1) == ALIGN and fwd(kind=F32, b=C + 2) == ALIGN
    assert fwd(mean=E + 2) == ALIGN
    assert fwd(out=A) == ALIAS and fwd(out=B) == ALIAS and fwd(rstd=E) == ALIAS and fwd(mean=C) == ALIAS
    assert fwd(rows=0, x=None, out=None) == OK

    def back(dy=A, lddy=16, x=B, ldx=16, w=C, mean=D, rstd=E, dtype=F16, kind=F32, rows=10, width=16, dx=F, lddx=16,
             dw=G, db=H, ws=I, wsb=1 << 20):
        return lib.layers_norm_backward(dy, lddy, x, ldx, w, mean, rstd, dtype, kind, rows, width, dx, lddx, dw, db,
                                        ws, wsb, None)

    assert back(dx=None, dw=None, db=None) == NULL and back(dy=None) == NULL and back(x=None) == NULL
    assert back(mean=None) == NULL and back(rstd=None) == NULL
    assert back(kind=BF16) == OP and back(dtype=9) == OP and back(lddx=15) == SHAPE and back(lddy=15) == SHAPE
    assert back(dx=F + 1) == ALIGN and back(dw=G + 2) == ALIGN and back(rstd=E + 1) == ALIGN
    assert back(ws=None) == WORKSPACE and back(wsb=100) == WORKSPACE
    assert back(dx=A) == ALIAS and back(dw=C) == ALIAS and back(db=G) == ALIAS and back(ws=B) == ALIAS
    assert back(dw=None, db=None, dx=A, ws=None, wsb=0) == ALIAS  # no sums: no workspace
    assert back(rows=0, dw=None, db=None, ws=None, wsb=0) == OK


@no_gpu
def test_route_validation(lib):
    def fwd(z=A, ld=64, dtype=BF16, tokens=10, n=64, top=2, score=0, bias=B, groups=8, kept=4, best=2, norm=1, ids=C,
            w=D):
        return lib.layers_route(z, ld, dtype, tokens, n, top, score, bias, groups, kept, best, norm, 1.0, ids, w, None)

    assert fwd(z=None) == NULL and fwd(ids=None) == NULL and fwd(w=None) == NULL
    assert fwd(dtype=3) == OP and fwd(score=2) == OP and fwd(best=0) == OP and fwd(best=3) == OP
    assert fwd(ld=63) == SHAPE and fwd(top=0) == SHAPE and fwd(top=65) == SHAPE and fwd(n=1, ld=1, groups=1, kept=1) == SHAPE
    assert fwd(groups=7) == SHAPE and fwd(kept=0) == SHAPE and fwd(kept=9) == SHAPE and fwd(groups=0) == SHAPE
    assert fwd(n=2049, ld=2049, groups=1, kept=1) == SHAPE  # more than the lanes hold
    assert fwd(n=2046, ld=2046, groups=33, kept=1) == SHAPE and fwd(n=130, ld=130, groups=65, kept=1) == SHAPE
    assert fwd(tokens=-1) == SHAPE and fwd(tokens=2 ** 26) == SHAPE
    assert fwd(z=A + 1) == ALIGN and fwd(bias=B + 2) == ALIGN and fwd(ids=C + 4) == ALIGN and fwd(w=D + 1) == ALIGN
    assert fwd(ids=A) == ALIAS and fwd(w=B) == ALIAS and fwd(w=C + 16) == ALIAS
    assert fwd(tokens=0, z=None, ids=None, w=None) == OK

    def back(g=A, z=B, ld=64, ids=C, dtype=F32, tokens=10, n=64, top=2, score=1, dz=D, lddz=64):
        return lib.layers_route_backward(g, z, ld, ids, dtype, tokens, n, top, score, 1, 1.0, dz, lddz, None)

    assert back(g=None) == NULL and back(z=None) == NULL and back(ids=None) == NULL and back(dz=None) == NULL
    assert back(score=-1) == OP and back(dtype=4) == OP and back(lddz=63) == SHAPE and back(top=65) == SHAPE
    assert back(ids=C + 4) == ALIGN and back(dz=D + 2) == ALIGN and back(g=A + 1) == ALIGN
    assert back(dz=A) == ALIAS and back(dz=B) == ALIAS and back(dz=C) == ALIAS and back(tokens=0, z=None) == OK


@no_gpu
def test_cross_entropy_validation(lib):
    def fwd(x=A, ldx=16, w=B, t=C, dtype=BF16, rows=100, classes=24, width=16, loss=D, lse=E, ws=F, wsb=1 << 20):
        return lib.layers_cross_entropy(x, ldx, w, t, dtype, rows, classes, width, loss, lse, ws, wsb, None)

    assert fwd(x=None) == NULL and fwd(w=None) == NULL and fwd(t=None) == NULL
    assert fwd(loss=None) == NULL and fwd(lse=None) == NULL
    assert fwd(dtype=3) == OP and fwd(rows=-1) == SHAPE and fwd(classes=0) == SHAPE and fwd(width=0) == SHAPE
    assert fwd(ldx=15) == SHAPE and fwd(ldx=2 ** 20 + 2) == SHAPE and fwd(classes=2 ** 20 + 1) == SHAPE
    assert fwd(x=A + 1) == ALIGN and fwd(t=C + 4) == ALIGN and fwd(loss=D + 2) == ALIGN
    assert fwd(ws=None) == WORKSPACE and fwd(wsb=1000) == WORKSPACE
    assert fwd(ldx=17, wsb=5000) == WORKSPACE  # rows off 4 bytes need room for their padded copies
    assert fwd(loss=A) == ALIAS and fwd(lse=D) == ALIAS and fwd(ws=B) == ALIAS and fwd(lse=C + 8) == ALIAS
    assert fwd(rows=0, x=None, t=None, loss=None) == OK

    def back(g=A, gl=B, x=C, ldx=16, w=D, t=E, lse=F, dtype=F16, rows=100, classes=24, width=16, dx=G, lddx=16, dw=H,
             ws=I, wsb=1 << 20):
        return lib.layers_cross_entropy_backward(g, gl, x, ldx, w, t, lse, dtype, rows, classes, width, dx, lddx, dw,
                                                 ws, wsb, None)

    assert back(dx=None, dw=None) == NULL and back(g=None) == NULL and back(x=None) == NULL and back(w=None) == NULL
    assert back(t=None) == NULL and back(lse=None) == NULL
    assert back(dtype=-1) == OP and back(lddx=15) == SHAPE and back(ldx=15) == SHAPE and back(width=0) == SHAPE
    assert back(g=A + 2) == ALIGN and back(gl=B + 1) == ALIGN and back(dw=H + 1) == ALIGN
    assert back(ws=None) == WORKSPACE and back(wsb=1000) == WORKSPACE
    assert back(dx=C) == ALIAS and back(dw=D) == ALIAS and back(dw=G) == ALIAS and back(ws=A) == ALIAS
    assert back(dx=B) == ALIAS and back(dx=F) == ALIAS
    assert back(rows=0, dw=None, g=None, x=None) == OK
