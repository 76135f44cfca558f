"""The experts' host side at its edges: what is validated, allocated and built
(no GPU: every call here fails validation before a kernel launch, or has nothing to
launch, or is let through where there is no device)."""
import ctypes
import os
import types

import pytest

from nearest_centroid_assignment_amd import build
from tests.test_experts_abi import (A, ALIAS, B, BF16, C, D, E, F, F16, F32, G, H, HIP, NULL, OK, SHAPE,  # noqa: F401
                                    experts, lib, no_gpu)


@no_gpu
def test_adamw_tensors_overlap(lib):
    """No tensor that is written may be given twice, or overlap any other tensor of
    the call; gradients may be shared."""
    def step(p, g, c=None, pt=F32, gt=F32, n=256, m=G, v=H):
        ptrs = lambda t: (ctypes.c_void_p * len(t))(*t)  # noqa: E731
        lengths = (ctypes.c_int64 * len(p))(*[n] * len(p))
        return lib.experts_adamw_step(ptrs(p), ptrs(g), ptrs(c) if c else None, lengths, len(p), pt, gt, m, v, None,
                                      None, 32, 1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, None)

    assert step((A, B), (C, D)) == HIP and step((A, B), (C, C)) == HIP  # let through: no device
    assert step((A, A + 1024), (C, D)) == HIP and step((A, A + 1020), (C, D)) == ALIAS
    assert step((A, A), (C, D)) == ALIAS  # tied weights
    assert step((A, B), (C, A)) == ALIAS and step((A, B), (B + 512, D)) == ALIAS
    assert step((A, B), (C, D), (E, E)) == ALIAS and step((A, B), (C, D), (E, A)) == ALIAS
    assert step((A, B), (C, D), (E, C)) == ALIAS
    assert step((A, B), (C, D), (A, B), pt=BF16) == HIP  # its own copy
    assert step((A, B), (C, D), (B, A), pt=BF16) == ALIAS
    assert step((A, G + 512), (C, D)) == ALIAS and step((A, B), (C, H + 4)) == ALIAS
    many = [A + 1024 * i for i in range(100)]
    grads = [C + 1024 * (i // 2) for i in range(100)]
    assert step(many, grads) == HIP
    assert step(many[::-1] + [many[7]], grads + [D]) == ALIAS and step(many, [*grads[:-1], many[0] + 4]) == ALIAS


def test_workspace_of_another_device(experts):
    """A workspace on another GPU than the call's is refused."""
    import torch

    from nearest_centroid_assignment_amd import binding

    class Bytes(torch.Tensor):
        device = property(lambda self: torch.device("cuda", 1))

    ws = torch.zeros(1000, dtype=torch.uint8).as_subclass(Bytes)
    like = types.SimpleNamespace(device=torch.device("cuda", 0))
    with pytest.raises(ValueError, match="cuda:0"):
        experts._scratch(ws, 300, like, None)
    with pytest.raises(ValueError, match="cuda:0"):
        binding._workspace(ws, 300, like.device)
    assert experts._scratch(ws, 300, types.SimpleNamespace(device=ws.device), None)[2] == 1000


@no_gpu
def test_columns_of_one_buffer(lib):
    """Column ranges of the same rows overlap only where they share a column."""
    def fwd(x, out, ld=40, ldo=40, rows=100, outs=16, ins=16):
        return lib.experts_linear(x, ld, C, None, None, 0, None, F32, 0, rows, outs, ins, 1, out, ldo, None, 0, G,
                                  1 << 24, None)

    for x, out, want in ((A, A + 64, HIP), (A + 64, A, HIP), (A, A + 96, HIP), (A + 96, A, HIP), (A, A + 160 + 64, HIP),
                         (A, A + 60, ALIAS), (A + 60, A, ALIAS), (A, A, ALIAS), (A, A + 100, ALIAS), (A + 100, A, ALIAS),
                         (A, A + 160 * 99 + 60, ALIAS), (A, A + 160 * 99 + 64, HIP)):
        assert fwd(x, out) == want, (x - A, out - A)
    assert fwd(A, A + 64, ldo=44) == ALIAS and fwd(A, A + 64, rows=1) == HIP and fwd(A, A + 60, rows=1) == ALIAS


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_state_types(experts, bits):
    """The moments are float32 whatever the process's default type is."""
    import torch

    kept = torch.get_default_dtype()
    try:
        torch.set_default_dtype(torch.float64)
        state = experts.adamw_state([torch.zeros(300), torch.zeros(5)], bits)
    finally:
        torch.set_default_dtype(kept)
    floats = ("m", "v") if bits == 32 else ("m_scale", "v_scale")
    assert all(state[k].dtype == torch.float32 and not state[k].any() for k in floats)
    assert state["m"].numel() == state["v"].numel() == 512 + 256


def test_workspace_of_few_rows(lib):
    """The kernel for few rows reads odd 16-bit rows in place: no room for copies."""
    for rows, outs, ins, n in ((1, 8192, 2047, 1), (16, 4096, 2047, 1), (3, 500, 777, 2)):
        for unaligned in (0, 1):
            assert lib.experts_linear_workspace_bytes(rows, outs, ins, n, BF16, 0, unaligned) == 256
    # Others still have it, and so have the gradients of few rows.
    assert lib.experts_linear_workspace_bytes(1000, 8192, 2047, 1, BF16, 0, 0) >= 2 * 2048 * 9192
    assert lib.experts_linear_workspace_bytes(1, 8192, 2047, 1, BF16, 1, 0) >= 2 * 2048 * 8193


@pytest.mark.parametrize("missing", ["compiler", "torch"])
def test_build_without_torch_module(missing, monkeypatch, tmp_path, capsys):
    """The libraries build where what only the torch module needs is missing; a
    module of another build does not stay."""
    import importlib.util

    old = tmp_path / "_experts_torch.so"
    old.write_text("")
    made = []
    monkeypatch.setattr(build, "TORCH_MODULE_PATH", str(old))
    monkeypatch.setattr(build, "_compile", lambda sources, path, *a: made.append(path) or path)
    monkeypatch.setattr(build, "_run", lambda *a, **k: pytest.fail("nothing is left to compile"))
    if missing == "compiler":
        exists = os.path.exists
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
        monkeypatch.setattr(build.os.path, "exists", lambda p: "clang" not in str(p) and exists(p))
    else:
        find = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == build.LIB_PATH
    monkeypatch.undo()
    assert made == [build.CALIB_PATH, build.LIB_PATH] and not old.exists()
    assert f"{missing} not found" in capsys.readouterr().err


def test_torch_module_compiler(monkeypatch):
    """Without a system compiler the module is left to ROCm's."""
    found = {"amdclang++": build.hipcc()}
    monkeypatch.setattr(build.shutil, "which", found.get)
    assert build.cxx() == found["amdclang++"] and build.torch_module_needs() is None


@no_gpu
def test_limits(lib):
    """The largest sizes that the header names are let through, the next are not."""
    def dispatch(tokens, top=1):
        return lib.experts_dispatch(A, 1, BF16, tokens, top, 1, B, C, D, 1, None)

    def gather(tokens):
        return lib.experts_dispatch_backward(A, 1, BF16, tokens, 1, 1, C, D, 1, None)

    def combine(tokens):
        return lib.experts_combine(A, 1, B, BF16, tokens, 1, 1, C, D, 1, None)

    def back(tokens, top):
        return lib.experts_combine_backward(A, 1, B, 1, C, BF16, tokens, top, 1, D, E, F, 1, G, None)

    for call in (dispatch, gather, combine):
        assert call(2**24 - 1) == HIP and call(2**24) == SHAPE
    assert back(2**26 - 5, 1) == HIP and back(2**26 - 3, 1) == SHAPE and back(2**24, 4) == SHAPE
    linear = lib.experts_linear_workspace_bytes
    rows = (2**35 - 2**12) // 8192
    assert linear(rows - 1, 8192, 64, 1, BF16, 0, 0) > 0 and linear(rows + 1, 8192, 64, 1, BF16, 0, 0) == 0
