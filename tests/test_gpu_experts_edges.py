"""The expert operators at their edges: errors of a launch, extreme values, sizes
between the ways that a call can be taken, and memory that is shared or viewed."""
import ctypes
import importlib.util
import os
import shutil

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from nearest_centroid_assignment_amd import binding, build, experts  # noqa: E402
from tests import gpu_util as gu  # noqa: E402
from tests.test_gpu_experts import (TYPES, close, encode, f64, make_ids, np32, randn,  # noqa: E402
                                    summed)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ------------------------------------------------------------- failed launches


def test_error_of_another_call():
    """An error that some other call of the process has left behind is not this
    step's: the step is applied, once."""
    L = experts.lib()
    ways = []
    for stale in (False, True):
        p, g = [randn(i, 3000) for i in range(70)], [randn(100 + i, 3000) for i in range(70)]
        state = experts.adamw_state(p)
        torch.cuda.synchronize()
        if stale:
            assert L.hipSetDevice(1 << 20) != 0
        try:
            experts.adamw_step(p, g, lr=0.1, **state)
        finally:
            L.hipGetLastError()
        ways.append(p + list(state.values()))
    for a, b in zip(*ways):
        assert torch.equal(a, b)


NATIVE = ("plan", "dispatch", "dispatch_backward", "combine", "combine_backward", "linear",
          "linear_backward", "adamw_step")


def native_copy(tmp_path, stubs):
    """A second copy of the native module, some of whose entry points are `stubs`."""
    path = shutil.copy(build.TORCH_MODULE_PATH, os.path.join(tmp_path, "_experts_torch.so"))
    spec = importlib.util.spec_from_file_location("_experts_torch", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    L = experts.lib()
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    names = [f"experts_{n}" for n in NATIVE] + [f"experts_{n}" for n in (
        "plan_workspace_bytes", "linear_workspace_bytes", "adamw_state_elements")]
    module.bind({n: address(stubs.get(n, getattr(L, n))) for n in names}, binding._check)
    return module


def ordinary_calls():
    ids, x = make_ids(1, 10, 2, 3).cuda(), randn(1, 10, 16)
    p = experts.plan(ids, 3)
    xs, w, weights = randn(2, 20, 16), randn(3, 24, 16), randn(4, 10, 2)
    q, g = [randn(5, 300)], [randn(6, 300)]
    s = experts.adamw_state(q)
    return dict(plan=(ids, 3), dispatch=(x, p), dispatch_backward=(xs, p), combine=(xs, weights, p),
                combine_backward=(x, xs, weights, p), linear=(xs, w, None, None, 0, None, False),
                linear_backward=(randn(7, 20, 24), xs, w, None, 0, None, None, 0, True, True, True),
                adamw_step=(q, g, s["m"], s["v"], 0.1, 0.9, 0.99, 1e-8, 0.0, 1, None, None, None, None))


@pytest.mark.parametrize("name", NATIVE)
def test_failed_launch_is_not_repeated(name, tmp_path):
    """A status that a launch may have preceded raises; one that validation gives
    leaves the call to Python."""
    counted, status = [], 0

    def entry():
        counted.append(name)
        return status

    stub = ctypes.CFUNCTYPE(ctypes.c_int)(entry)
    native, args = native_copy(tmp_path, {f"experts_{name}": stub}), ordinary_calls()[name]
    status = -2  # KM_ERR_SHAPE
    assert getattr(native, name)(*args) is None and len(counted) == 1
    status = -6  # KM_ERR_HIP
    with pytest.raises(binding.KMeansError) as e:
        getattr(native, name)(*args)
    assert e.value.status == -6 and len(counted) == 2


def test_incomplete_bind(tmp_path):
    """A bind that is refused leaves the entry points as they were."""
    native = native_copy(tmp_path, {})
    with pytest.raises(ValueError):
        native.bind({})
    ids = make_ids(1, 10, 2, 3).cuda()
    for a, b in zip(native.plan(ids, 3), experts.plan(ids, 3)):
        assert torch.equal(a, b)


# -------------------------------------------------------------- extreme values


def test_adamw_8_bit_scales():
    """Codes of blocks whose scales lie at either end of float32's range: those of
    the float32 formulas. With beta = 0 a block's moments are g and g^2."""
    sizes = [1e38, 3.2e38, 8.6e37, 8.4e37, 1.1e37, 9e36, 1.8e19, 1.2e19, 3.1e18, 1.0, 1e-15, 1e-16, 2e-19,
             0.9e-30, 1e-31, 1e-37, 1e-40, 0.0]
    rng = np.random.default_rng(5)
    g = (rng.uniform(-1, 1, (len(sizes), 256)) * np.array(sizes)[:, None]).astype(np.float32).reshape(-1)
    p = [torch.zeros(g.size, device="cuda")]
    state = experts.adamw_state(p, 8)
    experts.adamw_step(p, [torch.from_numpy(g).cuda()], lr=1e-3, betas=(0.0, 0.0), **state)
    with np.errstate(over="ignore", under="ignore"):
        mq, vq, ms, vs = encode(g, g * g)
    finite = np.isfinite(vs)
    vq = np.where(finite[:, None], vq.reshape(-1, 256), 0).reshape(-1)  # a NaN scale has codes 0
    assert finite.sum() == len(sizes) - 6
    assert np.array_equal(np32(state["m_scale"]), ms)
    assert np.array_equal(np32(state["v_scale"])[finite], vs[finite])
    assert np.isnan(np32(state["v_scale"])[~finite]).all()
    for name, want in (("m", mq), ("v", vq)):
        got = state[name].cpu().numpy()
        for i, size in enumerate(sizes):
            assert np.array_equal(got[256 * i:256 * i + 256], want[256 * i:256 * i + 256]), f"{name}, size {size}"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
@pytest.mark.parametrize("rows", [1, 130, 700])
def test_slope_far_from_zero(dtype, act, rows):
    """Far from zero the slopes are 1 and 0, also where z^2 leaves the range and,
    for a pre that was stored as an infinity, there."""
    n = 264
    far = [200.0, 65504.0, float("inf")] + ([] if dtype == torch.float16 else [1e13, 5e18, 2e19, 7e19, 1e25, 3.3e38])
    far = torch.tensor(far + [-v for v in far]).to(dtype).cuda()
    z = far[torch.arange(rows * n, device="cuda") % far.numel()].reshape(rows, n)
    dy = randn(1, rows, n, dtype=dtype)
    eye = torch.eye(n, device="cuda").to(dtype)
    want = torch.where(z > 0, dy, torch.zeros_like(dy))
    dx, dw, db = experts.linear_backward(dy, eye[:1].expand(rows, n).contiguous(), eye, pre=z, act=act)
    assert torch.equal(dx, want)
    close(db, f64(want).sum(0), summed(rows) * f64(want).abs().sum(0), "dbias")
    close(dw[:, 0], f64(want).sum(0), summed(rows) * f64(want).abs().sum(0), "dw")
    assert not dw[:, 1:].any()
    dx = experts.linear_backward(dy, dy, eye, in_pre=z, in_act=act, need_dw=False, need_dbias=False)[0]
    assert torch.equal(dx, want)
    z[0, 0] = float("nan")
    assert torch.isnan(experts.linear_backward(dy, dy, eye, pre=z, act=act)[0][0, 0])


# ------------------------------------------------------------- memory and views


def test_workspace_refusals():
    """A workspace that is a strided view would be written between its elements."""
    ids = torch.zeros(5000, 2, dtype=torch.int64, device="cuda")
    x, w = randn(1, 64, 4096), randn(2, 64, 4096)
    assert experts.lib().experts_linear_workspace_bytes(64, 64, 4096, 1, 0, 0, 0) > 256
    room = torch.full((1 << 24, 2), 7, dtype=torch.uint8, device="cuda")
    for bad in (room[:, 0], room.cpu()[:, 0].contiguous(), room[:, 0].contiguous().to(torch.int8), 5):
        with pytest.raises((TypeError, ValueError)):
            experts.plan(ids, 3, workspace=bad)
        with pytest.raises((TypeError, ValueError)):
            experts.linear(x, w, workspace=bad)
        with pytest.raises((TypeError, ValueError)):
            experts.linear_backward(randn(3, 64, 64), x, w, workspace=bad)
    with pytest.raises((TypeError, ValueError)):
        binding.kmeans_assign(x, w, torch.empty(64, dtype=torch.int64, device="cuda"), workspace=room[:, 0])
    assert bool((room == 7).all())
    flat = room.reshape(-1)
    assert torch.equal(experts.linear(x, w, workspace=flat), experts.linear(x, w))


def test_versions():
    """What a call writes in place counts as modified: autograd notices that a
    tensor it saved has changed."""
    side = torch.cuda.Stream()
    for bits, stream in ((32, None), (8, None), (32, side)):
        p = [torch.nn.Parameter(randn(i, 300)) for i in range(2)]
        g = [randn(9, 300) for _ in p]
        copies, state = [torch.zeros(300, dtype=torch.bfloat16, device="cuda") for _ in p], experts.adamw_state(p, bits)
        written, read = [*p, *copies, *state.values()], [*g]
        before = [t._version for t in written + read]
        loss = (p[0] * p[0]).sum()
        torch.cuda.synchronize()
        experts.adamw_step(p, g, lr=0.1, copies=copies, stream=stream, **state)
        torch.cuda.synchronize()
        after = [t._version for t in written + read]
        assert all(b > a for a, b in zip(before, after[:len(written)])) and after[len(written):] == before[len(written):]
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    plan = experts.plan(make_ids(1, 10, 2, 3).cuda(), 3)
    xs, y, z = torch.empty(20, 16, device="cuda"), torch.empty(10, 16, device="cuda"), torch.empty(20, 24, device="cuda")
    x, w, weights = randn(1, 10, 16), randn(2, 24, 16), randn(3, 10, 2)
    for out, call in ((xs, lambda: experts.dispatch(x, plan, out=xs)), (y, lambda: experts.combine(xs, weights, plan, out=y)),
                      (y, lambda: experts.dispatch_backward(xs, plan, out=y)), (z, lambda: experts.linear(xs, w, out=z))):
        before = out._version
        assert call() is out and out._version > before
    with torch.inference_mode():
        p = [randn(1, 300)]
        state = experts.adamw_state(p)
    experts.adamw_step(p, [randn(2, 300)], lr=0.1, **state)
    assert not torch.equal(p[0], randn(1, 300))


def test_lost_gradients_are_said():
    """The operators record no graph. An input that asks for one is answered, with
    a warning; without gradients being recorded there is none."""
    import warnings

    plan = experts.plan(make_ids(1, 10, 2, 3).cuda(), 3)
    x, xs, w, weights = randn(1, 10, 16), randn(2, 20, 16), randn(3, 24, 16), randn(4, 10, 2)
    bias, res = randn(5, 24), randn(6, 20, 24)
    calls = [(x, lambda **k: experts.dispatch(x, plan, **k)), (xs, lambda **k: experts.combine(xs, weights, plan, **k)),
             (weights, lambda **k: experts.combine(xs, weights, plan, **k))]
    calls += [(t, lambda **k: experts.linear(xs, w, bias, residual=res, **k)) for t in (xs, w, bias, res)]
    for t, call in calls:
        for stream in (None, torch.cuda.current_stream()):
            with warnings.catch_warnings():
                warnings.simplefilter("error")
                want = call(stream=stream)
                t.requires_grad_(True)
                with torch.no_grad():
                    call(stream=stream)
            with pytest.warns(UserWarning, match="explicit calls"):
                got = call(stream=stream)
            assert torch.equal(got, want) and not got.requires_grad
            t.requires_grad_(False)


@pytest.mark.parametrize("dtype", TYPES)
def test_halves_of_one_buffer(dtype):
    """An input and an output that are column ranges of the same rows do not overlap."""
    rows, k = 150, 70
    buf, w = randn(1, rows, 2 * k + 2, dtype=dtype), randn(2, k, k, dtype=dtype, scale=0.1)
    lo, hi = buf[:, :k], buf[:, k + 1:2 * k + 1]
    want = experts.linear(lo.contiguous(), w, residual=lo.contiguous(), act="silu")
    edge = buf[:, [k, 2 * k + 1]].clone()
    experts.linear(lo, w, residual=lo, act="silu", out=hi)
    assert torch.equal(hi, want) and torch.equal(buf[:, [k, 2 * k + 1]], edge)
    plan = experts.plan(make_ids(1, rows, 1, 5).cuda(), 5)
    experts.dispatch(hi, plan, out=lo)
    assert torch.equal(lo, experts.dispatch(want, plan))
    weights = randn(3, rows, 1)
    experts.combine(lo, weights, plan, out=hi)
    assert torch.equal(hi, experts.combine(lo.contiguous(), weights, plan))
    for bad in (buf[:, k - 1:2 * k - 1], buf[:, :k]):
        with pytest.raises(binding.KMeansError):
            experts.linear(lo, w, out=bad)


# ------------------------------------------- between the ways a call can be taken


@pytest.mark.parametrize("tokens,top,n,drop", [
    (64, 1, 65536, 0.1), (4096, 1, 1024, 0.1), (512, 8, 1024, 0), (4096, 1, 1025, 0), (131072, 1, 7, 0.1),
    (131073, 1, 7, 0.1), (70000, 2, 1024, 0.05), (65536, 2, 4096, 0.05), (32768, 4, 4097, 0.05), (65536, 8, 33, 0.1),
    (300000, 1, 5000, 0.02)])
def test_plan_between_sorts(tokens, top, n, drop):
    """Sizes that each way to sort takes, and the largest counts in LDS, against a stable sort."""
    gu.announce(f"plan {tokens} x {top}, {n} experts, drop {drop}")
    for lopsided in (False, True):
        ids = make_ids(tokens + n, tokens, top, n, drop, lopsided)
        p = experts.plan(ids.cuda(), n)
        flat = ids.reshape(-1)
        key = torch.where((flat >= 0) & (flat < n), flat, n)
        live = int((key < n).sum())
        order = key.sort(stable=True)[1].to(torch.int32)
        order[live:] = -1
        place = torch.full((tokens * top,), -1, dtype=torch.int32)
        place[order[:live].long()] = torch.arange(live, dtype=torch.int32)
        offsets = torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(key, minlength=n + 1)[:n].cumsum(0)])
        assert torch.equal(p.order.cpu(), order)
        assert torch.equal(p.place.cpu().reshape(-1), place)
        assert torch.equal(p.offsets.cpu().long(), offsets)


@pytest.mark.parametrize("dtype,tokens,width", [(torch.bfloat16, 40000, 2048), (torch.float16, 9000, 8192),
                                                (torch.float32, 20000, 2048)])
def test_rows_past_the_cache(dtype, tokens, width):
    """Row sets of more than 256 MB in whole lines, which pass the caches by: every
    row's outputs at sampled tokens in float64, and the places without a pair."""
    top, n = 2, 65
    gu.announce(f"rows past the cache: {dtype} {tokens} x {top} x {width}")
    ids = make_ids(3, tokens, top, n, 0.1)
    p = experts.plan(ids.cuda(), n)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, dy, ys = (torch.randn(rows, width, generator=gen, device="cuda").to(dtype)
                 for rows in (tokens, tokens, tokens * top))
    weights = randn(4, tokens, top)
    live = int(p.offsets[-1])
    ys[live:] = float("nan")
    xs, y = experts.dispatch(x, p), experts.combine(ys, weights, p)
    dx = experts.dispatch_backward(ys, p)
    dys, dweights = experts.combine_backward(dy, ys, weights, p)
    assert not xs[live:].any() and not dys[live:].any()
    assert torch.equal(xs[:live], x[p.order[:live].long() // top])
    for t in [0, 1, tokens - 1, *np.random.default_rng(1).integers(0, tokens, 200).tolist()]:
        places = p.place[t].tolist()
        g, total, plain = f64(dy[t]), torch.zeros(width, dtype=torch.float64), torch.zeros(width, dtype=torch.float64)
        size, plain_size = total.clone(), total.clone()
        for s, at in enumerate(places):
            if at < 0:
                assert float(dweights[t, s]) == 0
                continue
            row, w = f64(ys[at]), float(weights[t, s])
            total, size = total + w * row, size + abs(w) * row.abs()
            plain, plain_size = plain + row, plain_size + row.abs()
            close(dys[at], w * g, 2.0 ** -24 * (w * g).abs(), f"dys of {t}")
            close(dweights[t, s], (g * row).sum(), summed(width) * (g * row).abs().sum(), f"dweights of {t}")
        close(y[t], total, summed(top) * size, f"y of {t}")
        close(dx[t], plain, summed(top) * plain_size, f"dx of {t}")


@pytest.mark.parametrize("tokens,top,n", [
    (2048, 1, 33), (2049, 1, 33), (1024, 2, 2048), (1025, 2, 2048), (163840, 1, 1024), (163841, 1, 1024),
    (262144, 1, 300), (262145, 1, 300), (40960, 1, 2048), (40961, 1, 2048), (1100, 2, 2049)])
def test_plan_at_thresholds(tokens, top, n):
    """As above, at the sizes where the way to sort changes."""
    test_plan_between_sorts(tokens, top, n, 0.1)


@pytest.mark.parametrize("dtype,width", [(torch.float16, 1536), (torch.float16, 1537), (torch.float32, 768)])
@pytest.mark.parametrize("tokens", [1023, 1024, 2047, 2048])
def test_rows_at_thresholds(dtype, width, tokens):
    """Rows on both sides of where a wave or a block takes one, by length and number."""
    top, n = 2, 9
    p = experts.plan(make_ids(tokens, tokens, top, n, 0.1).cuda(), n)
    x, dy, ys = (randn(s, r, width, dtype=dtype) for s, r in ((1, tokens), (2, tokens), (3, tokens * top)))
    weights, live = randn(4, tokens, top), int(p.offsets[-1])
    ys[live:] = float("nan")
    at = p.place.long()
    rows = torch.where((at >= 0)[:, :, None], ys[at.clamp(min=0)].float(), 0.0)
    w = torch.where(at >= 0, weights, 0.0)
    token = p.order[:live].long() // top
    xs = experts.dispatch(x, p)
    assert torch.equal(xs[:live], x[token]) and not xs[live:].any()
    size = f64(rows).abs()
    w = f64(w)[:, :, None]
    close(experts.combine(ys, weights, p), (f64(rows) * w).sum(1), summed(top) * (size * w.abs()).sum(1), "y")
    close(experts.dispatch_backward(ys, p), f64(rows).sum(1), summed(top) * size.sum(1), "dx")
    dys, dweights = experts.combine_backward(dy, ys, weights, p)
    want = f64(dy)[token.cpu()] * f64(weights).reshape(-1)[p.order[:live].long().cpu()][:, None]
    close(dys[:live], want, 2.0 ** -24 * want.abs(), "dys")
    terms = f64(rows) * f64(dy)[:, None]
    close(dweights, terms.sum(2), summed(width) * terms.abs().sum(2), "dweights")
    assert not dys[live:].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,outs,ins", [(5, 72, 40), (70, 16, 24), (3, 264, 1100)])
def test_offsets_of_no_plan(dtype, n, outs, ins):
    """Offsets that are out of order, negative or past the rows: nothing is written
    outside the outputs, and the gradients of w read nothing around the inputs (NaN).
    Rows of out that no expert has are left to chance."""
    gu.announce(f"offsets of no plan: {dtype} {n} experts {outs} x {ins}")
    rows, rng = 300, np.random.default_rng(n)
    for kind in range(3):
        offsets = rng.integers(-50, rows + 50, n + 1) if kind else np.arange(n + 1) % 2 * rows
        if kind == 2:
            offsets = np.where(rng.random(n + 1) < 0.5, 2**31 - 1, -2**31)
        offsets = torch.from_numpy(offsets).to(torch.int32).cuda()
        # A guard of a row and more on every side of x, dy and out.
        full = [torch.full((rows + 4, k + 6), float("nan"), dtype=dtype, device="cuda") for k in (ins, outs, outs)]
        x, dy, out = (t[2:-2, 2:2 + k] for t, k in zip(full, (ins, outs, outs)))
        x.copy_(randn(1, rows, ins)), dy.copy_(randn(2, rows, outs)), out.zero_()
        w = randn(3, n, outs, ins, dtype=dtype, scale=0.1)
        experts.linear(x, w, offsets=offsets, act="silu", out=out)
        dw, db = experts.linear_backward(dy, x, w, offsets=offsets, need_dx=False)[1:]
        assert torch.isfinite(dw).all() and torch.isfinite(db).all()
        guard = torch.ones_like(full[2], dtype=torch.bool)
        guard[2:-2, 2:2 + outs] = False
        assert torch.isnan(full[2][guard]).all()


def test_more_tiles_than_an_int():
    """As above, where the tiles that the offsets describe pass 2^31."""
    rows, n, k = 1 << 23, 65536, 8
    offsets = (torch.arange(n + 1, device="cuda") % 2 * rows).to(torch.int32)
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(n, k, k, dtype=torch.bfloat16, device="cuda")
    assert (rows // 128) * (n // 2) >= 2**31  # (the tiles are of 64 to 256 rows)
    full = torch.full((rows + 1024, k), 7.0, dtype=torch.bfloat16, device="cuda")
    out = full[512:-512]
    gu.announce("more tiles than an int")
    experts.linear(x, w, offsets=offsets, out=out)
    assert bool((full[:512] == 7).all()) and bool((full[-512:] == 7).all())
    assert bool(((out == 0) | (out == 7)).all())
