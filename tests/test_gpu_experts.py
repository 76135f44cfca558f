"""The expert operators on the GPU against their formulas in float64 on the CPU.

Tolerances. With u the unit roundoff of the stored type (2^-24, 2^-8 for
bfloat16, 2^-11 for float16; and half its smallest subnormal step, which counts
only for float16), a value rounded once is off by at most u |value|. A float32 sum of n
products is off by (4 + 2 sqrt(n)) 2^-23 times the sum of their magnitudes: each
of its n roundings is at most 2^-24 of a partial sum, or twice that inside a
matrix instruction, and n independent ones add up like their square root; the
factor two is room. Activations and slopes are good to 2^-19 of their argument's
magnitude plus one, and no slope or second derivative exceeds 1.2.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from nearest_centroid_assignment_amd import binding, experts  # noqa: E402
from tests import gpu_util as gu  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def randn(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def f64(t):
    return t.detach().cpu().to(torch.float64)


def summed(n):
    return (4 + 2 * math.sqrt(n)) * 2.0 ** -23


def close(got, want, slack, what):
    """|got - want| <= slack + one rounding, elementwise (slack in float64)."""
    err = (f64(got) - want).abs()
    bound = slack + U[got.dtype] * (want.abs() + slack) + TINY[got.dtype]
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - bound)[bad].max())}"


def make_ids(seed, tokens, top, n, drop=0.0, lopsided=False):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, n, (tokens, top))
    if lopsided:
        ids[rng.random((tokens, top)) < 0.7] = n // 2
    out = rng.random((tokens, top))
    ids[out < drop] = -1
    ids[out > 1 - drop / 2] = n + 3
    return torch.from_numpy(ids).to(torch.int64)


def plan_ref(ids, n):
    flat = ids.reshape(-1).tolist()
    order = sorted((i for i, e in enumerate(flat) if 0 <= e < n), key=lambda i: (flat[i], i))
    place = [-1] * len(flat)
    for at, i in enumerate(order):
        place[i] = at
    offsets = [0] * (n + 1)
    for e in flat:
        if 0 <= e < n:
            offsets[e + 1] += 1
    for e in range(n):
        offsets[e + 1] += offsets[e]
    return order + [-1] * (len(flat) - len(order)), place, offsets


# ------------------------------------------------------------------ tokens


@pytest.mark.parametrize("tokens,top,n,drop", [
    (0, 2, 5, 0), (1, 1, 1, 0), (1, 8, 64, 0.2), (8, 2, 64, 0), (63, 1, 17, 0.3), (65, 3, 7, 0),
    (1024, 1, 300, 0.1), (1365, 3, 4096, 0), (2000, 2, 5, 0.1), (4096, 1, 4097, 0),
    (4097, 1, 33, 0), (5003, 3, 17, 0.1), (30000, 2, 1024, 0.05), (3000, 4, 20000, 0.05),
    (500, 2, 9, 2.0)])
def test_plan(tokens, top, n, drop):
    gu.announce(f"plan {tokens} x {top}, {n} experts, drop {drop}")
    for lopsided in (False, True):
        ids = make_ids(tokens + n, tokens, top, n, drop, lopsided)
        p = experts.plan(ids.cuda(), n)
        order, place, offsets = plan_ref(ids, n)
        assert p.order.cpu().tolist() == order
        assert p.place.cpu().reshape(-1).tolist() == place
        assert p.offsets.cpu().tolist() == offsets


def test_plan_of_labels():
    """The labels of the assignment are expert numbers; the offsets count them."""
    X, C = randn(1, 3000, 40), randn(2, 33, 40)
    labels, _ = binding.assign(X, C)
    p = experts.plan(labels, 33)
    assert torch.equal(p.offsets.long().diff(), torch.bincount(labels, minlength=33))
    assert torch.equal(labels[p.order.long()], labels.sort(stable=True)[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,top,n,width,drop", [
    (1, 1, 1, 1, 0), (1, 2, 4, 2048, 0), (8, 2, 64, 72, 0), (33, 3, 5, 7, 0.3), (100, 8, 17, 1001, 0.2),
    (130, 1, 3, 64, 0), (7, 2, 3, 5000, 0.2), (5000, 2, 9, 33, 0.2), (4100, 1, 300, 520, 0),
    (50, 2, 9, 24, 2.0)])
def test_rows(dtype, tokens, top, n, width, drop):
    """Dispatch, combine and their gradients; rows at places without a pair hold
    NaN in every input and must neither be read nor stay in an output."""
    gu.announce(f"rows {dtype} {tokens} x {top}, {n} experts, width {width}, drop {drop}")
    ids = make_ids(3 * tokens + width, tokens, top, n, drop)
    p = experts.plan(ids.cuda(), n)
    order, place, offsets = plan_ref(ids, n)
    live, pairs = offsets[-1], tokens * top
    x, dy = (randn(s, tokens, width, dtype=dtype) for s in (5, 6))
    ys, dxs = (randn(s, pairs, width, dtype=dtype) for s in (7, 8))
    ys[live:] = float("nan")
    dxs[live:] = float("nan")
    weights = randn(9, tokens, top)
    weights[torch.tensor(place).reshape(tokens, top) < 0] = float("nan")
    at = torch.tensor(order[:live], dtype=torch.long)
    token = at // top

    xs = experts.dispatch(x, p)
    assert xs.shape == (pairs, width)
    assert torch.equal(xs[:live].cpu(), x.cpu()[token]) and not xs[live:].any()

    w = f64(weights).reshape(-1)[at][:, None]
    zero = torch.zeros(tokens, width, dtype=torch.float64)
    y = experts.combine(ys, weights, p)
    terms = f64(ys[:live]) * w
    close(y, zero.index_add(0, token, terms), summed(top) * zero.index_add(0, token, terms.abs()), "y")

    dx = experts.dispatch_backward(dxs, p)
    terms = f64(dxs[:live])
    close(dx, zero.index_add(0, token, terms), summed(top) * zero.index_add(0, token, terms.abs()), "dx")

    dys, dweights = experts.combine_backward(dy, ys, weights, p)
    want = f64(dy)[token] * w
    close(dys[:live], want, 2.0 ** -24 * want.abs(), "dys")
    assert not dys[live:].any()
    terms = f64(dy)[token] * f64(ys[:live])
    full = torch.zeros(pairs, dtype=torch.float64)
    bound = full.clone()
    full[at], bound[at] = terms.sum(1), summed(width) * terms.abs().sum(1)
    close(dweights.reshape(-1), full, bound, "dweights")
    only, none = experts.combine_backward(dy, ys, weights, p, need_dweights=False)
    assert none is None and torch.equal(only, dys)
    none, only = experts.combine_backward(dy, ys, weights, p, need_dys=False)
    assert none is None and torch.equal(only, dweights)


def test_rows_strided():
    """Row strides, and rows that start on odd 2-byte addresses."""
    tokens, top, n, width = 90, 2, 7, 130
    p = experts.plan(make_ids(1, tokens, top, n).cuda(), n)
    wide = randn(1, tokens, width + 71, dtype=torch.bfloat16)
    x = wide[:, 3:3 + width]
    out = torch.full((tokens * top, width + 5), -7.0, dtype=torch.bfloat16, device="cuda")
    experts.dispatch(x, p, out=out[:, 1:1 + width])
    assert torch.equal(out[:, 1:1 + width], experts.dispatch(x.contiguous(), p))
    assert (out[:, 0] == -7).all() and (out[:, 1 + width:] == -7).all()
    weights = randn(2, tokens, top)
    y = torch.full((tokens, width + 9), -7.0, dtype=torch.bfloat16, device="cuda")
    experts.combine(out[:, 1:1 + width], weights, p, out=y[:, 9:])
    assert torch.equal(y[:, 9:], experts.combine(out[:, 1:1 + width].contiguous(), weights, p))
    assert (y[:, :9] == -7).all()


def test_rows_past_32_bits():
    """More than 2^31 elements: the last rows land where they belong."""
    tokens, top, width = 70000, 2, 16384
    gu.announce(f"rows {tokens} x {top} x {width}: {tokens * top * width / 2**31:.2f} x 2^31 elements")
    ids = torch.from_numpy(np.random.default_rng(0).integers(0, 5, (tokens, top))).cuda()
    p = experts.plan(ids, 5)
    x = torch.arange(tokens, device="cuda").remainder(2039).to(torch.bfloat16)[:, None].repeat(1, width)
    x[:, -1] = 3.0
    xs = experts.dispatch(x, p)
    token = p.order.long() // top
    assert torch.equal(xs[:, 0], x[token, 0]) and bool((xs[:, -1] == 3.0).all())
    assert torch.equal(xs[:, width // 2], x[token, width // 2])
    dx = experts.dispatch_backward(xs, p)
    assert bool((dx[:, -1] == 6.0).all()) and torch.equal(dx[:, 0], (2 * x[:, 0].float()).to(x.dtype))


# ------------------------------------------------------------------ linear


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    z = z.clone().requires_grad_(True)
    return torch.autograd.grad(act64(z, act).sum(), z)[0] if act != "none" else torch.ones_like(z)


def check_linear(dtype, rows, outs, ins, act, counts=None, residual=True, bias=True, seed=0, tail=0,
                 in_act=None):
    """Forward and backward against float64, per expert. Rows past the experts'
    hold NaN in every input."""
    n = rows if counts is None else sum(counts) + tail
    e = 1 if counts is None else len(counts)
    offsets = None if counts is None else torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32).cuda()
    lead = () if counts is None else (e,)
    x, w = randn(seed, n, ins, dtype=dtype), randn(seed + 1, *lead, outs, ins, dtype=dtype, scale=ins ** -0.5)
    b = randn(seed + 2, *lead, outs, dtype=dtype) if bias else None
    res = randn(seed + 3, n, outs, dtype=dtype) if residual else None
    dy = randn(seed + 4, n, outs, dtype=dtype)
    ip = randn(seed + 5, n, ins, dtype=dtype) if in_act else None
    live = n if counts is None else sum(counts)
    for t in (x, res, dy, ip):
        if t is not None:
            t[live:] = float("nan")
    out, pre = experts.linear(x, w, b, residual=res, act=act, offsets=offsets, save_pre=True)
    assert torch.equal(out, experts.linear(x, w, b, residual=res, act=act, offsets=offsets))
    dx, dw, db = experts.linear_backward(dy, x, w, pre=pre, act=act, offsets=offsets, in_pre=ip,
                                         in_act=in_act or "none")
    assert not out[live:].any() and not pre[live:].any() and not dx[live:].any()
    bounds = [0, n] if counts is None else [0] + list(np.cumsum(counts))
    for i in range(e):
        lo, hi = int(bounds[i]), int(bounds[i + 1])
        wi = f64(w if counts is None else w[i])
        xi, gi, pi = f64(x[lo:hi]), f64(dy[lo:hi]), f64(pre[lo:hi])
        z = xi @ wi.t()
        mag = xi.abs() @ wi.abs().t()
        if b is not None:
            bi = f64(b if counts is None else b[i])
            z, mag = z + bi, mag + bi.abs()
        zerr = summed(ins) * mag
        close(pre[lo:hi], z, zerr, f"pre of {i}")
        y, yerr = act64(z, act), 1.2 * zerr + (2.0 ** -19 * (1 + z.abs()) if act in ("silu", "gelu_tanh") else 0)
        if res is not None:
            y = y + f64(res[lo:hi])
            yerr = yerr + 2.0 ** -24 * y.abs()
        close(out[lo:hi], y, yerr, f"out of {i}")
        # From the stored pre, as linear_backward is given it.
        s = slope64(pi, act)
        dz = gi * s
        dzerr = gi.abs() * (2.0 ** -19 * (1 + pi.abs()) if act in ("silu", "gelu_tanh") else 0)
        close(db if counts is None else db[i], dz.sum(0), summed(hi - lo) * dz.abs().sum(0) + dzerr.sum(0), f"dbias of {i}")
        dzerr = dzerr + U[dtype] * dz.abs() + TINY[dtype]  # the products read dz rounded
        want, err = dz @ wi, summed(outs) * (dz.abs() @ wi.abs()) + dzerr @ wi.abs()
        if ip is not None:
            q = f64(ip[lo:hi])
            si = slope64(q, in_act)
            err = err * si.abs() + want.abs() * 2.0 ** -19 * (1 + q.abs())
            want = want * si
        close(dx[lo:hi], want, err, f"dx of {i}")
        close(dw if counts is None else dw[i], dz.t() @ xi,
              summed(hi - lo) * (dz.abs().t() @ xi.abs()) + dzerr.t() @ xi.abs(), f"dw of {i}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,outs,ins,act", [
    (1, 1, 1, "none"), (1, 8, 8, "relu"), (1, 200, 264, "gelu_tanh"), (2, 17, 33, "silu"), (15, 64, 128, "none"),
    (16, 100, 96, "gelu_tanh"), (17, 48, 1000, "silu"), (63, 65, 64, "relu"), (64, 64, 65, "none"),
    (65, 129, 127, "gelu_tanh"), (130, 257, 72, "silu"), (300, 31, 777, "relu"), (512, 520, 40, "gelu_tanh")])
def test_linear_dense(dtype, rows, outs, ins, act):
    gu.announce(f"linear {dtype} {rows} x {outs} x {ins} {act}")
    check_linear(dtype, rows, outs, ins, act)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,outs,ins,act,tail,in_act", [
    ([3], 8, 16, "none", 0, None), ([0, 0], 24, 8, "relu", 5, None), ([5, 0, 1, 70], 72, 136, "silu", 3, None),
    ([64, 64, 128], 64, 64, "none", 0, "silu"), ([1, 2, 3, 200, 0], 130, 33, "gelu_tanh", 9, None),
    ([100, 300, 17], 200, 129, "none", 40, "gelu_tanh"), ([1] * 70 + [0] * 5, 16, 24, "relu", 2, None)])
def test_linear_experts(dtype, counts, outs, ins, act, tail, in_act):
    gu.announce(f"linear experts {dtype} {counts[:6]} x {outs} x {ins} {act}")
    check_linear(dtype, 0, outs, ins, act, counts=counts, tail=tail, in_act=in_act)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,outs,ins,counts", [
    (2000, 2100, 136, None), (3400, 3608, 72, None), (200, 3600, 3400, None), (0, 1032, 520, [700, 0, 1300, 431]),
    (0, 3336, 3272, [100, 0, 260])])
def test_linear_large_tiles(dtype, rows, outs, ins, counts):
    """Sizes that the larger tiles take, each with partial tiles on every edge."""
    gu.announce(f"linear {dtype} {rows} x {outs} x {ins} {counts}")
    check_linear(dtype, rows, outs, ins, "gelu_tanh", counts=counts, tail=0 if counts is None else 21, residual=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,outs,ins,counts", [
    (200, 72, 1100, None), (100, 1096, 72, None), (140, 90, 1602, None), (600, 302, 1026, None), (258, 642, 2046, None), (1300, 40, 56, None), (90, 700, 2050, None),
    (0, 72, 1096, [100, 0, 700, 33]), (0, 1048, 136, [65, 0, 130]), (0, 33, 40, [1500, 3, 900])])
def test_linear_split_depth(dtype, rows, outs, ins, counts):
    """Few tiles with a long depth, in each direction: the depth is split."""
    gu.announce(f"linear split {dtype} {rows} x {outs} x {ins} {counts}")
    check_linear(dtype, rows, outs, ins, "silu", counts=counts, tail=0 if counts is None else 13,
                 in_act="silu")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,outs,ins,counts", [
    (1, 33, 4099, None), (16, 520, 2048, None), (30, 17, 1500, None), (64, 40, 4104, None), (33, 72, 31, None),
    (0, 136, 1032, [1, 0, 16, 17, 3]), (0, 24, 2056, [30, 0, 50, 2]), (0, 50, 777, [64, 70, 3, 0])])
def test_linear_few_rows(dtype, rows, outs, ins, counts):
    """Few rows an expert: the depth is split over a block's waves."""
    gu.announce(f"linear few rows {dtype} {rows} x {outs} x {ins} {counts}")
    check_linear(dtype, rows, outs, ins, "gelu_tanh", counts=counts, tail=0 if counts is None else 5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,outs,ins,counts", [
    (200, 72, 1100, None), (2000, 2100, 136, None), (258, 642, 2046, None), (1300, 40, 56, None), (269, 67, 1959, None),
    (700, 1000, 333, None), (65, 1030, 2000, None), (0, 72, 1096, [100, 0, 700, 33]), (0, 1048, 136, [65, 0, 130]),
    (0, 333, 520, [200, 700, 0, 120, 1]), (0, 130, 1954, [100, 400, 0, 900, 600, 15, 700, 300])])
def test_linear_gradients_apart(dtype, rows, outs, ins, counts):
    """dx and dw asked for alone, and together (one launch for most sizes)."""
    gu.announce(f"linear gradients apart {dtype} {rows} x {outs} x {ins} {counts}")
    tail = 0 if counts is None else 11
    live = rows if counts is None else sum(counts)
    n, e = live + tail, 1 if counts is None else len(counts)
    offsets = None if counts is None else torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32).cuda()
    x, dy, ip = randn(1, n, ins, dtype=dtype), randn(2, n, outs, dtype=dtype), randn(3, n, ins, dtype=dtype)
    w = randn(4, *(() if counts is None else (e,)), outs, ins, dtype=dtype, scale=ins ** -0.5)
    for t in (x, dy, ip):
        t[live:] = float("nan")
    call = lambda **k: experts.linear_backward(dy, x, w, offsets=offsets, in_pre=ip, in_act="silu", need_dbias=False, **k)  # noqa: E731
    ways = [call(), (call(need_dw=False)[0], call(need_dx=False)[1])]
    bounds = [0, n] if counts is None else [0] + list(np.cumsum(counts))
    for i in range(e):
        lo, hi = int(bounds[i]), int(bounds[i + 1])
        wi, xi, gi, q = f64(w if counts is None else w[i]), f64(x[lo:hi]), f64(dy[lo:hi]), f64(ip[lo:hi])
        si = slope64(q, "silu")
        want = gi @ wi
        err = summed(outs) * (gi.abs() @ wi.abs()) * si.abs() + want.abs() * 2.0 ** -19 * (1 + q.abs())
        want = want * si
        dw, dwerr = gi.t() @ xi, summed(hi - lo) * (gi.abs().t() @ xi.abs())
        for got in ways:
            close(got[0][lo:hi], want, err, f"dx of {i}")
            close(got[1] if counts is None else got[1][i], dw, dwerr, f"dw of {i}")
    for got in ways:
        assert not got[0][live:].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_options(dtype):
    """Row strides on and off 16 bytes, no bias, and gradients one at a time."""
    rows, outs, ins = 70, 88, 104
    for shift in (0, 8, 3):
        wide = randn(1, rows, ins + 16, dtype=dtype)
        x = wide[:, shift:shift + ins]
        w = randn(2, outs, ins, dtype=dtype, scale=0.1)
        buf = torch.full((rows, outs + 13), -7.0, dtype=dtype, device="cuda")
        experts.linear(x, w, act="silu", out=buf[:, shift:shift + outs])
        assert torch.equal(buf[:, shift:shift + outs], experts.linear(x.contiguous(), w, act="silu"))
        assert (buf[:, :shift] == -7).all() and (buf[:, shift + outs:] == -7).all()
        g = randn(3, rows, outs + 16, dtype=dtype)[:, shift:shift + outs]
        all3 = experts.linear_backward(g, x, w)
        for i, name in enumerate(("need_dx", "need_dw", "need_dbias")):
            needs = {k: k == name for k in ("need_dx", "need_dw", "need_dbias")}
            got = experts.linear_backward(g, x, w, **needs)
            assert [v is None for v in got] == [k != i for k in range(3)]
            assert torch.equal(got[i], all3[i])
    empty = experts.linear(x[:0], w)
    assert empty.shape == (0, outs)
    dx, dw, db = experts.linear_backward(g[:0], x[:0], w)
    assert dx.shape == (0, ins) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,outs,ins", [(130, 94, 102), (70, 333, 37), (600, 1026, 518)])
def test_linear_gaps(dtype, rows, outs, ins):
    """Rows that end inside a 16-byte chunk, NaN between them: nothing of a gap counts."""
    gu.announce(f"linear gaps {dtype} {rows} x {outs} x {ins}")
    wide_x, wide_dy = randn(1, rows, ins + 6, dtype=dtype), randn(2, rows, outs + 6, dtype=dtype)
    w = randn(3, outs, ins, dtype=dtype, scale=ins ** -0.5)
    x, dy = wide_x[:, :ins], wide_dy[:, :outs]
    want = (experts.linear(x.contiguous(), w), *experts.linear_backward(dy.contiguous(), x.contiguous(), w))
    wide_x[:, ins:] = float("nan")
    wide_dy[:, outs:] = float("nan")
    got = (experts.linear(x, w), *experts.linear_backward(dy, x, w))
    for name, g, v in zip(("out", "dx", "dw", "dbias"), got, want):
        assert torch.equal(g, v), name


def test_linear_values():
    """Infinities and NaN reach the outputs that depend on them, and no others."""
    x = torch.zeros(40, 24, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(32, 24, dtype=torch.bfloat16, device="cuda")
    x[3, 5], x[7, 0] = float("inf"), float("nan")
    out = experts.linear(x, w, act="relu")
    assert torch.isinf(out[3]).all() and torch.isnan(out[7]).all()
    rest = torch.ones(40, dtype=torch.bool)
    rest[[3, 7]] = False
    assert not out[rest.cuda()].any()


@pytest.mark.parametrize("act,in_act", [("silu", None), ("gelu_tanh", None), ("none", "silu")])
def test_linear_differences(act, in_act):
    """<gradient, direction> against the loss's central difference along it, for
    w, x and bias together. The float32 forward is off by about summed(ins) per
    output, so the loss of rows * outs random terms by noise = that times the
    norm of dy times 2, and the difference by noise / h; its third-order term is
    below h^2 times the norms involved."""
    rows, outs, ins, h = 90, 40, 72, 2.0 ** -6
    counts = [50, 0, 40]
    offsets = torch.tensor([0, 50, 50, 90], dtype=torch.int32).cuda()
    w, b = randn(1, 3, outs, ins, scale=ins ** -0.5), randn(2, 3, outs)
    x, dy = randn(3, rows, ins), randn(4, rows, outs)
    vw, vb, vx = randn(5, 3, outs, ins, scale=ins ** -0.5), randn(6, 3, outs, scale=0.1), randn(7, rows, ins)

    def loss(t):
        xi = x + t * vx
        if in_act:
            xi = (xi * torch.sigmoid(xi))
        y = experts.linear(xi, w + t * vw, b + t * vb, act=act, offsets=offsets)
        return float((f64(y) * f64(dy)).sum())

    x0 = x * torch.sigmoid(x) if in_act else x
    _, pre = experts.linear(x0, w, b, act=act, offsets=offsets, save_pre=True)
    dx, dw, db = experts.linear_backward(dy, x0, w, pre=pre, act=act, offsets=offsets,
                                         in_pre=x if in_act else None, in_act=in_act or "none")
    got = float((f64(dx) * f64(vx)).sum() + (f64(dw) * f64(vw)).sum() + (f64(db) * f64(vb)).sum())
    diff = (loss(h) - loss(-h)) / (2 * h)
    size = float(f64(dy).norm())
    assert len(counts) == 3
    assert abs(got - diff) <= 2 * size * summed(ins) * 8 / h + h * h * size * 60


# ------------------------------------------------------------------- adamw


def np32(t):
    return t.detach().float().cpu().numpy()


def encode(m, v):
    f = np.float32
    with np.errstate(invalid="ignore", divide="ignore"):
        mb, vb = m.reshape(-1, 256), v.reshape(-1, 256)
        ms, vs = np.abs(mb).max(1), vb.max(1)
        r = np.where(ms[:, None] > 0, mb / ms[:, None], f(0))
        mq = np.sign(r) * np.rint(np.sqrt(np.abs(r)) * f(127))
        r = np.where(vs[:, None] > 0, vb / vs[:, None], f(0))
        vq = np.rint(np.sqrt(np.sqrt(r)) * f(255))
        vq = np.where(vb > 0, np.maximum(vq, f(1)), vq)
    return mq.astype(np.int8).reshape(-1), vq.astype(np.uint8).reshape(-1), ms, vs


def decode(mq, vq, ms, vs):
    f = np.float32
    t = mq.astype(f) * f(1 / 127)
    m = ((t * np.abs(t)).reshape(-1, 256) * ms[:, None]).reshape(-1)
    t = vq.astype(f) * f(1 / 255)
    t = t * t
    return m, ((t * t).reshape(-1, 256) * vs[:, None]).reshape(-1)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,gt,copies", [
    (torch.float32, torch.float32, False), (torch.float32, torch.bfloat16, True),
    (torch.bfloat16, torch.float16, False), (torch.float16, torch.float32, True)])
def test_adamw(bits, pt, gt, copies):
    """Three steps over tensors of awkward lengths: the moments (codes and scales
    with 8 bits) equal the float32 formulas bit for bit, and so do parameters."""
    sizes = [(1,), (0,), (255,), (256,), (257,), (3, 1000), (70, 130), (5,), (4097,)] + [(7,)] * 70
    params = [randn(i, *s, dtype=pt) for i, s in enumerate(sizes)]
    outs = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in sizes] if copies else None
    state = experts.adamw_state(params, bits)
    total = state["m"].numel()
    f = np.float32
    ref = [np32(p).reshape(-1) for p in params]
    m, v = np.zeros(total, f), np.zeros(total, f)
    gs = torch.full((1,), 0.5, device="cuda")
    lr, b1, b2, eps, wd = 1e-2, 0.9, 0.95, 1e-8, 0.1
    starts, at = [], 0
    for s in sizes:
        starts.append(at)
        at += -(-int(np.prod(s)) // 256) * 256
    for step in (1, 2, 3):
        grads = [randn(100 * step + i, *s, dtype=gt, scale=1e-3 if i % 2 else 1.0) for i, s in enumerate(sizes)]
        grads[3].zero_()
        experts.adamw_step(params, grads, lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd, step=step,
                           copies=outs, grad_scale=gs, **state)
        g = np.zeros(total, f)
        for s, gi in zip(starts, grads):
            g[s:s + gi.numel()] = np32(gi).reshape(-1)
        g = g * f(0.5)
        m = m * f(b1) + g * f(1 - b1)
        v = v * f(b2) + (g * g) * f(1 - b2)
        move = (m * f(lr / (1 - b1 ** step))) / (np.sqrt(v) * f(1 / math.sqrt(1 - b2 ** step)) + f(eps))
        for i, (s, p) in enumerate(zip(starts, params)):
            new = ref[i] * f(1 - lr * wd) - move[s:s + ref[i].size]
            ref[i] = np32(torch.from_numpy(new).to(pt))
            assert np.array_equal(np32(p).reshape(-1), ref[i]), f"parameter {i} of step {step}"
            if copies:
                assert np.array_equal(np32(outs[i]).reshape(-1), np32(torch.from_numpy(new).bfloat16()))
        if bits == 8:
            mq, vq, ms, vs = encode(m, v)
            assert np.array_equal(state["m"].cpu().numpy(), mq) and np.array_equal(state["v"].cpu().numpy(), vq)
            assert np.array_equal(np32(state["m_scale"]), ms) and np.array_equal(np32(state["v_scale"]), vs)
            m, v = decode(mq, vq, ms, vs)
            gm, gv = experts.adamw_moments(**state)
            assert np.array_equal(np32(gm), m) and np.array_equal(np32(gv), v)
        else:
            assert np.array_equal(np32(state["m"]), m) and np.array_equal(np32(state["v"]), v)


def test_adamw_own_copy():
    """A bfloat16 parameter given as its own copy is updated once; a float32 one's
    memory is refused."""
    p = [randn(1, 1000, dtype=torch.bfloat16)]
    q, g = [p[0].clone()], [randn(2, 1000)]
    for params, copies in ((p, p), (q, None)):
        experts.adamw_step(params, g, lr=0.1, copies=copies, **experts.adamw_state(params))
    assert torch.equal(p[0], q[0])
    r = [randn(1, 1000)]
    with pytest.raises(binding.KMeansError):
        experts.adamw_step(r, g, lr=0.1, copies=[r[0].view(torch.bfloat16)[:1000]], **experts.adamw_state(r))


def test_adamw_8_bit_codes():
    """A second moment above zero never gets code 0, a block of zeros stays
    zeros, and a NaN or an infinity marks its block and no other."""
    p = [torch.zeros(5 * 256, device="cuda")]
    state = experts.adamw_state(p, 8)
    g = torch.zeros(5 * 256, device="cuda")
    g[:256] = 1e-9
    g[0] = 1.0
    g[2 * 256 + 3] = float("nan")
    g[3 * 256 + 3] = float("inf")
    experts.adamw_step(p, [g], lr=1e-3, **state)
    assert int(state["v"][:256].min()) >= 1
    assert not state["m"][256:512].any() and not state["v"][256:512].any() and float(state["m_scale"][1]) == 0
    assert torch.isnan(state["m_scale"][2:4]).all() and torch.isnan(state["v_scale"][2:4]).all()
    assert torch.isfinite(state["m_scale"][[0, 1, 4]]).all() and float(state["v_scale"][4]) == 0
    m, v = experts.adamw_moments(**state)
    assert torch.isnan(m[512:1024]).all() and torch.isfinite(m[:512]).all() and torch.isfinite(v[1024:]).all()
    assert float(p[0][256:512].abs().max()) == 0 and torch.isfinite(p[0][:256]).all()


# ------------------------------------------------- streams, graphs, refusals


def test_side_stream():
    """Calls on another stream than the inputs' own, their results read back
    after that stream is waited for."""
    tokens, top, n, width = 300, 2, 5, 136
    ids, x, w = make_ids(1, tokens, top, n), randn(2, tokens, width), randn(3, n, 64, width)
    want = experts.linear(experts.dispatch(x, experts.plan(ids.cuda(), n)), w, offsets=experts.plan(ids.cuda(), n).offsets)
    side = torch.cuda.Stream()
    ids = ids.cuda()
    side.wait_stream(torch.cuda.current_stream())
    p = experts.plan(ids, n, stream=side)
    xs = experts.dispatch(x, p, stream=side)
    got = experts.linear(xs, w, offsets=p.offsets, stream=side)
    del p, xs
    junk = [torch.full((tokens * top, width), 9.0, device="cuda") for _ in range(4)]
    side.synchronize()
    assert torch.equal(got, want) and len(junk) == 4


def test_graph():
    """The forward path, its gradients and a step in one captured graph, replayed
    on other inputs with eager work in between."""
    tokens, top, n, width, outs = 600, 2, 9, 72, 80
    ids, x = make_ids(1, tokens, top, n).cuda(), randn(2, tokens, width, dtype=torch.bfloat16)
    w, weights = randn(3, n, outs, width, dtype=torch.bfloat16, scale=0.1), randn(4, tokens, top)
    dy = randn(5, tokens, outs, dtype=torch.bfloat16)
    state = experts.adamw_state([w])

    def work():
        p = experts.plan(ids, n)
        xs = experts.dispatch(x, p)
        ys, pre = experts.linear(xs, w, act="silu", offsets=p.offsets, save_pre=True)
        y = experts.combine(ys, weights, p)
        dys, dweights = experts.combine_backward(dy, ys, weights, p)
        dxs, dw, db = experts.linear_backward(dys, xs, w, pre=pre, act="silu", offsets=p.offsets)
        dx = experts.dispatch_backward(dxs, p)
        return y, dweights, dx, dw, db

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
        experts.adamw_step([w], [got[3]], lr=1e-2, **state)
    for k in range(3):
        ids.copy_(make_ids(10 + k, tokens, top, n, 0.1))
        x.copy_(randn(20 + k, tokens, width, dtype=torch.bfloat16))
        w0, s0 = w.clone(), {key: t.clone() for key, t in state.items()}
        want = work()
        experts.adamw_step([w0], [want[3]], lr=1e-2, **s0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(w, w0) and all(torch.equal(state[key], s0[key]) for key in state)


def test_refusals():
    """Arguments that the binding refuses, each before anything is enqueued."""
    x, w = randn(1, 10, 16), randn(2, 24, 16)
    ids = torch.zeros(10, 2, dtype=torch.int64, device="cuda")
    p = experts.plan(ids, 3)
    with pytest.raises(TypeError):
        experts.plan(ids.int(), 3)
    with pytest.raises(binding.KMeansError):
        experts.plan(ids, 0)
    with pytest.raises(binding.KMeansError):
        experts.plan(torch.zeros(5000, 2, dtype=torch.int64, device="cuda"), 3,
                     workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        experts.plan(ids.cpu(), 3)
    with pytest.raises(TypeError):
        experts.dispatch(x.double(), p)
    with pytest.raises(ValueError):
        experts.dispatch(x[:9], p)
    with pytest.raises(ValueError):
        experts.dispatch(randn(1, 16, 10).t(), p)
    with pytest.raises(ValueError):
        experts.combine(randn(1, 20, 16), randn(2, 10, 3), p)
    with pytest.raises(TypeError):
        experts.combine(randn(1, 20, 16), randn(2, 10, 2, dtype=torch.float16), p)
    with pytest.raises(ValueError):
        experts.linear(x, w, act="tanh")
    with pytest.raises(TypeError):
        experts.linear(x, w.half())
    with pytest.raises(ValueError):
        experts.linear(x, w[:, :15].contiguous())
    with pytest.raises(ValueError):
        experts.linear(x, w, offsets=p.offsets)
    with pytest.raises(ValueError):
        experts.linear(x, w, randn(3, 23))
    with pytest.raises(ValueError):
        experts.linear_backward(randn(1, 10, 24), x, w, act="silu")
    q = randn(4, 24, 24)
    for kw in (dict(out=q), dict(residual=q, out=q)):
        with pytest.raises(binding.KMeansError):
            experts.linear(q, randn(5, 24, 24), **kw)
    with pytest.raises(binding.KMeansError):
        experts.linear_backward(q, q, q, act="relu", pre=q, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    params, grads = [randn(1, 300)], [randn(2, 300)]
    state = experts.adamw_state(params)
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(lr=1.0, betas=(1.0, 0.9)), dict(lr=1.0, step=0)):
        with pytest.raises(binding.KMeansError):
            experts.adamw_step(params, grads, **state, **bad)
    with pytest.raises(ValueError):
        experts.adamw_step(params, [randn(2, 299)], lr=1.0, **state)
    with pytest.raises(ValueError):
        experts.adamw_step(params, grads, lr=1.0, m_scale=randn(1, 2), **state)
    with pytest.raises(ValueError):
        experts.adamw_step(params, grads, state["m"][:256], state["v"], lr=1.0)
    with pytest.raises(binding.KMeansError):
        experts.adamw_step(params, params, lr=1.0, **state)
