"""The operators around the experts on the GPU against their formulas in float64.

Tolerances are those of tests/test_gpu_experts.py: u = 2^-24, 2^-8, 2^-11 for a value
rounded once to float32, bfloat16, float16, and (4 + 2 sqrt(n)) 2^-23 times the sum
of the magnitudes for a float32 sum of n values. What else enters a bound is derived where
it is used.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from nearest_centroid_assignment_amd import experts, layers  # noqa: E402
from tests import gpu_util as gu  # noqa: E402
from tests.test_gpu_experts import TYPES, U, close, f64, randn, summed  # noqa: E402

pytestmark = pytest.mark.gpu

FAR = [-1, -100, -2 ** 63, 2 ** 63 - 1, 2 ** 32]  # numbers that no table has


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def numbers(seed, n, classes, skip=0.0, hot=0.0):
    """int64 numbers on the CPU; a part of them outside the table, a part all the same."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(classes, (n,), generator=g)
    ids[torch.rand(n, generator=g) < hot] = classes // 2
    out = torch.rand(n, generator=g) < skip
    far = torch.tensor(FAR + [classes])
    ids[out] = far[torch.randint(len(far), (n,), generator=g)][out]
    return ids


def strided(t, extra=3, shift=1):
    """The same rows inside a wider buffer of NaN, off its start."""
    rows, cols = t.shape
    big = torch.full((rows, cols + extra), float("nan"), dtype=t.dtype, device=t.device)
    big[:, shift:shift + cols] = t
    return big[:, shift:shift + cols]


# ------------------------------------------------------------------- embed


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,classes,width,skip,hot", [
    (0, 5, 8, 0, 0), (1, 1, 1, 0, 0), (3, 7, 5, 0.5, 0), (8, 300, 2048, 0, 0), (100, 17, 1001, 0.2, 0),
    (5000, 33, 64, 0, 0.3), (1000, 1, 24, 0.1, 0), (4097, 3000, 40, 0.1, 0.5), (2100, 2048, 33, 0, 0),
    (70000, 50000, 24, 0.05, 0.2), (20000, 2049, 130, 0, 0.9), (300, 5000, 8, 2.0, 0), (40, 9, 9000, 0.1, 0.5),
    (8192, 2048, 16, 0.1, 0.1), (8193, 2048, 16, 0.1, 0.1), (30000, 700, 24, 0.1, 0.3), (1025, 200, 16, 0, 0.5)])
def test_embed(dtype, tokens, classes, width, skip, hot):
    """The products with the scale are rounded once in float32 and once to the type; a
    gradient sums up to as many rows as a number comes up, and is scaled once."""
    gu.announce(f"embed {dtype} {tokens} of {classes} x {width}, {skip} outside, {hot} the same")
    ids = numbers(tokens + classes, tokens, classes, skip, hot)
    live = (ids >= 0) & (ids < classes)
    w = randn(1, classes, width, dtype=dtype)
    dy = randn(2, tokens, width, dtype=dtype)
    dy[(~live).cuda()] = float("nan")  # never read into a sum
    scale = 3.7
    y = layers.embed(ids.cuda(), w, scale)
    dw = layers.embed_backward(dy, ids.cuda(), classes, scale)
    assert y.shape == (tokens, width) and dw.shape == (classes, width) and dw.dtype == dtype
    want = torch.zeros(tokens, width, dtype=torch.float64)
    want[live] = f64(w)[ids[live]] * scale
    close(y, want, want.abs() * 2.0 ** -23, "y")  # (the scale itself is a float32)
    grad = torch.zeros(classes, width, dtype=torch.float64)
    size = torch.zeros(classes, width, dtype=torch.float64)
    rows = f64(dy)[live]
    grad.index_add_(0, ids[live], rows * scale)
    size.index_add_(0, ids[live], rows.abs() * scale)
    most = int(torch.bincount(ids[live], minlength=1).max()) if live.any() else 0
    close(dw, grad, (summed(most) + 2.0 ** -22) * size, "dw")
    if dtype == torch.bfloat16 and tokens:
        # Rows apart and off their boundaries, an output inside a buffer, the same bits again.
        out = torch.full((tokens, width + 5), 7.0, dtype=dtype, device="cuda")
        assert torch.equal(layers.embed(ids.cuda(), w, scale, out=out[:, 2:2 + width]), y)
        assert (out[:, :2] == 7).all() and (out[:, 2 + width:] == 7).all()
        assert torch.equal(layers.embed_backward(strided(dy), ids.cuda(), classes, scale), dw)


def test_embed_of_centroids():
    """Codes of the assignment and their centroids: a sample's nearest centroid; and the
    gradient of one row a code, through every way to sort."""
    from nearest_centroid_assignment_amd import binding

    X, C = randn(1, 2000, 40), randn(2, 33, 40)
    labels, dist = binding.assign(X, C)
    near = layers.embed(labels, C)
    assert torch.equal(near, C[labels])
    assert torch.allclose(((X - near).double() ** 2).sum(1), dist.double(), rtol=1e-4, atol=1e-3)
    for n in (1, 2048, 2049, 70000):
        ids = torch.randperm(n, generator=torch.Generator().manual_seed(n)).cuda()
        dy = randn(n, n, 8)
        want = torch.empty_like(dy)
        want[ids] = dy
        assert torch.equal(layers.embed_backward(dy, ids, n), want)


# -------------------------------------------------------------- layer norm


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [
    (0, 9), (1, 1), (3, 5), (1, 2048), (7, 64), (2000, 129), (1030, 512), (33, 1001), (1100, 2048),
    (1500, 1025), (5, 4096), (70, 8192), (3, 8195), (2, 20000), (40, 17001), (4100, 24), (70, 128), (37, 130),
    (2000, 256), (600, 16384), (1, 7000), (20000, 72), (4100, 2055),
    (1030, 760), (500, 260)])
def test_layer_norm(dtype, rows, width):
    """mean is a float32 sum; d = x - mean is off by what the mean is and one rounding; the
    variance (its sum's roundings, twice d's) enters h by half. With e the error of d
    relative to the row's deviation: h is off by e + |h| (e + summed + 2^-22)."""
    gu.announce(f"layer_norm {dtype} {rows} x {width}")
    n = summed(width)
    for kind in dict.fromkeys((dtype, torch.float32)):
        x = (randn(1, rows, width) * 2 + randn(2, rows, 1)).to(dtype)
        weight, bias = randn(3, width).to(kind), randn(4, width).to(kind)
        y, mean, rstd = layers.layer_norm(x, weight, bias, save_stats=True)
        xd = f64(x)
        m = xd.mean(1, keepdim=True) if rows else xd.sum(1, keepdim=True)
        sd = (((xd - m) ** 2).mean(1, keepdim=True) + 1e-5).sqrt()
        off = n * xd.abs().mean(1, keepdim=True) + 2.0 ** -23 * (xd.abs() + m.abs())
        e = off.amax(1, keepdim=True) / sd if rows else off
        h = (xd - m) / sd
        eh = e + h.abs() * (e + n + 2.0 ** -22)
        close(mean, m[:, 0], n * xd.abs().mean(1), "mean")
        close(rstd, 1 / sd[:, 0], (e[:, 0] + n + 2.0 ** -22) / sd[:, 0], "rstd")
        wd, bd = f64(weight), f64(bias)
        slack = (eh * wd.abs()) + 2.0 ** -23 * ((h * wd).abs() + bd.abs())
        close(y, h * wd + bd, slack, "y")
        close(layers.layer_norm(x, None, bias), h + bd, eh + 2.0 ** -23 * (h.abs() + bd.abs()), "y without weight")
        close(layers.layer_norm(x, weight), h * wd, slack, "y without bias")

        # The gradient for the saved mean and rstd: h to two roundings, sums over the row,
        # and over the rows for the columns.
        dy = randn(5, rows, width, dtype=dtype)
        dx, dw, db = layers.layer_norm_backward(dy, x, weight, mean, rstd)
        assert dw.dtype == kind and db.dtype == kind and dx.dtype == dtype
        gd, md, rd = f64(dy), f64(mean)[:, None], f64(rstd)[:, None]
        h = (xd - md) * rd
        eh = 2.0 ** -23 * (xd.abs() + md.abs() + (xd - md).abs()) * rd
        g = gd * wd
        a, b = g.sum(1, keepdim=True) / width, (g * h).sum(1, keepdim=True) / width
        sa, sb = g.abs().sum(1, keepdim=True) / width, (g * h).abs().sum(1, keepdim=True) / width
        eb = (n + 2.0 ** -22) * sb + (g.abs() * eh).sum(1, keepdim=True) / width
        slack = rd * ((n + 2.0 ** -22) * sa + h.abs() * eb + eh * b.abs() + 2.0 ** -22 * (g.abs() + a.abs() + (h * b).abs()))
        close(dx, rd * (g - a - h * b), slack, "dx")
        r = summed(rows)
        close(dw, (gd * h).sum(0), (r + 2.0 ** -23) * (gd * h).abs().sum(0) + (gd.abs() * eh).sum(0), "dweight")
        close(db, gd.sum(0), r * gd.abs().sum(0), "dbias")
        if rows == 1030 or width == 17001:  # some of them, rows apart, and the same bits
            only = layers.layer_norm_backward(strided(dy), strided(x), weight, mean, rstd, need_dweight=False)
            assert only[1] is None and torch.equal(only[0], dx) and torch.equal(only[2], db)
            only = layers.layer_norm_backward(dy, x, weight, mean, rstd, need_dx=False, need_dbias=False)
            assert only[0] is None and only[2] is None and torch.equal(only[1], dw)
            only = layers.layer_norm_backward(dy, x, weight, mean, rstd, need_dweight=False, need_dbias=False)
            assert torch.equal(only[0], dx)
            out = torch.full((rows, width + 5), 7.0, dtype=dtype, device="cuda")
            layers.layer_norm(strided(x), weight, bias, out=out[:, 1:1 + width])
            assert torch.equal(out[:, 1:1 + width], y) and (out[:, 1 + width:] == 7).all() and (out[:, 0] == 7).all()


def test_layer_norm_far_from_zero():
    """Rows whose mean is a thousand times their deviation: the variance is that of what is
    left when the mean is taken off, so h is off by 1e3 float32 roundings (and the mean's), not
    by 1e6. Constant rows give the bias."""
    x = 1000.0 + randn(1, 300, 700)
    y = layers.layer_norm(x)
    xd = f64(x)
    want = (xd - xd.mean(1, keepdim=True)) / (xd.var(1, correction=0, keepdim=True) + 1e-5).sqrt()
    assert float((f64(y) - want).abs().max()) < 1001 * (summed(700) + 2.0 ** -23) * 1.1
    flat = torch.full((5, 300), 3.0, device="cuda")
    bias = randn(2, 300)
    assert torch.equal(layers.layer_norm(flat, randn(3, 300), bias), bias.expand(5, 300))


def test_layer_norm_gradient_is_the_derivative():
    """Against differences of the operator's own float64 formula by torch's autograd."""
    x, weight, bias = randn(1, 50, 200), randn(2, 200), randn(3, 200)
    dy = randn(4, 50, 200)
    _, mean, rstd = layers.layer_norm(x, weight, bias, save_stats=True)
    got = layers.layer_norm_backward(dy, x, weight, mean, rstd)
    leaves = [t.double().requires_grad_(True) for t in (x, weight, bias)]
    out = torch.nn.functional.layer_norm(leaves[0], (200,), leaves[1], leaves[2])
    for a, b in zip(got, torch.autograd.grad(out, leaves, dy.double())):
        assert float((a.double() - b).norm() / b.norm()) < 2.0 ** -19  # (rstd is off by a few 2^-24)


# ------------------------------------------------------------------- route


def route_ref(logits, top, score, bias, groups, kept, best, renormalize, scale):
    """The choice and the weights in float64 on the CPU, a token at a time."""
    z = f64(logits)
    t, e = z.shape
    live = z > -math.inf
    p = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1).nan_to_num(0.0)
    c = z if bias is None and (best == 1 or groups == 1) else p + (0 if bias is None else f64(bias))
    c = torch.where(live & ~c.isnan(), c, -math.inf)
    ids = torch.full((t, top), -1)
    for i in range(t):
        row = c[i].tolist()
        size = e // groups
        if groups > 1:
            rank = []
            for g in range(groups):
                part = sorted((v for v in row[g * size:(g + 1) * size] if v > -math.inf), reverse=True)[:best]
                rank.append((-(sum(part) if part else -math.inf), g))
            stay = {g for _, g in sorted(rank)[:kept]}
        order = sorted((-v, j) for j, v in enumerate(row)
                       if v > -math.inf and (groups == 1 or j // size in stay))[:top]
        for k, (_, j) in enumerate(order):
            ids[i, k] = j
    at = ids.clamp(min=0)
    s = torch.where(ids >= 0, p.gather(1, at), 0.0)
    if renormalize:
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    return ids, s * scale, p


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,n,top,groups,kept,best,biased,masked", [
    (1, 1, 1, 1, 1, 1, False, 0), (0, 8, 2, 1, 1, 1, False, 0), (3, 5, 2, 1, 1, 1, False, 0.3),
    (8, 64, 2, 1, 1, 1, False, 0), (100, 60, 3, 1, 1, 1, False, 0.5), (65, 256, 8, 8, 4, 2, True, 0),
    (33, 256, 8, 8, 4, 1, True, 0.2), (50, 160, 6, 8, 3, 1, False, 0), (40, 33, 16, 1, 1, 1, True, 0.9),
    (17, 300, 17, 3, 2, 2, False, 0.1), (20, 1024, 10, 1, 1, 1, True, 0.0), (9, 2048, 64, 64, 5, 2, True, 0.05),
    (30, 100, 3, 50, 20, 2, True, 0.3), (12, 48, 4, 16, 16, 2, False, 0), (300, 129, 4, 1, 1, 1, True, 0),
    (5, 64, 64, 1, 1, 1, False, 0.1), (21, 48, 20, 4, 1, 2, True, 0)])
def test_route(dtype, score, tokens, n, top, groups, kept, best, biased, masked):
    """The choice is that of float64, ties to the lower number (16-bit logits have many).
    Weights: s is off by its argument's rounding (2^-24 of up to 12) and the hardware's
    2^x and reciprocal (2^-22), the sum over n or top of them likewise: 2^-18 in all."""
    gu.announce(f"route {dtype} {score} {tokens} x {n}, {top} from {kept} of {groups} by {best}, bias {biased}, masked {masked}")
    logits = (randn(1, tokens, n) * 2).to(dtype)
    if masked:
        logits[randn(2, tokens, n) < torch.distributions.Normal(0, 1).icdf(torch.tensor(masked))] = -math.inf
        logits[: tokens // 5] = -math.inf  # rows with nothing left
    bias = randn(3, n) * 0.3 if biased else None
    dweights = randn(4, tokens, top)
    for renormalize in (True, False):
        kw = dict(score=score, renormalize=renormalize, scale=1.5)
        ids, weights = layers.route(logits, top, bias=bias, groups=groups, top_groups=kept, group_best=best, **kw)
        want, w, p = route_ref(logits, top, score, bias, groups, kept, best, renormalize, 1.5)
        assert torch.equal(ids.cpu(), want)
        close(weights, w, 2.0 ** -18 * w, "weights")
        assert (weights[ids < 0] == 0).all()
        got = layers.route_backward(dweights, logits, ids, **kw)
        # The gradient of the weights with the choice fixed, by autograd on s; what reaches dz
        # is a difference of terms of at most |share d| + share sum|share d|.
        z = torch.where(p > 0, f64(logits), torch.zeros_like(p)).requires_grad_(True)
        masks = torch.where(f64(logits) > -math.inf, 0.0, -math.inf)
        row = z + masks
        none = (masks == -math.inf).all(1, keepdim=True)
        s = torch.sigmoid(row) if score == "sigmoid" else torch.softmax(torch.where(none, z, row), 1)
        s = torch.where(want >= 0, s.gather(1, want.clamp(min=0)), torch.zeros(()))
        if renormalize:
            s = s / torch.where(s.sum(1, keepdim=True) > 0, s.sum(1, keepdim=True), torch.ones(()))
        d = f64(dweights) * 1.5
        grad = torch.autograd.grad((s * d).sum(), z)[0] if tokens else torch.zeros_like(z)
        terms = (s * d).abs().detach()
        size = torch.zeros(tokens, n + 1, dtype=torch.float64).scatter_add_(
            1, torch.where(want >= 0, want, n), terms + s.detach() * terms.sum(1, keepdim=True))[:, :n]
        if score == "softmax" and not renormalize:
            size = size + p * terms.sum(1, keepdim=True)
        # autograd's own terms cancel to within a few of float64's roundings (2^-53 of their
        # sizes each) where the formula gives zero: with renormalised softmax scores, s (d - sum)
        # of an expert that is not chosen is a difference of two equal sums of `top` terms.
        close(got, grad, 2.0 ** -17 * size + 2.0 ** -53 * (4 + top) * terms.sum(1, keepdim=True), "dlogits")
        assert (got[logits == -math.inf] == 0).all()
        assert torch.equal(layers.route_backward(dweights, strided(logits), ids, **kw), got)
        again = layers.route(strided(logits), top, bias=bias, groups=groups, top_groups=kept, group_best=best, **kw)
        assert torch.equal(again[0], ids) and torch.equal(again[1], weights)


def test_route_near_ties():
    """Choices apart by less than float32 holds next to the bias are told apart as in
    float64: sigmoids that differ by one unit of their logits, under a bias of 64."""
    n, tokens = 96, 400
    base = torch.linspace(-1, 1, tokens)[:, None].expand(tokens, n).clone()
    steps = torch.stack([torch.randperm(n, generator=torch.Generator().manual_seed(i)) for i in range(tokens)])
    logits = (base.view(torch.int32) + steps.int()).view(torch.float32).cuda()
    bias = torch.full((n,), 64.0, device="cuda")
    for score in ("softmax", "sigmoid"):
        for kw in (dict(bias=bias), dict(bias=bias, groups=8, top_groups=3, group_best=2)):
            ids, _ = layers.route(logits, 6, score=score, **kw)
            want = route_ref(logits, 6, score, bias, kw.get("groups", 1), kw.get("top_groups", 1),
                             kw.get("group_best", 1), True, 1.0)[0]
            assert torch.equal(ids.cpu(), want), score


def test_route_extremes():
    """All logits the type's lowest value: they are scores as any others, and the ties go to the
    lowest numbers. Far below zero the sigmoids' shares are those of e^z. A NaN is never
    chosen. -0 and 0 tie."""
    for dtype in TYPES:
        low = torch.full((3, 20), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        for score in ("softmax", "sigmoid"):
            ids, w = layers.route(low, 4, score=score)
            assert ids.tolist() == [[0, 1, 2, 3]] * 3
            assert torch.allclose(w, torch.full_like(w, 0.25))
    z = torch.tensor([[-200.0, -201.0, -300.0, -math.inf]], device="cuda")
    ids, w = layers.route(z, 3, score="sigmoid")
    e = math.exp(-1)
    assert ids.tolist() == [[0, 1, 2]] and torch.allclose(w[0, :2].cpu(), torch.tensor([1 / (1 + e), e / (1 + e)]))
    z = torch.tensor([[math.nan, 1.0, 2.0, math.nan, -math.inf]], device="cuda")
    for score in ("softmax", "sigmoid"):
        ids, w = layers.route(z, 3, score=score)
        assert ids.tolist() == [[2, 1, -1]] and w[0, 2] == 0
        assert float(w.sum()) == pytest.approx(1.0)
    z = torch.tensor([[-0.0, 0.0, -0.0, 0.0]], device="cuda")
    assert layers.route(z, 4)[0].tolist() == [[0, 1, 2, 3]]
    bias = torch.tensor([0.0, -math.inf, math.nan, 0.0], device="cuda")
    assert layers.route(z, 4, bias=bias)[0].tolist() == [[0, 3, -1, -1]]


@pytest.mark.parametrize("experts", [40, 700])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_of_repeated_experts(experts, score, renormalize):
    """Ids that no route gives, an expert more than once: its gradients add up. The terms of a
    sum of k values d r, |r| <= 1, are each off by a dozen float32 roundings (exponentials,
    division, inner sum), so all are by 16 of them at most of the largest."""
    z = randn(5, 9, experts)
    ids = numbers(6, 9 * 5, experts).reshape(9, 5)
    ids[0], ids[1] = 3, torch.tensor([4, 2, 4, 2, 4])
    ids[2, 1:], ids[3, 2] = -1, experts
    ids = ids.cuda()
    dw = randn(7, 9, 5)
    dz = layers.route_backward(dw, z, ids, score=score, renormalize=renormalize, scale=1.5)
    leaf = z.double().requires_grad_(True)
    live = (ids >= 0) & (ids < experts)
    s = torch.softmax(leaf, 1) if score == "softmax" else torch.sigmoid(leaf)
    w = torch.where(live, s.gather(1, ids.clamp(0, experts - 1)), 0.0)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    want, = torch.autograd.grad(1.5 * w, leaf, dw.double())
    most = 1.5 * 5 * float(dw.abs().max())
    assert float((dz.double() - want).abs().max()) <= 16 * 2.0 ** -24 * most
    assert torch.equal(dz, layers.route_backward(dw, z, ids, score=score, renormalize=renormalize, scale=1.5))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_infinite_bias(score):
    """A bias of +inf takes its experts first, one of -inf takes them out, in any groups."""
    z = randn(77, 50, 40)
    bias = 0.1 * randn(78, 40)
    bias[[7, 23]], bias[[2, 30, 31]] = math.inf, -math.inf
    for groups, kept, best in ((1, 1, 1), (4, 2, 1), (4, 2, 2)):
        ids, w = layers.route(z, 5, score=score, bias=bias, groups=groups, top_groups=kept, group_best=best)
        assert (ids[:, :2] == torch.tensor([7, 23], device="cuda")).all() and w.isfinite().all()
        s = (torch.softmax(z.double(), 1) if score == "softmax" else torch.sigmoid(z.double())) + bias.double()
        if groups > 1:  # those of 7 and 23
            s[:, 10:20], s[:, 30:] = -math.inf, -math.inf
        s[:, [7, 23]] = -math.inf
        assert (ids[:, 2:] == s.topk(3, 1).indices).all()


# ----------------------------------------------------------- cross entropy


def entropy_ref(x, w, targets, dloss, dlse, dtype):
    """float64 values and bounds (on the tensors' device). A logit z is a float32 sum; lse is
    off by as much as the logits and the roundings of e^(z - largest) and its sum; dz by p times
    those, and rounded once to the operands' type."""
    x, w = x.double(), w.double()
    classes = w.shape[0]
    z = x @ w.t()
    ez = summed(x.shape[1]) * (x.abs() @ w.abs().t())
    live = (targets >= 0) & (targets < classes)
    lse = torch.logsumexp(z, 1)
    el = ez.amax(1) + 2.0 ** -23 * (z.amax(1) - z.amin(1)).clamp(max=120) + summed(classes) + 2.0 ** -23 * lse.abs() + 2.0 ** -21
    at = torch.where(live, targets, torch.zeros_like(targets))[:, None]
    loss = torch.where(live, lse - z.gather(1, at)[:, 0], 0.0)
    eloss = torch.where(live, el + ez.gather(1, at)[:, 0], 0.0)
    out = dict(lse=(lse, el), loss=(loss, eloss))
    if dloss is not None:
        b = torch.where(live, dloss.double(), 0.0)
        a = b if dlse is None else b + dlse.double()
        p = torch.exp(z - lse[:, None])
        hit = torch.zeros_like(p).scatter_(1, at, b[:, None])
        dz = a[:, None] * p - hit
        ep = a.abs()[:, None] * p * (ez + el[:, None] + 2.0 ** -23 * (z - lse[:, None]).abs() + 2.0 ** -21)
        edz = ep + (U[dtype] + 2.0 ** -23) * (dz.abs() + ep)
        # 2^x below float32's smallest normal, 2^-126, is zero, and so is a dz that small.
        edz = edz + 2.0 ** -126 * (1 + a.abs()[:, None])
        if dtype == torch.float16:  # what falls below float16's steps at the common scale
            edz = edz + 2.0 ** -24 * 2.0 ** -13 * torch.maximum(a.abs().max(), b.abs().max())
        out["dx"] = dz @ w, edz @ w.abs() + summed(classes) * (dz.abs() @ w.abs())
        out["dw"] = dz.t() @ x, edz.t() @ x.abs() + summed(len(x)) * (dz.t().abs() @ x.abs())
    return out


def check_entropy(dtype, rows, classes, width, skip=0.0, lse_grad=False, scale=1.0, views=False):
    gu.announce(f"cross_entropy {dtype} {rows} x {classes} x {width}, {skip} ignored, dlse {lse_grad}, scale {scale}")
    x = randn(1, rows, width, dtype=dtype, scale=scale)
    w = randn(2, classes, width, dtype=dtype, scale=2 / math.sqrt(width))
    targets = numbers(3, rows, classes, skip).cuda()
    dloss = randn(4, rows) * (0.5 if dtype == torch.float16 else 1.0 / max(rows, 1))
    dlse = randn(5, rows) * 0.1 * dloss.abs().amax() if lse_grad else None
    want = entropy_ref(x, w, targets, dloss, dlse, dtype)
    loss, lse = layers.cross_entropy(x, w, targets)
    dx, dw = layers.cross_entropy_backward(dloss, x, w, targets, lse, dlse)
    for name, got in (("lse", lse), ("loss", loss), ("dx", dx), ("dw", dw)):
        close(got, *(t.cpu() for t in want[name]), name)
    live = (targets >= 0) & (targets < classes)
    assert (loss[~live] == 0).all()
    if not lse_grad:
        assert (dx[~live] == 0).all()
    if views:  # rows apart and off their boundaries: the same bits; one output (cut otherwise)
        sx = strided(x)
        again = layers.cross_entropy(sx, w, targets)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
        again = layers.cross_entropy_backward(dloss, sx, w, targets, lse, dlse)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
        only = layers.cross_entropy_backward(dloss, sx, w, targets, lse, dlse, need_dw=False)
        assert only[1] is None
        close(only[0], *(t.cpu() for t in want["dx"]), "dx alone")
        only = layers.cross_entropy_backward(dloss, sx, w, targets, lse, dlse, need_dx=False)
        assert only[0] is None
        close(only[1], *(t.cpu() for t in want["dw"]), "dw alone")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,classes,width,skip", [
    (1, 1, 1, 0), (1, 5, 7, 0), (3, 64, 64, 0.5), (16, 1000, 129, 0.2), (65, 257, 40, 0), (100, 3000, 72, 0.1),
    (300, 513, 1001, 0.3), (1000, 1111, 777, 0.1), (2, 20000, 64, 0), (16, 70001, 96, 0.1), (513, 130, 2048, 0),
    (2100, 2304, 256, 0.05), (5000, 7, 24, 0.1), (40, 900, 33, 2.0), (128, 4096, 3000, 0), (658, 119, 2944, 0.1),
    (100, 33, 4097, 0.1), (1100, 17, 2050, 0.1), (203, 24640, 192, 0), (33, 8191, 520, 0)])
def test_cross_entropy(dtype, rows, classes, width, skip):
    check_entropy(dtype, rows, classes, width, skip, lse_grad=rows % 2 == 0, views=rows in (16, 65, 1000))


@pytest.mark.parametrize("dtype", TYPES)
def test_cross_entropy_in_pieces(dtype):
    """So many rows that dz takes several pieces of the classes, the last one shorter."""
    size = torch.finfo(dtype).bits // 8
    check_entropy(dtype, 300000, 2600 // size, 24, 0.05, lse_grad=True)


def test_cross_entropy_no_rows():
    x, w = torch.empty(0, 24, device="cuda"), randn(1, 50, 24)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = layers.cross_entropy(x, w, none)
    assert loss.shape == lse.shape == (0,)
    dx, dw = layers.cross_entropy_backward(loss, x, w, none, lse)
    assert dx.shape == (0, 24) and dw.shape == w.shape and (dw == 0).all()
    x, w = x[:, :23].bfloat16(), w[:, :23].bfloat16()  # of rows that a product would copy
    dx, dw = layers.cross_entropy_backward(loss, x, w.contiguous(), none, lse)
    assert dx.shape == (0, 23) and dw.shape == w.shape and (dw == 0).all()


def test_cross_entropy_large_logits():
    """Logits of thousands: the largest is taken off first. Rows with infinities keep to themselves."""
    check_entropy(torch.float32, 70, 700, 40, scale=500.0)
    check_entropy(torch.bfloat16, 70, 700, 40, scale=500.0)
    x, w = randn(1, 130, 40), randn(2, 300, 40).abs() + 0.1
    targets = numbers(3, 130, 300).cuda()
    want = layers.cross_entropy(x, w, targets)
    x[5, 3], x[6, 3], x[7, 3] = math.inf, -math.inf, math.nan
    loss, lse = layers.cross_entropy(x, w, targets)
    assert lse[5] == math.inf and lse[6] == -math.inf and lse[7].isnan()
    assert not loss[5:8].isfinite().any()
    for got, ref in ((loss, want[0]), (lse, want[1])):
        assert torch.equal(got[:5], ref[:5]) and torch.equal(got[8:], ref[8:])


def test_cross_entropy_is_the_derivative():
    """Against torch's autograd in float64, and against differences of the loss itself."""
    x, w = randn(1, 60, 30), randn(2, 90, 30)
    targets = numbers(3, 60, 90, 0.1)
    lam = 1e-2
    loss, lse = layers.cross_entropy(x, w, targets.cuda())
    live = (targets >= 0) & (targets < 90)
    n = int(live.sum())
    dloss = torch.full((60,), 1.0 / n, device="cuda")
    dx, dw = layers.cross_entropy_backward(dloss, x, w, targets.cuda(), lse, dlse=2 * lam / 60 * lse)

    def total(x, w):
        z = x @ w.t()
        ce = torch.nn.functional.cross_entropy(z[live], targets[live], reduction="sum") / n
        return ce + lam * (torch.logsumexp(z, 1) ** 2).mean()

    leaves = [f64(t).requires_grad_(True) for t in (x, w)]
    for got, want in zip((dx, dw), torch.autograd.grad(total(*leaves), leaves)):
        assert float((f64(got) - want).norm() / want.norm()) < 2.0 ** -17
    h = 1e-4
    with torch.no_grad():
        for t, got, at in ((0, dx, (7, 3)), (1, dw, (11, 5))):
            up, down = [[f64(a) for a in (x, w)] for _ in range(2)]
            up[t][at] += h
            down[t][at] -= h
            slope = float(total(*up) - total(*down)) / (2 * h)
            assert float(got[at]) == pytest.approx(slope, rel=1e-4, abs=1e-7)


# --------------------------------------------------- together and elsewhere


def run_of_them(s, stream=None):
    """The operators as a model calls them, one after another."""
    kw = dict(stream=stream)
    e = layers.embed(s["ids"], s["w"], 2.0, **kw)
    y, mean, rstd = layers.layer_norm(e, s["weight"], s["bias"], save_stats=True, **kw)
    logits = experts.linear(y, s["wr"], **kw)
    ids, weights = layers.route(logits, 2, score="sigmoid", bias=s["balance"], groups=4, top_groups=2,
                                group_best=2, **kw)
    plan = experts.plan(ids, 16, **kw)
    ys = experts.linear(experts.dispatch(y, plan, **kw), s["we"], offsets=plan.offsets, **kw)
    out = experts.combine(ys, weights, plan, **kw)
    loss, lse = layers.cross_entropy(out, s["w"], s["ids"], **kw)
    dout, dw = layers.cross_entropy_backward(s["dloss"], out, s["w"], s["ids"], lse, **kw)
    dys, dweights = experts.combine_backward(dout, ys, weights, plan, **kw)
    dlogits = layers.route_backward(dweights, logits, ids, score="sigmoid", **kw)
    dy, dwr, _ = experts.linear_backward(dlogits, y, s["wr"], need_dbias=False, **kw)
    de, dweight, dbias = layers.layer_norm_backward(dy, e, s["weight"], mean, rstd, **kw)
    table = layers.embed_backward(de, s["ids"], s["w"].shape[0], 2.0, **kw)
    return [e, y, mean, rstd, ids, weights, out, loss, lse, dout, dw, dweights, dlogits, de, dweight, dbias, table]


def state_of(seed, tokens=700, classes=3000, width=136):
    t = torch.bfloat16
    return dict(ids=numbers(seed, tokens, classes, 0.05).cuda(), w=randn(seed + 1, classes, width, dtype=t),
                weight=randn(seed + 2, width, dtype=t), bias=randn(seed + 3, width, dtype=t),
                wr=randn(seed + 4, 16, width, dtype=t, scale=0.1), balance=randn(seed + 5, 16) * 0.1,
                we=randn(seed + 6, 16, width, width, dtype=t, scale=0.1),
                dloss=torch.full((tokens,), 1.0 / tokens, device="cuda"))


def test_streams():
    """A side stream gives the same bits as the current one, also when the inputs' memory is
    given back right after the call."""
    s = state_of(1)
    want = run_of_them(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    copy = {k: v.clone() for k, v in s.items()}
    side.wait_stream(torch.cuda.current_stream())
    got = run_of_them(copy, stream=side)
    del copy
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del junk
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_graph():
    """A step captured once and replayed on new inputs, with eager work between the
    replays, gives the eager step's bits."""
    static = state_of(1)
    run_of_them(static)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_of_them(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run_of_them(static)
    for seed in (20, 40, 60, 20):
        new = state_of(seed)
        for k, v in new.items():
            static[k].copy_(v)
        want = run_of_them(new)
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), seed


def test_warns_of_autograd():
    w = randn(1, 20, 8).requires_grad_(True)
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    x = randn(2, 3, 8)
    for call in (lambda: layers.embed(ids, w), lambda: layers.layer_norm(x, w[0]), lambda: layers.route(w, 2),
                 lambda: layers.cross_entropy(x, w, ids)):
        with pytest.warns(UserWarning, match="layers.*not recorded"):
            call()
        with torch.no_grad():
            call()


def test_refusals():
    """What a call cannot take it refuses before a kernel is enqueued."""
    x, w = randn(1, 6, 8), randn(2, 20, 8)
    ids = torch.zeros(6, dtype=torch.int64, device="cuda")
    f = torch.zeros(6, device="cuda")
    bad = [
        (TypeError, lambda: layers.embed(ids.int(), w)), (TypeError, lambda: layers.embed(ids[::2], w)),
        (ValueError, lambda: layers.embed(ids, w.t())), (TypeError, lambda: layers.embed(ids, w.double())),
        (ValueError, lambda: layers.embed(ids.cpu(), w)), (ValueError, lambda: layers.embed(ids, w.cpu())),
        (layers.KMeansError, lambda: layers.embed(ids, w, out=w[:6])),
        (ValueError, lambda: layers.embed_backward(x, ids[:5], 20)),
        (layers.KMeansError, lambda: layers.embed_backward(x, ids, 0)),
        (layers.KMeansError, lambda: layers.embed_backward(x, ids, 2 ** 20 + 1)),
        (layers.KMeansError, lambda: layers.embed_backward(x, ids, 20, workspace=torch.empty(300, dtype=torch.uint8, device="cuda"))),
        (ValueError, lambda: layers.layer_norm(x, w[0, :7])), (TypeError, lambda: layers.layer_norm(x, w[0].half())),
        (TypeError, lambda: layers.layer_norm(x, w[0], w[0].half())),
        (layers.KMeansError, lambda: layers.layer_norm(x, eps=-1.0)),
        (layers.KMeansError, lambda: layers.layer_norm(x, eps=math.nan)),
        (layers.KMeansError, lambda: layers.layer_norm(x, out=x)),
        (ValueError, lambda: layers.layer_norm_backward(x, x[:5], None, f, f)),
        (ValueError, lambda: layers.layer_norm_backward(x, x, None, f[:5], f)),
        (layers.KMeansError, lambda: layers.route(w, 0)), (layers.KMeansError, lambda: layers.route(w, 9)),
        (layers.KMeansError, lambda: layers.route(w, 2, groups=3)), (ValueError, lambda: layers.route(w, 2, score="relu")),
        (layers.KMeansError, lambda: layers.route(w, 2, groups=2, top_groups=3)),
        (layers.KMeansError, lambda: layers.route(w, 2, groups=2, group_best=3)),
        (layers.KMeansError, lambda: layers.route(randn(1, 2, 2049), 2)),
        (TypeError, lambda: layers.route(w, 2, bias=w[0].half())), (ValueError, lambda: layers.route(w.t(), 2)),
        (TypeError, lambda: layers.route_backward(f[:, None], x, ids[:, None].int())),
        (ValueError, lambda: layers.route_backward(f[:, None], x, ids[:5, None])),
        (ValueError, lambda: layers.cross_entropy(x, w[:, :7].contiguous(), ids)),
        (ValueError, lambda: layers.cross_entropy(x, w, ids[:5])), (TypeError, lambda: layers.cross_entropy(x, w.half(), ids)),
        (ValueError, lambda: layers.cross_entropy(x, w[::2], ids)),
        (ValueError, lambda: layers.cross_entropy_backward(f[:5], x, w, ids, f)),
        (TypeError, lambda: layers.cross_entropy_backward(f, x, w, ids, f.double())),
        (layers.KMeansError, lambda: layers.cross_entropy_backward(f, x, w, ids, f, workspace=torch.empty(300, dtype=torch.uint8, device="cuda"))),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
