"""Edges of the operators around the experts on the GPU: rows whose answer must not depend on
their neighbours, the orders of the lanes that the other sizes leave out, the largest sizes."""
import math

import pytest

torch = pytest.importorskip("torch")

from nearest_centroid_assignment_amd import experts, layers  # noqa: E402
from tests import gpu_util as gu  # noqa: E402
from tests.test_gpu_experts import TYPES, close, randn  # noqa: E402
from tests.test_gpu_layers import entropy_ref, route_ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ------------------------------------------------------------------- route


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,top,kw", [
    (40, 4, dict(bias=True)), (40, 4, dict(groups=8, top_groups=3, group_best=2)),
    (256, 8, dict(bias=True, groups=8, top_groups=4, group_best=2)), (600, 5, dict(bias=True))])
def test_route_nan_beside_ties(dtype, score, n, top, kw):
    """Rows with a NaN (or, of softmax scores, an infinite) logit among rows of equal logits, whose
    choices need float64: every row is answered as it is alone. By the formulas each s of such
    a softmax row is NaN and nothing is chosen; a sigmoid's NaN takes out its own expert."""
    gu.announce(f"route beside ties {dtype} {score} {top} of {n} {kw}")
    kw = dict(kw, score=score)
    if kw.pop("bias", False):
        kw["bias"] = torch.full((n,), 0.5, device="cuda")
    tokens = 37  # waves of four tokens with none, one or more of them
    z = torch.ones(tokens, n, device="cuda").to(dtype)
    z[2::3] = randn(1, len(range(2, tokens, 3)), n, dtype=dtype)
    odd = torch.zeros(tokens, dtype=torch.bool)
    odd[[1, 6, 11, 12, 20, 21, 22, 31, 36]] = True
    z[odd.cuda(), 3] = math.nan
    if score == "softmax":
        z[[6, 36], 3] = math.inf
    ids, weights = layers.route(z, top, **kw)
    for t in range(tokens):
        alone = layers.route(z[t:t + 1].contiguous(), top, **kw)
        assert torch.equal(alone[0][0], ids[t]) and torch.equal(alone[1][0], weights[t]), t
    if score == "softmax":
        assert (ids[odd.cuda()] == -1).all() and (weights[odd.cuda()] == 0).all()
    else:
        assert (ids[odd.cuda()] >= 0).all() and (ids[odd.cuda()] != 3).all()
    assert (ids[~odd.cuda()] >= 0).all() and weights.isfinite().all()
    assert ids[0].tolist() == list(range(top))


@pytest.mark.parametrize("dtype", TYPES)
def test_route_nan_by_the_logits(dtype):
    """Where nothing is added the logits choose, and a softmax row with a NaN gives its others:
    shares among the chosen, or NaN where they need the row's own s."""
    z = torch.tensor([[1.0, math.nan, 2.0, 0.0], [1.0, math.inf, 2.0, 0.0]], device="cuda").to(dtype)
    for kw in (dict(), dict(group_best=2)):
        ids, w = layers.route(z, 2, **kw)
        assert ids.tolist() == [[2, 0], [1, 2]]
        e = math.exp(-1)
        assert torch.allclose(w[0].cpu(), torch.tensor([1 / (1 + e), e / (1 + e)])) and w[1].isnan().all()
        ids, w = layers.route(z, 2, renormalize=False, **kw)
        assert ids.tolist() == [[2, 0], [1, 2]] and w.isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,size,kept,best,biased,masked", [
    (3, 70, 2, 2, True, 0.0), (5, 41, 2, 1, False, 0.3), (5, 48, 3, 2, False, 0.0), (6, 32, 4, 1, True, 0.2),
    (7, 11, 3, 2, True, 0.5), (9, 16, 2, 2, False, 0.1), (11, 3, 5, 1, True, 0.0), (13, 1, 6, 2, True, 0.3),
    (15, 16, 14, 2, True, 0.0)])
def test_route_of_groups_that_leave_lanes(dtype, score, groups, size, kept, best, biased, masked):
    """Sixteen lanes that the groups do not divide: 5, 3, 2 or 1 to a group and one to seven
    without any. The choice is that of float64; weights as in test_route."""
    gu.announce(f"route {dtype} {score} {kept} of {groups} x {size} by {best}, bias {biased}, masked {masked}")
    tokens, n = 45, groups * size
    top = min(6, kept * size)
    logits = (randn(1, tokens, n) * 2).to(dtype)
    if masked:
        logits[torch.rand(tokens, n, generator=torch.Generator().manual_seed(2)).cuda() < masked] = -math.inf
        logits[:3] = -math.inf
    bias = randn(3, n) * 0.3 if biased else None
    kw = dict(score=score, bias=bias, groups=groups, top_groups=kept, group_best=best)
    for renormalize in (True, False):
        ids, weights = layers.route(logits, top, renormalize=renormalize, scale=1.5, **kw)
        want, w, _ = route_ref(logits, top, score, bias, groups, kept, best, renormalize, 1.5)
        assert torch.equal(ids.cpu(), want)
        close(weights, w, 2.0 ** -18 * w, "weights")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [4, 40])  # groups of 16 lanes to a token, and of a wave
def test_route_group_ranks_of_large_biases(dtype, score, size):
    """Sums of two choices that float32 does not hold, of biases that are the type's lowest or
    largest value: the groups are those of the formulas in float64, where they are finite."""
    low, high = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    tokens, groups = 9, 4 if size == 4 else 20
    logits = randn(1, tokens, groups * size, dtype=dtype)
    for first, kept in (((-math.inf, low, 0.0, -math.inf), 2), ((2e38, 3e38, -math.inf, 2.5e38), 1),
                        ((low, low, low, low), 3), ((low, 0.9 * low, low, -math.inf), 1),
                        ((0.8 * high, high, high, 0.0), 2)):
        bias = torch.full((groups, size), -math.inf)
        bias[:4] = torch.tensor(first)[:, None] * (1 - 1e-3 * torch.arange(size))  # no two alike
        bias = bias.reshape(-1).cuda()
        kw = dict(score=score, bias=bias, groups=groups, top_groups=kept, group_best=2)
        ids, weights = layers.route(logits, min(6, kept * size), **kw)
        want, w, _ = route_ref(logits, min(6, kept * size), score, bias, groups, kept, 2, True, 1.0)
        assert torch.equal(ids.cpu(), want), first
        close(weights, w, 2.0 ** -18 * w, "weights")


# ----------------------------------------------------------- cross entropy


def test_cross_entropy_of_very_many_rows():
    """More rows than one dispatch of the kernel that joins their sums holds (2^28): a sample
    of them, both sides of every border among it, against the formulas in float64."""
    rows, classes, width, dtype = 2 ** 28 + 21, 40, 2, torch.bfloat16
    gu.announce(f"cross_entropy {rows} x {classes} x {width}")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=gen, device="cuda", dtype=dtype)
    w = randn(2, classes, width, dtype=dtype)
    targets = torch.randint(-1, classes, (rows,), generator=gen, device="cuda")
    loss, lse = layers.cross_entropy(x, w, targets)
    dloss = torch.rand(rows, generator=gen, device="cuda")
    gu.announce("its gradient")
    dx, _ = layers.cross_entropy_backward(dloss, x, w, targets, lse, need_dw=False)
    assert loss.isfinite().all() and lse.isfinite().all() and dx.isfinite().all()
    at = torch.randint(rows, (2000,), generator=gen, device="cuda")
    at[:64] = torch.arange(64)
    at[64:128] = torch.arange(2 ** 27 - 32, 2 ** 27 + 32)
    at[128:181] = torch.arange(2 ** 28 - 32, rows)
    want = entropy_ref(x[at], w, targets[at], dloss[at], None, dtype)
    for name, got in (("loss", loss), ("lse", lse), ("dx", dx)):
        close(got[at], *(t.cpu() for t in want[name]), name)


# --------------------------------------------------------------- tangents


def test_warns_of_tangents():
    """Both ways to a kernel say that the result has no tangent, and give the primal's result."""
    from torch.autograd import forward_ad

    w, ids = randn(1, 20, 8), torch.arange(3, device="cuda")
    want = layers.embed(ids, w)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(w, randn(2, 20, 8))
        for kw in (dict(), dict(stream=torch.cuda.current_stream())):
            for call in (lambda: layers.embed(ids, dual, **kw), lambda: layers.layer_norm(dual, **kw),
                         lambda: layers.route(dual, 2, **kw), lambda: layers.cross_entropy(w, dual, ids[:1].expand(20).contiguous(), **kw)):
                with pytest.warns(UserWarning, match="tangent"):
                    out = call()
                assert forward_ad.unpack_dual(out if torch.is_tensor(out) else out[1]).tangent is None
        with pytest.warns(UserWarning, match="tangent"):
            assert torch.equal(layers.embed(ids, dual), want)


# --------------------------------------------------------------- refusals


def test_refusals_allocate_nothing():
    """A count that no call takes is refused before memory for its outputs is asked for."""
    z, ids, dy = randn(1, 8, 16), torch.zeros(8, dtype=torch.int64, device="cuda"), randn(2, 8, 16)
    before = torch.cuda.memory_reserved()
    torch.cuda.reset_peak_memory_stats()
    at = torch.cuda.memory_allocated()
    for call in (lambda: layers.route(z, 10 ** 8), lambda: layers.route(z, 17), lambda: layers.route(z, -1),
                 lambda: layers.embed_backward(dy, ids, 10 ** 8), lambda: layers.embed_backward(dy, ids, -1)):
        with pytest.raises(layers.KMeansError):
            call()
    assert torch.cuda.max_memory_allocated() <= at + 4096 and torch.cuda.memory_reserved() == before


def test_flags_that_are_no_truth_values():
    """What Python itself raises for them, by the native way as by the other."""
    x, ids = randn(1, 8, 16), torch.zeros(8, dtype=torch.int64, device="cuda")
    f, flag = torch.ones(8, device="cuda"), torch.ones(2)
    for call in (lambda: layers.layer_norm(x, save_stats=flag),
                 lambda: layers.layer_norm_backward(x, x, None, f, f, need_dx=flag),
                 lambda: layers.route(x, 2, renormalize=flag),
                 lambda: layers.route_backward(f[:, None], x, ids[:, None], renormalize=flag),
                 lambda: layers.cross_entropy_backward(f, x, x, ids, f, need_dw=flag)):
        with pytest.raises(RuntimeError, match="Boolean value"):
            call()
    with pytest.raises(RuntimeError, match="Boolean value"):
        experts.linear(x, x, save_pre=flag)
    with pytest.raises(RuntimeError, match="Boolean value"):
        experts.linear_backward(x[:, :8].contiguous(), x, randn(3, 8, 16), need_dx=flag)
