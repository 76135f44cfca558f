"""The model of cluster codes: one step's gradients against torch's own differentiation of
the same formulas in float64, and a short run."""
import math

import pytest

torch = pytest.importorskip("torch")

from nearest_centroid_assignment_amd import train_codes  # noqa: E402
from tests import gpu_util as gu  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_step_gradients():
    """bfloat16 rounds what the operators hand on: forward e, y, logits, xs, hidden, pre, ys,
    moe, h and out, backward dz of the head, dout, dh, dys, dz, dxs, dlogits and dy twice, and
    every gradient once. Each rounding is 2^-8 of its value at most; what a value's error does
    to a gradient is of the size of the gradient, but for the two norms and the softmax, which
    at most double it. So with 20 independent ones the norm is off by at most
    2 sqrt(20) 2^-8 of the gradient's, taken twice for room."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    tokens, classes, count, width, hidden = 700, 50, 6, 72, 136
    model = train_codes.Model(classes, count, width, hidden, 32, gen)
    model.balance += 0.05 * torch.randn(count, generator=gen, device="cuda")
    for p, c in zip(model.masters, model.copies):  # norms and shifts that are not 1 and 0
        if p.dim() == 1:
            p += 0.1 * torch.randn(p.shape, generator=gen, device="cuda")
            c.copy_(p)
    codes = torch.randint(classes, (tokens,), generator=gen, device="cuda")
    targets = torch.randint(classes, (tokens,), generator=gen, device="cuda")
    targets[::7] = -1
    dloss = torch.rand(tokens, generator=gen, device="cuda") / tokens
    loss, saved = train_codes.forward(model, codes, targets)
    got = train_codes.backward(model, dloss, saved)
    ids = saved[6]

    leaves = [p.double().requires_grad_(True) for p in model.copies]
    table, n1, s1, router, w1, b1, w2, b2, n2, s2, head = leaves
    norm = torch.nn.functional.layer_norm
    e = table[codes]
    y = norm(e, (width,), n1, s1)
    s = torch.sigmoid(y @ router.t()).gather(1, ids)  # the choice as it was made
    s = s / s.sum(1, keepdim=True)
    z = torch.einsum("tw,khw->tkh", y, w1) + b1
    each = torch.einsum("tkh,kwh->tkw", z * torch.sigmoid(z), w2) + b2
    moe = (each.gather(1, ids[:, :, None].expand(-1, -1, width)) * s[:, :, None]).sum(1)
    out = norm(e + moe, (width,), n2, s2)
    want = torch.nn.functional.cross_entropy(out @ head.t(), targets, ignore_index=-1, reduction="none")
    grads = torch.autograd.grad(want, leaves, dloss.double())
    bound = 4 * math.sqrt(20) * 2.0 ** -8
    for name, a, b in zip(("loss", *train_codes.NAMES), (loss, *got), (want, *grads)):
        off = float((a.double() - b.detach()).norm() / b.detach().norm())
        gu.announce(f"{name}: {off:.2e} of its norm")
        assert off <= bound, name


@pytest.mark.parametrize("bits", [32, 8])
def test_runs(bits):
    first, last, walk = train_codes.train(steps=6, samples=2048, width=64, hidden=128, clusters=17, count=4,
                                          batch=512, bits=bits, log=gu.announce)
    assert math.isfinite(first) and math.isfinite(last) and 0 < walk < math.log(17)
