"""The mixture of experts behind a nearest-centroid router, trained end to end:
one step's gradients against torch's own differentiation of the same formulas in
float64, and the loss over a short run."""
import pytest

torch = pytest.importorskip("torch")

from nearest_centroid_assignment_amd import train_experts  # noqa: E402
from tests import gpu_util as gu  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_step_gradients():
    """bfloat16 rounds each of h, pre, ys, dys and dz once (2^-8 each), and the
    returned gradients once: with independent roundings their norm is off by at
    most sqrt(6) 2^-8 of the gradient's, taken twice for room."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    tokens, width, hidden, clusters = 500, 72, 136, 5
    model = train_experts.Experts(clusters + 1, width, hidden, 32, gen)
    x = torch.randn(tokens, width, generator=gen, device="cuda").to(torch.bfloat16)
    labels = torch.randint(clusters, (tokens,), generator=gen, device="cuda")
    dy = torch.randn(tokens, width, generator=gen, device="cuda").to(torch.bfloat16)
    y, saved = train_experts.forward(model, x, labels, clusters)
    got = train_experts.backward(model, dy, saved)

    leaves = [p.double().requires_grad_(True) for p in model.copies[:4] + [model.masters[4]]]
    w1, b1, w2, b2, logits = leaves
    xd = x.double()

    def expert(rows, e):
        h = xd[rows] @ w1[e].t() + b1[e]
        return (h * torch.sigmoid(h)) @ w2[e].t() + b2[e]

    mix = torch.softmax(logits[labels], 1)
    own = torch.zeros(tokens, width, dtype=torch.float64, device="cuda")
    for e in range(clusters):
        rows = (labels == e).nonzero()[:, 0]
        own = own.index_add(0, rows, expert(rows, e))
    everyone = torch.arange(tokens, device="cuda")
    want_y = mix[:, :1] * own + mix[:, 1:] * expert(everyone, clusters)
    want = torch.autograd.grad(want_y, leaves, dy.double())
    bound = 2 * 6 ** 0.5 * 2.0 ** -8
    for name, a, b in zip(("y", "dw1", "db1", "dw2", "db2", "dlogits"), (y, *got), (want_y, *want)):
        off = float((a.double() - b.detach()).norm() / b.detach().norm())
        gu.announce(f"{name}: {off:.2e} of its norm")
        assert off <= bound, name


@pytest.mark.parametrize("bits", [32, 8])
def test_loss_falls(bits):
    first, last, mean = train_experts.train(steps=120, samples=8192, width=64, hidden=128, clusters=9,
                                            batch=2048, bits=bits, log=gu.announce)
    assert last < 0.25 * mean < first
