"""One update of the model of cluster codes: AdamW's step, the copies and the balance of the
experts, each against its formula in float64."""
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


def _gradients(model, gen, norm):
    """One a parameter, of the types that backward gives, together of this norm (but for their
    rounding)."""
    grads = [(i + 1) * torch.randn(c.shape, generator=gen, device="cuda") for i, c in enumerate(model.copies)]
    size = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    return [(g * (norm / size)).to(c.dtype) for g, c in zip(grads, model.copies)]


def test_update():
    """Three steps with float32 moments against AdamW (decay first, both biases corrected) in
    float64, the gradients clipped to a norm of 1 together. Each parameter is off by at most a few
    dozen float32 roundings of itself and of the step of lr (moments, root, division: 2^-18 of the
    step, the sums of the norm among them); the copies are the masters, rounded."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    model = train_codes.Model(50, 6, 72, 136, 32, gen)
    lr, b1, b2, decay, eps = 3e-3, 0.9, 0.99, 0.01, 1e-8
    want = [p.double() for p in model.masters]
    m, v = [torch.zeros_like(p) for p in want], [torch.zeros_like(p) for p in want]
    slack = [torch.zeros_like(p) for p in want]
    for step, size in enumerate((40.0, 0.5, 1.3)):
        gu.announce(f"update {step}")
        grads = _gradients(model, gen, size)
        loads = torch.tensor([30, 0, 20, 20, 40, 10], device="cuda")  # of a mean of 20
        offsets = torch.cat([loads.new_zeros(1), loads.cumsum(0)]).int()
        before = model.balance.clone()
        model.update(grads, offsets, lr)
        g64 = [g.double() for g in grads]
        norm = math.sqrt(sum(float((g * g).sum()) for g in g64))
        clip = min(1.0, 1.0 / (norm + 1e-6))
        assert (clip < 1.0) == (size > 1.0)
        for i, g in enumerate(g64):
            g = g * clip
            m[i] = b1 * m[i] + (1 - b1) * g
            v[i] = b2 * v[i] + (1 - b2) * g * g
            move = lr * (m[i] / (1 - b1 ** (step + 1))) / ((v[i] / (1 - b2 ** (step + 1))).sqrt() + eps)
            want[i] = want[i] * (1 - lr * decay) - move
            # A moment that cancels is off by 2^-18 of the largest of its terms, which is what a
            # step of lr (1 / (1 - b2^t))^(1/2) stands for at most.
            slack[i] += 2.0 ** -22 * want[i].abs() + 2.0 ** -18 * (move.abs() + lr)
        for name, got, copy, ref, off in zip(train_codes.NAMES, model.masters, model.copies, want, slack):
            assert ((got.double() - ref).abs() <= off).all(), (name, step)
            assert torch.equal(copy, got.to(copy.dtype)), (name, step)
        # Experts with more than the mean's load are liked less, those with less more.
        sign = torch.tensor([-1.0, 1.0, 0.0, 0.0, -1.0, 1.0], device="cuda")
        assert torch.equal(torch.sign(model.balance - before), sign)
        assert torch.allclose((model.balance - before).abs(), 1e-3 * sign.abs())


def test_balance_counts_in_the_choice():
    """A bias that is moved against one expert takes its tokens away: the loads that update reads
    are those of the choice that the bias is part of."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    model = train_codes.Model(50, 6, 72, 136, 32, gen)
    codes = torch.randint(50, (600,), generator=gen, device="cuda")
    plan = train_codes.forward(model, codes, codes)[1][8]
    loads = plan.offsets.diff()
    most = int(loads.argmax())
    assert int(loads.sum()) == 1200 and int(loads[most]) > 200
    model.balance[most] -= 2.0  # more than the sigmoids' range
    loads = train_codes.forward(model, codes, codes)[1][8].offsets.diff()
    assert int(loads[most]) == 0 and int(loads.sum()) == 1200
