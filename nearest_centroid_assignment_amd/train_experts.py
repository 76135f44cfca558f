"""Train a mixture of experts behind a nearest-centroid router, end to end on
the GPU:

    python -m nearest_centroid_assignment_amd.train_experts [--steps 200] [--bits 8]

The data are Gaussian blobs (``datagen``); what is learned is a different
nonlinear map in every blob. ``kmeans_fit`` finds the centroids, and every batch
is routed by ``assign``: each sample goes to the expert of its nearest centroid
and to one expert that all samples share, mixed with weights that are learned per
expert. An expert is two layers with a silu between them. One step:

    assign -> plan -> dispatch -> linear (silu) -> linear -> combine -> loss
    combine_backward -> linear_backward (its dx times silu') -> linear_backward
    -> adamw_step (float32 masters, bfloat16 copies that the products read)

The learned maps are compared at the end with the error of predicting the mean.
"""
from __future__ import annotations

import argparse

import torch

from . import binding, datagen, experts


class Experts:
    """The parameters: float32 masters, the bfloat16 copies that the products
    read, and AdamW's moments."""

    def __init__(self, count, width, hidden, bits, gen):
        def draw(*shape, scale):
            return torch.randn(shape, generator=gen, device="cuda") * scale

        self.masters = [draw(count, hidden, width, scale=width ** -0.5),
                        torch.zeros(count, hidden, device="cuda"),
                        draw(count, width, hidden, scale=hidden ** -0.5),
                        torch.zeros(count, width, device="cuda"),
                        torch.zeros(count, 2, device="cuda")]  # mixing logits: own expert, shared
        self.copies = [p.to(torch.bfloat16) for p in self.masters]
        self.state = experts.adamw_state(self.masters, bits)
        self.step = 0

    def update(self, grads, lr, clip=1.0):
        norm = torch.stack(torch._foreach_norm(grads)).norm()
        scale = (clip / (norm + 1e-6)).clamp(max=1.0).reshape(1).float()
        self.step += 1
        experts.adamw_step(self.masters, grads, lr=lr, betas=(0.9, 0.99), weight_decay=0.01,
                           step=self.step, copies=self.copies, grad_scale=scale, **self.state)


def forward(model, x, labels, shared):
    """Predictions for x (tokens, width) and what the gradients need."""
    ids = torch.stack([labels, torch.full_like(labels, shared)], 1)
    plan = experts.plan(ids, shared + 1)
    w1, b1, w2, b2, _ = model.copies
    xs = experts.dispatch(x, plan)
    h, pre = experts.linear(xs, w1, b1, act="silu", offsets=plan.offsets, save_pre=True)
    ys = experts.linear(h, w2, b2, offsets=plan.offsets)
    weights = torch.softmax(model.masters[4][labels], 1)
    return experts.combine(ys, weights, plan), (plan, xs, h, pre, ys, weights, labels)


def backward(model, dy, saved):
    """Gradients of the masters, float32, given dy (tokens, width)."""
    plan, xs, h, pre, ys, weights, labels = saved
    w1, _, w2, _, logits = model.copies
    dys, dweights = experts.combine_backward(dy, ys, weights, plan)
    dz, dw2, db2 = experts.linear_backward(dys, h, w2, offsets=plan.offsets, in_pre=pre,
                                           in_act="silu")
    _, dw1, db1 = experts.linear_backward(dz, xs, w1, offsets=plan.offsets, need_dx=False)
    dsoft = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
    dlogits = torch.zeros_like(logits, dtype=torch.float32).index_add_(0, labels, dsoft)
    return [g.float() for g in (dw1, db1, dw2, db2)] + [dlogits]


def train(steps=200, samples=16384, width=256, hidden=512, clusters=17, batch=4096, bits=32,
          lr=3e-3, seed=0, log=print):
    """Returns (first loss, last loss, loss of predicting the mean)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    X, C0 = datagen.make_blobs(samples, clusters, width, kb=clusters, sigma_c=1.0, sigma=0.5, seed=seed)
    X, C0 = torch.from_numpy(X).cuda(), torch.from_numpy(C0).cuda()
    fit = binding.fit(X, C0, max_iter=20, tol=1e-3)
    centres = fit["centres"]
    log(f"router: {clusters} centroids in {fit['n_iter']} iterations, inertia {fit['inertia']:.4g}")
    maps = torch.randn(clusters, width, width, generator=gen, device="cuda") * width ** -0.5
    target = torch.empty_like(X)
    for c in range(clusters):
        rows = fit["labels"] == c
        target[rows] = torch.tanh(X[rows] @ maps[c])
    model = Experts(clusters + 1, width, hidden, bits, gen)
    losses = []
    for step in range(steps):
        at = torch.randint(samples, (batch,), generator=gen, device="cuda")
        x, want = X[at], target[at]
        labels, _ = binding.assign(x, centres, min_dist=False)
        y, saved = forward(model, x.to(torch.bfloat16), labels, clusters)
        diff = y.float() - want
        losses.append((diff * diff).mean())
        dy = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        model.update(backward(model, dy, saved), lr)
        if step % 50 == 0 or step == steps - 1:
            log(f"step {step}: loss {float(losses[-1]):.5f}")
    return float(losses[0]), float(torch.stack(losses[-5:]).mean()), float(target.var())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--batch", type=int, default=4096)
    ap.add_argument("--clusters", type=int, default=17)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--bits", type=int, choices=(8, 32), default=32)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)
    first, last, mean = train(steps=a.steps, batch=a.batch, clusters=a.clusters, width=a.width,
                              hidden=a.hidden, bits=a.bits, seed=a.seed)
    print(f"loss {first:.5f} -> {last:.5f}; predicting the mean {mean:.5f}")


if __name__ == "__main__":
    main()
