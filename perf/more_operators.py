"""Cases of the operators around the experts: what is timed, in the framework's kernels and in plain torch.

Four operators that a model of cluster codes (or of any tokens) needs around its
mixture of experts, from the codes that go in to the loss over the codes that come out:

  embed    rows of a table by code, scaled; the table's gradient
  norm     layer norm; gradients, the weight's and bias's summed over the rows
  route    scores of the experts to expert numbers and weights: softmax or sigmoid, a bias
           for balance, groups, renormalised; the scores' gradient
  entropy  softmax cross entropy of x w^T against codes, the logits never kept; gradients

With ``own`` false, ``run`` computes the plain form: elementary torch operations
in float32 (the choice of experts in float64), rounded once where the operator returns.
With ``own`` true it calls ``nearest_centroid_assignment_amd.layers``.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
EPS = 1e-5


# ------------------------------------------------------------------- cases


def listed():
    return [
        # A decoding step of 8 sequences over the codes of 16384 centroids. Latency.
        dict(name="embed decode bf16", op="embed", tokens=8, classes=16384, width=2048, dtype="bfloat16",
             pad=0.0, grad=False),
        # float32 rows as the rest of the framework has them, odd sizes, padded places.
        dict(name="embed odd f32", op="embed", tokens=5003, classes=1111, width=777, dtype="float32",
             pad=0.1, grad=True),
        # A training batch over a large vocabulary, codes as uneven as words are.
        dict(name="embed train bf16", op="embed", tokens=65536, classes=50000, width=2048, dtype="bfloat16",
             pad=0.02, grad=True),
        # The norm before the experts of a decoding step. Latency.
        dict(name="norm decode bf16", op="norm", rows=16, width=2048, dtype="bfloat16", wide=False, bias=True,
             grad=False),
        # Odd sizes; float32 weights beside 16-bit rows.
        dict(name="norm odd f16", op="norm", rows=5003, width=1001, dtype="float16", wide=True, bias=True,
             grad=True),
        # A training batch at the mid workload's size.
        dict(name="norm train bf16", op="norm", rows=65536, width=2048, dtype="bfloat16", wide=False, bias=True,
             grad=True),
        # A decoding step's choice of 2 experts of 64. Latency.
        dict(name="route decode bf16", op="route", tokens=8, experts=64, top=2, score="softmax", biased=False,
             groups=1, kept=1, best=1, renormalize=True, masked=0.0, dtype="bfloat16", grad=False),
        # Plain softmax weights, experts that a mask takes out, rows that it leaves nothing.
        dict(name="route odd f32", op="route", tokens=5003, experts=60, top=3, score="softmax", biased=False,
             groups=1, kept=1, best=1, renormalize=False, masked=0.2, dtype="float32", grad=True),
        # A training batch: 8 of 256 experts from 4 of 8 groups, balanced by a bias.
        dict(name="route train bf16", op="route", tokens=65536, experts=256, top=8, score="sigmoid", biased=True,
             groups=8, kept=4, best=2, renormalize=True, masked=0.0, dtype="bfloat16", grad=True),
        # How likely 16 continuations are: no gradient, the table is read once. Latency and bandwidth.
        dict(name="entropy score bf16", op="entropy", rows=16, classes=16384, width=2048, dtype="bfloat16",
             ignored=0.0, lse_grad=False, grad=False),
        # float32, odd sizes, ignored places, a term on the log of the sum.
        dict(name="entropy odd f32", op="entropy", rows=1000, classes=1111, width=777, dtype="float32",
             ignored=0.1, lse_grad=True, grad=True),
        # The head of a training step over a large vocabulary: forward and backward.
        dict(name="entropy train bf16", op="entropy", rows=8192, classes=65536, width=2048, dtype="bfloat16",
             ignored=0.05, lse_grad=False, grad=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A size of the range: half of them multiples of 64, the others as they fall."""
    v = _log(rng, lo, hi)
    return max(lo, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(("embed", "norm", "route", "entropy", "entropy"))
    dtype = rng.choice(("bfloat16", "bfloat16", "float16", "float32"))
    size = 4 if dtype == "float32" else 2
    if op == "embed":
        width, classes = _width(rng, 64, 8192), _log(rng, 16, 200000)
        while classes * width * size > 50000 * 2048 * 2:
            classes //= 2
        tokens = _log(rng, 1, max(1, min(262144, 65536 * 2048 * 2 // (width * size))))
        return dict(op=op, tokens=tokens, classes=classes, width=width, dtype=dtype, pad=rng.choice((0.0, 0.05)),
                    grad=rng.random() < 0.7)
    if op == "norm":
        width = _width(rng, 16, 16384)
        rows = _log(rng, 1, max(1, min(262144, 65536 * 2048 * 2 // (width * size))))
        return dict(op=op, rows=rows, width=width, dtype=dtype, wide=rng.random() < 0.4, bias=rng.random() < 0.7,
                    grad=rng.random() < 0.7)
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * _log(rng, 4, 1024 // groups)
        kept = rng.randint(1, groups)
        tokens = _log(rng, 1, min(262144, 65536 * 256 * 2 // (experts * size)))
        return dict(op=op, tokens=tokens, experts=experts, top=rng.randint(1, min(8, experts // groups * kept)),
                    score=rng.choice(("softmax", "sigmoid")), biased=rng.random() < 0.5, groups=groups, kept=kept,
                    best=rng.choice((1, 2)), renormalize=rng.random() < 0.7, masked=rng.choice((0.0, 0.0, 0.1)),
                    dtype=dtype, grad=rng.random() < 0.7)
    rows, classes, width = _log(rng, 1, 8192), _width(rng, 64, 131072), _width(rng, 64, 4096)
    most = 8192 * 65536 * 2048 // (12 if dtype == "float32" else 1)
    while rows * classes * width > most or rows * classes > 8192 * 65536 or classes * width > 65536 * 2048:
        classes = max(1, classes // 2)
    return dict(op=op, rows=rows, classes=classes, width=width, dtype=dtype, ignored=rng.choice((0.0, 0.1)),
                lse_grad=rng.random() < 0.3, grad=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(scale).to(dtype)


def _frequency(classes, device):
    """How often each code comes up: the r-th as 1 / (r + 10)."""
    p = 1.0 / (torch.arange(classes, device=device, dtype=torch.float64) + 10.0)
    return p / p.sum()


def _codes(g, n, classes, none):
    """Codes with those frequencies; a part `none` of them is -1."""
    ids = torch.searchsorted(_frequency(classes, DEV).cumsum(0).float(),
                             torch.rand(n, generator=g, device=DEV)).clamp_(max=classes - 1)
    if none:
        ids = torch.where(torch.rand(n, generator=g, device=DEV) < none, -1, ids)
    return ids


def prepare(case, seed):
    g = _gen(seed)
    op, dtype = case["op"], TYPES[case["dtype"]]
    if op == "embed":
        t, d = case["tokens"], case["width"]
        s = dict(ids=_codes(g, t, case["classes"], case["pad"]), scale=math.sqrt(d),
                 w=_randn(g, (case["classes"], d), dtype, 0.02))
        if case["grad"]:
            s["dy"] = _randn(g, (t, d), dtype)
    elif op == "norm":
        r, d = case["rows"], case["width"]
        weights = torch.float32 if case["wide"] else dtype
        # Rows of a residual stream: sizes and means differ, some columns are large.
        x = torch.randn((r, d), generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn((r, 1), generator=g, device=DEV))
        x += 0.5 * torch.randn((r, 1), generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn((1, d), generator=g, device=DEV))
        s = dict(x=x.to(dtype), weight=(1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(weights),
                 bias=_randn(g, d, weights, 0.1) if case["bias"] else None)
        if case["grad"]:
            s["dy"] = _randn(g, (r, d), dtype)
    elif op == "route":
        t, e = case["tokens"], case["experts"]
        logits = torch.randn((t, e), generator=g, device=DEV)
        logits += 0.5 * torch.randn((1, e), generator=g, device=DEV)  # some experts are liked
        if case["masked"]:
            logits[torch.rand((t, e), generator=g, device=DEV) < case["masked"]] = -math.inf
            logits[torch.rand(t, generator=g, device=DEV) < 0.01] = -math.inf
        s = dict(logits=logits.to(dtype), scale=1.5 if case["score"] == "sigmoid" else 1.0,
                 bias=_randn(g, e, torch.float32, 0.1) if case["biased"] else None)
        if case["grad"]:
            s["dweights"] = _randn(g, (t, case["top"]), torch.float32)
    else:
        r, v, d = case["rows"], case["classes"], case["width"]
        s = dict(x=_randn(g, (r, d), dtype), w=_randn(g, (v, d), dtype, 2.0 / math.sqrt(d)),
                 targets=_codes(g, r, v, case["ignored"]))
        if case["grad"]:
            # The mean over the batch; float16 gradients come with a loss scale.
            s["dloss"] = torch.full((r,), (4096.0 if dtype == torch.float16 else 1.0) / r, device=DEV)
            s["dlse"] = _randn(g, (r,), torch.float32, 0.1 / r) * (4096.0 if dtype == torch.float16 else 1.0) \
                if case["lse_grad"] else None
    s["case"] = dict(case)
    return s


# ------------------------------------------------- the plain form, float32


def _plain_embed(s):
    case, ids, w = s["case"], s["ids"], s["w"]
    live = (ids >= 0) & (ids < case["classes"])
    at = torch.where(live, ids, 0)
    y = torch.where(live[:, None], w[at].float() * s["scale"], 0.0)
    out = dict(y=y.to(w.dtype))
    if case["grad"]:
        g = torch.where(live[:, None], s["dy"].float() * s["scale"], 0.0)
        dw = torch.zeros((case["classes"], case["width"]), device=ids.device)
        out["dw"] = dw.index_add_(0, at, g).to(w.dtype)
    return out


def _plain_norm(s):
    x = s["x"].float()
    weight = s["weight"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    h = c * rstd[:, None]
    y = h * weight
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out = dict(y=y.to(s["x"].dtype))
    if s["case"]["grad"]:
        dy = s["dy"].float()
        g = dy * weight
        dx = (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True)) * rstd[:, None]
        out.update(mean=mean, rstd=rstd, dx=dx.to(s["x"].dtype), dweight=(dy * h).sum(0).to(s["weight"].dtype))
        if s["bias"] is not None:
            out["dbias"] = dy.sum(0).to(s["weight"].dtype)
    return out


def _choose(case, logits, bias):
    """Expert numbers, largest choice first and ties to the lowest number, in float64; -1 where none is left."""
    z = logits.double()
    live = z > -math.inf
    if case["score"] == "sigmoid":
        c = 1.0 / (1.0 + torch.exp(-z))
    else:
        c = torch.exp(z - torch.where(live, z, -1e300).amax(1, keepdim=True))
        c = torch.where(live, c, 0.0)
        c = c / c.sum(1, keepdim=True)
    if bias is not None:
        c = c + bias.double()
    c = torch.where(live, c, -math.inf)
    if case["groups"] > 1:
        t, e = c.shape
        parts = c.reshape(t, case["groups"], e // case["groups"])
        best = parts.sort(dim=2, descending=True)[0][:, :, :case["best"]]
        total = torch.where(best > -math.inf, best, 0.0).sum(2)
        total = torch.where(best[:, :, 0] > -math.inf, total, -math.inf)
        kept = total.sort(dim=1, descending=True, stable=True)[1][:, :case["kept"]]
        keep = torch.zeros_like(total, dtype=torch.bool).scatter_(1, kept, True)
        c = torch.where(keep[:, :, None], parts, -math.inf).reshape(t, e)
    value, at = c.sort(dim=1, descending=True, stable=True)
    return torch.where(value > -math.inf, at, -1)[:, :case["top"]].contiguous()


def _plain_route(s):
    case = s["case"]
    z = s["logits"].float()
    ids = _choose(case, s["logits"], s["bias"])
    live = ids >= 0
    at = ids.clamp(min=0)
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-z))
    else:
        top = z.amax(1, keepdim=True)
        p = torch.exp(z - torch.where(top > -math.inf, top, 0.0))
        p = p / p.sum(1, keepdim=True).clamp(min=1e-30)
    r = torch.where(live, p.gather(1, at), 0.0)
    total = r.sum(1, keepdim=True).clamp(min=1e-30)
    if case["renormalize"]:
        r = r / total
    out = dict(ids=ids, weights=r * s["scale"])
    if case["grad"]:
        dr = torch.where(live, s["dweights"], 0.0) * s["scale"]
        if case["renormalize"]:
            dr = (dr - (r * dr).sum(1, keepdim=True)) / total
        dp = torch.zeros_like(p).scatter_add_(1, at, torch.where(live, dr, 0.0))
        if case["score"] == "sigmoid":
            dz = dp * p * (1.0 - p)
        else:
            dz = p * (dp - (p * dp).sum(1, keepdim=True))
        out["dlogits"] = dz.to(s["logits"].dtype)
    return out


def _plain_entropy(s):
    case, dtype = s["case"], s["x"].dtype
    x, w, targets = s["x"].float(), s["w"].float(), s["targets"]
    live = (targets >= 0) & (targets < case["classes"])
    at = torch.where(live, targets, 0)[:, None]
    z = x @ w.t()
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
    out = dict(loss=torch.where(live, lse - z.gather(1, at)[:, 0], 0.0), lse=lse)
    if case["grad"]:
        b = torch.where(live, s["dloss"], 0.0)
        a = b if s["dlse"] is None else b + s["dlse"]
        dz = torch.exp(z.sub_(lse[:, None])).mul_(a[:, None])
        dz.scatter_add_(1, at, -b[:, None])
        out["dx"], out["dw"] = (dz @ w).to(dtype), (dz.t() @ x).to(dtype)
    return out


# ------------------------------------------------------- the framework's


def _own_embed(s):
    from nearest_centroid_assignment_amd import layers

    out = dict(y=layers.embed(s["ids"], s["w"], scale=s["scale"]))
    if s["case"]["grad"]:
        out["dw"] = layers.embed_backward(s["dy"], s["ids"], s["case"]["classes"], scale=s["scale"])
    return out


def _own_norm(s):
    from nearest_centroid_assignment_amd import layers

    if not s["case"]["grad"]:
        return dict(y=layers.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS))
    y, mean, rstd = layers.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, save_stats=True)
    dx, dweight, dbias = layers.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd,
                                                    need_dbias=s["bias"] is not None)
    out = dict(y=y, mean=mean, rstd=rstd, dx=dx, dweight=dweight)
    if s["bias"] is not None:
        out["dbias"] = dbias
    return out


def _own_route(s):
    from nearest_centroid_assignment_amd import layers

    case = s["case"]
    ids, weights = layers.route(s["logits"], case["top"], score=case["score"], bias=s["bias"],
                                groups=case["groups"], top_groups=case["kept"], group_best=case["best"],
                                renormalize=case["renormalize"], scale=s["scale"])
    out = dict(ids=ids, weights=weights)
    if case["grad"]:
        out["dlogits"] = layers.route_backward(s["dweights"], s["logits"], ids, score=case["score"],
                                               renormalize=case["renormalize"], scale=s["scale"])
    return out


def _own_entropy(s):
    from nearest_centroid_assignment_amd import layers

    loss, lse = layers.cross_entropy(s["x"], s["w"], s["targets"])
    out = dict(loss=loss, lse=lse)
    if s["case"]["grad"]:
        out["dx"], out["dw"] = layers.cross_entropy_backward(s["dloss"], s["x"], s["w"], s["targets"], lse,
                                                             dlse=s["dlse"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"embed": _own_embed, "norm": _own_norm, "route": _own_route, "entropy": _own_entropy}[op](state)
    return {"embed": _plain_embed, "norm": _plain_norm, "route": _plain_route,
            "entropy": _plain_entropy}[op](state)


# ------------------------------------------------------------------- work


def work(case):
    b = {"float32": 4, "bfloat16": 2, "float16": 2}[case["dtype"]]
    if case["op"] == "embed":
        t, v, d = case["tokens"], case["classes"], case["width"]
        hit = float((1.0 - (1.0 - _frequency(v, "cpu")) ** t).sum())  # rows of the table that come up
        nbytes, flops = 8 * t + (hit + t) * d * b, t * d
        if case["grad"]:
            nbytes, flops = nbytes + (t + v) * d * b, flops + 2 * t * d
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "norm":
        r, d = case["rows"], case["width"]
        params = d * (4 if case["wide"] else b) * (2 if case["bias"] else 1)
        nbytes, flops = 2 * r * d * b + params, 7 * r * d
        if case["grad"]:
            nbytes, flops = nbytes + 2 * r * d * b + 8 * r + params, flops + 15 * r * d
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top"]
        nbytes, flops = t * e * b + 12 * t * k + (4 * e if case["biased"] else 0), 6 * t * e
        if case["grad"]:
            nbytes, flops = nbytes + 4 * t * k + t * e * b, flops + 6 * t * e
        return {"bytes": nbytes, "flops": flops}
    r, v, d = case["rows"], case["classes"], case["width"]
    nbytes, flops = (r + v) * d * b + 16 * r, 2.0 * r * v * d
    if case["grad"]:
        nbytes, flops = nbytes + (r + v) * d * b + 4 * r * (2 if case["lse_grad"] else 1), 3 * flops
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------- the definitions, in 64 bits


def _exact_embed(case, s):
    ids = s["ids"]
    at = ((ids >= 0) & (ids < case["classes"])).nonzero()[:, 0]
    y = torch.zeros((case["tokens"], case["width"]), dtype=torch.float64, device=DEV)
    y[at] = s["w"][ids[at]].double() * s["scale"]
    out = dict(y=y)
    if case["grad"]:
        dw = torch.zeros((case["classes"], case["width"]), dtype=torch.float64, device=DEV)
        out["dw"] = dw.index_add_(0, ids[at], s["dy"][at].double()) * s["scale"]
    return out


def _exact_norm(case, s):
    x, weight = s["x"].double(), s["weight"].double()
    var, mean = torch.var_mean(x, 1, correction=0)
    sigma = torch.sqrt(var + EPS)
    h = (x - mean[:, None]) / sigma[:, None]
    out = dict(y=h * weight if s["bias"] is None else h * weight + s["bias"].double())
    if case["grad"]:
        dy, n = s["dy"].double(), case["width"]
        g = dy * weight
        dx = (n * g - g.sum(1)[:, None] - h * torch.linalg.vecdot(g, h)[:, None]) / (n * sigma[:, None])
        out.update(mean=mean, rstd=1.0 / sigma, dx=dx, dweight=torch.linalg.vecdot(dy, h, dim=0))
        if s["bias"] is not None:
            out["dbias"] = dy.sum(0)
    return out


def _exact_route(case, s):
    z = s["logits"].double()
    t, e = z.shape
    masked = torch.isneginf(z)
    p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(z, 1), nan=0.0)
    c = (p if s["bias"] is None else p + s["bias"].double()).masked_fill(masked, -math.inf)
    if case["groups"] > 1:
        size = e // case["groups"]
        rank = []
        for i in range(case["groups"]):
            part = c[:, i * size:(i + 1) * size]
            first = part.max(1)
            if case["best"] == 2 and size > 1:
                second = part.scatter(1, first.indices[:, None], -math.inf).amax(1)
                rank.append(first.values + torch.where(torch.isneginf(second), 0.0, second))
            else:
                rank.append(first.values)
        rank = torch.stack(rank, 1)
        for i in range(case["groups"]):  # a group stays if fewer than `kept` come before it
            before = (rank > rank[:, i:i + 1]).sum(1) + (rank[:, :i] == rank[:, i:i + 1]).sum(1)
            c[before >= case["kept"], i * size:(i + 1) * size] = -math.inf
    ids, rows = [], torch.arange(t, device=DEV)
    for _ in range(case["top"]):  # the first of the largest, taken out, and again
        best = c.amax(1)
        at = (c == best[:, None]).to(torch.int8).argmax(1)
        ids.append(torch.where(torch.isneginf(best), -1, at))
        c[rows, at] = -math.inf
    ids = torch.stack(ids, 1)
    chosen = torch.zeros((t, e + 1), dtype=torch.bool, device=DEV).scatter_(1, torch.where(ids < 0, e, ids), True)[:, :e]
    denom = (p * chosen).sum(1, keepdim=True) if case["renormalize"] else torch.ones(t, 1, dtype=torch.float64, device=DEV)
    denom = torch.where(denom == 0, 1.0, denom)
    share = p * chosen / denom * s["scale"]
    pick = lambda v: torch.where(ids < 0, 0.0, v.gather(1, ids.clamp(min=0)))  # noqa: E731
    out = dict(ids=ids, weights=pick(share))
    if case["grad"]:
        g = torch.zeros((t, e + 1), dtype=torch.float64, device=DEV)
        g = g.scatter_(1, torch.where(ids < 0, e, ids), s["dweights"].double())[:, :e] * chosen
        inner = (share * g).sum(1, keepdim=True)  # over the chosen
        if case["renormalize"]:
            slope = 1.0 - p if case["score"] == "sigmoid" else torch.ones_like(p)
            out["dlogits"] = share * slope * (g - inner / s["scale"])
        elif case["score"] == "sigmoid":
            out["dlogits"] = share * (1.0 - p) * g
        else:
            out["dlogits"] = share * g - p * inner
    return out


def _exact_entropy(case, s):
    if case["rows"] * case["classes"] > 2 ** 29 + 2 ** 20:
        return None
    x, w, targets = s["x"].double(), s["w"].double(), s["targets"]
    rows = ((targets >= 0) & (targets < case["classes"])).nonzero()[:, 0]
    z = x @ w.t()
    lse = torch.logsumexp(z, 1)
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - z[rows, targets[rows]]
    out = dict(loss=loss, lse=lse)
    if case["grad"]:
        z = torch.exp(z.sub_(lse[:, None]))
        outer = torch.zeros_like(lse)
        outer[rows] = s["dloss"][rows].double()
        back = outer.clone()
        if s["dlse"] is not None:
            outer = outer + s["dlse"].double()
        z *= outer[:, None]
        z[rows, targets[rows]] -= back[rows]
        out["dx"], out["dw"] = z @ w, z.t() @ x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "norm": _exact_norm, "route": _exact_route,
            "entropy": _exact_entropy}[case["op"]](case, s)
