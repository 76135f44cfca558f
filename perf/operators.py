"""Cases of the expert operators: what is timed, in the framework's kernels and in plain torch.

Three operators that train and run a mixture of experts whose router is a
nearest-centroid assignment (or any other source of expert numbers):

  tokens   (token, expert) pairs sorted by expert, the token rows gathered in
           that order, the experts' rows summed back with weights; gradients
  linear   act(x w^T + b) + residual, for all rows or per expert; gradients
  adamw    one AdamW step over many tensors, moments in 32 or in 8 bits

With ``own`` false, ``run`` computes the plain form: elementary torch
operations in float32, rounded once where the operator returns. With ``own``
true it calls ``nearest_centroid_assignment_amd.experts``.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BLOCK = 256  # values that share a scale in an 8-bit moment
GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715


# ------------------------------------------------------------------- cases


def listed():
    return [
        # A decoding step of 8 sequences: two experts of 64 for each token. Latency.
        dict(name="tokens decode bf16", op="tokens", tokens=8, top=2, experts=64, width=2048,
             dtype="bfloat16", drop=0.0, grad=False),
        # The probe workload's samples grouped by their nearest centroid (one label a row).
        dict(name="tokens probe f32", op="tokens", tokens=4096, top=1, experts=256, width=512,
             dtype="float32", drop=0.0, grad=True),
        # Odd sizes, a width that is not a multiple of any vector, pairs dropped by a capacity rule.
        dict(name="tokens odd f16", op="tokens", tokens=5003, top=3, experts=17, width=1001,
             dtype="float16", drop=0.1, grad=True),
        # A training batch at the mid workload's size, two of 1024 experts for each sample.
        dict(name="tokens train bf16", op="tokens", tokens=65536, top=2, experts=1024, width=2048,
             dtype="bfloat16", drop=0.0, grad=True),
        # One token through a wide layer: the weights are read once. Latency and bandwidth.
        dict(name="linear token bf16", op="linear", rows=1, outs=8192, ins=2048, experts=0,
             dtype="bfloat16", act="gelu_tanh", residual=True, inner=False, drop=0.0, grad=False),
        # The 16 pairs of a decoding step through their experts of 64.
        dict(name="linear decode bf16", op="linear", rows=16, outs=4096, ins=2048, experts=64,
             dtype="bfloat16", act="silu", residual=False, inner=False, drop=0.0, grad=False),
        # float32 samples as the rest of the framework has them, odd sizes, trained.
        dict(name="linear odd f32", op="linear", rows=1000, outs=1111, ins=777, experts=0,
             dtype="float32", act="relu", residual=True, inner=False, drop=0.0, grad=True),
        # A dense layer of a training step: forward and backward.
        dict(name="linear train bf16", op="linear", rows=8192, outs=8192, ins=2048, experts=0,
             dtype="bfloat16", act="gelu_tanh", residual=False, inner=False, drop=0.0, grad=True),
        # The experts' second product, ragged row counts; its input's activation is differentiated with it.
        dict(name="linear experts f16", op="linear", rows=32768, outs=2048, ins=4096, experts=17,
             dtype="float16", act="none", residual=False, inner=True, drop=0.02, grad=True),
        # A small model's step: many short tensors, where launches count.
        dict(name="adamw small f32", op="adamw", tensors=10, largest=32768, bits=32,
             param="float32", grad_type="float32", copy=False),
        # The weights of experts of a training run: float32 masters, bfloat16 gradients and copies.
        dict(name="adamw large f32", op="adamw", tensors=12, largest=67108864, bits=32,
             param="float32", grad_type="bfloat16", copy=True),
        # The same with moments in 8 bits; the step and the export of its moments.
        dict(name="adamw large 8 bit", op="adamw", tensors=12, largest=67108864, bits=8,
             param="float32", grad_type="bfloat16", copy=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A size of the range: half of them multiples of 64, the others as they fall."""
    v = _log(rng, lo, hi)
    return max(lo, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(("tokens", "linear", "linear", "adamw"))
    dtype = rng.choice(("bfloat16", "bfloat16", "float16", "float32"))
    if op == "tokens":
        width = _width(rng, 64, 8192)
        most = 65536 * 2 * 2048 // (2 if dtype == "float32" else 1)
        top = rng.choice((1, 2, 2, 3, 4, 8))
        tokens = _log(rng, 1, max(1, min(65536, most // (width * top))))
        return dict(op=op, tokens=tokens, top=top, experts=_log(rng, 8, 1024), width=width,
                    dtype=dtype, drop=rng.choice((0.0, 0.0, 0.1)), grad=rng.random() < 0.7)
    if op == "linear":
        experts = rng.choice((0, 0, _log(rng, 2, 64)))
        rows, outs, ins = _log(rng, 1, 16384), _width(rng, 64, 8192), _width(rng, 64, 8192)
        most = 8192 * 8192 * 2048 // (8 if dtype == "float32" else 1)
        while rows * outs * ins > most:
            rows //= 2
        while experts * outs * ins > 2 ** 28:
            experts //= 2
        grad = rng.random() < 0.6
        inner = experts > 1 and grad and rng.random() < 0.5
        return dict(op=op, rows=rows, outs=outs, ins=ins, experts=experts if experts > 1 else 0,
                    dtype=dtype, act="none" if inner else rng.choice(("none", "relu", "silu", "gelu_tanh")),
                    residual=rng.random() < 0.5, inner=inner, drop=rng.choice((0.0, 0.05)) if experts > 1 else 0.0,
                    grad=grad)
    return dict(op=op, tensors=rng.randint(1, 12), largest=_log(rng, 300, 67108864),
                bits=rng.choice((8, 32)), param=rng.choice(("float32", "float32", "bfloat16")),
                grad_type=rng.choice(("float32", "bfloat16", "float16")), copy=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(scale).to(dtype)


def _expert_ids(g, pairs, experts, drop):
    """Expert numbers with the uneven loads that routers give; dropped pairs are -1."""
    load = torch.randn(experts, generator=g, device=DEV).mul_(0.4).exp_()
    edges = (load / load.sum()).cumsum(0)
    ids = torch.searchsorted(edges, torch.rand(pairs, generator=g, device=DEV)).clamp_(max=experts - 1)
    if drop:
        ids = torch.where(torch.rand(pairs, generator=g, device=DEV) < drop, -1, ids)
    return ids


def _sizes(case):
    """Lengths of the tensors of an adamw case: matrices of falling size and short vectors."""
    n, big = case["tensors"], case["largest"]
    return [max(1, big >> (i // 3)) if i % 3 == 0 else max(1, (big >> (i // 3)) // 2 + 17 * i)
            if i % 3 == 1 else max(1, int(math.sqrt(big)) // 2 + 5 * i) for i in range(n)]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "tokens":
        dtype, t, k = TYPES[case["dtype"]], case["tokens"], case["top"]
        ids = _expert_ids(g, t * k, case["experts"], case["drop"]).reshape(t, k)
        rows = t * k
        s = dict(ids=ids, x=_randn(g, (t, case["width"]), dtype), ys=_randn(g, (rows, case["width"]), dtype),
                 weights=torch.softmax(torch.randn((t, k), generator=g, device=DEV), 1))
        if case["grad"]:
            s["dy"] = _randn(g, (t, case["width"]), dtype)
            s["dxs"] = _randn(g, (rows, case["width"]), dtype)
    elif op == "linear":
        dtype, r, n, k, e = TYPES[case["dtype"]], case["rows"], case["outs"], case["ins"], case["experts"]
        s = dict(w=_randn(g, (e, n, k) if e else (n, k), dtype, 1.0 / math.sqrt(k)),
                 bias=_randn(g, (e, n) if e else (n,), dtype, 0.1), offsets=None, residual=None)
        if e:
            ids = _expert_ids(g, r, e, case["drop"])
            counts = (ids[:, None] == torch.arange(e, device=DEV)).sum(0)
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            s["capacity"] = max(1, int(counts.max()))
        x = _randn(g, (r, k), torch.float32)
        if case["inner"]:
            s["in_pre"] = x.to(dtype)
            x = _act(s["in_pre"].float(), "silu")
        s["x"] = x.to(dtype)
        if case["residual"]:
            s["residual"] = _randn(g, (r, n), dtype)
        if case["grad"]:
            s["dy"] = _randn(g, (r, n), dtype)
    else:
        sizes = _sizes(case)
        padded = [-(-v // BLOCK) * BLOCK for v in sizes]
        total = sum(padded)
        s = dict(params=[_randn(g, v, TYPES[case["param"]], 0.02) for v in sizes],
                 grads=[_randn(g, v, TYPES[case["grad_type"]], 1e-3) for v in sizes],
                 copies=None, padded=padded, m_scale=None, v_scale=None,
                 grad_scale=torch.full((1,), 0.7, device=DEV))
        if case["copy"]:
            s["copies"] = [p.to(torch.bfloat16) for p in s["params"]]
        m = torch.randn(total, generator=g, device=DEV).mul_(2e-4)
        v = torch.randn(total, generator=g, device=DEV).mul_(1e-3).square_()
        at = 0
        for size, room in zip(sizes, padded):  # what pads a tensor to whole blocks is zero
            m[at + size:at + room] = 0.0
            v[at + size:at + room] = 0.0
            at += room
        if case["bits"] == 8:
            s["m"], s["m_scale"] = _encode_m(m)
            s["v"], s["v_scale"] = _encode_v(v)
        else:
            s["m"], s["v"] = m, v
        s["hyper"] = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, step=100)
    s["case"] = dict(case)
    return s


# ------------------------------------------------- the plain form, float32


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(GELU_A * (z + GELU_B * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu_tanh":
        t = torch.tanh(GELU_A * (z + GELU_B * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * (GELU_A * (1.0 + 3.0 * GELU_B * z * z))
    return torch.ones_like(z)


def _plain_plan(ids, experts):
    """order: the pair at each sorted place (-1 past the last); place: a pair's sorted place (-1 if dropped)."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    ranked, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ranked, torch.arange(experts + 1, device=flat.device))
    at = torch.arange(flat.numel(), device=flat.device)
    place = torch.empty_like(order).scatter_(0, order, at)
    place = torch.where(key < experts, place, -1).reshape(ids.shape)
    order = torch.where(at < offsets[-1], order, -1)
    return order.to(torch.int32), place.to(torch.int32), offsets.to(torch.int32)


def _gathered(rows, at):
    """rows[at] in float32, zero where at is negative."""
    got = rows[at.clamp(min=0).long()].float()
    return torch.where((at >= 0).unsqueeze(-1), got, torch.zeros_like(got))


def _plain_tokens(s):
    case, dtype = s["case"], s["x"].dtype
    order, place, offsets = _plain_plan(s["ids"], case["experts"])
    token = torch.where(order >= 0, torch.div(order, case["top"], rounding_mode="floor"), -1)
    out = dict(order=order, place=place, offsets=offsets, xs=_gathered(s["x"], token).to(dtype),
               y=(_gathered(s["ys"], place) * s["weights"].unsqueeze(-1)).sum(1).to(dtype))
    if case["grad"]:
        out["dx"] = _gathered(s["dxs"], place).sum(1).to(dtype)
        weight = torch.where(order >= 0, s["weights"].reshape(-1)[order.clamp(min=0).long()], 0.0)
        out["dys"] = (_gathered(s["dy"], token) * weight.unsqueeze(-1)).to(dtype)
        out["dweights"] = (_gathered(s["ys"], place) * s["dy"].float().unsqueeze(1)).sum(2)
    return out


def _pages(s):
    """The row at each (expert, slot) of a padded batch (-1: none), and the (expert, slot) of each row."""
    offsets, e, cap, r = s["offsets"].long(), s["case"]["experts"], s["capacity"], s["case"]["rows"]
    at = offsets[:-1, None] + torch.arange(cap, device=offsets.device)
    at = torch.where(at < offsets[1:, None], at, -1)
    row = torch.arange(r, device=offsets.device)
    owner = torch.searchsorted(offsets, row, right=True) - 1
    live = row < offsets[-1]
    owner = torch.where(live, owner, 0)
    slot = torch.where(live, owner * cap + row - offsets[owner], -1)
    return at, slot


def _plain_linear(s):
    case, dtype = s["case"], s["x"].dtype
    w, bias = s["w"].float(), s["bias"].float()
    if case["experts"]:
        at, slot = _pages(s)
        x = _gathered(s["x"], at)
        z = torch.baddbmm(bias.unsqueeze(1), x, w.transpose(1, 2))
        flat = lambda v: _gathered(v.reshape(-1, v.shape[-1]), slot)  # noqa: E731
        live = (slot >= 0).unsqueeze(-1)
    else:
        x = s["x"].float()
        z = torch.addmm(bias, x, w.t())
        flat = lambda v: v  # noqa: E731
        live = None
    z = flat(z)
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if live is not None:
        y = torch.where(live, y, torch.zeros_like(y))
    out = dict(y=y.to(dtype))
    if case["grad"]:
        dz = s["dy"].float()
        if case["act"] != "none":
            out["pre"] = z.to(dtype)  # an output of the forward call, and what the backward call is given
            dz = dz * _act_slope(out["pre"].float(), case["act"])
        if case["experts"]:
            dz = _gathered(dz, at)
            dx = flat(torch.bmm(dz, w))
            out["dw"] = torch.bmm(dz.transpose(1, 2), x).to(dtype)
            out["dbias"] = dz.sum(1).to(dtype)
        else:
            dx = dz @ w
            out["dw"] = (dz.t() @ x).to(dtype)
            out["dbias"] = dz.sum(0).to(dtype)
        if case["inner"]:
            dx = dx * _act_slope(s["in_pre"].float(), "silu")
        out["dx"] = dx.to(dtype)
    return out


def _decode_m(q, scale):
    t = q.float() * (1.0 / 127.0)
    return ((t * t.abs()).reshape(-1, BLOCK) * scale[:, None]).reshape(-1)


def _encode_m(m):
    b = m.reshape(-1, BLOCK)
    scale = b.abs().amax(1)
    r = b / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
    q = torch.round(torch.sqrt(r.abs()) * 127.0) * torch.sign(r)
    return q.to(torch.int8).reshape(-1), scale


def _decode_v(q, scale):
    t = q.float() * (1.0 / 255.0)
    t = t * t
    return ((t * t).reshape(-1, BLOCK) * scale[:, None]).reshape(-1)


def _encode_v(v):
    b = v.reshape(-1, BLOCK)
    scale = b.amax(1)
    r = b / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
    q = torch.round(torch.sqrt(torch.sqrt(r)) * 255.0)
    q = torch.where(b > 0, torch.clamp(q, min=1.0), q)
    return q.to(torch.uint8).reshape(-1), scale


def _factors(h):
    b1, b2 = h["betas"]
    rate = h["lr"] / (1.0 - b1 ** h["step"])
    return b1, 1.0 - b1, b2, 1.0 - b2, 1.0 - h["lr"] * h["weight_decay"], rate, \
        1.0 / math.sqrt(1.0 - b2 ** h["step"]), h["eps"]


def _plain_adamw(s):
    case = s["case"]
    b1, c1, b2, c2, keep, rate, root, eps = _factors(s["hyper"])
    sizes = [p.numel() for p in s["params"]]
    m, v = s["m"], s["v"]
    if case["bits"] == 8:
        m, v = _decode_m(m, s["m_scale"]), _decode_v(v, s["v_scale"])
    g = torch.cat([torch.nn.functional.pad(x.float(), (0, room - x.numel())) for x, room in zip(s["grads"], s["padded"])])
    p = torch.cat([torch.nn.functional.pad(x.float(), (0, room - x.numel())) for x, room in zip(s["params"], s["padded"])])
    g = g * s["grad_scale"]
    m = m * b1 + g * c1
    v = v * b2 + (g * g) * c2
    p = p * keep - (m * rate) / (torch.sqrt(v) * root + eps)
    if case["bits"] == 8:
        for name, (q, scale) in (("m", _encode_m(m)), ("v", _encode_v(v))):
            s[name].copy_(q)
            s[name + "_scale"].copy_(scale)
        m, v = _decode_m(s["m"], s["m_scale"]), _decode_v(s["v"], s["v_scale"])
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    new = [x[:size] for x, size in zip(p.split(s["padded"]), sizes)]
    torch._foreach_copy_(s["params"], new)
    if s["copies"] is not None:
        torch._foreach_copy_(s["copies"], new)
    return dict(params=s["params"], copies=s["copies"], m=m, v=v)


# ------------------------------------------------------- the framework's


def _own_tokens(s):
    from nearest_centroid_assignment_amd import experts

    plan = experts.plan(s["ids"], s["case"]["experts"])
    out = dict(order=plan.order, place=plan.place, offsets=plan.offsets,
               xs=experts.dispatch(s["x"], plan), y=experts.combine(s["ys"], s["weights"], plan))
    if s["case"]["grad"]:
        out["dx"] = experts.dispatch_backward(s["dxs"], plan)
        out["dys"], out["dweights"] = experts.combine_backward(s["dy"], s["ys"], s["weights"], plan)
    return out


def _own_linear(s):
    from nearest_centroid_assignment_amd import experts

    case = s["case"]
    keep = case["grad"] and case["act"] != "none"
    y = experts.linear(s["x"], s["w"], s["bias"], residual=s["residual"], act=case["act"],
                       offsets=s["offsets"], save_pre=keep)
    out = {}
    if keep:
        y, out["pre"] = y
    out["y"] = y
    if case["grad"]:
        out["dx"], out["dw"], out["dbias"] = experts.linear_backward(
            s["dy"], s["x"], s["w"], pre=out.get("pre"), act=case["act"], offsets=s["offsets"],
            in_pre=s.get("in_pre"), in_act="silu" if case["inner"] else "none")
    return out


def _own_adamw(s):
    from nearest_centroid_assignment_amd import experts

    experts.adamw_step(s["params"], s["grads"], s["m"], s["v"], m_scale=s["m_scale"], v_scale=s["v_scale"],
                       copies=s["copies"], grad_scale=s["grad_scale"], **s["hyper"])
    m, v = s["m"], s["v"]
    if s["case"]["bits"] == 8:
        m, v = experts.adamw_moments(m, v, s["m_scale"], s["v_scale"])
    return dict(params=s["params"], copies=s["copies"], m=m, v=v)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tokens": _own_tokens, "linear": _own_linear, "adamw": _own_adamw}[op](state)
    return {"tokens": _plain_tokens, "linear": _plain_linear, "adamw": _plain_adamw}[op](state)


# ------------------------------------------------------------------- work


def work(case):
    size = lambda name: {"float32": 4, "bfloat16": 2, "float16": 2}[name]  # noqa: E731
    if case["op"] == "tokens":
        t, k, d, b = case["tokens"], case["top"], case["width"], size(case["dtype"])
        rows = t * k
        tok, row = t * d * b, rows * d * b
        nbytes = 16 * rows + 4 * case["experts"] + tok + row + row + tok + 4 * rows
        flops = 2 * rows * d
        if case["grad"]:  # dxs, ys (with its forward read), dy in; dx, dys, dweights out
            nbytes += row + tok + tok + row + 4 * rows
            flops += 4 * rows * d
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "linear":
        r, n, k, b = case["rows"], case["outs"], case["ins"], size(case["dtype"])
        e = case["experts"]
        live = r * (1.0 - case["drop"])
        hit = min(e, live) if e else 1  # experts with a row at most
        nbytes = (r * k + hit * n * (k + 1) + r * n * (2 if case["residual"] else 1)) * b
        flops = 2 * live * n * k
        if case["grad"]:
            nbytes += (r * n + (e or 1) * n * (k + 1) + r * k * (2 if case["inner"] else 1)
                       + (r * n if case["act"] != "none" else 0)) * b
            flops *= 3
        return {"bytes": nbytes, "flops": flops}
    total = sum(_sizes(case))
    moments = 16 if case["bits"] == 32 else 4 + 8 + 16.0 / BLOCK  # 8 bits: read, written, exported
    return {"bytes": total * (2 * size(case["param"]) + size(case["grad_type"]) + moments + (2 if case["copy"] else 0)),
            "flops": 16 * total}


# ------------------------------------------- the definitions, in 64 bits


def _exact_tokens(case, s):
    e, top = case["experts"], case["top"]
    ids = s["ids"].cpu().reshape(-1).tolist()
    groups = [[] for _ in range(e)]
    for pair, expert in enumerate(ids):
        if 0 <= expert < e:
            groups[expert].append(pair)
    order = [pair for group in groups for pair in group]
    place = [-1] * len(ids)
    for at, pair in enumerate(order):
        place[pair] = at
    starts = [0]
    for group in groups:
        starts.append(starts[-1] + len(group))
    live = torch.tensor(order, dtype=torch.long, device=DEV)
    token, n = live // top, len(order)
    x, ys, weights = s["x"].double(), s["ys"].double(), s["weights"].double().reshape(-1)
    rows = len(ids)

    def spread(v):
        full = torch.zeros((rows, v.shape[1]), dtype=torch.float64, device=DEV)
        full[:n] = v
        return full

    def gather(v):
        total = torch.zeros_like(x)
        return total.index_add_(0, token, v)

    out = dict(order=torch.tensor(order + [-1] * (rows - n), dtype=torch.int32, device=DEV),
               place=torch.tensor(place, dtype=torch.int32, device=DEV).reshape(s["ids"].shape),
               offsets=torch.tensor(starts, dtype=torch.int32, device=DEV),
               xs=spread(x[token]), y=gather(ys[:n] * weights[live, None]))
    if case["grad"]:
        dy = s["dy"].double()
        out["dx"] = gather(s["dxs"][:n].double())
        out["dys"] = spread(dy[token] * weights[live, None])
        dw = torch.zeros(rows, dtype=torch.float64, device=DEV)
        dw[live] = (dy[token] * ys[:n]).sum(1)
        out["dweights"] = dw.reshape(s["weights"].shape)
    return out


def _exact_linear(case, s):
    def slope(z, act):
        z = z.detach().requires_grad_(True)
        with torch.enable_grad():
            return torch.autograd.grad(_exact_act(z, act).sum(), z)[0] if act != "none" else torch.ones_like(z)

    bounds = s["offsets"].cpu().tolist() if case["experts"] else [0, case["rows"]]
    w = s["w"] if case["experts"] else s["w"][None]
    bias = s["bias"] if case["experts"] else s["bias"][None]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=DEV)  # noqa: E731
    r, n, k = case["rows"], case["outs"], case["ins"]
    out = dict(y=new(r, n))
    grad = case["grad"]
    keep = grad and case["act"] != "none"
    if keep:
        out["pre"] = new(r, n)
    if grad:
        out.update(dx=new(r, k), dw=new(*w.shape), dbias=new(*bias.shape))
    for e, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        if lo == hi:
            continue
        x, we = s["x"][lo:hi].double(), w[e].double()
        z = x @ we.t() + bias[e].double()
        out["y"][lo:hi] = _exact_act(z, case["act"])
        if s["residual"] is not None:
            out["y"][lo:hi] += s["residual"][lo:hi].double()
        if keep:
            out["pre"][lo:hi] = z
        if grad:
            dz = s["dy"][lo:hi].double() * slope(z, case["act"])
            dx = dz @ we
            out["dx"][lo:hi] = dx * slope(s["in_pre"][lo:hi].double(), "silu") if case["inner"] else dx
            out["dw"][e] = dz.t() @ x
            out["dbias"][e] = dz.sum(0)
    if grad and not case["experts"]:
        out["dw"], out["dbias"] = out["dw"][0], out["dbias"][0]
    return out


def _exact_act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def _exact_adamw(case, s):
    h = s["hyper"]
    b1, b2 = h["betas"]
    codes = case["bits"] == 8
    out = dict(params=[], copies=None if s["copies"] is None else [], m=[], v=[])
    at = 0
    for p, g, room in zip(s["params"], s["grads"], s["padded"]):
        n = p.numel()
        here = slice(at, at + room)
        blocks = slice(at // BLOCK, (at + room) // BLOCK)
        m, v = s["m"][here].double(), s["v"][here].double()
        if codes:
            m = (m / 127) * (m / 127).abs() * s["m_scale"][blocks].double().repeat_interleave(BLOCK)
            v = (v / 255) ** 4 * s["v_scale"][blocks].double().repeat_interleave(BLOCK)
        g = torch.cat([g.double() * s["grad_scale"].double(), g.new_zeros(room - n, dtype=torch.float64)])
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g ** 2
        step = m / (1 - b1 ** h["step"]) / ((v / (1 - b2 ** h["step"])).sqrt() + h["eps"])
        new = p.double() * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * step[:n]
        out["params"].append(new)
        if out["copies"] is not None:
            out["copies"].append(new)
        # An 8-bit moment has no exact value: which of two codes a value that lies between them
        # gets is settled by the last bit of the float32 arithmetic.
        out["m"].append(m)
        out["v"].append(v)
        at += room
    out["m"] = None if codes else torch.cat(out["m"])
    out["v"] = None if codes else torch.cat(out["v"])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"tokens": _exact_tokens, "linear": _exact_linear, "adamw": _exact_adamw}[case["op"]](case, s)
