"""Cases for measuring projections with low-rank adapters and the expert router.

``listed()`` names fixed cases, ``draw(rng)`` gives more of the same ranges.
``prepare(case, seed)`` makes a case's inputs on the GPU, ``run(state)`` is one
pass (plain torch in fp32, or this package's kernels where ``own`` is true),
``work(case)`` what the pass cannot do without, and ``exact(case, seed)`` its
result in 64 bits.

Operators (``op``):

- ``lora``     out[t] = x[t] @ w^T + bias + scale[l] * (x[t] @ A[l]^T) @ B[l]^T, l the
               adapter of row t (none: the projection alone); with ``grad`` the
               gradients of x and of every adapter's A and B too
- ``route``    the top_k largest probabilities softmax(logits[t]), renormalised or
               not, and their experts
- ``balance``  counts[e] = choices of expert e, the loss coef * E * sum_e f[e] P[e]
               with f the share of the choices and P the mean probability, and its
               gradient; tokens that are padding take no part
- ``router``   a training step's route and balance, and one gradient of the
               logits through both
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ES = {"bf16": 2, "f16": 2, "f32": 4}
COEF = 0.01


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request's decode step through a projection
        {"name": "adapters one token", "op": "lora", "t": 1, "n": 4096, "k": 4096, "l": 8, "r": 16, "dt": "bf16", "out": "bf16", "runs": False, "bias": False, "grad": False},
        # a decode step of many requests, about as many adapters
        {"name": "adapters decode batch", "op": "lora", "t": 64, "n": 4096, "k": 4096, "l": 64, "r": 16, "dt": "bf16", "out": "bf16", "runs": False, "bias": False, "grad": False},
        # prompts and single tokens mixed, sizes that end inside a tile, logits-like fp32 results
        {"name": "adapters ragged", "op": "lora", "t": 333, "n": 1744, "k": 2064, "l": 5, "r": 24, "dt": "f16", "out": "f32", "runs": True, "bias": True, "grad": False},
        # a prefill batch of several prompts
        {"name": "adapters prefill", "op": "lora", "t": 8192, "n": 4096, "k": 4096, "l": 16, "r": 64, "dt": "bf16", "out": "bf16", "runs": True, "bias": False, "grad": False},
        # a training step of a few adapters at once
        {"name": "adapters training", "op": "lora", "t": 8192, "n": 4096, "k": 4096, "l": 4, "r": 16, "dt": "bf16", "out": "bf16", "runs": True, "bias": False, "grad": True},
        # an odd batch, gradients kept in fp32
        {"name": "adapters training ragged", "op": "lora", "t": 1111, "n": 1528, "k": 2560, "l": 3, "r": 40, "dt": "f16", "out": "f16", "runs": True, "bias": True, "grad": True},
        # a decode step's routing
        {"name": "route decode", "op": "route", "t": 16, "e": 128, "top": 8, "dt": "bf16", "renorm": True},
        # a large prefill batch's routing
        {"name": "route prefill", "op": "route", "t": 32768, "e": 128, "top": 8, "dt": "bf16", "renorm": True},
        # a small training batch's balance
        {"name": "balance small", "op": "balance", "t": 512, "e": 64, "top": 8, "dt": "f32", "pad": 0.0},
        # a large one with many experts, padded sequences
        {"name": "balance padded", "op": "balance", "t": 16411, "e": 256, "top": 8, "dt": "f32", "pad": 0.2},
        # a training step's router
        {"name": "router training", "op": "router", "t": 16384, "e": 64, "top": 6, "dt": "f32", "renorm": False, "pad": 0.1},
    ]


def draw(rng):
    def log(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
        return min(hi, max(lo, int(v) // step * step))

    op = rng.choice(["lora", "lora", "lora", "lora", "route", "balance", "router"])
    if op == "lora":
        grad = rng.random() < 0.4
        n, k = log(64, 8192, 8), log(256, 8192, 8)
        t = min(log(1, 8192), (1 << 37) // (n * k))
        dt = rng.choice(["bf16", "bf16", "f16"])
        r = log(8, 128, 8)
        return {"op": op, "t": t, "n": n, "k": k, "l": log(1, min(64, 1024 // r)), "r": r, "dt": dt, "out": dt if grad or rng.random() < 0.7 else "f32",
                "runs": t > 64 or rng.random() < 0.5, "bias": rng.random() < 0.3, "grad": grad}
    dt = rng.choice(["bf16", "f16", "f32", "f32"])
    t, e = log(1, 32768), log(8, 256)
    top = rng.randint(1, min(8, e))
    if op == "route":
        return {"op": op, "t": t, "e": e, "top": top, "dt": dt, "renorm": rng.random() < 0.7}
    pad = rng.choice([0.0, 0.1, 0.4])
    if op == "balance":
        return {"op": op, "t": t, "e": e, "top": top, "dt": dt, "pad": pad}
    return {"op": op, "t": t, "e": e, "top": top, "dt": dt, "renorm": rng.random() < 0.5, "pad": pad}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, shape, dt=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)


def _adapters_of_rows(case, seed):
    """Adapter of every row: prompts of unequal length one after another
    (``runs``) or a request a row; one in ten requests has none (-1)."""
    g = torch.Generator().manual_seed(seed)
    t, l = case["t"], case["l"]
    if not case["runs"]:
        ids = torch.randint(0, l, (t,), generator=g)
        return torch.where(torch.rand(t, generator=g) < 0.1, -1, ids)
    parts = 2 * l
    cuts = torch.randint(0, t + 1, (parts - 1,), generator=g).sort()[0]
    length = torch.diff(cuts, prepend=torch.zeros(1, dtype=torch.long), append=torch.full((1,), t))
    who = torch.cat([torch.randperm(l, generator=g), torch.randperm(l, generator=g)])
    who = torch.where(torch.rand(parts, generator=g) < 0.1, -1, who)
    return who.repeat_interleave(length)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dt = DT[case["dt"]]
    if case["op"] == "lora":
        t, n, k, l, r = (case[c] for c in "tnklr")
        s["x"] = _normal(g, (t, k), dt)
        s["w"] = _normal(g, (n, k), dt, k ** -0.5)
        s["a"] = _normal(g, (l, r, k), dt, k ** -0.5)
        s["b"] = _normal(g, (l, n, r), dt, 0.1)
        s["ids"] = _adapters_of_rows(case, seed).to("cuda", torch.int32)
        s["scale"] = torch.exp(0.3 * _normal(g, (l,)))
        s["beside"] = _normal(g, (n,), dt, 0.1) if case["bias"] else None
        if case["grad"]:
            s["go"] = _normal(g, (t, n), dt, 0.1)
        return s
    t, e, top = case["t"], case["e"], case["top"]
    # a router's logits: some experts liked by most tokens
    s["logits"] = (_normal(g, (t, e)) * 1.5 + _normal(g, (e,))).to(dt)
    if case["op"] == "route":
        return s
    s["mask"] = None
    if case["pad"]:
        s["mask"] = torch.rand(t, generator=g, device="cuda") >= case["pad"]
    s["gl"] = torch.ones((), device="cuda") + 0.1 * _normal(g, ())
    if case["op"] == "balance":
        s["ids"] = s["logits"].float().argsort(dim=1, descending=True, stable=True)[:, :top].to(torch.int32).contiguous()
    else:
        s["gw"] = _normal(g, (t, top), std=1e-3)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain_lora(s):
    t, n, k, l, r = (s[c] for c in "tnklr")
    dt, res = DT[s["dt"]], DT[s["out"]]
    x, w = s["x"].float(), s["w"].float()
    a = s["a"].float().reshape(l * r, k)
    b = s["b"].float().transpose(1, 2).reshape(l * r, n)
    # every adapter's product, scaled where it is the row's own, zero elsewhere
    of = (s["ids"].long()[:, None] == torch.arange(l, device="cuda")) * s["scale"]
    of = of.repeat_interleave(r, 1)
    v = (x @ a.t()) * of
    out = x @ w.t() + v @ b
    if s["beside"] is not None:
        out = out + s["beside"].float()
    if not s["grad"]:
        return out.to(res)
    go = s["go"].float()
    u = (go @ b.t()) * of
    grad_x = go @ w + u @ a
    grad_a = (u.t() @ x).reshape(l, r, k)
    grad_b = (v.t() @ go).reshape(l, r, n).transpose(1, 2).contiguous()
    return out.to(res), grad_x.to(dt), grad_a, grad_b


def _plain_softmax(logits):
    z = logits.float()
    p = torch.exp(z - z.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _plain_route(s, p):
    ids = s["logits"].float().argsort(dim=1, descending=True, stable=True)[:, : s["top"]]
    w = p.gather(1, ids)
    return ids, w / w.sum(1, keepdim=True) if s["renorm"] else w


def _plain_balance(s, p, ids):
    """Loss, counts and the loss's derivative by every real token's probabilities."""
    e = s["e"]
    real = torch.ones(s["t"], device="cuda") if s["mask"] is None else s["mask"].float()
    counts = ((ids[:, :, None] == torch.arange(e, device="cuda")).sum(1) * real[:, None].long()).sum(0)
    tokens = real.sum().clamp(min=1)
    f = counts.float() / counts.sum().clamp(min=1)
    slopes = COEF * e * f / tokens
    loss = (p * real[:, None]).sum(0) @ slopes
    return loss, counts.to(torch.int32), slopes, real


def _plain(s):
    if s["op"] == "lora":
        return _plain_lora(s)
    p = _plain_softmax(s["logits"])
    if s["op"] == "route":
        ids, w = _plain_route(s, p)
        return w, ids.to(torch.int32)
    if s["op"] == "balance":
        loss, counts, slopes, real = _plain_balance(s, p, s["ids"].long())
        g = s["gl"] * p * (slopes - (p * slopes).sum(1, keepdim=True)) * real[:, None]
        return loss, counts, g.to(DT[s["dt"]])
    ids, w = _plain_route(s, p)
    loss, counts, slopes, real = _plain_balance(s, p, ids)
    if s["renorm"]:
        local = w * (s["gw"] - (s["gw"] * w).sum(1, keepdim=True))
        g = torch.zeros_like(p).scatter(1, ids, local)
    else:
        gp = torch.zeros_like(p).scatter(1, ids, s["gw"])
        g = p * (gp - (p * gp).sum(1, keepdim=True))
    g = (g + s["gl"] * p * (slopes - (p * slopes).sum(1, keepdim=True))) * real[:, None]
    here = real[:, None] > 0
    return torch.where(here, w, 0.0), torch.where(here, ids, -1).to(torch.int32), loss, counts, g.to(DT[s["dt"]])


def _own(s):
    import moe_expert_grouped_amd as mi

    if s["op"] == "lora":
        args = (s["w"], s["a"], s["b"], s["ids"], s["scale"])
        if not s["grad"]:
            return mi.mm_lora(s["x"], *args, bias=s["beside"], out_dtype=DT[s["out"]])
        out, act = mi.mm_lora(s["x"], *args, bias=s["beside"], with_act=True)
        return out, *mi.mm_lora_backward(s["go"], s["x"], *args, act=act, grad_dtype=torch.float32)
    if s["op"] == "route":
        return mi.moe_route_topk(s["logits"], s["top"], renormalize=s["renorm"])
    if s["op"] == "balance":
        loss, counts, slopes = mi.moe_balance_loss(s["logits"], s["ids"], coef=COEF, token_mask=s["mask"])
        return loss, counts, mi.moe_route_backward(s["logits"], slopes=slopes, grad_loss=s["gl"], token_mask=s["mask"])
    w, ids = mi.moe_route_topk(s["logits"], s["top"], renormalize=s["renorm"], token_mask=s["mask"])
    loss, counts, slopes = mi.moe_balance_loss(s["logits"], ids, coef=COEF, token_mask=s["mask"])
    g = mi.moe_route_backward(s["logits"], topk_ids=ids, topk_weights=w, grad_weights=s["gw"], renormalize=s["renorm"], slopes=slopes, grad_loss=s["gl"], token_mask=s["mask"])
    return w, ids, loss, counts, g


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    es = ES[case["dt"]]
    if case["op"] == "lora":
        t, n, k, l, r = (case[c] for c in "tnklr")
        used = min(l, 2 * l * 0.9) if case["runs"] else l * (1 - (1 - 0.9 / l) ** t)
        bank = used * r * (n + k) * es
        small = t * 4 + l * 4 + (n * es if case["bias"] else 0)
        size = t * k * es + n * k * es + bank + small + t * n * ES[case["out"]]
        flops = 2 * t * n * k + 2 * t * r * (n + k)
        if case["grad"]:
            size += t * n * es + t * k * es + l * r * (n + k) * 4
            flops += 2 * t * n * k + 4 * t * r * (n + k)
        return {"bytes": size, "flops": flops}
    t, e, top = case["t"], case["e"], case["top"]
    row, picks = t * e * es, t * top
    if case["op"] == "route":
        return {"bytes": row + picks * 8, "flops": 4 * t * e}
    mask = t if case["pad"] else 0
    if case["op"] == "balance":
        return {"bytes": 2 * row + picks * 4 + mask, "flops": 8 * t * e}
    return {"bytes": 2 * row + picks * 12 + mask, "flops": 10 * t * e}


# ---------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------

def _exact_lora(case, s):
    t, n, k = case["t"], case["n"], case["k"]
    w = s["w"].double()
    x = s["x"].double()
    out = x @ w.t()
    if s["beside"] is not None:
        out += s["beside"].double()
    if case["grad"]:
        go = s["go"].double()
        grad_x = go @ w
        grad_a = torch.zeros(case["l"], case["r"], k, dtype=torch.float64, device="cuda")
        grad_b = torch.zeros(case["l"], n, case["r"], dtype=torch.float64, device="cuda")
    for l in range(case["l"]):
        rows = (s["ids"] == l).nonzero()[:, 0]
        if not rows.numel():
            continue
        a, b, c = s["a"][l].double(), s["b"][l].double(), s["scale"][l].double()
        v = x[rows] @ a.t()
        out[rows] += c * (v @ b.t())
        if case["grad"]:
            u = go[rows] @ b
            grad_x[rows] += c * (u @ a)
            grad_a[l] = c * (u.t() @ x[rows])
            grad_b[l] = c * (go[rows].t() @ v)
    return (out, grad_x, grad_a, grad_b) if case["grad"] else out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        return _exact_lora(case, s)
    e, top = case["e"], case["top"]
    z = s["logits"].double()
    p = torch.softmax(z, 1)
    if case["op"] != "balance":
        order = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :top]
        w = torch.gather(p, 1, order)
        total = w.sum(1, keepdim=True)
        if case["renorm"]:
            w = w / total
        if case["op"] == "route":
            return w, order
    else:
        order = s["ids"].long()
    here = slice(None) if s["mask"] is None else s["mask"]
    counts = torch.bincount(order[here].reshape(-1), minlength=e)
    tokens = order[here].shape[0]
    slopes = COEF * e * counts.double() / max(1, tokens * top) / max(1, tokens)
    loss = (p[here].sum(0) * slopes).sum()
    # the derivative by the probabilities, then through the softmax
    gp = s["gl"].double() * slopes.expand_as(p)
    if case["op"] == "router":
        gw = s["gw"].double()
        if case["renorm"]:
            gw = (gw - (gw * w).sum(1, keepdim=True)) / total
        gp = gp.scatter_add(1, order, gw)
    g = p * (gp - (gp * p).sum(1, keepdim=True))
    if s["mask"] is not None:
        g[~s["mask"]] = 0.0
    if case["op"] == "balance":
        return loss, counts, g
    if s["mask"] is not None:
        w, order = w.clone(), order.clone()
        w[~s["mask"]] = 0.0
        order[~s["mask"]] = -1
    return w, order, loss, counts, g
