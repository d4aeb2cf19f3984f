"""Cases for measuring the 8-bit block-scaled operators and the combine of expert rows.

``listed()`` names fixed cases, ``draw(rng)`` gives more of the same ranges.
``prepare(case, seed)`` makes a case's inputs on the GPU, ``run(state)`` is one
pass (plain torch in fp32, or this package's kernels where ``own`` is true),
``work(case)`` what the pass cannot do without, and ``exact(case, seed)`` its
result in 64 bits.

Operators (``op``):

- ``norm``     h = x (+ residual); y = h / sqrt(mean(h^2) + eps) * weight; y as
               e4m3 codes with one fp32 scale per 128 columns (and y itself)
- ``quant``    x, or silu(gate) * up of x = [gate | up], as e4m3 codes with one
               scale per 1 x 128 block (activations) or 128 x 128 block (weights)
- ``mm``       out[m, n] = sum_B sa[m, B] sb[n/128, B] sum_{k in B} a[m, k] b[n, k]
- ``grouped``  the same product for every expert's rows with its own b
- ``combine``  out[t] = sum_j w[t, j] rows[perm[t, j]], and with ``grad`` the
               gradients of rows, of w and of the permuted copy of the tokens

Scales have one column per 128 columns, padded with zeros to a multiple of 4.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ES = {"bf16": 2, "f16": 2, "f32": 4}
MIN_SCALE = 2.0 ** -126
EPS = 1e-6


def _cols(k):
    """Scale columns of k values: one per 128, padded to a multiple of 4."""
    return 4 * -(-k // 512)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step, before its projections
        {"name": "norm one token", "op": "norm", "t": 1, "h": 4096, "dt": "bf16", "residual": True, "keep": False},
        # a prefill batch before its MoE layer: the router reads y, the experts the codes
        {"name": "norm prefill", "op": "norm", "t": 8192, "h": 7168, "dt": "bf16", "residual": True, "keep": True},
        # the activation between FC1 and FC2 of a prefill batch, 8 experts a token
        {"name": "quant swiglu rows", "op": "quant", "batch": 1, "rows": 65536, "k": 2048, "dt": "bf16", "br": 1, "glu": True},
        # a few experts' weights when they are loaded, sizes that end inside a block
        {"name": "quant weights ragged", "op": "quant", "batch": 8, "rows": 2000, "k": 4112, "dt": "f32", "br": 128, "glu": False},
        # a few decoded tokens through one projection: the weights' bytes count
        {"name": "mm decode", "op": "mm", "m": 4, "n": 8192, "k": 8192, "dt": "bf16"},
        # an odd batch and sizes that end inside a tile and a block, kept in fp32
        {"name": "mm ragged", "op": "mm", "m": 333, "n": 1744, "k": 2064, "dt": "f32"},
        # a prefill batch through one projection
        {"name": "mm prefill", "op": "mm", "m": 4096, "n": 8192, "k": 8192, "dt": "bf16"},
        # 16 decoded tokens with 8 experts each: few rows an expert, some experts empty
        {"name": "grouped decode", "op": "grouped", "e": 64, "m": 128, "n": 2048, "k": 4096, "dt": "bf16", "skew": 0.0},
        # FC2 of a prefill batch over many experts of very unequal load
        {"name": "grouped skewed", "op": "grouped", "e": 128, "m": 32768, "n": 7168, "k": 2048, "dt": "bf16", "skew": 1.0},
        # the end of a decode step's MoE layer
        {"name": "combine decode", "op": "combine", "t": 16, "top": 8, "h": 7168, "dt": "bf16", "grad": False},
        # the end of a prefill batch's MoE layer
        {"name": "combine prefill", "op": "combine", "t": 8192, "top": 8, "h": 4096, "dt": "bf16", "grad": False},
        # a training step's combine, with every gradient; an odd batch
        {"name": "combine training", "op": "combine", "t": 4099, "top": 6, "h": 4096, "dt": "bf16", "grad": True},
    ]


def draw(rng):
    def log(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
        return min(hi, max(lo, int(v) // step * step))

    op = rng.choice(["norm", "quant", "mm", "mm", "grouped", "grouped", "combine", "combine"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        return {"op": op, "t": log(1, 8192), "h": log(256, 7168, 16), "dt": dt, "residual": rng.random() < 0.7, "keep": rng.random() < 0.5}
    if op == "quant":
        if rng.random() < 0.5:
            return {"op": op, "batch": 1, "rows": log(1, 32768), "k": log(128, 4096, 16), "dt": dt, "br": 1, "glu": rng.random() < 0.5}
        return {"op": op, "batch": rng.randint(1, 8), "rows": log(128, 2048), "k": log(256, 4096, 16), "dt": dt, "br": 128, "glu": False}
    if op == "mm":
        return {"op": op, "m": log(1, 4096), "n": log(256, 8192, 16), "k": log(256, 8192, 16), "dt": dt}
    if op == "grouped":
        return {"op": op, "e": log(4, 64), "m": log(8, 16384), "n": log(256, 4096, 16), "k": log(256, 4096, 16), "dt": dt, "skew": rng.choice([0.0, 0.0, 0.7, 1.0])}
    return {"op": op, "t": log(1, 4096), "top": rng.randint(1, 8), "h": log(128, 4096, 16), "dt": dt, "grad": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, shape, dt=torch.float32, std=1.0):
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * std).to(dt)


def _codes(g, shape, std):
    """e4m3 codes as a quantiser leaves them: blocks that reach to 448."""
    return _normal(g, shape, std=std).clamp_(-448.0, 448.0).to(FP8)


def _scales(g, lead, k, mid):
    """Scales of rows of k values, log-normal around `mid`, zero in the padding."""
    s = torch.zeros(*lead, _cols(k), device="cuda")
    s[..., : -(-k // 128)] = torch.exp(0.5 * _normal(g, (*lead, -(-k // 128)))) * mid
    return s


def _route(g, t, top, experts, absent):
    """Distinct experts of each token, a share of the slots routed elsewhere:
    the stable sort's place of each slot (-1: none), and its inverse."""
    ids = torch.rand(t, experts, generator=g, device="cuda").argsort(1)[:, :top].reshape(-1)
    ids = torch.where(torch.rand(t * top, generator=g, device="cuda") < absent, experts, ids)
    order = ids.argsort(stable=True)
    perm = torch.empty_like(order)
    perm[order] = torch.arange(t * top, device="cuda")
    perm = torch.where(ids < experts, perm, -1)
    inverse = torch.where(ids[order] < experts, order, -1)
    return perm.to(torch.int32), inverse.to(torch.int32)


def _counts(case, seed):
    """Rows of each expert: a skewed share of m rows in a seeded order of the
    experts, drawn as a router's choices fall."""
    g = torch.Generator().manual_seed(seed)
    e = case["e"]
    p = (torch.randperm(e, generator=g) + 1).double() ** -case["skew"]
    ids = torch.multinomial(p, case["m"], replacement=True, generator=g)
    return torch.bincount(ids, minlength=e)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DT[case["dt"]]
    s = dict(case)
    if op == "norm":
        t, h = case["t"], case["h"]
        s["x"] = _normal(g, (t, h), dt)
        s["r"] = _normal(g, (t, h), dt, 3.0) if case["residual"] else None
        s["w"] = (1.0 + 0.3 * _normal(g, (h,))).to(dt)
    elif op == "quant":
        shape = (case["rows"], case["k"] * (2 if case["glu"] else 1))
        s["x"] = _normal(g, shape if case["br"] == 1 else (case["batch"], *shape), dt, 2.0 if case["glu"] else 0.05)
    elif op == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = _codes(g, (m, k), 150.0), _scales(g, (m,), k, 0.01)
        s["b"], s["sb"] = _codes(g, (n, k), 110.0), _scales(g, (-(-n // 128),), k, 3e-4)
    elif op == "grouped":
        e, m, n, k = case["e"], case["m"], case["n"], case["k"]
        counts = _counts(case, seed)
        s["counts"] = counts.tolist()
        s["indptr"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to("cuda", torch.int32)
        s["a"], s["sa"] = _codes(g, (m, k), 150.0), _scales(g, (m,), k, 0.01)
        s["b"], s["sb"] = _codes(g, (e, n, k), 110.0), _scales(g, (e, -(-n // 128)), k, 3e-4)
    else:
        t, top, h = case["t"], case["top"], case["h"]
        s["perm"], s["inverse"] = _route(g, t, top, 64, 0.05)
        s["w"] = torch.softmax(_normal(g, (t, top)), 1)
        s["rows"] = _normal(g, (t * top, h), dt)
        if case["grad"]:
            s["go"] = _normal(g, (t, h), dt)
            s["gp"] = _normal(g, (t * top, h), dt)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _quantise(y, br):
    """Codes and scales of y [..., rows, k] in fp32, blocks of br x 128."""
    rows, k = y.shape[-2:]
    nb, kb = -(-rows // br), -(-k // 128)
    p = torch.nn.functional.pad(y, (0, kb * 128 - k, 0, nb * br - rows))
    p = p.reshape(*y.shape[:-2], nb, br, kb, 128)
    sc = (p.abs().amax((-3, -1)) / 448.0).clamp(min=MIN_SCALE)
    q = (p / sc[..., :, None, :, None]).reshape(*y.shape[:-2], nb * br, kb * 128)[..., :rows, :k]
    return q.to(FP8), torch.nn.functional.pad(sc, (0, _cols(k) - kb))


def _spread(sc, k):
    return sc.repeat_interleave(128, -1)[..., :k]


def _product(a, sa, b, sb):
    k = a.shape[1]
    x = a.float() * _spread(sa, k)
    w = b.float() * _spread(sb, k).repeat_interleave(128, 0)[: b.shape[0]]
    return x @ w.t()


def _plain(s):
    op, dt = s["op"], DT[s["dt"]]
    if op == "norm":
        h = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].float()
        codes, sc = _quantise(y, 1)
        out = [codes, sc]
        if s["r"] is not None:
            out.append(h.to(dt))
        return out + [y.to(dt)] if s["keep"] else out
    if op == "quant":
        x = s["x"].float()
        if s["glu"]:
            gate, up = x[..., : s["k"]], x[..., s["k"]:]
            x = gate / (1.0 + torch.exp(-gate)) * up
        return _quantise(x, s["br"])
    if op == "mm":
        return _product(s["a"], s["sa"], s["b"], s["sb"]).to(dt)
    if op == "grouped":
        out = torch.empty(s["m"], s["n"], dtype=dt, device="cuda")
        at = 0
        for e, c in enumerate(s["counts"]):
            if c:
                out[at:at + c] = _product(s["a"][at:at + c], s["sa"][at:at + c], s["b"][e], s["sb"][e])
            at += c
        return out
    t, top, h = s["t"], s["top"], s["h"]
    perm = s["perm"].long()
    here = (perm >= 0).float()
    at = perm.clamp(min=0)
    picked = s["rows"][at].float().reshape(t, top, h)
    w = (s["w"].reshape(-1) * here).reshape(t, top, 1)
    out = (picked * w).sum(1).to(dt)
    if not s["grad"]:
        return out
    go = s["go"].float()
    grad_w = (picked * go[:, None]).sum(2) * here.reshape(t, top)
    grad_rows = torch.zeros(t * top + 1, h, dtype=dt, device="cuda")
    grad_rows[torch.where(perm >= 0, perm, t * top)] = (go[:, None] * w).reshape(t * top, h).to(dt)
    grad_x = (s["gp"][at].float() * here[:, None]).reshape(t, top, h).sum(1).to(dt)
    return out, grad_rows[: t * top], grad_w, grad_x


def _own(s):
    import moe_expert_grouped_amd as mi

    op, dt = s["op"], DT[s["dt"]]
    if op == "norm":
        got = mi.add_rmsnorm_fp8(s["x"], s["w"], s["r"], eps=EPS, with_norm=s["keep"])
        return [v for v in got if v is not None]
    if op == "quant":
        return mi.fp8_quantize(s["x"], block_rows=s["br"], swiglu=s["glu"])
    if op == "mm":
        return mi.mm_fp8_block(s["a"], s["b"], s["sa"], s["sb"], out_dtype=dt)
    if op == "grouped":
        return mi.grouped_mm_fp8_block(s["a"], s["sa"], s["b"], s["sb"], s["indptr"], out_dtype=dt)
    out = mi.moe_combine_rows(s["rows"], s["perm"], s["w"])
    if not s["grad"]:
        return out
    grad_rows, grad_w = mi.moe_combine_rows_backward(s["go"], s["rows"], s["perm"], s["w"], permuted_idx_to_expanded_idx=s["inverse"])
    return out, grad_rows, grad_w, mi.moe_permute_rows_backward(s["gp"], s["perm"], s["top"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, es = case["op"], ES[case["dt"]]
    if op == "norm":
        t, h = case["t"], case["h"]
        streams = 1 + (2 if case["residual"] else 0) + (1 if case["keep"] else 0)
        return {"bytes": t * h * (streams * es + 1) + t * _cols(h) * 4 + h * es, "flops": 8 * t * h}
    if op == "quant":
        v = case["batch"] * case["rows"] * case["k"]
        sc = case["batch"] * -(-case["rows"] // case["br"]) * _cols(case["k"]) * 4
        return {"bytes": v * (es * (2 if case["glu"] else 1) + 1) + sc, "flops": v * (10 if case["glu"] else 4)}
    if op in ("mm", "grouped"):
        m, n, k, c = case["m"], case["n"], case["k"], _cols(case["k"])
        # the experts that have rows: all of them, or as many as uniform choices reach
        e = 1 if op == "mm" else case["e"] * (1 - (1 - 1 / case["e"]) ** m) if not case["skew"] else min(case["e"], m)
        return {"bytes": m * (k + 4 * c) + e * (n * k + -(-n // 128) * c * 4) + m * n * es, "flops": 2 * m * n * k}
    t, top, h = case["t"], case["top"], case["h"]
    rows, small = t * top * h * es, t * top * 8
    if not case["grad"]:
        return {"bytes": rows + t * h * es + small, "flops": 2 * t * top * h}
    return {"bytes": 3 * rows + 3 * t * h * es + 2 * small, "flops": 6 * t * top * h}


# ---------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------

def _to_e4m3(v):
    """The e4m3 value nearest to v, ties to even: 3 mantissa bits, exponents from -6."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quantise(y, br):
    """Block by block over the last two axes; y is [..., rows, k] in 64 bits."""
    rows, k = y.shape[-2:]
    q = torch.empty_like(y)
    sc = torch.zeros(*y.shape[:-2], -(-rows // br), _cols(k), dtype=torch.float64, device=y.device)
    for c in range(0, k, 128):
        cut = y[..., c:c + 128]
        top = cut.abs().amax(-1)
        if br > 1:
            top = torch.stack([part.amax(-1) for part in top.split(br, -1)], -1)
        one = torch.clamp(top / 448, min=MIN_SCALE)
        sc[..., c // 128] = one
        each = one if br == 1 else one.repeat_interleave(br, -1)[..., :rows]
        q[..., c:c + 128] = _to_e4m3(cut / each[..., None])
    return q, sc


def _exact_product(a, sa, b, sb):
    out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    of = torch.arange(b.shape[0], device=a.device) // 128
    for c in range(0, a.shape[1], 128):
        part = a[:, c:c + 128].double() @ b[:, c:c + 128].double().t()
        out += part * sa[:, c // 128, None].double() * sb[of, c // 128].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = h + s["r"].double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["h"] + EPS) * s["w"].double()
        got = [*_exact_quantise(y, 1)]
        if s["r"] is not None:
            got.append(h)
        return got + [y] if case["keep"] else got
    if op == "quant":
        x = s["x"].double()
        if case["glu"]:
            gate, up = x.split(case["k"], -1)
            x = gate * torch.sigmoid(gate) * up
        return _exact_quantise(x, case["br"])
    if op == "mm":
        return _exact_product(s["a"], s["sa"], s["b"], s["sb"])
    if op == "grouped":
        parts = zip(s["a"].split(s["counts"]), s["sa"].split(s["counts"]), s["b"], s["sb"])
        return torch.cat([_exact_product(*p) for p in parts])
    t, top, h = case["t"], case["top"], case["h"]
    perm, w = s["perm"].long().reshape(t, top), s["w"].double()
    out = torch.zeros(t, h, dtype=torch.float64, device="cuda")
    grad_x, grad_w = torch.zeros_like(out), torch.zeros_like(w)
    grad_rows = torch.zeros(t * top, h, dtype=torch.float64, device="cuda") if case["grad"] else None
    for j in range(top):
        slots = (perm[:, j] >= 0).nonzero()[:, 0]
        at = perm[slots, j]
        out[slots] += w[slots, j, None] * s["rows"][at].double()
        if case["grad"]:
            go = s["go"][slots].double()
            grad_rows[at] = w[slots, j, None] * go
            grad_w[slots, j] = (s["rows"][at].double() * go).sum(1)
            grad_x[slots] += s["gp"][at].double()
    return (out, grad_rows, grad_w, grad_x) if case["grad"] else out
