"""A projection with many requests' adapters on the GPU against the fp64 oracle.

Exact cases: every operand a small integer, so that each product, sum and piece of the
second product is an integer below 2^24 and fp32 holds all of them; outputs are then
the rounding of an exact value, bit by bit.

Tolerances of the others, u = 2^-24, sums taken as chains: k u of the magnitude for
the product over k, (k + rank) u for the adapters' part (its pieces leave 2^-16 of v for 16-bit
outputs, 2^-24 for fp32), and half a step of the output's type.
"""
import numpy as np
import pytest
import torch

import moe_expert_grouped_amd as mi
import synth
from oracle import lora_mm as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
HALVES = [torch.bfloat16, torch.float16]


def _np(t):
    return t.detach().cpu().double().numpy()


def _near(got, ref, tol, dtype, what):
    t = tol + HALF[dtype] * np.abs(ref) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    err = np.abs(_np(got) - ref)
    assert (err <= t).all(), f"{what}: {np.argwhere(~(err <= t))[:4]} {np.nanmax(err / t)}"


def _ids(g, T, L, kind):
    """Adapters of the rows: at random, in runs, or a few of many; some rows have none."""
    if kind == "runs":
        cuts = torch.randint(0, T + 1, (2 * L,), generator=g).sort()[0]
        ids = torch.bucketize(torch.arange(T), cuts, right=True) % (L + 1) - 1
    else:
        ids = torch.randint(0, L if kind == "mixed" else min(L, 3), (T,), generator=g)
    off = torch.rand(T, generator=g)
    ids[off < 0.1] = -1
    ids[(off >= 0.1) & (off < 0.15)] = L + 2
    return ids.to(torch.int32)


def _case(T, N, K, L, R, dtype, kind, exact, seed):
    g = synth.gen(seed)

    def t(*shape, top, std):
        if exact:
            return torch.randint(-top, top + 1, shape, generator=g).to(dtype)
        return (torch.randn(shape, generator=g) * std).to(dtype)

    x, w = t(T, K, top=2, std=1.0), t(N, K, top=2, std=K ** -0.5)
    a, b = t(L, R, K, top=1, std=K ** -0.5), t(L, N, R, top=2, std=0.3)
    if exact:  # few of a's entries, so that v stays small
        a = torch.where(torch.rand(a.shape, generator=g) < 24.0 / K, a.float(), 0.0).to(dtype)
    scale = (torch.randint(1, 4, (L,), generator=g).float() if exact
             else torch.exp(0.5 * torch.randn(L, generator=g)))
    return x, w, a, b, _ids(g, T, L, kind), scale, t(N, top=3, std=0.5), t(T, N, top=1, std=1.0)


# rows from one to several tiles, sizes that end inside a step, a tile and an item
SHAPES = [(1, 8, 8, 1, 8, "mixed"), (1, 520, 1032, 4, 16, "mixed"), (1, 4104, 72, 2, 24, "mixed"), (1, 64, 4096, 3, 32, "few"),
          (1, 136, 520, 1, 40, "few"), (2, 4104, 264, 3, 32, "mixed"),
          # tiles of few rows that start at their own step, the last of them short
          (150, 4104, 2600, 3, 16, "mixed"), (150, 2600, 4104, 3, 16, "mixed"), (3, 136, 72, 5, 8, "mixed"),
          (15, 64, 264, 2, 24, "few"), (16, 256, 512, 16, 16, "mixed"), (17, 264, 640, 9, 40, "mixed"),
          (33, 1024, 136, 64, 64, "mixed"), (64, 512, 256, 64, 16, "mixed"), (65, 128, 96, 3, 72, "few"),
          (100, 392, 328, 7, 32, "runs"), (130, 264, 200, 2, 128, "runs"), (257, 200, 456, 1, 16, "few"),
          (333, 328, 160, 40, 48, "mixed"), (520, 520, 264, 5, 256, "runs"), (700, 72, 1024, 600, 8, "mixed"),
          (1100, 304, 120, 3, 16, "runs")]


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("T,N,K,L,R,kind", SHAPES)
def test_exact(gpu, T, N, K, L, R, kind, dtype):
    print(f"mm_lora exact T={T} N={N} K={K} L={L} R={R} {kind} {dtype}", flush=True)
    x, w, a, b, ids, scale, bias, go = _case(T, N, K, L, R, dtype, kind, True, T + N)
    ref, mag, act, _ = O.mm_lora(x.double(), w.double(), a.double(), b.double(), ids, scale, bias.double())
    assert mag.max() < 2 ** 24
    dev = [t.to(gpu) for t in (x, w, a, b, ids, scale)]
    for od in (torch.float32, dtype):
        out = torch.full((T, N), 7.0, dtype=od, device=gpu)
        got, ga = mi.mm_lora(*dev, bias=bias.to(gpu), out=out, out_dtype=od, with_act=True)
        torch.cuda.synchronize()
        assert got is out
        assert torch.equal(got.cpu(), torch.from_numpy(ref).to(od)), np.argwhere(_np(got) != _np(torch.from_numpy(ref).to(od)))[:5]
        assert np.array_equal(_np(ga), act)
    plain = mi.mm_lora(*dev[:5], out_dtype=torch.float32)
    ref = O.mm_lora(x.double(), w.double(), a.double(), b.double(), ids)[0]
    assert np.array_equal(_np(plain), ref)


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("T,N,K,L,R,kind", SHAPES)
def test_exact_backward(gpu, T, N, K, L, R, kind, dtype):
    print(f"mm_lora_backward exact T={T} N={N} K={K} L={L} R={R} {kind} {dtype}", flush=True)
    x, w, a, b, ids, scale, _, go = _case(T, N, K, L, R, dtype, kind, True, T + K)
    # u = go b stays small where b has few entries
    b = torch.where(torch.rand(b.shape, generator=synth.gen(T)) < 24.0 / N, b.float(), 0.0).to(dtype)
    refs = O.mm_lora_backward(go.double(), x.double(), w.double(), a.double(), b.double(), ids, scale)
    assert all(m.max() < 2 ** 24 for _, m in refs)
    dev = [t.to(gpu) for t in (go, x, w, a, b, ids, scale)]
    act = mi.mm_lora(*dev[1:], with_act=True)[1]
    torch.cuda.synchronize()
    for gd in (torch.float32, dtype):
        for v in (act, None):
            got = mi.mm_lora_backward(*dev, act=v, grad_dtype=gd)
            torch.cuda.synchronize()
            for what, t, (ref, _) in zip(("grad_x", "grad_a", "grad_b"), got, refs):
                want = torch.from_numpy(ref).to(t.dtype)
                assert torch.equal(t.cpu(), want), (what, gd, v is None, np.argwhere(_np(t) != _np(want))[:5])
    gx, none, none2 = mi.mm_lora_backward(*dev, with_adapters=False)
    assert none is None and none2 is None and torch.equal(gx, got[0])
    none, ga, gb = mi.mm_lora_backward(*dev, act=act, with_x=False)
    assert none is None and torch.equal(ga, got[1]) and torch.equal(gb, got[2])


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("T,N,K,L,R,kind", SHAPES)
def test_against_oracle(gpu, T, N, K, L, R, kind, dtype):
    print(f"mm_lora T={T} N={N} K={K} L={L} R={R} {kind} {dtype}", flush=True)
    x, w, a, b, ids, scale, bias, go = _case(T, N, K, L, R, dtype, kind, False, T + N + 1)
    ref, mag, act, amag = O.mm_lora(x.double(), w.double(), a.double(), b.double(), ids, scale, bias.double())
    dev = [t.to(gpu) for t in (x, w, a, b, ids, scale)]
    for od in (torch.float32, dtype):
        got, ga = mi.mm_lora(*dev, bias=bias.to(gpu), out_dtype=od, with_act=True)
        left = U if od == torch.float32 else 2.0 ** -16
        _near(got, ref, ((K + R + 8) * U + left) * mag, od, "out")
        _near(ga, act, K * U * amag, torch.float32, "act")
    refs = O.mm_lora_backward(go.double(), x.double(), w.double(), a.double(), b.double(), ids, scale)
    dev = [go.to(gpu)] + dev
    for gd in (torch.float32, dtype):
        got = mi.mm_lora_backward(*dev, act=ga, grad_dtype=gd)
        (gx, mx), (rga, ma), (rgb, mb) = refs
        _near(got[0], gx, ((N + R + 8) * U + 2.0 ** -16) * mx, dtype, "grad_x")
        _near(got[1], rga, ((N + T + 8) * U + U) * ma, gd, "grad_a")
        _near(got[2], rgb, ((K + T + 8) * U + U) * mb, gd, "grad_b")


@pytest.mark.parametrize("T,N,K,L,R,kind", [(4096, 64, 64, 5, 16, "runs"), (4097, 72, 72, 1024, 8, "mixed"),
                                            (9000, 64, 136, 7, 8, "mixed"), (70001, 64, 64, 3, 16, "runs"),
                                            (5000, 1024, 64, 1, 24, "few"), (2100, 72, 2056, 3, 16, "runs"),
                                            (1500, 2056, 72, 9, 40, "mixed"), (4500, 128, 4104, 4, 8, "few")])
def test_exact_many_rows(gpu, T, N, K, L, R, kind):
    """Rows past what one workgroup sorts, past the rows of a chunk, and narrow results, whose
    product is split."""
    print(f"mm_lora many rows T={T} N={N} K={K} L={L} R={R} {kind}", flush=True)
    dtype = torch.bfloat16
    x, w, a, b, ids, scale, bias, go = _case(T, N, K, L, R, dtype, kind, True, T)
    x, b = x.clamp(-1, 1), torch.where(torch.rand(b.shape, generator=synth.gen(T)) < 8.0 / N, b.float(), 0.0).to(dtype)
    go = torch.where(torch.rand(go.shape, generator=synth.gen(T + 1)) < 0.1, go.float(), 0.0).to(dtype)
    ref, mag, act, _ = O.mm_lora(x.double(), w.double(), a.double(), b.double(), ids, scale, bias.double())
    refs = O.mm_lora_backward(go.double(), x.double(), w.double(), a.double(), b.double(), ids, scale)
    assert mag.max() < 2 ** 24 and all(m.max() < 2 ** 24 for _, m in refs)
    dev = [t.to(gpu) for t in (x, w, a, b, ids, scale)]
    out, ga = mi.mm_lora(*dev, bias=bias.to(gpu), out_dtype=torch.float32, with_act=True)
    torch.cuda.synchronize()
    assert np.array_equal(_np(out), ref) and np.array_equal(_np(ga), act)
    got = mi.mm_lora_backward(go.to(gpu), *dev, act=ga, grad_dtype=torch.float32)
    for what, t, (want, _) in zip(("grad_x", "grad_a", "grad_b"), got, refs):
        assert torch.equal(t.cpu(), torch.from_numpy(want).to(t.dtype)), what
