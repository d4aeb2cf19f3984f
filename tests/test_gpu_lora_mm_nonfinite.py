"""Infinities in one request's rows or adapter: the projection and its gradients hold +inf,
-inf and NaN exactly where the 64-bit formula does, on every path.

All finite values are whole numbers whose products and sums stay below 2^24, so that the
fp32 sums are exact: a result is finite and exact, infinite of the right sign, or NaN.  The
activations pass 2^8 and the fp16 values 2^8, so that each has several bf16 pieces of either
sign.
"""
import numpy as np
import pytest
import torch

import moe_expert_grouped_amd as mi
import synth
from oracle import lora_mm as O

pytestmark = pytest.mark.gpu

INF = float("inf")
HALVES = [torch.bfloat16, torch.float16]
# one launch, few rows, 64 x 64 tiles, 128 x 128 (forward, backward), 256 x 256 (forward, backward),
# a split k axis (forward, backward); ranks up to 16 on the large tiles
SIZES = [(1, 136, 264, 3, 32), (20, 136, 264, 3, 16), (1100, 264, 520, 4, 40), (1100, 2056, 136, 3, 24),
         (1100, 72, 2056, 3, 16), (4100, 2056, 72, 3, 72), (4100, 72, 2056, 3, 56),
         (1100, 72, 4680, 3, 16), (1100, 4680, 72, 3, 40),
         (1100, 2056, 136, 3, 16), (4100, 2056, 72, 3, 8), (4100, 72, 2056, 3, 16)]


def _case(T, N, K, L, R, dtype, seed):
    g = synth.gen(seed)

    def whole(*shape, top, share=1.0):
        t = torch.randint(-top, top + 1, shape, generator=g).float()
        return torch.where(torch.rand(shape, generator=g) < share, t, 0.0).to(dtype)

    x, w = whole(T, K, top=40), whole(N, K, top=1)
    a, b = whole(L, R, K, top=3, share=8 / K), whole(L, N, R, top=2)
    go = whole(T, N, top=1, share=4 / N)
    # fp16 values of two bf16 pieces, the second of either sign or 0 (bf16 has the nearest)
    odd = torch.tensor([255.0, 257.0, 259.0, -257.0, -259.0])
    b[1, 8:13, 0] = x[0, :5] = go[0, :5] = odd.to(dtype)
    ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32)
    ids[T // 2] = ids[0] = 1
    return x, w, a, b, ids, torch.randint(1, 4, (L,), generator=g).float(), go


def _plant(what, x, w, a, b, go, row):
    """One kind of infinity for adapter 1, beside values that make some results infinite."""
    N, K, R = w.shape[0], w.shape[1], a.shape[1]
    one = torch.where(torch.arange(R) % 3 == 0, -1.0, 1.0)  # a sign for every rank
    size = torch.ones(R)
    size[:3] = torch.tensor([255.0, 257.0, 259.0])
    some = torch.arange(20, 26)
    by = torch.tensor([-1.0, 1.0, 1.0, -1.0, -1.0, 1.0])
    if what == "a":
        a[1, 3, 5], a[1, R - 1, K - 1] = INF, -INF
    if what == "b":
        b[1, 7, 2], b[1, N - 1, R - 1] = INF, -INF
    if what == "x":  # every term of the row's outputs `some` has the sign of by
        x[row, 5] = INF
        a[1, :, 5] = one.to(a.dtype)
        w[some, 5] = by.to(w.dtype)
        b[1, some] = (by[:, None] * one * size).to(b.dtype)
    if what == "go":  # and of its gradients `some`
        go[row, 3] = -INF
        b[1, 3] = one.to(b.dtype)
        w[3, some] = by.to(w.dtype)
        a[1][:, some] = (by * (one * size)[:, None]).to(a.dtype)
        x[:, some] = x[:, some].clamp(-1, 1)


def _equal(got, ref, what):
    want = torch.from_numpy(ref).to(got.dtype)
    same = torch.equal(torch.nan_to_num(got.cpu(), nan=7e4), torch.nan_to_num(want, nan=7e4)) and \
        torch.equal(got.cpu().isnan(), want.isnan()) and torch.equal(got.cpu().isinf(), want.isinf())
    if not same:
        bad = ~((got.cpu() == want) | (got.cpu().isnan() & want.isnan()))
        at = bad.nonzero()[:4]
        raise AssertionError((what, int(bad.sum()), [(i.tolist(), got[tuple(i)].item(), want[tuple(i)].item()) for i in at]))


@pytest.mark.parametrize("what", ["a", "b", "x", "go"])
@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("T,N,K,L,R", SIZES)
def test_infinities_as_the_formula(gpu, T, N, K, L, R, dtype, what):
    print(f"mm_lora infinity in {what} T={T} N={N} K={K} R={R} {dtype}", flush=True)
    x, w, a, b, ids, scale, go = _case(T, N, K, L, R, dtype, T + N)
    _plant(what, x, w, a, b, go, T // 2)
    cpu = [t.double().numpy() for t in (x, w, a, b)] + [ids, scale]
    with np.errstate(invalid="ignore"):
        ref, mag, act, _ = O.mm_lora(*cpu)
        refs = O.mm_lora_backward(go.double().numpy(), *cpu)
    for m in (mag, *(m for _, m in refs)):
        assert m[np.isfinite(m)].max(initial=0) < 2 ** 24
    if what in ("x", "go"):
        assert np.isinf((ref if what == "x" else refs[0][0])[T // 2, 20:26]).all()
    dev = [t.to(gpu) for t in (x, w, a, b, ids, scale)]
    for od in (torch.float32, dtype):
        out, v = mi.mm_lora(*dev, out_dtype=od, with_act=True)
        _equal(v, act, "act")
        _equal(out, ref, "out")
    for gd in (torch.float32, dtype):
        for given in (v, None):
            got = mi.mm_lora_backward(go.to(gpu), *dev, act=given, grad_dtype=gd)
            for t, (r, _), name in zip(got, refs, ("grad_x", "grad_a", "grad_b")):
                _equal(t, r, (name, gd))


@pytest.mark.parametrize("T", [1, 20, 1100])
def test_finite_activations_past_the_largest_bf16(gpu, T):
    """Sums in fp32 may lie between the largest bf16, 255 / 128 * 2^127, and the largest fp32:
    they are finite, and so are their products."""
    print(f"mm_lora largest activations T={T}", flush=True)
    N, K, L, R = 136, 72, 2, 16
    big = torch.tensor([255 / 128], dtype=torch.float64) * 2.0 ** 127
    x, w = torch.zeros(T, K, dtype=torch.bfloat16), torch.zeros(N, K, dtype=torch.bfloat16)
    a, b = torch.zeros(L, R, K, dtype=torch.bfloat16), torch.zeros(L, N, R, dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = big.item(), 1.5 * 2.0 ** 119  # v = big + 3/4 of bf16's step there
    a[:, 3, :2] = 1.0
    a[:, 4, :2] = -1.0
    b[:, ::2, 3], b[:, 1::2, 4] = 2.0 ** -100, 3 * 2.0 ** -101
    go = torch.zeros(T, N, dtype=torch.bfloat16)
    go[:, :2] = 2.0 ** -110
    ids = torch.arange(T, dtype=torch.int32) % L
    cpu = [t.double().numpy() for t in (x, w, a, b)] + [ids]
    ref, _, act, _ = O.mm_lora(*cpu)
    refs = O.mm_lora_backward(go.double().numpy(), *cpu)
    dev = [t.to(gpu) for t in (x, w, a, b, ids)]
    out, v = mi.mm_lora(*dev, out_dtype=torch.float32, with_act=True)
    _equal(v, act, "act")
    _equal(out, ref, "out")
    _equal(mi.mm_lora(*dev), ref, "out")
    gb = mi.mm_lora_backward(go.to(gpu), *dev, act=v, grad_dtype=torch.float32)[2].cpu().double()
    # T terms of one sign, each exact in its pieces
    assert ((gb - torch.from_numpy(refs[2][0])).abs() <= T * 2.0 ** -24 * torch.from_numpy(refs[2][1])).all()
