"""CPU pins of the oracles of the adapters' projection and the router (hand-made cases,
differences, library special cases), and what their entry points refuse."""
import numpy as np
import pytest
import torch

import moe_expert_grouped_amd as mi
from moe_expert_grouped_amd import _lib
from oracle import lora_mm as OL
from oracle import router as OR

FAKE = 0x10000000  # never dereferenced: validation fails before any launch


def _err(status):
    with pytest.raises((ValueError, NotImplementedError)) as ei:
        _lib.check(status)
    return str(ei.value)


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


# ---------------------------------------------------------------------------
# the oracles
# ---------------------------------------------------------------------------

def test_lora_oracle_row_by_row():
    x, w, a, b = _rand(6, 5), _rand(4, 5, seed=1), _rand(3, 2, 5, seed=2), _rand(3, 4, 2, seed=3)
    ids, scale, bias = [2, -1, 0, 2, 3, 1], [0.5, 2.0, -1.0], _rand(4, seed=4)
    out, mag, act, _ = OL.mm_lora(x, w, a, b, ids, scale, bias)
    for t, l in enumerate(ids):
        full = w + (scale[l] * b[l] @ a[l] if 0 <= l < 3 else 0.0)
        assert np.allclose(out[t], full @ x[t] + bias, rtol=1e-13)
        assert np.allclose(act[t], a[l] @ x[t] if 0 <= l < 3 else 0.0)
    assert (mag >= np.abs(out) - 1e-12).all()


def test_lora_oracle_gradients_against_differences():
    x, w, a, b = _rand(6, 5), _rand(4, 5, seed=1), _rand(3, 2, 5, seed=2), _rand(3, 4, 2, seed=3)
    ids, scale, go = [2, -1, 0, 2, 3, 0], [0.5, 2.0, -1.0], _rand(6, 4, seed=5)
    grads = [g for g, _ in OL.mm_lora_backward(go, x, w, a, b, ids, scale)]
    assert not grads[1][1].any() and not grads[2][1].any()  # adapter 1 has no row
    for t, grad in zip((x, a, b), grads):
        for i in np.ndindex(t.shape):
            def at(d):
                keep = t[i]
                t[i] = keep + d
                v = (OL.mm_lora(x, w, a, b, ids, scale)[0] * go).sum()
                t[i] = keep
                return v
            # bilinear: the central difference is the derivative
            assert abs((at(0.5) - at(-0.5)) - grad[i]) < 1e-12


def test_router_oracle_by_hand():
    inf = float("inf")
    z = np.array([[0.0, np.log(3.0), -inf, np.log(3.0)], [-inf] * 4, [1.0, 2.0, 3.0, 4.0], [-0.0, 0.0, -1.0, 0.0]])
    w, ids = OR.topk(z, 3, renormalize=False)
    assert ids.tolist() == [[1, 3, 0], [-1, -1, -1], [3, 2, 1], [0, 1, 3]]
    assert np.allclose(w[0], [3 / 7, 3 / 7, 1 / 7]) and not w[1].any()
    w, _ = OR.topk(z, 2)
    assert np.allclose(w[0], [0.5, 0.5]) and np.allclose(w.sum(1), [1, 0, 1, 1])
    w, ids = OR.topk(z, 2, mask=[True, True, False, True])
    assert ids[2].tolist() == [-1, -1] and not w[2].any()
    # even choices and even probabilities: the loss is coef
    even = np.zeros((8, 4))
    loss, counts, slopes = OR.balance(even, np.arange(16).reshape(8, 2) % 4, 0.25)
    assert counts.tolist() == [4, 4, 4, 4] and abs(loss - 0.25) < 1e-15 and np.allclose(slopes, 0.25 / 8)
    # all on one expert that all prefer: E times as much
    loss, counts, _ = OR.balance(np.where(np.arange(4) == 1, 100.0, 0.0) * np.ones((8, 1)), np.ones((8, 1), int), 1.0)
    assert counts.tolist() == [0, 8, 0, 0] and abs(loss - 4.0) < 1e-12
    assert OR.balance(even, np.full((8, 2), -1), 1.0)[0] == 0.0
    assert OR.balance(even, np.zeros((8, 2), int), 1.0, mask=[False] * 8)[0] == 0.0


@pytest.mark.parametrize("renorm", [True, False])
def test_router_oracle_gradient_against_differences(renorm):
    T, E, k, coef = 5, 7, 3, 0.3
    z, gw, gl = _rand(T, E), _rand(T, k, seed=1), 0.7
    mask = [True, True, False, True, True]
    w, ids = OR.topk(z, k, renorm, mask)
    loss, counts, slopes = OR.balance(z, ids, coef, mask)
    grad, mag = OR.backward(z, k, ids, w, gw, renorm, slopes, gl, mask)

    def value(z):
        ws = np.zeros((T, k))
        for t in range(T):
            if mask[t]:
                p = OR.softmax(z[t])[ids[t]]
                ws[t] = p / p.sum() if renorm else p
        return (ws * gw).sum() + gl * OR.balance(z, ids, coef, mask)[0]

    for i in np.ndindex(z.shape):
        d = np.zeros_like(z)
        d[i] = 1e-5
        assert abs((value(z + d) - value(z - d)) / 2e-5 - grad[i]) < 1e-9
    assert not grad[2].any() and (mag >= np.abs(grad) - 1e-15).all()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def far(i):
    return FAKE + (i << 28)


MM = dict(x=far(1), m=40, k=64, dt=_lib.MI_BF16, w=far(2), n=72, a=far(3), b=far(4), L=3, R=16, ids=far(5),
          scale=far(6), bias=far(7), out=far(8), odt=_lib.MI_BF16, act=far(9), ws=far(10), wsb=1 << 24, stream=None)
BACK = dict(go=far(1), x=far(2), m=40, k=64, dt=_lib.MI_BF16, w=far(3), n=72, a=far(4), b=far(5), L=3, R=16,
            ids=far(6), scale=far(7), act=far(8), gx=far(9), ga=far(10), gb=far(11), gdt=_lib.MI_F32, ws=far(12),
            wsb=1 << 24, stream=None)
TOPK = dict(z=far(1), dt=_lib.MI_BF16, T=40, E=16, k=4, renorm=1, mask=far(2), w=far(3), ids=far(4), stream=None)
BAL = dict(z=far(1), dt=_lib.MI_F32, T=40, E=16, ids=far(2), k=4, mask=far(3), given=far(4), coef=1.0, loss=far(5),
           counts=far(6), slopes=far(7), ws=far(8), wsb=1 << 20, stream=None)
RBACK = dict(z=far(1), dt=_lib.MI_F32, T=40, E=16, ids=far(2), w=far(3), gw=far(4), k=4, renorm=1, slopes=far(5),
             gl=far(6), mask=far(7), out=far(8), odt=_lib.MI_F32, stream=None)


def _call(name, base, **kw):
    assert set(kw) <= set(base)
    return getattr(_lib.lib(), name)(*{**base, **kw}.values())


def test_lora_refusals():
    c = lambda **kw: _err(_call("mi_mm_lora", MM, **kw))
    assert "bf16 or fp16" in c(dt=_lib.MI_F32)
    assert "rows out of range" in c(m=-1)
    assert "n % 8" in c(n=60) and "n % 8" in c(n=0)
    assert "k % 8" in c(k=12)
    assert "rank must be" in c(R=12) and "rank must be" in c(R=264) and "rank must be" in c(R=0)
    assert "num_adapters" in c(L=0) and "num_adapters" in c(L=1025)
    assert "below 2^20" in c(n=1 << 20) and "below 2^20" in c(n=1 << 16, k=1 << 14)
    assert "x's type or fp32" in c(odt=_lib.MI_F16)
    for t in ("x", "w", "a", "b", "ids", "out"):
        assert "is null" in c(**{t: None})
    for t in ("x", "w", "a", "b", "bias", "out", "act"):
        assert "16-byte aligned" in c(**{t: MM[t] + 8})
    assert "workspace needs" in c(wsb=100) and "workspace needs" in c(ws=None) and "workspace needs" in c(ws=far(10) + 16)
    assert _call("mi_mm_lora", MM, m=0, x=None, out=None) == _lib.MI_OK
    c = lambda **kw: _err(_call("mi_mm_lora_backward", BACK, **kw))
    assert "bf16 or fp16" in c(dt=_lib.MI_F32)
    assert "fp32 or of x's type" in c(gdt=_lib.MI_F16)
    assert "given together" in c(ga=None)
    assert "no gradient" in c(gx=None, ga=None, gb=None)
    for t in ("a", "b", "go", "ids", "w", "x"):
        assert "is null" in c(**{t: None})
    for t in ("go", "x", "w", "a", "b", "act", "gx", "ga", "gb"):
        assert "16-byte aligned" in c(**{t: BACK[t] + 8})
    assert "workspace needs" in c(wsb=100)
    assert "take at most" in c(m=1 << 20, n=1 << 14, go=1 << 40, x=1 << 44, gx=1 << 45, act=1 << 46, ids=1 << 47,
                               ws=1 << 50, wsb=1 << 48)
    for m in (20, 0):  # banks whose gradients a launch could not cover
        assert "below 2^35" in c(m=m, n=(1 << 20) - 8, k=1016, L=1024, R=256)
    assert _call("mi_mm_lora_backward", BACK, m=0, ga=None, gb=None) == _lib.MI_OK
    L = _lib.lib()
    assert L.mi_mm_lora_workspace_size(40, 72, 64, 3, 12, 0) == 0
    assert L.mi_mm_lora_workspace_size(5000, 72, 64, 3, 16, 1) > L.mi_mm_lora_workspace_size(5000, 72, 64, 3, 16, 0)


def test_router_refusals():
    c = lambda **kw: _err(_call("mi_moe_route_topk", TOPK, **kw))
    assert "top_k must be" in c(k=0) and "top_k must be" in c(k=17) and "top_k must be" in c(k=65, E=128)
    assert "num_experts" in c(E=1025)
    assert "[0, 2^31)" in c(T=1 << 30) and "[0, 2^31)" in c(T=-1)
    assert "bf16, fp16 or fp32" in c(dt=3)
    for t in ("z", "w", "ids"):
        assert "is null" in c(**{t: None})
    assert _call("mi_moe_route_topk", TOPK, T=0, z=None) == _lib.MI_OK
    c = lambda **kw: _err(_call("mi_moe_balance_loss", BAL, **kw))
    assert "top_k" in c(k=0)
    assert "num_experts" in c(E=0)
    for t in ("loss", "counts", "slopes", "z", "ids"):
        assert "is null" in c(**{t: None})
    assert "workspace needs" in c(wsb=8) and "workspace needs" in c(ws=far(8) + 2)
    c = lambda **kw: _err(_call("mi_moe_route_backward", RBACK, **kw))
    assert "is needed" in c(gw=None, slopes=None, gl=None)
    assert "given together" in c(gl=None)
    assert "top_k" in c(k=0)
    assert "bf16, fp16 or fp32" in c(odt=5) and "bf16, fp16 or fp32" in c(dt=5)
    assert "is null" in c(z=None) and "is null" in c(out=None)
    assert "needs topk_ids" in c(ids=None) and "needs topk_ids" in c(w=None)
    assert "may be logits itself" in c(out=far(1) + 16)
    assert "may be logits itself" in c(out=far(1), odt=_lib.MI_BF16)
    assert _call("mi_moe_route_backward", RBACK, T=0, z=None, out=None) == _lib.MI_OK


def test_outputs_apart_from_the_inputs():
    """Every output against every tensor it may not share memory with, at its start and at
    its last bytes."""
    def each(fn, base, outs, size):
        for out in outs:
            for other in size:
                if other == out:
                    continue
                for at in (0, (size[other] - 1) // 16 * 16):
                    assert "overlap" in _err(_call(fn, base, **{out: base[other] + at})), (out, other)

    bank = 3 * 16 * 2
    each("mi_mm_lora", MM, ["out", "act"], dict(x=40 * 128, w=72 * 128, a=bank * 64, b=bank * 72, ids=160, scale=12,
                                               bias=144, out=40 * 144, act=40 * 64, ws=1 << 24))
    each("mi_mm_lora_backward", BACK, ["gx", "ga", "gb"],
         dict(go=40 * 144, x=40 * 128, w=72 * 128, a=bank * 64, b=bank * 72, ids=160, scale=12, act=40 * 64,
              gx=40 * 128, ga=2 * bank * 64, gb=2 * bank * 72, ws=1 << 24))
    each("mi_moe_route_topk", TOPK, ["w", "ids"], dict(z=40 * 32, mask=40, w=640, ids=640))
    each("mi_moe_balance_loss", BAL, ["loss", "counts", "slopes"],
         dict(z=40 * 64, ids=640, mask=40, given=64, loss=4, counts=64, slopes=64,
              ws=_lib.lib().mi_moe_balance_loss_workspace_size(40, 16)))
    each("mi_moe_route_backward", RBACK, ["out"], dict(ids=640, w=640, gw=640, slopes=64, gl=4, mask=40))


def test_python_refusals_before_the_gpu():
    bf = torch.bfloat16
    x, w = torch.zeros(3, 16, dtype=bf), torch.zeros(8, 16, dtype=bf)
    a, b = torch.zeros(2, 8, 16, dtype=bf), torch.zeros(2, 8, 8, dtype=bf)
    ids, sc, go = torch.zeros(3, dtype=torch.int32), torch.ones(2), torch.zeros(3, 8, dtype=bf)

    def bad(match, f, *args, **kw):
        with pytest.raises(ValueError, match=match):
            f(*args, **kw)

    bad("bfloat16 or float16", mi.mm_lora, x.float(), w, a, b, ids, sc)
    bad("w must be", mi.mm_lora, x, w[:, :8], a, b, ids, sc)
    bad("lora_a must be", mi.mm_lora, x, w, a.half(), b, ids, sc)
    bad("lora_b must be", mi.mm_lora, x, w, a, b[:1], ids, sc)
    bad("lora_ids must be", mi.mm_lora, x, w, a, b, ids.long(), sc)
    bad("lora_scale must be", mi.mm_lora, x, w, a, b, ids, sc[:1])
    bad("out_dtype", mi.mm_lora, x, w, a, b, ids, sc, out_dtype=torch.float16)
    bad("bias must be", mi.mm_lora, x, w, a, b, ids, sc, bias=torch.zeros(8))
    bad("on the GPU", mi.mm_lora, x, w, a, b, ids, sc)
    bad("x must be", mi.mm_lora_backward, go, x[:2], w, a, b, ids, sc)
    bad("grad_dtype", mi.mm_lora_backward, go, x, w, a, b, ids, sc, grad_dtype=torch.float16)
    bad("no gradient", mi.mm_lora_backward, go, x, w, a, b, ids, sc, with_x=False, with_adapters=False)
    bad("needs with_x", mi.mm_lora_backward, go, x, w, a, b, ids, sc, with_x=False, grad_x=x)
    bad("need with_adapters", mi.mm_lora_backward, go, x, w, a, b, ids, sc, with_adapters=False, grad_a=a)
    bad("act must be", mi.mm_lora_backward, go, x, w, a, b, ids, sc, act=go)
    bad("on the GPU", mi.mm_lora_backward, go, x, w, a, b, ids, sc)
    z, k = torch.zeros(3, 16), torch.zeros(3, 2, dtype=torch.int32)
    gw = torch.zeros(3, 2)
    bad("logits must be", mi.moe_route_topk, z[0], 2)
    bad("token_mask must be", mi.moe_route_topk, z, 2, token_mask=torch.ones(3))
    bad("on the GPU", mi.moe_route_topk, z, 2)
    bad("topk_ids must be", mi.moe_balance_loss, z, k.long())
    bad("given_counts must be", mi.moe_balance_loss, z, k, given_counts=k[0])
    bad("on the GPU", mi.moe_balance_loss, z, k)
    bad("is needed", mi.moe_route_backward, z)
    bad("given together", mi.moe_route_backward, z, slopes=z[0])
    bad("slopes must be", mi.moe_route_backward, z, slopes=z[0, :4], grad_loss=torch.ones(()))
    bad("needs topk_ids", mi.moe_route_backward, z, grad_weights=gw)
    bad("need topk_weights", mi.moe_route_backward, z, grad_weights=gw, topk_ids=k)
    bad("on the GPU", mi.moe_route_backward, z, grad_weights=gw, topk_ids=k, renormalize=False)
