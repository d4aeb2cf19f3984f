"""The router's top_k, balance loss and gradients on the GPU against the fp64 oracle.

Tolerances, u = 2^-24.  A probability is an exponential (3 u with its argument's error: the
rest of the product with log2 e is carried, two roundings of it and the function's own
step), a sum of E of them in at most E / 8 + 6 steps, and one quotient: (E / 8 + 12) u
relative.  A gradient adds E / 8 + top_k + 8 steps on the magnitude of its terms.
"""
import numpy as np
import pytest
import torch

import moe_expert_grouped_amd as mi
import synth
from oracle import router as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _np(t):
    return t.detach().cpu().double().numpy()


def _near(got, ref, tol, dtype, what):
    t = tol + HALF[dtype] * np.abs(ref) + TINY[dtype]
    err = np.abs(_np(got) - ref)
    assert (err <= t).all(), f"{what}: {np.argwhere(~(err <= t))[:4]} {np.nanmax(err / t)}"


def _case(T, E, dtype, seed, pad):
    g = synth.gen(seed)
    z = (torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)).to(dtype)
    if E > 2:  # ties, experts that are switched off, equal zeros of both signs
        z[:, E // 2] = z[:, 0]
        z[torch.rand(T, E, generator=g) < 0.1] = -float("inf")
        z[::3, E - 1], z[::3, E - 2] = 0.0, -0.0
    if T > 2:
        z[T // 2] = -float("inf")
    mask = torch.rand(T, generator=g) >= pad if pad else None
    return z, mask


SHAPES = [(1, 1, 1), (1, 8, 2), (1, 64, 6), (3, 5, 3), (7, 60, 4), (16, 128, 8), (33, 72, 8), (64, 256, 8),
          (65, 200, 64), (130, 64, 1), (129, 33, 33), (40, 384, 17), (20, 512, 8), (19, 1000, 10),
          (9, 1024, 64), (600, 16, 2)]


@pytest.mark.parametrize("pad", [0.0, 0.3])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_against_oracle(gpu, T, E, k, dtype, pad):
    print(f"router T={T} E={E} k={k} {dtype} pad={pad}", flush=True)
    z, mask = _case(T, E, dtype, T + E, pad)
    dev, dmask = z.to(gpu), None if mask is None else mask.to(gpu)
    eps = (E / 8 + 12) * U
    g = synth.gen(7)
    gw, gl = torch.randn(T, k, generator=g), torch.randn((), generator=g)
    for renorm in (True, False):
        w, ids = mi.moe_route_topk(dev, k, renormalize=renorm, token_mask=dmask)
        rw, rids = O.topk(z.double(), k, renorm, mask)
        assert np.array_equal(ids.cpu().numpy(), rids)
        _near(w, rw, (eps + k * U) * rw, torch.float32, "weights")
        loss, counts, slopes = mi.moe_balance_loss(dev, ids, coef=0.5, token_mask=dmask)
        rl, rc, rs = O.balance(z.double(), rids, 0.5, mask)
        assert counts.dtype == torch.int32 and np.array_equal(counts.cpu().numpy(), rc)
        _near(slopes, rs, 4 * U * rs, torch.float32, "slopes")
        _near(loss, np.float64(rl), (eps + (T / 8 + 40) * U) * abs(rl), torch.float32, "loss")
        grads = dict(topk_ids=ids, topk_weights=w, grad_weights=gw.to(gpu), renormalize=renorm)
        bal = dict(slopes=slopes, grad_loss=gl.to(gpu))
        for through, by in ((grads, 0), (bal, 1), ({**grads, **bal}, 2)):
            for gd in (None, torch.float32):
                got = mi.moe_route_backward(dev, token_mask=dmask, grad_dtype=gd, **through)
                assert got.dtype == (gd or dtype)
                ref, mag = O.backward(z.double(), k, rids, rw, gw.double() if by != 1 else None, renorm,
                                      rs if by else None, float(gl), mask)
                _near(got, ref, (2 * eps + (E / 8 + 2 * k + 12) * U) * mag, got.dtype, "gradient")
