"""The combine of permuted rows and its gradients on the GPU against the fp64 oracle.

Tolerances, u = 2^-24: the combine is top_k fp32 fmas, so at most top_k u times
the sum of the terms' absolute values, and half a step of the output's type.  A
row's gradient is one fp32 product and one rounding to its type.  A weight's
gradient is a chain of at most H / 64 fmas a lane (and 6 additions across the
lanes): (H / 64 + 8) u times the sum of absolute values.
"""
import numpy as np
import pytest
import torch

import synth
from moe_expert_grouped_amd import (moe_combine_rows, moe_combine_rows_backward, moe_permute_rows,
                                    moe_permute_rows_backward, moe_route_permutation)
from oracle import combine as C

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _np(t):
    return t.detach().cpu().double().numpy()


def _near(got, ref, tol, dtype, what):
    t = tol + HALF[dtype] * np.abs(ref) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    err = np.abs(_np(got) - ref)
    assert (err <= t).all(), f"{what}: {np.argwhere(~(err <= t))[:4]}"


def _case(T, k, H, P, dtype, seed):
    """A permutation into P rows with absent slots: entries -1 and past the rows."""
    g = synth.gen(seed)
    perm = torch.full((T * k,), -1, dtype=torch.int32)
    n = min(T * k, P)
    slots = torch.randperm(T * k, generator=g)[:n]
    perm[slots] = torch.randperm(P, generator=g)[:n].to(torch.int32)
    off = torch.rand(T * k, generator=g)
    perm[off < 0.1] = -1
    perm[off > 0.95] = P + 5
    rows = torch.randn(P, H, generator=g).to(dtype)
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    w.view(-1)[perm < 0] = float("nan")  # an absent slot's weight is not looked at
    return perm, rows, w


SHAPES = [(1, 1, 8, 1), (1, 8, 4096, 8), (3, 2, 264, 6), (17, 6, 528, 80), (64, 8, 1024, 600),
          (5, 33, 72, 170), (130, 3, 2056, 390), (2, 9, 7168, 18), (40, 4, 136, 0)]


@pytest.mark.parametrize("out_dtype", [None, torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,k,H,P", SHAPES)
def test_combine_against_oracle(gpu, T, k, H, P, dtype, out_dtype):
    print(f"moe_combine_rows T={T} k={k} H={H} P={P} {dtype} -> {out_dtype}", flush=True)
    perm, rows, w = _case(T, k, H, P, dtype, T + H)
    od = out_dtype or dtype
    out = torch.full((T, H), 7.0, dtype=od, device=gpu)
    got = moe_combine_rows(rows.to(gpu), perm.to(gpu), w.to(gpu), out_dtype=out_dtype, out=out)
    ref, mag = C.combine_rows(rows.double(), perm, w, T, k)
    _near(got, ref, k * U * mag, od, "combine")
    got = moe_permute_rows_backward(rows.to(gpu), perm.to(gpu), k, out_dtype=out_dtype)
    ref, mag = C.combine_rows(rows.double(), perm, None, T, k)
    _near(got, ref, k * U * mag, od, "permute backward")


@pytest.mark.parametrize("go_dtype", DTYPES, ids=str)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,k,H,P", SHAPES)
def test_combine_backward_against_oracle(gpu, T, k, H, P, dtype, go_dtype):
    print(f"moe_combine_rows_backward T={T} k={k} H={H} P={P} {dtype} {go_dtype}", flush=True)
    perm, rows, w = _case(T, k, H, P, dtype, T + H + 1)
    go = torch.randn(T, H, generator=synth.gen(T)).to(go_dtype)
    gr = torch.full((P, H), 7.0, dtype=dtype, device=gpu)
    dev = [t.to(gpu) for t in (go, rows, perm, w)]
    grad_rows, grad_w = moe_combine_rows_backward(*dev, grad_rows=gr)
    torch.cuda.synchronize()
    rr, rw, mag, hit = C.combine_rows_backward(go.double(), rows.double(), perm, w)
    _near(grad_rows[torch.from_numpy(hit).to(gpu)], rr[hit], U * np.abs(rr[hit]), dtype, "rows")
    assert (_np(grad_rows)[~hit] == 7.0).all()
    _near(grad_w, rw, (H / 64 + 8) * U * mag, torch.float32, "weights")
    # the inverse: every row is written, zeros where no slot points
    inv = torch.full((P,), -1, dtype=torch.int32)
    here = (perm >= 0) & (perm < P)
    inv[perm[here].long()] = torch.nonzero(here)[:, 0].to(torch.int32)
    gr2 = torch.full((P, H), 7.0, dtype=dtype, device=gpu)
    again, grad_w2 = moe_combine_rows_backward(*dev, permuted_idx_to_expanded_idx=inv.to(gpu),
                                               grad_rows=gr2)
    assert torch.equal(grad_w2, grad_w)
    assert not _np(again)[~hit].any()
    fresh, none = moe_combine_rows_backward(*dev, with_weights=False)
    assert none is None and torch.equal(fresh, again)


def test_gradients_against_differences(gpu):
    """fp32: the combine is linear in the rows and in the weights, so central
    differences along a direction are exact up to the roundings of the two
    sums of T * k * H terms, each at most (k + 1) u of its size."""
    T, k, H, P = 6, 3, 72, 18
    perm, rows, w = _case(T, k, H, P, torch.float32, 11)
    w = torch.nan_to_num(w)
    g = synth.gen(12)
    go, dr, dw = (torch.randn(s, generator=g) for s in ((T, H), (P, H), (T, k)))
    dev = lambda *ts: [t.to(gpu) for t in ts]
    print("combine gradients against differences", flush=True)
    gr, gw = moe_combine_rows_backward(*dev(go, rows, perm, w))
    gx = moe_permute_rows_backward(*dev(rows, perm), k)

    def loss(r, v):
        return float((_np(moe_combine_rows(*dev(r, perm, v))) * go.double().numpy()).sum())

    size = np.abs(_np(rows)).max() * H * T * k * 4
    tol = 8 * (k + 2) * U * size
    assert abs((loss(rows + dr, w) - loss(rows - dr, w)) / 2 - (_np(gr) * _np(dr)).sum()) <= tol
    assert abs((loss(rows, w + dw) - loss(rows, w - dw)) / 2 - (_np(gw) * _np(dw)).sum()) <= tol
    # the copy to expert order: <permute(x), rows> = <x, its gradient at rows>
    x = torch.randn(T, H, generator=g)
    px = moe_permute_rows(x.to(gpu), perm.to(gpu), k, P)
    hit = (perm >= 0) & (perm < P)
    left = (_np(px) * _np(rows)).sum()
    assert abs(left - (_np(x) * _np(gx)).sum()) <= tol
    assert hit.any()


def test_route_permute_combine_round_trip(gpu):
    """Routing, the copy to expert order and the way back: weights that sum
    to one over the routed slots give the tokens back."""
    T, k, E, H = 515, 8, 24, 264
    ids = synth.routing_ids(seed=3, T=T, top_k=k, E=E, invalid_frac=0.0).to(gpu)
    x = synth.bf16_normal((T, H), 1.0, synth.gen(4)).to(gpu)
    print("route, permute, combine", flush=True)
    _, perm, inv = moe_route_permutation(ids, E, with_inverse=True)
    rows = moe_permute_rows(x, perm, k)
    w = torch.full((T, k), 1.0 / k, device=gpu)
    out = moe_combine_rows(rows, perm, w)
    assert torch.equal(out.view(torch.int16), x.view(torch.int16))  # 1/8 and its sums are exact
    gr, _ = moe_combine_rows_backward(x, rows, perm, w, permuted_idx_to_expanded_idx=inv)
    gx = moe_permute_rows_backward(gr, perm, k)
    assert torch.equal(gx.view(torch.int16), x.view(torch.int16))


def test_empty_calls(gpu):
    print("combine, empty inputs", flush=True)
    i = torch.empty(0, dtype=torch.int32, device=gpu)
    rows, w = torch.ones(3, 16, device=gpu), torch.empty(0, 2, device=gpu)
    assert moe_combine_rows(rows, i, w).shape == (0, 16)
    go = torch.empty(0, 16, device=gpu)
    gr, gw = moe_combine_rows_backward(go, rows, i, w)
    assert not gr.any() and gw.shape == (0, 2)
    inv = torch.full((3,), -1, dtype=torch.int32, device=gpu)
    gr, _ = moe_combine_rows_backward(go, rows, i, w, permuted_idx_to_expanded_idx=inv,
                                      grad_rows=torch.ones_like(rows))
    assert not gr.any()
    torch.cuda.synchronize()


def test_views_broadcast_gradients_and_shared_rows(gpu):
    """Strided and broadcast inputs give what their copies give; two slots may read
    the same row on the way back to the tokens."""
    T, k, H, P = 9, 3, 264, 20
    g = synth.gen(81)
    rows = torch.randn(P, 2 * H, generator=g).to(torch.bfloat16).to(gpu)[:, ::2]
    perm = torch.randint(0, P, (T, k), generator=g, dtype=torch.int32)
    w = torch.rand(k, T, generator=g).to(gpu).t()
    print("moe_combine_rows of shared rows, views", flush=True)
    got = moe_combine_rows(rows, perm.to(gpu), w, out_dtype=torch.float32)
    ref, mag = C.combine_rows(_np(rows), perm.numpy(), _np(w), T, k)
    _near(got, ref, (k + 1) * U * mag, torch.float32, "shared rows")
    gx = moe_permute_rows_backward(rows, perm.to(gpu), k, out_dtype=torch.float32)
    ref, mag = C.combine_rows(_np(rows), perm.numpy(), None, T, k)
    _near(gx, ref, (k + 1) * U * mag, torch.float32, "gradient of a shared copy")

    print("moe_combine_rows_backward of a broadcast gradient", flush=True)
    own = torch.randperm(T * k, generator=g).to(torch.int32).to(gpu)
    rows = torch.randn(T * k, 2 * H, generator=g).to(gpu)[:, ::2]
    for go in (torch.randn(1, H, generator=g).to(gpu).expand(T, H),
               torch.randn(T, 1, generator=g).to(gpu).expand(T, H),
               torch.ones((), device=gpu).expand(T, H)):
        a = moe_combine_rows_backward(go, rows, own, w)
        b = moe_combine_rows_backward(go.contiguous(), rows.contiguous(), own, w.contiguous())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        ref, ref_w, mag, _ = C.combine_rows_backward(_np(go), _np(rows), own.cpu().numpy(), _np(w))
        _near(a[0], ref, 0.0, torch.float32, "rows' gradient")
        _near(a[1], ref_w, (H + 1) * U * mag, torch.float32, "weights' gradient")
