"""The combine's gradient with an inverse permutation that does not go with the
permutation: every row is written, by one slot.

Tolerances as in test_gpu_combine: a row's gradient is one fp32 product and one
rounding to its type, a weight's at most H / 64 + 8 roundings of the terms' absolute
sum.
"""
import numpy as np
import pytest
import torch

import synth
from moe_expert_grouped_amd import moe_combine_rows_backward, moe_route_permutation
from oracle import combine as C

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def _np(t):
    return t.detach().cpu().double().numpy()


def _inputs(T, k, H, dtype, seed, gpu):
    g = synth.gen(seed)
    go = torch.randn(T, H, generator=g).to(dtype).to(gpu)
    rows = torch.randn(T * k, H, generator=g).to(dtype).to(gpu)
    return go, rows, torch.rand(T, k, generator=g).to(gpu)


def _by_definition(go, w, perm, inv):
    """Row p: the gradient of slot inv[p] where that slot points at p, else zeros."""
    k, out = w.shape[1], np.zeros((inv.size, go.shape[1]))
    for p, s in enumerate(inv):
        if 0 <= s < perm.size and perm[s] == p:
            out[p] = w[s // k, s % k] * go[s // k]
    return out


def _check(go, rows, perm, w, inv, what):
    gr = torch.full_like(rows, 7.0)
    got, gw = moe_combine_rows_backward(go, rows, perm, w, permuted_idx_to_expanded_idx=inv,
                                        grad_rows=gr)
    torch.cuda.synchronize()
    p, i = perm.cpu().numpy(), inv.cpu().numpy()
    want = _by_definition(_np(go), _np(w), p, i)
    step = 2.0 ** -25 if rows.dtype == torch.float16 else 0.0
    tol = (U + HALF[rows.dtype]) * np.abs(want) + step * (want != 0)
    assert (np.abs(_np(got) - want) <= tol).all(), what
    _, rw, mag, _ = C.combine_rows_backward(_np(go), _np(rows), p, _np(w))
    tol = (go.shape[1] / 64 + 8) * U * mag + U * np.abs(rw)
    assert (np.abs(_np(gw) - rw) <= tol).all(), what
    again, gw2 = moe_combine_rows_backward(go, rows, perm, w, permuted_idx_to_expanded_idx=inv)
    assert torch.equal(again, got) and torch.equal(gw2, gw)


@pytest.mark.parametrize("dtype", list(HALF), ids=str)
def test_slots_taken_out_after_the_routing(gpu, dtype):
    """Tokens dropped by setting their slots to -1: their rows, which the routing's
    inverse still names, get zeros."""
    T, k, E, H = 77, 4, 9, 264
    ids = synth.routing_ids(seed=5, T=T, top_k=k, E=E, invalid_frac=0.1).to(gpu)
    _, perm, inv = moe_route_permutation(ids, E, with_inverse=True)
    go, rows, w = _inputs(T, k, H, dtype, 6, gpu)
    perm.view(T, k)[::3] = -1
    print(f"moe_combine_rows_backward, dropped tokens {dtype}", flush=True)
    _check(go, rows, perm, w, inv, "dropped tokens")


@pytest.mark.parametrize("dtype", list(HALF), ids=str)
def test_inverse_of_another_permutation(gpu, dtype):
    """Entries that name no slot, a slot past the end, or a slot with another row."""
    T, k, H = 50, 3, 520
    g = synth.gen(8)
    perm = torch.randperm(T * k, generator=g).to(torch.int32)
    inv = torch.empty_like(perm)
    inv[perm.long()] = torch.arange(T * k, dtype=torch.int32)
    inv[::7], inv[3::11], inv[5::13] = -1, T * k + 9, 2 ** 31 - 1
    inv[20:40] = inv[20:40].flip(0)
    go, rows, w = _inputs(T, k, H, dtype, 9, gpu)
    print(f"moe_combine_rows_backward, another inverse {dtype}", flush=True)
    _check(go, rows, perm.to(gpu), w, inv.to(gpu), "another inverse")


@pytest.mark.parametrize("dtype", list(HALF), ids=str)
def test_shared_rows_have_the_named_slot_s_gradient(gpu, dtype):
    T, k, H = 40, 4, 2056
    g = synth.gen(10)
    perm = torch.randint(0, T * k, (T * k,), generator=g).to(torch.int32)
    inv = torch.full((T * k,), -1, dtype=torch.int32)
    inv[perm.long()] = torch.arange(T * k, dtype=torch.int32)
    go, rows, w = _inputs(T, k, H, dtype, 11, gpu)
    print(f"moe_combine_rows_backward, shared rows {dtype}", flush=True)
    _check(go, rows, perm.to(gpu), w, inv.to(gpu), "shared rows")
