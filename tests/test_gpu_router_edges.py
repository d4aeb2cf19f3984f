"""The router where it can go wrong: NaN, infinities and masked rows, equal logits, ids
outside the experts and repeated ones, given counts, unaligned rows, outputs in place, equal bits,
graphs, and gradients against differences of the 64-bit loss."""
import numpy as np
import pytest
import torch

import moe_expert_grouped_amd as mi
import synth
from oracle import router as O

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("E", [6, 64, 129, 520])
def test_special_values(gpu, E, dtype):
    print(f"router special values E={E} {dtype}", flush=True)
    low = torch.finfo(dtype).min
    z = torch.zeros(9, E, dtype=dtype)
    z[0] = low                       # a mask of the type's lowest value: an even softmax
    z[1], z[1, E - 1] = low, 1.0
    z[2], z[2, 3] = -INF, 2.0        # one expert left
    z[3, 4] = NAN
    z[4, 2] = INF
    z[5] = -INF
    z[6] = -0.0                      # equal to the zeros beside them
    z[6, 1::2] = 0.0
    z[7] = torch.arange(E, dtype=torch.float32).to(dtype)
    z[8, 5], z[8, 1] = NAN, -NAN
    w, ids = mi.moe_route_topk(z.to(gpu), 3)
    w, ids = w.cpu(), ids.cpu()
    assert ids[0].tolist() == [0, 1, 2] and torch.allclose(w[0], torch.full((3,), 1 / 3))
    assert ids[1].tolist() == [E - 1, 0, 1] and w[1].tolist() == [1.0, 0.0, 0.0]
    assert ids[2].tolist() == [3, -1, -1] and w[2].tolist() == [1.0, 0.0, 0.0]
    assert ids[3, 0] == 4 and w[3].isnan().all()
    assert ids[4, 0] == 2 and w[4, 0].isnan()
    assert ids[5].tolist() == [-1] * 3 and not w[5].any()
    assert ids[6].tolist() == [0, 1, 2]
    want = O.topk(z[7:8].double().numpy(), 3)
    assert ids[7].tolist() == want[1][0].tolist() and np.allclose(w[7], want[0][0], rtol=1e-5)
    assert ids[8, :2].tolist() == [1, 5] and w[8].isnan().all()
    # the gradient of rows that leave nothing
    gw, gl = torch.ones(9, 3, device=gpu), torch.ones((), device=gpu)
    sl = torch.rand(E, device=gpu)
    for renorm in (True, False):
        ww, ii = mi.moe_route_topk(z.to(gpu), 3, renormalize=renorm)
        g = mi.moe_route_backward(z.to(gpu), topk_ids=ii, topk_weights=ww, grad_weights=gw, renormalize=renorm,
                                  slopes=sl, grad_loss=gl, grad_dtype=torch.float32).cpu()
        assert not g[5].any() and g[3].isnan().any() and torch.isfinite(g[[0, 1, 2, 6, 7]]).all()
        assert not g[2].any()  # one expert's softmax is 1 whatever its logit


def test_masked_tokens_are_not_looked_at(gpu):
    print("router masked tokens", flush=True)
    T, E, k = 50, 72, 4
    z = torch.randn(T, E, generator=synth.gen(1)).to(gpu)
    mask = (torch.rand(T, generator=synth.gen(2)) < 0.6).to(gpu)
    bad = z.clone()
    bad[~mask] = NAN
    gw, gl = torch.randn(T, k, device=gpu), torch.ones((), device=gpu)

    def run(z, mask):
        w, ids = mi.moe_route_topk(z, k, token_mask=mask)
        loss, counts, slopes = mi.moe_balance_loss(z, ids, token_mask=mask, coef=0.3)
        g = mi.moe_route_backward(z, topk_ids=ids, topk_weights=w, grad_weights=gw, slopes=slopes, grad_loss=gl, token_mask=mask)
        return w, ids, loss, counts, slopes, g

    ref, got = run(z, mask), run(bad, mask.to(torch.uint8))
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    assert not got[0][~mask].any() and (got[1][~mask] == -1).all() and not got[5][~mask].any()
    # masked tokens whose ids are still there count nowhere; no token left: zeros
    ids = torch.zeros(T, k, dtype=torch.int32, device=gpu)
    loss, counts, slopes = mi.moe_balance_loss(bad, ids, token_mask=mask)
    assert counts[0] == k * mask.sum() and counts.sum() == counts[0] and torch.isfinite(loss)
    loss, counts, slopes = mi.moe_balance_loss(bad, ids, token_mask=torch.zeros_like(mask))
    assert loss == 0 and not counts.any() and not slopes.any()


@pytest.mark.parametrize("T", [0, 1, 40, 700])
def test_counts_and_given_counts(gpu, T):
    print(f"balance given counts T={T}", flush=True)
    E, k = 70, 5
    g = synth.gen(T)
    z = torch.randn(T, E, generator=g)
    ids = torch.randint(-3, E + 4, (T, k), generator=g).to(torch.int32)
    given = torch.randint(0, 2 ** 30, (E,), generator=g).to(torch.int32)  # their sum passes 32 bits
    for by in (None, given):
        loss, counts, slopes = mi.moe_balance_loss(z.to(gpu), ids.to(gpu), coef=2.0, given_counts=None if by is None else by.to(gpu))
        rl, rc, rs = O.balance(z.double().numpy(), ids.numpy(), 2.0, given=None if by is None else by.numpy())
        assert np.array_equal(counts.cpu().numpy(), rc)
        assert np.allclose(slopes.cpu().double(), rs, rtol=4 * 2.0 ** -24, atol=0)
        assert abs(loss.item() - rl) <= (T / 8 + 60) * 2.0 ** -24 * abs(rl)


def test_repeated_and_foreign_ids(gpu):
    """Two slots of a token with one expert, and slots with none."""
    print("router backward repeated ids", flush=True)
    T, E, k = 33, 24, 20
    g = synth.gen(4)
    z, gw = torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    ids = torch.randint(-2, 6, (T, k), generator=g).to(torch.int32)
    w = torch.rand(T, k, generator=g)
    for renorm in (True, False):
        got = mi.moe_route_backward(z.to(gpu), topk_ids=ids.to(gpu), topk_weights=w.to(gpu), grad_weights=gw.to(gpu), renormalize=renorm)
        ref, mag = O.backward(z.double().numpy(), k, ids.numpy(), w.double().numpy(), gw.double().numpy(), renorm)
        assert (np.abs(got.cpu().double().numpy() - ref) <= (2 * (E / 8 + 12) + E / 8 + 2 * k + 12) * 2.0 ** -24 * mag + 1e-30).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("E", [64, 61, 1000])
def test_unaligned_rows_and_in_place(gpu, E, dtype):
    print(f"router unaligned E={E} {dtype}", flush=True)
    T, k = 45, 6
    flat = torch.randn(T * E + 1, generator=synth.gen(E)).to(dtype).to(gpu)
    odd = flat[1:].view(T, E)  # contiguous, not 16-byte aligned
    z = odd.clone()
    w, ids = mi.moe_route_topk(z, k)
    w2, ids2 = mi.moe_route_topk(odd, k)
    assert torch.equal(w, w2) and torch.equal(ids, ids2)
    assert all(torch.equal(a, b) for a, b in zip(mi.moe_balance_loss(z, ids), mi.moe_balance_loss(odd, ids)))
    _, _, slopes = mi.moe_balance_loss(z, ids)
    kw = dict(topk_ids=ids, topk_weights=w, grad_weights=torch.ones_like(w), slopes=slopes, grad_loss=torch.ones((), device=gpu))
    ref = mi.moe_route_backward(z, **kw)
    assert torch.equal(ref, mi.moe_route_backward(odd, **kw))
    for gd in DTYPES:
        out = torch.zeros(T * E + 1, dtype=gd, device=gpu)[1:].view(T, E)
        assert torch.equal(mi.moe_route_backward(z, grad_logits=out, **kw), mi.moe_route_backward(z, grad_dtype=gd, **kw))
    wide = torch.cat([z, z], 1)[:, :E]  # rows apart
    assert torch.equal(mi.moe_route_topk(wide, k)[1], ids)
    mi.moe_route_backward(z, grad_logits=z, **kw)
    assert torch.equal(z, ref)


def test_equal_calls_equal_bits(gpu):
    print("router repeated", flush=True)
    for T, E in ((5000, 200), (40000, 64), (300, 1024)):
        z = torch.randn(T, E, generator=synth.gen(T)).to(gpu)
        w, ids = mi.moe_route_topk(z, 4)
        ref = mi.moe_balance_loss(z, ids)
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(ref, mi.moe_balance_loss(z, ids)))
        again = mi.moe_route_topk(z, 4)
        assert torch.equal(again[0], w) and torch.equal(again[1], ids)


def test_many_tokens(gpu):
    """More rows than one round of workgroups, sums against torch in 64 bits."""
    T, E, k = 150001, 40, 3
    print(f"router many tokens T={T}", flush=True)
    z = torch.randn(T, E, generator=synth.gen(5, gpu), device=gpu)
    w, ids = mi.moe_route_topk(z, k, renormalize=False)
    p = torch.softmax(z.double(), 1)
    want = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(ids.long(), want)
    assert torch.allclose(w.double(), p.gather(1, want), rtol=(E / 8 + 12) * 2.0 ** -24, atol=0)
    loss, counts, slopes = mi.moe_balance_loss(z, ids, coef=0.1)
    c = torch.bincount(want.flatten(), minlength=E)
    assert torch.equal(counts.long(), c)
    rs = 0.1 * E * c.double() / (T * k) / T
    rl = (p.sum(0) @ rs).item()
    # a lane adds T / (256 * 16) rows, a workgroup 16 and the second launch 16 + 16 partial sums
    assert abs(loss.item() - rl) <= (E / 8 + 12 + T / 4096 + 64) * 2.0 ** -24 * rl
    g = mi.moe_route_backward(z, slopes=slopes, grad_loss=torch.ones((), device=gpu))
    ref = p * (rs - (p * rs).sum(1, keepdim=True))
    mag = p * (rs + (p * rs).sum(1, keepdim=True))
    assert ((g.double() - ref).abs() <= (4 * E / 8 + 40) * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(gpu, renorm):
    """The kernels' gradient against central differences of the 64-bit value; the step's
    own error is its square times a third derivative of order 1 of the same terms."""
    print(f"router differences renorm={renorm}", flush=True)
    T, E, k, coef = 6, 20, 4, 0.5
    g = synth.gen(8)
    z, gw = torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    mask = torch.tensor([1, 1, 0, 1, 1, 1], dtype=torch.bool)
    w, ids = mi.moe_route_topk(z.to(gpu), k, renormalize=renorm, token_mask=mask.to(gpu))
    loss, counts, slopes = mi.moe_balance_loss(z.to(gpu), ids, coef=coef, token_mask=mask.to(gpu))
    got = mi.moe_route_backward(z.to(gpu), topk_ids=ids, topk_weights=w, grad_weights=gw.to(gpu), renormalize=renorm,
                                slopes=slopes, grad_loss=torch.full((), 0.7, device=gpu), token_mask=mask.to(gpu)).cpu().double().numpy()
    i, zd, gd = ids.cpu().numpy(), z.double().numpy(), gw.double().numpy()

    def value(z):
        v = 0.7 * O.balance(z, i, coef, mask)[0]
        for t in range(T):
            if mask[t]:
                p = O.softmax(z[t])[i[t]]
                v += ((p / p.sum() if renorm else p) * gd[t]).sum()
        return v

    for at in np.ndindex(z.shape):
        d = np.zeros_like(zd)
        d[at] = 1e-4
        assert abs((value(zd + d) - value(zd - d)) / 2e-4 - got[at]) < 1e-6 * (1 + np.abs(gd).max())


def test_in_a_graph(gpu):
    print("router in a graph", flush=True)
    T, E, k = 900, 96, 6
    z = torch.randn(T, E, device=gpu)
    gw, gl = torch.randn(T, k, device=gpu), torch.ones((), device=gpu)
    w, ids = torch.empty(T, k, device=gpu), torch.empty(T, k, dtype=torch.int32, device=gpu)
    loss, counts, slopes = torch.empty((), device=gpu), torch.empty(E, dtype=torch.int32, device=gpu), torch.empty(E, device=gpu)
    grad = torch.empty(T, E, device=gpu)
    ws = torch.empty(mi.balance_workspace_bytes(T, E), dtype=torch.uint8, device=gpu)

    def step(w, ids, loss, counts, slopes, grad, ws=None):
        mi.moe_route_topk(z, k, topk_weights=w, topk_ids=ids)
        mi.moe_balance_loss(z, ids, loss=loss, counts=counts, slopes=slopes, workspace=ws)
        mi.moe_route_backward(z, topk_ids=ids, topk_weights=w, grad_weights=gw, slopes=slopes, grad_loss=gl, grad_logits=grad)

    bufs = (w, ids, loss, counts, slopes, grad)
    step(*bufs, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*bufs, ws=ws)
    for rnd in range(4):
        z.copy_(torch.randn(T, E, generator=synth.gen(rnd, gpu), device=gpu) * (1 + rnd))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = [torch.empty_like(t) for t in bufs]
        step(*ref)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bufs, ref)), f"replay {rnd}"
