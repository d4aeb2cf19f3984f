"""The adapters' projection where it can go wrong: rows without adapters, empty calls, NaN
and infinities of one request, strides, several passes over the rows, equal bits of
equal calls, exact differences, other streams and captured graphs."""
import numpy as np
import pytest
import torch

import moe_expert_grouped_amd as mi
import synth
from oracle import lora_mm as O

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16
ONE = (1, 136, 264, 3, 32)  # a single row (one launch)
# few rows (two launches) and many (the plan and the MFMA tiles)
SIZES = [(20, 136, 264, 3, 16), (400, 520, 264, 5, 40), (1500, 264, 136, 4, 24)]


def _case(T, N, K, L, R, dtype, gpu, seed=0):
    g = synth.gen(seed + T)
    n = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(dtype).to(gpu)
    ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32).to(gpu)
    scale = torch.exp(0.3 * torch.randn(L, generator=g)).to(gpu)
    return (n(T, K), n(N, K, std=K ** -0.5), n(L, R, K, std=K ** -0.5), n(L, N, R, std=0.3), ids, scale), n(T, N)


def _all(args, go, **kw):
    out, act = mi.mm_lora(*args, with_act=True, **kw)
    return (out, act, *mi.mm_lora_backward(go, *args, act=act, grad_dtype=torch.float32))


def _same(p, q):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(p, q))


@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
@pytest.mark.parametrize("T,N,K,L,R", [ONE, *SIZES])
def test_no_row_has_an_adapter(gpu, T, N, K, L, R, dtype):
    print(f"mm_lora without adapters T={T} {dtype}", flush=True)
    (x, w, a, b, ids, scale), go = _case(T, N, K, L, R, dtype, gpu)
    a[:], b[:] = float("nan"), float("inf")  # not looked at
    for off in (-1, L, 2 ** 31 - 1, -2 ** 31):
        none = torch.full_like(ids, off)
        out, act, gx, ga, gb = _all((x, w, a, b, none, scale), go)
        torch.cuda.synchronize()
        assert not act.any() and not ga.any() and not gb.any()
        assert torch.allclose(out.float(), x.float() @ w.float().t(), rtol=0.02, atol=0.02)
        assert torch.allclose(gx.float(), go.float() @ w.float(), rtol=0.02, atol=0.05 * N ** 0.5 * K ** -0.5)


@pytest.mark.parametrize("R", [8, 16, 24, 32])
def test_one_rows_own_adapter(gpu, R):
    """Small whole numbers, so that every sum is exact; the other adapters hold NaN."""
    print(f"mm_lora of one row R={R}", flush=True)
    g = synth.gen(R)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g).to(BF).to(gpu)
    for N, K in ((8, 8), (24, 520), (136, 1032)):
        for l in (0, 2):
            x, w, a, b = whole(1, K), whole(N, K), whole(3, R, K), whole(3, N, R)
            others = [i for i in range(3) if i != l]
            a[others], b[others] = float("nan"), float("nan")
            ids = torch.tensor([l], dtype=torch.int32, device=gpu)
            out, act = mi.mm_lora(x, w, a, b, ids, out_dtype=torch.float32, with_act=True)
            torch.cuda.synchronize()
            v = x.double().cpu() @ a[l].double().cpu().t()
            assert torch.equal(act.double().cpu(), v)
            assert torch.equal(out.double().cpu(), x.double().cpu() @ w.double().cpu().t() + v @ b[l].double().cpu().t())


@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
def test_empty_calls(gpu, dtype):
    print(f"mm_lora with no rows {dtype}", flush=True)
    (x, w, a, b, ids, scale), go = _case(20, 136, 264, 3, 16, dtype, gpu)
    args = (x[:0], w, a, b, ids[:0], scale)
    out, act = mi.mm_lora(*args, with_act=True)
    assert out.shape == (0, 136) and act.shape == (0, 16)
    ga, gb = torch.full((3, 16, 264), 7.0, device=gpu), torch.full((3, 136, 16), 7.0, device=gpu)
    gx, _, _ = mi.mm_lora_backward(go[:0], *args, grad_a=ga, grad_b=gb, grad_dtype=torch.float32)
    torch.cuda.synchronize()
    assert gx.shape == (0, 264) and not ga.any() and not gb.any()


@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
@pytest.mark.parametrize("T,N,K,L,R", SIZES)
def test_one_requests_nan_is_its_own(gpu, T, N, K, L, R, dtype):
    """NaN and infinities in one adapter's bank, and in one row, leave every other
    request's bits as they were."""
    print(f"mm_lora with NaN T={T} {dtype}", flush=True)
    (x, w, a, b, ids, scale), go = _case(T, N, K, L, R, dtype, gpu)
    ref = _all((x, w, a, b, ids, scale), go)
    for bad in (float("nan"), float("inf")):
        a2, b2 = a.clone(), b.clone()
        a2[1, 3, 5], b2[1, 7, 2] = bad, bad
        got = _all((x, w, a2, b2, ids, scale), go)
        torch.cuda.synchronize()
        rest = ids != 1
        for i in (0, 1, 2):
            assert _same([got[i][rest]], [ref[i][rest]]), (bad, i)
            assert not torch.isfinite(got[i][~rest]).all()
        others = torch.arange(L, device=gpu) != 1
        assert _same([got[3][others], got[4][others]], [ref[3][others], ref[4][others]])
        x2, go2, row = x.clone(), go.clone(), T // 2
        x2[row, 3], go2[row, 1] = bad, bad
        ids2 = ids.clone()
        ids2[row] = 2
        ref2, got = _all((x, w, a, b, ids2, scale), go), _all((x2, w, a, b, ids2, scale), go2)
        torch.cuda.synchronize()
        rest = torch.arange(T, device=gpu) != row
        others = torch.arange(L, device=gpu) != 2
        for i in (0, 1, 2):
            assert _same([got[i][rest]], [ref2[i][rest]]), (bad, i)
        assert _same([got[3][others], got[4][others]], [ref2[3][others], ref2[4][others]])
        # the row's own products, as in 64 bits: +-inf or NaN where they are
        want = x2[row].double().cpu() @ w.double().cpu().t()
        v = x2[row].double().cpu() @ a[2].double().cpu().t()
        want = want + scale[2].double().cpu() * (v @ b[2].double().cpu().t())
        assert torch.equal(torch.isnan(got[0][row].cpu()), torch.isnan(want)), bad


@pytest.mark.parametrize("T,N,K,L,R", SIZES)
def test_strides_and_given_outputs(gpu, T, N, K, L, R):
    print(f"mm_lora strides T={T}", flush=True)
    args, go = _case(T, N, K, L, R, BF, gpu)
    ref = _all(args, go)
    wide = lambda t: torch.cat([t, torch.full_like(t, 9.0)], -1)[..., : t.shape[-1]]
    turned = lambda t: t.transpose(-1, -2).contiguous().transpose(-1, -2)
    x, w, a, b, ids, scale = args
    got = _all((wide(x), turned(w), turned(a), wide(b), torch.stack([ids, ids], 1)[:, 0], wide(scale)), wide(go))
    assert _same(ref, got)
    out, act = torch.full_like(ref[0], 3.0), torch.full_like(ref[1], 3.0)
    ws = torch.full((mi.lora_mm_workspace_bytes(T, N, K, L, R),), 255, dtype=torch.uint8, device=gpu)
    assert mi.mm_lora(*args, out=out, act=act, workspace=ws)[0] is out
    grads = [torch.full_like(t, 3.0) for t in ref[2:]]
    ws = torch.full((mi.lora_mm_workspace_bytes(T, N, K, L, R, backward=True),), 255, dtype=torch.uint8, device=gpu)
    mi.mm_lora_backward(go, *args, act=act, grad_x=grads[0], grad_a=grads[1], grad_b=grads[2],
                        grad_dtype=torch.float32, workspace=ws)
    assert _same(ref, [out, act, *grads])
    with pytest.raises(ValueError, match="workspace needs"):
        mi.mm_lora(*args, workspace=ws[:8])
    with pytest.raises(ValueError, match="out must be"):
        mi.mm_lora(*args, out=out.float())


def test_equal_calls_equal_bits(gpu):
    """The sums' order depends on sizes and ids alone; rows in another order give the
    same rows."""
    print("mm_lora repeated", flush=True)
    for T, N, K, L, R in SIZES + [(3000, 512, 512, 2, 16)]:
        args, go = _case(T, N, K, L, R, BF, gpu)
        ref = _all(args, go)
        for _ in range(3):
            assert _same(ref, _all(args, go))
        order = torch.randperm(T, generator=synth.gen(3)).to(gpu)
        x, w, a, b, ids, scale = args
        got = _all((x[order], w, a, b, ids[order], scale), go[order])
        assert _same([t[order] for t in ref[:3]], got[:3])


@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
@pytest.mark.parametrize("T", [12, 300])
def test_gradients_against_differences(gpu, T, dtype):
    """Small integers: the forward is exact, and bilinear, so the difference of its products
    with grad_out over a step of 2 is twice the gradient, exactly."""
    print(f"mm_lora differences T={T} {dtype}", flush=True)
    N, K, L, R = 72, 64, 3, 8
    g = synth.gen(T)
    i = lambda *s, top=2: torch.randint(-top, top + 1, s, generator=g).to(dtype).to(gpu)
    x, w, a, b, go = i(T, K), i(N, K), i(L, R, K, top=1), i(L, N, R, top=1), i(T, N, top=1)
    ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32).to(gpu)
    scale = torch.tensor([1.0, 2.0, 3.0], device=gpu)
    grads = mi.mm_lora_backward(go, x, w, a, b, ids, scale, grad_dtype=torch.float32)
    value = lambda: (mi.mm_lora(x, w, a, b, ids, scale, out_dtype=torch.float32).double() * go.double()).sum().item()
    for t, grad, at in ((x, grads[0], [(0, 0), (T - 1, K - 1), (T // 2, 7)]), (a, grads[1], [(0, 0, 0), (2, 7, 63), (1, 3, 9)]),
                        (b, grads[2], [(0, 0, 0), (2, 71, 7), (1, 30, 5)])):
        for p in at:
            keep = t[p].item()
            t[p] = keep + 1
            up = value()
            t[p] = keep - 1
            down = value()
            t[p] = keep
            want = torch.tensor((up - down) / 2).to(grad.dtype)
            assert grad[p].item() == want.item(), (p, grad[p].item(), want.item())


def test_rows_past_a_31_bit_offset(gpu):
    """x of more than 2 GB is taken in several passes, each with its own plan."""
    N, K, L, R = 64, 65536, 2, 8
    T = 2 ** 30 // K + 300
    print(f"mm_lora several passes T={T} K={K}", flush=True)
    g = synth.gen(9, gpu)
    x = torch.randint(-1, 2, (T, K), generator=g, device=gpu, dtype=torch.int8).to(BF)
    w = torch.randint(-1, 2, (N, K), generator=g, device=gpu).to(BF)
    a = (torch.rand((L, R, K), generator=g, device=gpu) < 2e-4).to(BF)
    b = torch.randint(-2, 3, (L, N, R), generator=g, device=gpu).to(BF)
    ids = torch.randint(-1, L, (T,), generator=g, device=gpu).to(torch.int32)
    out, act = mi.mm_lora(x, w, a, b, ids, out_dtype=torch.float32, with_act=True)
    torch.cuda.synchronize()
    rows = torch.cat([torch.arange(3), torch.arange(2 ** 30 // K - 260, T, 7)])
    ref, mag, ra, _ = O.mm_lora(x[rows].double().cpu(), w.double().cpu(), a.double().cpu(), b.double().cpu(), ids[rows].cpu())
    assert mag.max() < 2 ** 24
    assert np.array_equal(out[rows].double().cpu().numpy(), ref) and np.array_equal(act[rows].double().cpu().numpy(), ra)
    # the gradient of the rows of a wide output, in passes too; the adapters' are refused
    w2, a2, b2 = w.t().contiguous(), torch.zeros((L, R, N), dtype=BF, device=gpu), torch.zeros((L, K, R), dtype=BF, device=gpu)
    gx, _, _ = mi.mm_lora_backward(x, out[:, :N].to(BF), w2, a2, b2, ids, with_adapters=False)
    torch.cuda.synchronize()
    want = torch.from_numpy(x[rows].double().cpu().numpy() @ w2.double().cpu().numpy()).to(BF)
    assert torch.equal(gx[rows].cpu(), want)
    with pytest.raises(NotImplementedError, match="take at most"):
        mi.mm_lora_backward(x, out[:, :N].to(BF), w2, a2, b2, ids)


@pytest.mark.parametrize("T,N,K,L,R", [ONE, *SIZES])
def test_in_a_graph(gpu, T, N, K, L, R):
    print(f"mm_lora in a graph T={T}", flush=True)
    args, go = _case(T, N, K, L, R, BF, gpu)
    x, w, a, b, ids, scale = args
    new = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=gpu)
    bufs = [new(T, N, dt=BF), new(T, R), new(T, K, dt=BF), new(L, R, K), new(L, N, R)]
    wf = torch.empty(mi.lora_mm_workspace_bytes(T, N, K, L, R), dtype=torch.uint8, device=gpu)
    wb = torch.empty(mi.lora_mm_workspace_bytes(T, N, K, L, R, backward=True), dtype=torch.uint8, device=gpu)

    def step(o):
        mi.mm_lora(*args, out=o[0], act=o[1], workspace=wf)
        mi.mm_lora_backward(go, *args, act=o[1], grad_x=o[2], grad_a=o[3], grad_b=o[4], grad_dtype=torch.float32, workspace=wb)

    step(bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(bufs)
    for rnd in range(4):
        g = synth.gen(50 + rnd, gpu)
        x.copy_(torch.randn(x.shape, generator=g, device=gpu))
        go.copy_(torch.randn(go.shape, generator=g, device=gpu))
        b.copy_(torch.randn(b.shape, generator=g, device=gpu) * 0.2)
        ids.copy_(torch.randint(-1, L if rnd else 1, ids.shape, generator=g, device=gpu))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(bufs, _all(args, go)), f"replay {rnd}"


def test_two_streams(gpu):
    """Calls on two streams at once, each with its own workspace, on the streams that
    are current."""
    print("mm_lora on two streams", flush=True)
    cases = [_case(*s, BF, gpu, seed=7) for s in (SIZES[1], SIZES[2])]
    refs = [_all(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(gpu) for _ in cases]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _all(*cases[i])
    torch.cuda.synchronize()
    assert _same(refs[0], got[0]) and _same(refs[1], got[1])
