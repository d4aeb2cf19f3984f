"""Rows whose shared product and adapter's part cancel: 16-bit outputs hold the rounding of the
sum, whatever the number of rows, because x a^T and grad_out b keep their 24 bits.

Whole numbers below 2^24 throughout, so fp32 holds every product and sum: outputs are the
rounding of an exact value.  The activations have up to 20 bits, and w is the negative of
adapter 0's product but for a few entries, which leaves small sums.
"""
import pytest
import torch

import moe_expert_grouped_amd as mi
import synth
from oracle import lora_mm as O

pytestmark = pytest.mark.gpu

HALVES = [torch.bfloat16, torch.float16]
# one launch, few rows, 64 x 64, 128 x 128 and 256 x 256 tiles, a split k axis
SIZES = [(1, 136, 264, 2, 16), (20, 136, 264, 3, 16), (1100, 264, 520, 4, 40), (1100, 2056, 136, 3, 24),
         (4100, 2056, 136, 3, 64), (1100, 72, 2056, 3, 16), (1100, 72, 4680, 3, 16),
         (1100, 2056, 136, 3, 16), (4100, 2056, 136, 3, 16)]


def _whole(g, *shape, share=1.0):
    t = torch.randint(-200, 201, shape, generator=g)
    return torch.where(torch.rand(shape, generator=g) < share, t, 0)


def _ids(g, T, L):
    ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32)
    ids[::2] = 0
    return ids


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("T,N,K,L,R", SIZES)
def test_cancelling_outputs(gpu, T, N, K, L, R, dtype):
    print(f"mm_lora cancelling T={T} N={N} K={K} R={R} {dtype}", flush=True)
    g = synth.gen(T + N)
    x, a = _whole(g, T, K), _whole(g, L, R, K, share=24 / K)
    to = torch.arange(N) % R
    b = (to[:, None] == torch.arange(R)).long().expand(L, N, R)
    w = -a[0, to] + torch.randint(-1, 2, (N, K), generator=g) * (torch.rand(N, K, generator=g) < 4 / K)
    ids = _ids(g, T, L)
    ref, mag, act, _ = O.mm_lora(*(t.double().numpy() for t in (x, w, a, b)), ids)
    assert mag.max() < 2 ** 24 and (T == 1 or abs(act).max() > 2 ** 17)
    dev = [t.to(dtype).to(gpu) for t in (x, w, a, b)] + [ids.to(gpu)]
    for od in (dtype, torch.float32):
        out = mi.mm_lora(*dev, out_dtype=od).cpu()
        want = torch.from_numpy(ref).to(od)
        bad = (out != want).nonzero()
        assert not len(bad), (od, len(bad), [(i.tolist(), out[tuple(i)].item(), want[tuple(i)].item()) for i in bad[:4]])


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("T,K,N,L,R", SIZES)
def test_cancelling_gradients(gpu, T, N, K, L, R, dtype):
    print(f"mm_lora_backward cancelling T={T} N={N} K={K} R={R} {dtype}", flush=True)
    g = synth.gen(T + N)
    x, go, b = _whole(g, T, K, share=4 / K), _whole(g, T, N), _whole(g, L, N, R, share=24 / N)
    to = torch.arange(K) % R
    a = (torch.arange(R)[:, None] == to).long().expand(L, R, K)
    w = -b[0][:, to] + torch.randint(-1, 2, (N, K), generator=g) * (torch.rand(N, K, generator=g) < 4 / N)
    ids = _ids(g, T, L)
    ref, mag = O.mm_lora_backward(*(t.double().numpy() for t in (go, x, w, a, b)), ids)[0]
    assert mag.max() < 2 ** 24
    dev = [t.to(dtype).to(gpu) for t in (go, x, w, a, b)] + [ids.to(gpu)]
    got = mi.mm_lora_backward(*dev, with_adapters=False)[0].cpu()
    want = torch.from_numpy(ref).to(dtype)
    bad = (got != want).nonzero()
    assert not len(bad), (len(bad), [(i.tolist(), got[tuple(i)].item(), want[tuple(i)].item()) for i in bad[:4]])
