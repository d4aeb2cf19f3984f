"""The adapters' projection on its large tiles, over many k steps: every tile's loop refills
each of its stages several times, with an odd and an even number of steps and a short last
one, adapters of several staged steps and several adapters in a tile; and the first products
of wide ranks over more steps than their wavefronts have stages.

Every operand is a small whole number, all products and sums stay below 2^24, and fp32 holds
them: outputs are the rounding of an exact value, bit by bit.
"""
import numpy as np
import pytest
import torch

import moe_expert_grouped_amd as mi
import synth
from oracle import lora_mm as O

pytestmark = pytest.mark.gpu

HALVES = [torch.bfloat16, torch.float16]
# T, N, K, L, R.  256 x 256 and 128 x 128 tiles of x w^T (9 and 10 steps of 64), of grad_out w
# (the same of N), and first products of 16 steps and more at ranks with a short last block
SHAPES = [(4100, 2056, 520, 5, 72), (4100, 2056, 584, 9, 64), (4100, 520, 2056, 5, 40), (4100, 584, 2056, 9, 136),
          (1100, 2056, 520, 5, 72), (1100, 2056, 584, 9, 64), (1100, 520, 2056, 5, 72), (1100, 584, 2056, 9, 24),
          (4200, 264, 1000, 7, 40), (4200, 1000, 264, 7, 64), (4128, 136, 1096, 3, 136), (4128, 1096, 136, 3, 72),
          (2500, 200, 1608, 4, 32), (2500, 1608, 200, 4, 32),
          # ranks up to 16, whose pieces lie side by side, in each tile
          (4100, 2056, 520, 9, 16), (4100, 584, 2056, 40, 8), (1100, 2056, 584, 40, 16), (4128, 584, 1096, 5, 8), (1100, 264, 520, 70, 16),
          # narrow results over 74 steps, in four parts
          (1100, 72, 4680, 3, 40), (1100, 4680, 72, 3, 40)]


def _case(T, N, K, L, R, dtype):
    g = synth.gen(T + N + R)

    def whole(*shape, top, share=1.0):
        t = torch.randint(-top, top + 1, shape, generator=g).float()
        return torch.where(torch.rand(shape, generator=g) < share, t, 0.0).to(dtype)

    ids = torch.randint(-1, L + 1, (T,), generator=g).to(torch.int32)
    ids[: T // 3] = torch.arange(T // 3, dtype=torch.int32) // 200 % L  # prompts, then single rows
    return (whole(T, K, top=3), whole(N, K, top=2), whole(L, R, K, top=2, share=16 / K),
            whole(L, N, R, top=2, share=min(1.0, 16 / N + 16 / R)), ids,
            torch.randint(1, 4, (L,), generator=g).float(), whole(N, top=3), whole(T, N, top=1))


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("T,N,K,L,R", SHAPES)
def test_many_steps_exactly(gpu, T, N, K, L, R, dtype):
    print(f"mm_lora tiles T={T} N={N} K={K} L={L} R={R} {dtype}", flush=True)
    x, w, a, b, ids, scale, bias, go = _case(T, N, K, L, R, dtype)
    cpu = [t.double().numpy() for t in (x, w, a, b)] + [ids, scale]
    ref, mag, act, _ = O.mm_lora(*cpu, bias.double().numpy())
    refs = O.mm_lora_backward(go.double().numpy(), *cpu)
    assert mag.max() < 2 ** 24 and all(m.max() < 2 ** 24 for _, m in refs)
    dev = [t.to(gpu) for t in (x, w, a, b, ids, scale)]
    for od in (torch.float32, dtype):
        out, v = mi.mm_lora(*dev, bias=bias.to(gpu), out_dtype=od, with_act=True)
        torch.cuda.synchronize()
        want = torch.from_numpy(ref).to(od)
        assert torch.equal(out.cpu(), want), ("out", od, (out.cpu() != want).nonzero()[:4])
        assert np.array_equal(v.double().cpu().numpy(), act)
    for gd in (torch.float32, dtype):
        for given in (v, None):
            got = mi.mm_lora_backward(go.to(gpu), *dev, act=given, grad_dtype=gd)
            torch.cuda.synchronize()
            for t, (r, _), what in zip(got, refs, ("grad_x", "grad_a", "grad_b")):
                want = torch.from_numpy(r).to(t.dtype)
                assert torch.equal(t.cpu(), want), (what, gd, (t.cpu() != want).nonzero()[:4])
