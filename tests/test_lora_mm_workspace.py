"""The projection's workspace: what its query gives for a number of rows is enough for every
smaller one, so that one workspace serves a caller's largest batch and all others."""
import re

import pytest
import torch

import moe_expert_grouped_amd as mi
from moe_expert_grouped_amd import _lib

FAKE = 0x10000000  # never dereferenced: validation fails before any launch
# n, k, adapters, rank
SIZES = [(4096, 4096, 16, 16), (4096, 4096, 16, 64), (96, 4760, 3, 16), (4760, 96, 64, 8), (64, 64, 1024, 8),
         (28672, 4096, 4, 256), (72, 65536, 2, 8), (1528, 2560, 3, 40), (8, 8, 1, 8)]
ROWS = sorted({*range(0, 130), *range(130, 1100, 23), *(2 ** i + d for i in range(7, 17) for d in (-1, 0, 1)),
               16384, 16385, 16447, 40000, 131073, 200001})


def _need(m, n, k, L, R, backward):
    """What a call of m rows asks for, from its refusal of one byte."""
    p = [FAKE + (i << 44) for i in range(16)]
    if backward:
        st = _lib.lib().mi_mm_lora_backward(p[0], p[1], m, k, _lib.MI_BF16, p[2], n, p[3], p[4], L, R, p[5], p[6],
                                            p[7], p[8], p[9], p[10], _lib.MI_F32, p[11], 1, None)
    else:
        st = _lib.lib().mi_mm_lora(p[0], m, k, _lib.MI_BF16, p[1], n, p[2], p[3], L, R, p[4], p[5], p[6], p[7],
                                   _lib.MI_BF16, p[8], p[9], 1, None)
        if m == 0:
            return 0
    with pytest.raises(ValueError, match="workspace needs") as e:
        _lib.check(st)
    return int(re.search(r"needs (\d+) bytes", str(e.value)).group(1))


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("n,k,L,R", SIZES)
def test_enough_for_fewer_rows(n, k, L, R, backward):
    most = 0
    for m in ROWS:
        most = max(most, _need(m, n, k, L, R, backward))
        have = mi.lora_mm_workspace_bytes(m, n, k, L, R, backward=backward)
        assert have >= most, (m, have, most)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_one_workspace_for_all_batches(gpu, dtype):
    n, k, L, R, most = 256, 4096, 5, 16, 2048
    g = torch.Generator().manual_seed(1)

    def new(*shape):
        return (torch.randn(shape, generator=g) * 0.1).to(dtype).to(gpu)

    x, w, a, b, go = new(most, k), new(n, k), new(L, R, k), new(L, n, R), new(most, n)
    ids = torch.randint(-1, L, (most,), generator=g).to(torch.int32).to(gpu)
    ws = torch.empty(mi.lora_mm_workspace_bytes(most, n, k, L, R), dtype=torch.uint8, device=gpu)
    wb = torch.empty(mi.lora_mm_workspace_bytes(most, n, k, L, R, backward=True), dtype=torch.uint8, device=gpu)
    for m in (0, 1, 2, 30, 64, 256, 300, 600, 1024, 1025, 1500, most):
        print(f"mm_lora one workspace m={m}", flush=True)
        args = (x[:m], w, a, b, ids[:m])
        ws.fill_(255)
        wb.fill_(255)
        out, act = mi.mm_lora(*args, with_act=True, workspace=ws)
        got = (out, act, *mi.mm_lora_backward(go[:m], *args, workspace=wb))
        out, act = mi.mm_lora(*args, with_act=True)
        ref = (out, act, *mi.mm_lora_backward(go[:m], *args))
        assert all(torch.equal(p, q) for p, q in zip(got, ref)), m


@pytest.mark.parametrize("m,n,k", [(8192, 128, 4096), (1500, 576, 4096), (1100, 896, 4096)])
def test_no_parts_where_the_tiles_fill_the_card(m, n, k):
    """Unsplit, a call needs no fp32 partial sums of its result."""
    assert _need(m, n, k, 4, 16, False) < m * n * 4 + m * 250
