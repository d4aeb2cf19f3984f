"""The stated precision of the block products' sums, at groups of 8 products that are
worst for it: fp32 outputs are exact there, 16-bit ones within the stated bound.

Values are multiples of 2^-3 and every sum stays below 2^21, so fp32 holds all of them.
A 16-bit output drops, in each 8 consecutive products, less than 2^-13 of the largest
from each of the 7 others; then half a step of the output's type.
"""
import numpy as np
import pytest
import torch

from moe_expert_grouped_amd import grouped_mm_fp8_block, mm_fp8_block
from oracle import fp8 as F

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}
# a's and b's 8 values: small products beside a large one, and beside two that cancel
GROUPS = {
    "one large": ([256] + [1.125] * 7, [256] + [7] * 7),
    "two that cancel": ([256, -256] + [1.25] * 6, [256, 256] + [6] * 6),
    "large last": ([1.125] * 7 + [-256], [7] * 7 + [256]),
}


@pytest.mark.parametrize("dtype", list(HALF), ids=str)
@pytest.mark.parametrize("m,n", [(3, 272), (130, 2064), (1100, 2064), (3400, 2576)])
@pytest.mark.parametrize("which", list(GROUPS))
def test_sums_of_eight_products(gpu, which, m, n, dtype):
    k = 128
    ga, gb = (torch.tensor(v, dtype=torch.float32) for v in GROUPS[which])
    a, b = ga.repeat(m, k // 8).to(F8), gb.repeat(n, k // 8).to(F8)
    sa = torch.zeros(m, 4)
    sa[:, 0] = 2.0 ** (-6 - torch.arange(m) % 3)   # fp16 outputs stay below 65504
    sb = torch.tensor([[1.0, 0, 0, 0]]).repeat(-(-n // 128), 1)
    print(f"mm_fp8_block sums of eight, {which} {m}x{n} {dtype}", flush=True)
    ops = (a.to(gpu), b.to(gpu), sa.to(gpu), sb.to(gpu))
    got = mm_fp8_block(*ops, out_dtype=dtype).cpu().double().numpy()
    ind = torch.tensor([0, m // 2, m], dtype=torch.int32, device=gpu)
    two = torch.stack([ops[1], ops[1]]), torch.stack([ops[3], ops[3]])
    grouped = grouped_mm_fp8_block(ops[0], ops[2], *two, ind, out_dtype=dtype)
    # 3 rows of each scale and one column stand for all: the others are copies
    ref, _ = F.mm_fp8_block(a[:3].view(torch.uint8).numpy(), sa[:3].numpy(),
                            b[:1].view(torch.uint8).numpy(), sb[:1].numpy())
    ref = ref[np.arange(m) % 3]
    top = (ga * gb).abs().max().item() * (k // 8) * sa[:, :1].double().numpy()
    lost = 0.0 if dtype == torch.float32 else 7 * 2.0 ** -13 * top
    for v in (got, grouped.cpu().double().numpy()):
        assert (np.abs(v - ref) <= lost + HALF[dtype] * np.abs(ref)).all()
