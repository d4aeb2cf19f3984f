"""The block products on small integers with scales that are powers of two: every
product and every partial sum is a multiple of one power of two and below 2^24 of it,
and the products of 8 consecutive columns lie within 2^4 of each other, so nothing is
dropped anywhere and the result is the exact one rounded once, bitwise, for every
output type.  The plain product is torch's in 64 bits.

Cases reach each kernel and tile height, with and without a streamed b, with own first
steps over more than 64 steps, and more steps than one register of b's scales holds
(fp32 outputs have 128 x 128 tiles where 16-bit ones have 256 x 256).
"""
import pytest
import torch

import synth
from moe_expert_grouped_amd import fp8_scale_cols, grouped_mm_fp8_block, mm_fp8_block

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _ints(g, gpu, top, *shape):
    v = torch.randint(-top, top + 1, shape, generator=g, device=gpu, dtype=torch.int8)
    return v.to(torch.float32).to(F8)


def _scales(g, gpu, lead, k):
    s = torch.full((*lead, fp8_scale_cols(k)), float("nan"), device=gpu)  # padding is not used
    kb = -(-k // 128)
    s[..., :kb] = 2.0 ** torch.randint(-1, 2, (*lead, kb), generator=g, device=gpu).float()
    return s


def _exact(a, sa, b, sb):
    (m, k), n = a.shape, b.shape[0]
    x = a.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    w = b.double() * sb.double().repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n]
    out = x @ w.t()
    assert out.abs().max() < 2.0 ** 22  # 2^24 of the unit, 1 / 4
    return out


DENSE = [
    ("few rows, 16 columns", 3, 272, 1040), ("few rows, 16 columns, scales refilled", 3, 32, 65680),
    ("few rows, 32 columns", 5, 4112, 656), ("few rows, 32 columns, scales refilled", 2, 4112, 65680),
    ("64 x 64", 130, 2064, 656), ("64 x 64, more than 64 steps", 130, 2064, 8464),
    ("128 x 128", 1100, 2064, 400), ("128 x 128, a low last tile", 1070, 2064, 528),
    ("128 x 128, more than 64 steps", 1070, 2064, 8464),
    ("256 x 256, a last tile of 72 rows", 3400, 2576, 400),
    ("256 x 256, a last tile of 52 rows", 3380, 2576, 272),
    ("256 x 256, more than 64 steps", 3380, 2576, 8720),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("what,m,n,k", DENSE, ids=lambda v: str(v))
def test_dense(gpu, what, m, n, k, dtype):
    print(f"mm_fp8_block exact, {what}: {m}x{n}x{k} {dtype}", flush=True)
    g = synth.gen(m + n + k, gpu)
    a, b = _ints(g, gpu, 4, m, k), _ints(g, gpu, 3, n, k)
    sa, sb = _scales(g, gpu, (m,), k), _scales(g, gpu, (-(-n // 128),), k)
    got = mm_fp8_block(a, b, sa, sb, out_dtype=dtype)
    torch.cuda.synchronize()
    assert torch.equal(got, _exact(a, sa, b, sb).to(dtype))


LOW = [0, 1, 2, 15, 16, 17, 3, 9]                       # groups of few rows
MIXED = [64, 0, 1, 63, 17, 40, 48, 5, 33, 64, 2, 30, 16, 21, 64, 60]
TALL = [60, 128, 65, 1, 64, 100, 129, 61, 90, 40, 32, 127, 0, 33, 62, 70]
LARGE = [256, 1, 129, 300, 64, 255, 200, 65, 0, 256, 128, 600, 33, 250, 190, 256]

# rows of the groups, n, k; b is streamed where all of it has 128 MiB or more, with own
# first steps where k is a multiple of 4096
GROUPED = [
    ("few rows, 16 columns", [3, 0, 17, 11], 272, 1040),
    ("few rows, 32 columns", LOW, 912, 656),
    ("64 x 64", [40, 64, 0, 1, 65, 100], 400, 656),
    ("64 x 64, streamed", MIXED, 1040, 8208),
    ("64 x 64, own first steps", MIXED, 2048, 4096),
    ("64 x 64, own first steps, more than 64 steps", MIXED[:-1] + [200], 1040, 12288),
    ("128 x 128", [60, 128, 0, 1, 129, 62], 400, 656),
    ("128 x 128, streamed", TALL, 1040, 8208),
    ("128 x 128, own first steps", TALL, 2064, 4096),
    ("128 x 128, own first steps, more than 64 steps", TALL, 1040, 12288),
    ("256 x 256", [700, 100, 30, 0, 167], 9872, 400),
    ("256 x 256, streamed", LARGE, 2064, 4112),
    ("256 x 256, own first steps", LARGE, 2064, 4096),
    ("256 x 256, own first steps, more than 64 steps", LARGE, 2064, 12288),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("what,counts,n,k", GROUPED, ids=lambda v: str(v) if not isinstance(v, list) else "groups")
def test_grouped(gpu, what, counts, n, k, dtype):
    first, E, m = 2, len(counts), sum(counts) + 5
    print(f"grouped_mm_fp8_block exact, {what}: {E} groups, {m} rows, {n}x{k} {dtype}", flush=True)
    g = synth.gen(m + n + k, gpu)
    a, b = _ints(g, gpu, 4, m, k), _ints(g, gpu, 3, E, n, k)
    sa, sb = _scales(g, gpu, (m,), k), _scales(g, gpu, (E, -(-n // 128)), k)
    ends = [first]
    for c in counts:
        ends.append(ends[-1] + c)
    out = torch.full((m, n), 7.0, dtype=dtype, device=gpu)
    grouped_mm_fp8_block(a, sa, b, sb, torch.tensor(ends, dtype=torch.int32, device=gpu), out=out,
                         out_dtype=dtype)
    torch.cuda.synchronize()
    assert (out[:first] == 7.0).all() and (out[ends[-1]:] == 7.0).all()
    for e, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        if lo < hi:
            want = _exact(a[lo:hi], sa[lo:hi], b[e], sb[e]).to(dtype)
            assert torch.equal(out[lo:hi], want), f"group {e}"
