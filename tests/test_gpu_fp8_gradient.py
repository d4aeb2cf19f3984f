"""The gradient of a product's rows: the same product with the weights' codes and
scales transposed, as the docstrings give it.

    y[m, n] = sum_k x[m, k] w[n, k]   gives   dx[m, k] = sum_n dy[m, n] w[n, k]

Checked against 64 bits on the values that the codes and scales stand for, with the
product's tolerance; and against the unquantised dy: a code is off by at most half a
step around its value (twice that allowed, for a value next to a power of two).
"""
import numpy as np
import pytest
import torch

import synth
from moe_expert_grouped_amd import (fp8_quantize, fp8_scale_cols, grouped_mm_fp8_block,
                                    mm_fp8_block)
from oracle import fp8 as F
from tests.test_gpu_fp8 import U, _check, _np, _u8

pytestmark = pytest.mark.gpu


def transposed(codes, scales):
    """Weights [..., N, K] and their 128 x 128 scales as those of [..., K, N]."""
    N, K = codes.shape[-2:]
    s = scales[..., :-(-K // 128)].transpose(-1, -2)
    s = torch.nn.functional.pad(s, (0, fp8_scale_cols(N) - s.shape[-1]))
    return codes.transpose(-1, -2).contiguous(), s.contiguous()


SHAPES = [(5, 144, 272), (70, 400, 256), (300, 528, 1040), (33, 2064, 400), (9, 512, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gradient_of_the_rows(gpu, m, n, k, dtype):
    print(f"mm_fp8_block gradient {m}x{n}x{k} {dtype}", flush=True)
    g = synth.gen(m + n + k)
    w = (torch.randn(n, k, generator=g) * k ** -0.5).to(gpu)
    dy = torch.randn(m, n, generator=g).to(gpu)
    b, sb = fp8_quantize(w, block_rows=128)
    bt, sbt = transposed(b, sb)
    a, sa = fp8_quantize(dy)
    dx = mm_fp8_block(a, bt, sa, sbt, out_dtype=dtype)
    # transposed codes stand for the transposed values
    wq = F.decode(_u8(b)) * F.spread(_np(sb), n, k, 128)
    assert np.array_equal(F.decode(_u8(bt)) * F.spread(_np(sbt), k, n, 128), wq.T)
    dyq = F.decode(_u8(a)) * F.spread(_np(sa), m, n)
    ref, mag = dyq @ wq, np.abs(dyq) @ np.abs(wq)
    _check(dx, ref, mag, F.group_maxima(_u8(a), _np(sa), _u8(bt), _np(sbt)), n, dtype, "dx")
    # and dy's own rounding, at most half a step of each code
    half = F.half_step(_np(dy) / F.spread(_np(sa), m, n)) * F.spread(_np(sa), m, n) * (1 + 2.0 ** -20)
    assert (np.abs(dyq - _np(dy)) <= 2 * half).all()
    assert (np.abs(ref - _np(dy) @ wq) <= 2 * half @ np.abs(wq)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_gradient_of_the_experts_rows(gpu, dtype):
    counts, n, k = [7, 0, 130, 1, 64], 272, 528
    E, m = len(counts), sum(counts)
    print(f"grouped_mm_fp8_block gradient {dtype}", flush=True)
    g = synth.gen(17)
    w = (torch.randn(E, n, k, generator=g) * k ** -0.5).to(gpu)
    dy = torch.randn(m, n, generator=g).to(gpu)
    ind = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device=gpu)
    b, sb = fp8_quantize(w, block_rows=128)
    bt, sbt = transposed(b, sb)
    a, sa = fp8_quantize(dy)
    dx = grouped_mm_fp8_block(a, sa, bt, sbt, ind, out_dtype=dtype)
    ref, mag, top, _ = F.grouped_mm_fp8_block(_u8(a), _np(sa), _u8(bt), _np(sbt), ind.tolist())
    _check(dx, ref, mag, top, n, dtype, "dx")
    at = 0
    for e, c in enumerate(counts):
        wq = F.decode(_u8(b[e])) * F.spread(_np(sb[e]), n, k, 128)
        dyq = F.decode(_u8(a[at:at + c])) * F.spread(_np(sa[at:at + c]), c, n)
        assert np.allclose(ref[at:at + c], dyq @ wq, rtol=1e-12, atol=1e-12)
        at += c


def test_gradient_against_differences(gpu):
    """The product is linear in x: along a direction the difference quotient in 64 bits
    and <dx, direction> agree up to the kernel's fp32 sums."""
    m, n, k = 20, 272, 400
    g = synth.gen(19)
    print("mm_fp8_block gradient against differences", flush=True)
    b, sb = fp8_quantize((torch.randn(n, k, generator=g) * 0.05).to(gpu), block_rows=128)
    a, sa = fp8_quantize(torch.randn(m, n, generator=g).to(gpu))
    dx = _np(mm_fp8_block(a, transposed(b, sb)[0], sa, transposed(b, sb)[1],
                          out_dtype=torch.float32))
    wq = F.decode(_u8(b)) * F.spread(_np(sb), n, k, 128)
    dy = F.decode(_u8(a)) * F.spread(_np(sa), m, n)
    x, d = (torch.randn(m, k, generator=g).double().numpy() for _ in range(2))
    loss = lambda v: ((v @ wq.T) * dy).sum()
    diff = (loss(x + d) - loss(x - d)) / 2
    size = (np.abs(d) * (np.abs(dy) @ np.abs(wq))).sum()
    assert abs(diff - (dx * d).sum()) <= (2 * 128 + 8) * U * size + 1e-9
