"""SwiGLU of the 8-bit quantiser at large gates, as accurate as a plain fp32 evaluation.

u = 2^-24.  exp is good to one step of its result and one rounding (3 u); the sum, its
reciprocal, three products and the scale's division are a rounding each: 9 u relative
at every gate whose exp is a normal number.
"""
import numpy as np
import pytest
import torch

import synth
from moe_expert_grouped_amd import fp8_quantize
from oracle import fp8 as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
def test_swiglu_scales_at_every_gate(gpu, dtype):
    """Blocks of one gate each: the scale is that value over 448."""
    n = 4096
    gate = (torch.rand(n, generator=synth.gen(21)) * 174 - 87).to(dtype)
    x = torch.cat([gate[:, None].expand(n, 128), torch.full((n, 128), 1.5).to(dtype)], 1)
    print(f"fp8_quantize swiglu gates {dtype}", flush=True)
    codes, scales = fp8_quantize(x.contiguous().to(gpu), swiglu=True)
    want = np.abs(F.swiglu(x.double().numpy())[:, 0]) / 448
    got = scales.cpu().double().numpy()[:, 0]
    # below 448 * 2^-126 the scale is the smallest one
    far = want > 2.0 ** -125
    assert far.sum() > n // 2
    err = np.abs(got[far] / want[far] - 1) / U
    assert (err <= 9).all(), f"{err.max()} u at gate {gate.double().numpy()[far][err.argmax()]}"
    sign = np.where(gate.double().numpy() > 0, 1, -1)
    v = F.decode(codes.cpu().view(torch.uint8).numpy())
    assert (v[far] == 448 * sign[far][:, None]).all()


def test_swiglu_tail(gpu):
    """Gates whose exp is subnormal: silu itself is rounded to a subnormal number, at
    most half a step of those in each of two products (2^-149 in all, times up)."""
    n = 512
    gate = -torch.linspace(87, 110, n)
    x = torch.cat([gate[:, None].expand(n, 128), torch.full((n, 128), 2.0 ** 40)], 1)
    print("fp8_quantize swiglu tail", flush=True)
    codes, scales = fp8_quantize(x.contiguous().to(gpu), swiglu=True)
    want = np.abs(F.swiglu(x.double().numpy())[:, 0])
    v = F.decode(codes.cpu().view(torch.uint8).numpy())[:, 0]
    got = -v * scales.cpu().double().numpy()[:, 0]
    big = want > 2.0 ** -100
    tol = 9 * U * want + 2.0 ** -149 * 2.0 ** 40
    assert big.sum() > n // 2 and (v[big] == -448).all()
    assert (np.abs(got - want)[big] <= tol[big]).all()
    assert (got[~big] <= 2.0 ** -99).all()


def test_swiglu_gates_without_a_number(gpu):
    """+inf stays the block's scale; NaN and -inf (0 times infinity) make it NaN; up's
    infinity meets a gate of zero as NaN."""
    x = torch.ones(6, 256)
    x[0, 5], x[1, 5], x[2, 5] = float("inf"), float("nan"), -float("inf")
    x[3, 5], x[3, 133] = 0.0, float("inf")
    x[4, 5] = 3e38
    x[5, 5] = -3e38
    print("fp8_quantize swiglu infinities", flush=True)
    codes, scales = fp8_quantize(x.to(gpu), swiglu=True)
    s = scales.cpu().numpy()[:, 0]
    assert s[0] == np.inf and np.isnan(s[1:4]).all()
    with np.errstate(invalid="ignore"):
        v = F.decode(codes.cpu().view(torch.uint8).numpy()) * s[:, None]
    assert np.isnan(v[:4]).all()
    assert s[4] == np.float32(3e38) / np.float32(448) and v[4, 5] == 448 * float(s[4])
    assert v[5, 5] == 0 and np.isfinite(v[4:]).all()
