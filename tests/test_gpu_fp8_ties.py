"""Codes of values next to a tie between two codes: they are those of the fp32 quotient
y / scale, rounded once, bitwise.

The blocks' largest values are arbitrary, so the scales are; the other values are the
midpoints of neighbouring codes times the scale, and up to 3 fp32 steps to either side,
where a quotient taken as y * (1 / scale) falls on the wrong side now and then.
"""
import numpy as np
import pytest
import torch

import synth
from moe_expert_grouped_amd import add_rmsnorm_fp8, fp8_quantize
from oracle import fp8 as F

pytestmark = pytest.mark.gpu


def _near_ties(blocks, seed):
    """[blocks, 128] fp32: a largest value and 127 values at and around ties."""
    rng = np.random.default_rng(seed)
    amax = np.exp(rng.uniform(-20, 20, blocks)).astype(np.float32)
    s = amax / np.float32(448)
    v = np.unique(np.abs(F.e4m3_values()[:127]))
    mid = (0.5 * (v[:-1] + v[1:]))[rng.integers(0, v.size - 1, (blocks, 127))]
    y = (mid * s[:, None].astype(np.float64)).astype(np.float32)
    step = rng.integers(-3, 4, y.shape)
    y = (y.view(np.int32) + step.astype(np.int32)).view(np.float32)
    y *= rng.choice(np.array([-1, 1], np.float32), y.shape)
    return np.concatenate([amax[:, None], y], axis=1), s


def _want(y, s):
    """e4m3 of the fp32 quotient, by torch's conversion on the CPU."""
    return torch.from_numpy(y / s).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _u8(t):
    return t.cpu().view(torch.uint8).numpy()


def test_rows(gpu):
    y, s = _near_ties(40000, 1)
    print("fp8_quantize near ties, rows", flush=True)
    codes, scales = fp8_quantize(torch.from_numpy(y).to(gpu))
    assert np.array_equal(scales.cpu().numpy()[:, 0], s)
    assert np.array_equal(_u8(codes), _want(y, s[:, None]))


def test_weight_blocks(gpu):
    y, s = _near_ties(300 * 128, 2)
    # one scale a 128 x 128 block: the first row's, its values next to ties of that scale
    y = y.reshape(300, 128, 128)
    s0 = s.reshape(300, 128)[:, :1, None]
    y[:, 1:] = (y[:, 1:].astype(np.float64) / s.reshape(300, 128, 1)[:, 1:] * s0).astype(np.float32)
    y[:, 1:, 0] = 0
    print("fp8_quantize near ties, weight blocks", flush=True)
    codes, scales = fp8_quantize(torch.from_numpy(y).to(gpu), block_rows=128)
    assert np.array_equal(scales.cpu().numpy()[:, 0, 0], s0[:, 0, 0])
    assert np.array_equal(_u8(codes), _want(y, s0))


@pytest.mark.parametrize("h", [512, 16400])
def test_norm(gpu, h):
    """The norm's codes are those of its own fp32 y, which norm_out shows for fp32 rows."""
    x = torch.randn(300, h, generator=synth.gen(h)).to(gpu)
    w = torch.ones(h, device=gpu)
    print(f"add_rmsnorm_fp8 codes of its y, {h}", flush=True)
    codes, scales, _, y = add_rmsnorm_fp8(x, w, with_norm=True)
    yv, sv = y.cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(sv, F.block_scales(yv))
    assert np.array_equal(_u8(codes), _want(yv, np.repeat(sv, 128, 1)[:, :h]))


def test_infinite_blocks_keep_their_codes(gpu):
    """A block with an infinity: code 0 for its numbers, NaN for the infinity."""
    x = torch.ones(1, 128)
    x[0, 7] = float("inf")
    print("fp8_quantize infinite block", flush=True)
    codes, scales = fp8_quantize(x.to(gpu))
    c = _u8(codes)[0]
    assert scales[0, 0].item() == float("inf")
    assert c[7] & 0x7F == 0x7F and not np.delete(c, 7).any()
