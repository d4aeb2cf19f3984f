"""The 8-bit block-scaled operators on the GPU against the fp64 oracle.

Tolerances.  u = 2^-24 is an fp32 rounding.

Product: a block's 128 products are exact in fp32 and summed in fp32 in an
order of the hardware's, at most two roundings of a partial sum per term; the
factor sa * sb is one rounding and each block's fma one more.  Against S, the
sum of the absolute values of all terms, that is at most (2 * 128 + 1 + KB) u S
for KB blocks.  For a 16-bit output the hardware sums 8 consecutive products
aligned to the largest exponent E among them and drops what lies under
2^(E - 13): each of the 7 others by less than that, so 7 * 2^-13 times the largest
product of each 8 (at most the row's largest |a| times the column's largest |b|),
summed over the groups of 8.  Then half a step of the output's type.

Quantisation: a scale is one correctly rounded division of the block's amax,
so it is compared bitwise.  y * (1 / s) is two roundings from y / s, so the
code is the nearest to some value within 2 u |y / s| of it (4 u is allowed):
half a step around y / s plus that.

SwiGLU: exp in fp32 from a hardware exp2 of one rounded product: its argument
is off by |g| u, a few ulp more for the exp2, the sum, the division and the
products: (|g| + 16) u relative.

Norm: squares are summed in fp32 over at most ceil(H / 2048) * 8 + 9 additions per
chain, halved by the root; then the root, the division and two products:
(ceil(H / 2048) * 8 + 24) u relative.
"""
import numpy as np
import pytest
import torch

import synth
from moe_expert_grouped_amd import (add_rmsnorm_fp8, fp8_quantize, fp8_scale_cols,
                                    grouped_mm_fp8_block, mm_fp8_block)
from oracle import fp8 as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
F8 = torch.float8_e4m3fn


def _codes(g, shape, lo=0):
    """Any finite code; `lo` > 0 keeps out codes below it (large values only)."""
    c = torch.randint(lo, 0x7F, shape, generator=g)
    return (c + 128 * torch.randint(0, 2, shape, generator=g)).to(torch.uint8)


def _scale_rows(g, lead, k):
    s = torch.full((*lead, fp8_scale_cols(k)), float("nan"))  # the padding is never used
    s[..., : -(-k // 128)] = torch.exp(torch.randn((*lead, -(-k // 128)), generator=g) - 3)
    return s


def _np(t):
    return t.detach().cpu().double().numpy()


def _u8(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def _check(got, ref, mag, top, k, dtype, what):
    kb = -(-k // 128)
    tol = (2 * 128 + 1 + kb) * U * mag + HALF[dtype] * np.abs(ref)
    if dtype != torch.float32:
        tol = tol + 7 * 2.0 ** -13 * top
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25  # subnormal step
    err = np.abs(_np(got) - ref)
    assert np.isfinite(_np(got)).all(), what
    assert (err <= tol).all(), f"{what}: worst {np.max(err / np.maximum(tol, 1e-300))}"


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

MM_SHAPES = [(1, 16, 16), (1, 128, 128), (2, 256, 512), (15, 112, 144), (16, 144, 128),
             (17, 128, 528), (33, 400, 256), (64, 256, 1024), (65, 272, 640), (127, 128, 384),
             (129, 384, 400), (200, 1040, 272), (257, 512, 2064), (300, 16, 4096),
             (520, 784, 208), (1, 2048, 8320), (5, 4112, 1040), (1100, 1296, 336)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m,n,k", MM_SHAPES)
def test_mm_against_oracle(gpu, m, n, k, dtype):
    print(f"mm_fp8_block {m}x{n}x{k} {dtype}", flush=True)
    g = synth.gen(m * 31 + n * 7 + k)
    a, b = _codes(g, (m, k)), _codes(g, (n, k))
    sa, sb = _scale_rows(g, (m,), k), _scale_rows(g, (-(-n // 128),), k)
    if dtype == torch.float16:
        sa, sb = sa * 2.0 ** -8, sb * 2.0 ** -8  # the sums stay below 65504
    out = torch.full((m + 2, n), 7.0, dtype=dtype, device=gpu)
    got = mm_fp8_block(a.to(gpu).view(F8), b.to(gpu).view(F8), sa.to(gpu), sb.to(gpu),
                       out=out[:m], out_dtype=dtype)
    torch.cuda.synchronize()
    assert (out[m:] == 7.0).all()
    ops = (a.numpy(), np.nan_to_num(sa.numpy()), b.numpy(), np.nan_to_num(sb.numpy()))
    ref, mag = F.mm_fp8_block(*ops)
    _check(got, ref, mag, F.group_maxima(*ops), k, dtype, f"{m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", [(3, 272, 1040), (130, 272, 1040), (600, 528, 656)])
def test_mm_integers_are_exact(gpu, m, n, k):
    """Small integers and scales that are powers of two: every partial sum is
    an integer multiple of one power of two below 2^24, so fp32 is exact."""
    print(f"mm_fp8_block integers {m}x{n}x{k}", flush=True)
    g = synth.gen(k)
    av = torch.randint(-4, 5, (m, k), generator=g).float()
    bv = torch.randint(-3, 4, (n, k), generator=g).float()
    kb, cols = -(-k // 128), fp8_scale_cols(k)
    sa, sb = torch.zeros(m, cols), torch.zeros(-(-n // 128), cols)
    sa[:, :kb] = 2.0 ** torch.randint(-1, 2, (m, kb), generator=g).float()
    sb[:, :kb] = 2.0 ** torch.randint(-1, 2, (sb.shape[0], kb), generator=g).float()
    a, b = av.to(F8), bv.to(F8)
    got = mm_fp8_block(a.to(gpu), b.to(gpu), sa.to(gpu), sb.to(gpu), out_dtype=torch.float32)
    ref, _ = F.mm_fp8_block(_u8(a), sa.numpy(), _u8(b), sb.numpy())
    assert np.array_equal(_np(got), ref)


def test_mm_nan_and_infinite_scales_reach_only_their_rows_and_columns(gpu):
    g = synth.gen(77)
    m, n, k = 70, 272, 400
    a, b = _codes(g, (m, k)), _codes(g, (n, k))
    sa, sb = torch.ones(m, 4), torch.ones(3, 4)
    a[3, 17], b[200, 399] = 0x7F, 0xFF
    sa[9, 2], sa[40, 3] = float("nan"), float("inf")
    print("mm_fp8_block NaN codes and scales", flush=True)
    got = mm_fp8_block(a.to(gpu).view(F8), b.to(gpu).view(F8), sa.to(gpu), sb.to(gpu))
    bad = ~torch.isfinite(got).cpu().numpy()
    want = np.zeros((m, n), bool)
    want[[3, 9, 40]] = True
    want[:, 200] = True
    assert np.array_equal(bad, want)


GROUPS = [
    ([0, 5, 5, 21], 24),                     # an empty group, rows behind the last
    ([3, 3, 3, 3], 10),                      # nothing at all
    ([2, 130, 131, 400, 400], 402),          # rows before the first, one row, none
    ([0, 64, 128, 192, 256], 256),
    ([0, 1, 2, 3, 4, 5, 6, 7, 8], 8),
    ([0, 700, 701, 1100], 1100),
    ([5, 9, 40, 33, 60], 50),                # decreasing and past the rows: clamped
    ([-4, 7, 30], 20),
    ([0, 257, 769, 1000, 1512, 2600], 2600),
]


@pytest.mark.parametrize("n,k", [(256, 512), (144, 272), (1040, 400)])
@pytest.mark.parametrize("indptr,m", GROUPS, ids=str)
def test_grouped_against_oracle(gpu, indptr, m, n, k):
    print(f"grouped_mm_fp8_block {indptr} rows {m} n {n} k {k}", flush=True)
    g = synth.gen(m + n + k)
    E = len(indptr) - 1
    a, b = _codes(g, (m, k)), _codes(g, (E, n, k))
    sa, sb = _scale_rows(g, (m,), k), _scale_rows(g, (E, -(-n // 128)), k)
    dtype = [torch.bfloat16, torch.float32][m % 2]
    out = torch.full((m, n), 7.0, dtype=dtype, device=gpu)
    ind = torch.tensor(indptr, dtype=torch.int32)
    grouped_mm_fp8_block(a.to(gpu).view(F8), sa.to(gpu), b.to(gpu).view(F8), sb.to(gpu),
                         ind.to(gpu), out=out, out_dtype=dtype)
    torch.cuda.synchronize()
    owner = np.zeros(m, int) - 1
    for e in range(E):
        s = min(max(indptr[e], 0), m)
        owner[s:max(min(indptr[e + 1], m), s)] += 1
    if (owner > 0).any():  # overlapping groups (an invalid m_indptr) leave either's rows
        once = owner <= 0
    else:
        once = np.ones(m, bool)
    ref, mag, top, written = F.grouped_mm_fp8_block(a.numpy(), np.nan_to_num(sa.numpy()), b.numpy(),
                                               np.nan_to_num(sb.numpy()), indptr)
    assert (_np(out)[~written] == 7.0).all()
    rows = written & once
    if rows.any():
        _check(out[torch.from_numpy(rows).to(gpu)], ref[rows], mag[rows], top[rows], k, dtype,
               str(indptr))


# (m_indptr, rows of each of 64 groups, or None, m, n, k): enough tiles of 256 x 256 to fill the chip, groups
# that end in tiles of every height, more than 64 blocks of k and a last one of 16,
# a last panel of one 128-column block and of a little more; b streamed (128 MiB or
# more, groups of one m-tile) with an own first step per panel (k = 4096, 8192)
LARGE = [
    ([3, 703, 803, 833, 833, 1000], 1004, 9872, 8704),
    ([0, 700, 828, 892, 892, 1000], 1000, 9856, 8208),
    ([0, 1500, 1628, 1692, 6000], 6000, 2064, 528),
    ([0, 257, 300, 300, 1100], 1101, 9984, 144),
    (None, 3400, 3984, 400),
    (None, 2500, 5008, 8464),
    ([0, 200, 300, 340, 340, 1200], 1200, 6160, 8192),
    (21, 1344, 528, 4096),
    (21, 1344, 1040, 4096),
    (70, 4480, 1040, 4096),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("indptr,m,n,k", LARGE, ids=str)
def test_large_tiles_against_oracle(gpu, indptr, m, n, k, dtype):
    """The rows at the ends of every tile and the columns at the ends of some panels."""
    print(f"large tiles {indptr} rows {m} n {n} k {k} {dtype}", flush=True)
    g = synth.gen(m + n + k, gpu)
    if isinstance(indptr, int):
        indptr = list(range(0, m + 1, indptr))
    E = 1 if indptr is None else len(indptr) - 1
    code = lambda *shape: (torch.randint(0, 0x7F, shape, generator=g, device=gpu, dtype=torch.uint8) +
                           128 * torch.randint(0, 2, shape, generator=g, device=gpu, dtype=torch.uint8))
    small = 2.0 ** -8 if dtype == torch.float16 else 1.0
    scale = lambda *lead: small * torch.rand(*lead, fp8_scale_cols(k), generator=g, device=gpu)
    a, b, sa, sb = code(m, k), code(E, n, k), scale(m), scale(E, -(-n // 128))
    out = torch.full((m, n), 7.0, dtype=dtype, device=gpu)
    if indptr is None:
        mm_fp8_block(a.view(F8), b[0].view(F8), sa, sb[0], out=out, out_dtype=dtype)
        groups = [(0, m)]
    else:
        grouped_mm_fp8_block(a.view(F8), sa, b.view(F8), sb,
                             torch.tensor(indptr, dtype=torch.int32, device=gpu), out=out,
                             out_dtype=dtype)
        groups = list(zip(indptr[:-1], indptr[1:]))
        assert (out[:indptr[0]] == 7.0).all() and (out[indptr[-1]:] == 7.0).all()
    torch.cuda.synchronize()
    blocks = sorted({0, 1, 2, 3, n // 256, -(-n // 128) - 2, -(-n // 128) - 1})
    for e, (lo, hi) in enumerate(groups):
        if E > 8 and e % 9:
            continue
        rows = sorted({r for t in range(lo, hi, 64) for r in (t, t + 17, t + 63) if r < hi} |
                      ({hi - 1} if hi > lo else set()))[-60:]
        if not rows:
            continue
        for blk in blocks:
            cols = slice(blk * 128, min(blk * 128 + 128, n))
            ops = (_u8(a[rows]), _np(sa[rows]), _u8(b[e, cols]), _np(sb[e, blk:blk + 1]))
            ref, mag = F.mm_fp8_block(*ops)
            _check(out[rows][:, cols], ref, mag, F.group_maxima(*ops), k, dtype,
                   f"group {e} block {blk}")


def test_grouped_many_experts_and_fresh_out(gpu):
    """1024 experts, most of them empty; a fresh out is zero outside the groups."""
    g = synth.gen(6)
    E, n, k = 1024, 32, 48
    counts = torch.where(torch.rand(E, generator=g) < 0.7, 0, torch.randint(1, 9, (E,), generator=g))
    ind = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32)
    m = int(ind[-1]) + 5
    a, b = _codes(g, (m, k)), _codes(g, (E, n, k))
    sa, sb = _scale_rows(g, (m,), k), _scale_rows(g, (E, 1), k)
    print(f"grouped_mm_fp8_block 1024 experts, {m} rows", flush=True)
    got = grouped_mm_fp8_block(a.to(gpu).view(F8), sa.to(gpu), b.to(gpu).view(F8), sb.to(gpu),
                               ind.to(gpu), out_dtype=torch.float32)
    ref, mag, top, written = F.grouped_mm_fp8_block(a.numpy(), np.nan_to_num(sa.numpy()), b.numpy(),
                                               np.nan_to_num(sb.numpy()), ind.numpy())
    _check(got, ref, mag, top, k, torch.float32, "1024 experts")
    assert not _np(got)[~written].any()


def test_grouped_of_one_expert_is_the_dense_product(gpu):
    g = synth.gen(8)
    for m, n, k in ((7, 512, 1024), (300, 784, 656)):
        a, b = _codes(g, (m, k)).to(gpu).view(F8), _codes(g, (n, k)).to(gpu).view(F8)
        sa, sb = _scale_rows(g, (m,), k).to(gpu), _scale_rows(g, (-(-n // 128),), k).to(gpu)
        print(f"grouped against dense {m}x{n}x{k}", flush=True)
        ind = torch.tensor([0, m], dtype=torch.int32, device=gpu)
        x = mm_fp8_block(a, b, sa, sb, out_dtype=torch.float32)
        y = grouped_mm_fp8_block(a, sa, b[None], sb[None], ind, out_dtype=torch.float32)
        tol = (2 * 128 + 1 + -(-k // 128)) * 2 * U
        scale = F.mm_fp8_block(_u8(a), np.nan_to_num(_np(sa)), _u8(b), np.nan_to_num(_np(sb)))[1]
        assert (np.abs(_np(x) - _np(y)) <= tol * scale).all()


def test_mm_views_and_streams(gpu):
    """Strided views are copied; a side stream's call is ordered on it."""
    g = synth.gen(9)
    m, n, k = 40, 128, 256
    a, b = _codes(g, (m, 2 * k)).to(gpu).view(F8), _codes(g, (n, k)).to(gpu).view(F8)
    sa, sb = _scale_rows(g, (2 * m,), k).to(gpu), _scale_rows(g, (1,), k).to(gpu)
    print("mm_fp8_block views and a side stream", flush=True)
    want = mm_fp8_block(a[:, :k].contiguous(), b, sa[::2].contiguous(), sb)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = mm_fp8_block(a[:, :k], b, sa[::2], sb)
    s.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------

def _check_codes(codes, scales, y, block_rows, what, rel=0.0):
    """Codes nearest to y / s, `rel` the relative error allowed in y."""
    rows, k = y.shape
    s = F.spread(scales, rows, k, block_rows)
    v = y / s
    err = np.abs(F.decode(codes) - v)
    tol = F.half_step(v) + (4 * U + 2 * rel) * np.abs(v)
    # a value rounded up across a power of two may be half of the larger step away
    tol = np.where(err > tol, F.half_step(v * (1 + 4 * U + 2 * rel)) + (4 * U + 2 * rel) * np.abs(v),
                   tol)
    assert (err <= tol).all(), f"{what}: {np.argwhere(err > tol)[:4]}"


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,k", [(1, 16), (1, 128), (3, 144), (127, 512), (128, 528),
                                    (130, 1040), (300, 2000), (2, 7168)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantise_against_oracle(gpu, rows, k, dtype, block_rows):
    print(f"fp8_quantize {rows}x{k} {dtype} blocks of {block_rows}", flush=True)
    g = synth.gen(rows + k)
    x = (torch.randn(2, rows, k, generator=g) *
         torch.exp(3 * torch.randn(2, rows, 1, generator=g))).to(dtype)
    x[0, 0] = 0
    x[1, rows // 2, k // 2] *= 30
    codes = torch.full((2, rows, k), 9.0, device=gpu).to(F8)
    scales = torch.full((2, -(-rows // block_rows), fp8_scale_cols(k)), 9.0, device=gpu)
    fp8_quantize(x.to(gpu), block_rows=block_rows, codes=codes, scales=scales)
    torch.cuda.synchronize()
    for i in range(2):
        y = x[i].float().numpy()
        want = F.block_scales(y, block_rows)
        assert np.array_equal(scales[i].cpu().numpy(), want)
        _check_codes(_u8(codes[i]), want, y.astype(np.float64), block_rows, f"{rows}x{k}")
    one = fp8_quantize(x[1].to(gpu), block_rows=block_rows)
    assert np.array_equal(_u8(one[0]), _u8(codes[1])) and torch.equal(one[1], scales[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,k", [(1, 16), (5, 272), (130, 1040), (64, 2048)])
def test_quantise_swiglu_against_oracle(gpu, rows, k, dtype):
    print(f"fp8_quantize swiglu {rows}x{k} {dtype}", flush=True)
    g = synth.gen(rows * 3 + k)
    x = (4 * torch.randn(rows, 2 * k, generator=g)).to(dtype)
    codes, scales = fp8_quantize(x.to(gpu), swiglu=True)
    y = F.swiglu(x.double().numpy())
    rel = (np.abs(x.double().numpy()).max() + 16) * U
    want = F.block_scales(y).astype(np.float64)
    got = scales.cpu().double().numpy()
    assert (np.abs(got - want) <= (rel + 2 * U) * want).all()
    _check_codes(_u8(codes), got, y, 1, f"swiglu {rows}x{k}", rel)


def test_swiglu_of_large_gates(gpu):
    """Gates far from zero: silu is the gate itself or a (possibly zero) tail,
    never NaN, and exp overflowing to infinity gives zero."""
    x = torch.zeros(4, 256)
    x[0, :128], x[0, 128:] = 3e4, 2.0
    x[1, :128], x[1, 128:] = -3e4, 2.0
    x[2, :128], x[2, 128:] = -80.0, 2.0
    x[3, :128], x[3, 128:] = 90.0, -1.0
    print("fp8_quantize swiglu large gates", flush=True)
    codes, scales = fp8_quantize(x.cuda(), swiglu=True)
    v = F.decode(_u8(codes)) * F.spread(scales.cpu().numpy(), 4, 128)
    want = F.swiglu(x.double().numpy())
    assert np.allclose(v, want, rtol=2.0 ** -4, atol=1e-30)


def test_quantise_special_values(gpu):
    x = torch.zeros(7, 128)
    x[0, 3] = float("nan")
    x[1, 3], x[1, 4] = float("inf"), 5.0
    x[2, 3] = -float("inf")
    x[3, :4] = torch.tensor([1e-40, -1e-41, 0.0, 1e-44])   # subnormal in fp32
    x[4, :4] = torch.tensor([3.4e38, -3.4e38, 1e38, 1.0])
    x[5, :3] = torch.tensor([448.0, 2.0 ** -9, 2.0 ** -10])  # the smallest code, and half of it
    print("fp8_quantize special values", flush=True)
    for br in (1, 128):
        rows = range(7) if br == 1 else (None,)
        for r in rows:
            part = x[r:r + 1] if br == 1 else x[3:]
            codes, scales = fp8_quantize(part.to(gpu), block_rows=br)
            c, s = F.decode(_u8(codes)), scales.cpu().numpy()
            want = F.block_scales(part.numpy(), br)
            assert np.array_equal(s, want, equal_nan=True)
            if br == 1 and r < 3:
                with np.errstate(invalid="ignore"):
                    assert np.isnan(c * s[0, 0]).all()
            else:
                _check_codes(_u8(codes), s, part.double().numpy(), br, f"row {r}")
    codes, scales = fp8_quantize(x[6:].to(gpu))
    assert not _u8(codes).any() and scales[0, 0].item() == 2.0 ** -126
    codes, _ = fp8_quantize(x[5:6].to(gpu))
    assert _u8(codes)[0, :3].tolist() == [0x7E, 0x01, 0x00]


def test_quantise_every_e4m3_value_and_tie(gpu):
    """A block with scale 1 that holds every value and every midpoint: values
    keep their codes, midpoints go to the even code."""
    v = np.unique(np.abs(F.e4m3_values()[:127]))
    mid = 0.5 * (v[:-1] + v[1:])
    flat = np.concatenate([v, mid, -v, -mid])
    pad = -(-flat.size // 127) * 127 - flat.size
    x = np.concatenate([flat, np.zeros(pad)]).reshape(-1, 127)
    x = np.concatenate([x, np.full((x.shape[0], 1), 448.0)], axis=1)
    print("fp8_quantize every value and tie", flush=True)
    codes, scales = fp8_quantize(torch.from_numpy(x).float().to(gpu))
    assert (scales[:, 0] == 1.0).all()
    got = F.decode(_u8(codes))[:, :127].reshape(-1)[:flat.size]
    even = np.where(np.arange(mid.size) % 2 == 0, v[:-1], v[1:])  # code i of value i
    assert np.array_equal(got, np.concatenate([v, even, -v, -even]))


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("t,h", [(1, 16), (3, 128), (5, 528), (2, 2048), (7, 2064), (4, 4096),
                                 (3, 7168), (2, 8192), (2, 8208), (3, 16400), (300, 512)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_against_oracle(gpu, t, h, dtype, residual):
    print(f"add_rmsnorm_fp8 {t}x{h} {dtype} residual {residual}", flush=True)
    g = synth.gen(t * 5 + h)
    x = (torch.randn(t, h, generator=g) * torch.exp(2 * torch.randn(t, 1, generator=g))).to(dtype)
    r = (3 * torch.randn(t, h, generator=g)).to(dtype) if residual else None
    wf = h % 32 == 0  # the weight in fp32, or in x's type
    w = (1 + 0.5 * torch.randn(h, generator=g)).to(torch.float32 if wf else dtype)
    eps = 1e-5
    dev = lambda v: None if v is None else v.to(gpu)
    codes, scales, ro, y = add_rmsnorm_fp8(dev(x), dev(w), dev(r), eps=eps, with_norm=True)
    hr, yr = F.add_rmsnorm(x.double().numpy(), w.double().numpy(),
                           None if r is None else r.double().numpy(), np.float32(eps))
    step = 2.0 ** -25 if dtype == torch.float16 else 0.0
    if residual:
        assert (np.abs(_np(ro) - hr) <= (HALF[dtype] + U) * np.abs(hr) + step).all()
    else:
        assert ro is None
    # the sum x + r is one fp32 rounding of its own size (cancellation keeps it absolute)
    rel = (-(-h // 2048) * 8 + 24) * U
    assert (np.abs(_np(y) - yr) <= (HALF[dtype] + rel) * np.abs(yr) + step).all()
    want, got = F.block_scales(yr).astype(np.float64), scales.cpu().double().numpy()
    assert (np.abs(got - want) <= (rel + 2 * U) * want).all()
    _check_codes(_u8(codes), got, yr, 1, f"norm {t}x{h}", rel)


@pytest.mark.parametrize("h", [512, 16400])
def test_norm_in_place_and_without_norm_out(gpu, h):
    """residual_out may be residual or x; the outputs do not change."""
    g = synth.gen(h)
    x, r = (synth.bf16_normal((9, h), 1.0, g).to(gpu) for _ in range(2))
    w = torch.ones(h, dtype=torch.bfloat16, device=gpu)
    print(f"add_rmsnorm_fp8 in place {h}", flush=True)
    c0, s0, r0 = add_rmsnorm_fp8(x, w, r)
    for which in (0, 1):
        xx, rr = x.clone(), r.clone()
        c1, s1, r1 = add_rmsnorm_fp8(xx, w, rr, residual_out=(xx, rr)[which])
        assert r1.data_ptr() == (xx, rr)[which].data_ptr()
        assert torch.equal(r1.view(torch.int16), r0.view(torch.int16))
        assert np.array_equal(_u8(c1), _u8(c0)) and torch.equal(s1, s0)
    with pytest.raises(ValueError, match="norm_out may not overlap"):
        add_rmsnorm_fp8(x, w, r, norm_out=x)


def test_norm_rows_without_a_number(gpu):
    """A zero row has zero codes; a NaN or infinite row is NaN throughout and
    leaves the others alone."""
    x = torch.randn(5, 272, generator=synth.gen(4))
    x[1] = 0
    x[2, 100], x[3, 271] = float("nan"), float("inf")
    w = torch.ones(272)
    print("add_rmsnorm_fp8 rows without a number", flush=True)
    codes, scales, _, y = add_rmsnorm_fp8(x.to(gpu), w.to(gpu), with_norm=True)
    v = F.decode(_u8(codes))
    assert not v[1].any() and np.isfinite(v[[0, 1, 4]]).all()
    with np.errstate(invalid="ignore"):
        deq = v * F.spread(scales.cpu().numpy(), 5, 272)
    assert np.isnan(deq[2]).all()
    # an infinite sum of squares scales finite values to zero, the infinity to NaN
    assert np.isnan(_np(y)[3, 271]) and not _np(y)[3, :271].any()
    assert np.isnan(deq[3, 256:]).all()


def test_empty_calls(gpu):
    print("8-bit operators, empty inputs", flush=True)
    e = torch.empty(0, 256, device=gpu)
    c, s = fp8_quantize(e)
    assert c.shape == (0, 256) and s.shape == (0, 4)
    c, s, r = add_rmsnorm_fp8(e, torch.ones(256, device=gpu), e)
    assert c.shape == (0, 256) and r.shape == (0, 256)
    b, sb = fp8_quantize(torch.ones(64, 256, device=gpu), block_rows=128)
    assert mm_fp8_block(c, b, s, sb).shape == (0, 64)
    ind = torch.zeros(2, dtype=torch.int32, device=gpu)
    assert grouped_mm_fp8_block(c, s, b[None], sb[None], ind).shape == (0, 64)
    torch.cuda.synchronize()


@pytest.mark.parametrize("indptr,m", [([4, 4, 9], 40), ([0, 0, 0], 7), ([0, 33, 33], 33),
                                      ([2, 200, 500], 700)], ids=str)
def test_grouped_fresh_out_is_zero_outside_the_groups(gpu, indptr, m):
    """A fresh out holds zeros before the first group and behind the last, also
    where its memory held something else."""
    g = synth.gen(m)
    n, k = 272, 144
    E = len(indptr) - 1
    a, b = _codes(g, (m, k)).to(gpu).view(F8), _codes(g, (E, n, k)).to(gpu).view(F8)
    sa, sb = _scale_rows(g, (m,), k).to(gpu), _scale_rows(g, (E, 3), k).to(gpu)
    ind = torch.tensor(indptr, dtype=torch.int32, device=gpu)
    for dtype in DTYPES:
        print(f"grouped_mm_fp8_block fresh out {indptr} {dtype}", flush=True)
        torch.full((m, n), float("nan"), dtype=dtype, device=gpu)  # freed: reused by out
        got = grouped_mm_fp8_block(a, sa * 2.0 ** -8, b, sb * 2.0 ** -8, ind, out_dtype=dtype)
        v = _np(got)
        inside = np.zeros(m, bool)
        inside[indptr[0]:indptr[-1]] = True
        assert not v[~inside].any() and np.isfinite(v).all()
        assert not inside.any() or (v[inside] != 0).any(axis=1).all()


def test_quantise_and_norm_views(gpu):
    """Strided views give what their copies give, on a side stream too."""
    g = synth.gen(83)
    x = torch.randn(70, 3, 544, generator=g).to(torch.bfloat16).to(gpu)
    w = torch.randn(2 * 544, generator=g).to(gpu)[::2]
    u8 = lambda t: t.view(torch.uint8)
    torch.cuda.synchronize()
    print("fp8_quantize and add_rmsnorm_fp8 of views", flush=True)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [fp8_quantize(x[:, 1]), fp8_quantize(x.transpose(0, 1), block_rows=128),
               fp8_quantize(x[:, 0], swiglu=True),
               add_rmsnorm_fp8(x[:, 1], w, x[:, 2], with_norm=True)]
    s.synchronize()
    c = lambda t: t.contiguous()
    want = [fp8_quantize(c(x[:, 1])), fp8_quantize(c(x.transpose(0, 1)), block_rows=128),
            fp8_quantize(c(x[:, 0]), swiglu=True),
            add_rmsnorm_fp8(c(x[:, 1]), c(w), c(x[:, 2]), with_norm=True)]
    for a, b in zip(got, want):
        assert all(p.is_contiguous() and torch.equal(u8(p), u8(q)) for p, q in zip(a, b))
