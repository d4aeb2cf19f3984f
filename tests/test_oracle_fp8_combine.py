"""CPU pins of the 8-bit oracle and the combine oracle, and the host-side
refusals of their entry points (no GPU: they fail before any launch)."""
import numpy as np
import pytest
import torch

import moe_expert_grouped_amd as mi
from moe_expert_grouped_amd import _lib
from oracle import combine as C
from oracle import fp8 as F

FAKE = 0x100000  # never dereferenced: validation fails before any launch


def test_e4m3_values_are_torch_s():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(F.decode(codes.numpy()), want, equal_nan=True)
    assert np.nanmax(F.e4m3_values()) == 448.0


def test_half_step_is_half_the_gap():
    v = np.unique(F.e4m3_values()[:127])
    for lo, hi in zip(v[:-1], v[1:]):
        assert F.half_step(0.5 * (lo + hi)) == 0.5 * (hi - lo)
    assert F.half_step(0.0) == 2.0 ** -10


def test_scales_by_hand():
    y = np.zeros((3, 144), dtype=np.float32)
    y[0, 5], y[1, 130], y[2, 0] = -448.0, 896.0, 1.0
    s = F.block_scales(y)
    assert s.shape == (3, 4) and s[0, 0] == 1.0 and s[1, 1] == 2.0
    assert s[0, 1] == np.float32(2.0 ** -126) and not s[:, 2:].any()
    whole = F.block_scales(y, 128)
    assert whole.shape == (1, 4) and whole[0, 0] == 1.0 and whole[0, 1] == 2.0
    y[1, 3] = np.nan
    assert np.isnan(F.block_scales(y)[1, 0]) and F.block_scales(y)[0, 0] == 1.0
    assert [F.scale_cols(k) for k in (16, 512, 528, 7168)] == [4, 4, 8, 56]
    assert [mi.fp8_scale_cols(k) for k in (16, 512, 528, 7168)] == [4, 4, 8, 56]
    assert [_lib.lib().mi_fp8_scale_cols(k) for k in (0, 16, 512, 528, 7168)] == [0, 4, 4, 8, 56]


def test_product_by_hand():
    one, two = 0x38, 0x40  # 1.0 and 2.0
    a = np.full((2, 144), one, dtype=np.uint8)
    b = np.full((130, 144), two, dtype=np.uint8)
    sa = np.array([[1, 10, 0, 0], [2, 20, 0, 0]], np.float32)
    sb = np.array([[1, 3, 0, 0], [5, 7, 0, 0]], np.float32)
    out, _ = F.mm_fp8_block(a, sa, b, sb)
    assert out[0, 0] == 2 * (128 * 1 * 1 + 16 * 10 * 3)
    assert out[1, 129] == 2 * (128 * 2 * 5 + 16 * 20 * 7)
    got, _, top, written = F.grouped_mm_fp8_block(a, sa, np.stack([b, b]), np.stack([sb, sb]), [0, 0, 1])
    assert written.tolist() == [True, False] and got[0, 0] == out[0, 0]
    assert top[0, 0] == out[0, 0] / 8


def test_norm_against_torch():
    g = torch.Generator().manual_seed(3)
    x, r, w = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 48), (5, 48), (48,)))
    h, y = F.add_rmsnorm(x.numpy(), w.numpy(), r.numpy(), 1e-5)
    want = torch.nn.functional.rms_norm(x + r, (48,), w, 1e-5)
    assert np.allclose(y, want.numpy(), rtol=1e-13, atol=0) and np.array_equal(h, (x + r).numpy())


def test_combine_gradients_against_differences():
    """The combine is linear in the rows and in the weights, so central
    differences are exact up to fp64 rounding."""
    rng = np.random.default_rng(5)
    T, k, H, P = 4, 3, 6, 11
    perm = rng.permutation(P + 2)[:T * k] - 1   # one entry -1, one past the rows
    perm[0] = P + 3
    rows, w, go = rng.normal(size=(P, H)), rng.normal(size=(T, k)), rng.normal(size=(T, H))
    gr, gw, _, hit = C.combine_rows_backward(go, rows, perm, w)
    f = lambda r, v: (C.combine_rows(r, perm, v, T, k)[0] * go).sum()
    for idx in np.ndindex(*rows.shape):
        d = np.zeros_like(rows)
        d[idx] = 0.5
        assert abs(f(rows + d, w) - f(rows - d, w) - gr[idx]) < 1e-12
    for idx in np.ndindex(*w.shape):
        d = np.zeros_like(w)
        d[idx] = 0.5
        assert abs(f(rows, w + d) - f(rows, w - d) - gw[idx]) < 1e-12
    assert hit.sum() == ((perm >= 0) & (perm < P)).sum()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def _err(status):
    with pytest.raises(ValueError) as ei:
        _lib.check(status)
    return str(ei.value)


def _call(fn, defaults, **kw):
    assert set(kw) <= set(defaults)
    return getattr(_lib.lib(), fn)(*{**defaults, **kw}.values())


def _mm(**kw):
    return _call("mi_mm_fp8_block", dict(a=FAKE, sa=FAKE, m=5, k=128, b=FAKE, sb=FAKE, n=64,
                                         out=FAKE, dt=_lib.MI_BF16, stream=None), **kw)


def _gmm(**kw):
    return _call("mi_grouped_mm_fp8_block", dict(a=FAKE, sa=FAKE, m=5, k=128, b=FAKE, sb=FAKE, e=4,
                                                 n=64, ind=FAKE, zero=0, out=FAKE, dt=_lib.MI_BF16,
                                                 stream=None), **kw)


@pytest.mark.parametrize("f,name", [(_mm, "mm_fp8_block"), (_gmm, "grouped_mm_fp8_block")])
def test_product_refusals(f, name):
    assert f"{name}: n % 16 == 0" in _err(f(n=40))
    assert f"{name}: n % 16 == 0" in _err(f(n=0))
    assert f"{name}: k % 16 == 0" in _err(f(k=136))
    assert f"{name}: k % 16 == 0" in _err(f(k=0))
    assert "rows out of range" in _err(f(m=-1))
    assert "rows out of range" in _err(f(m=1 << 31))
    assert "out_dtype" in _err(f(dt=7))
    assert "b or b_scale is null" in _err(f(sb=None))
    assert "a, a_scale or out is null" in _err(f(sa=None))
    for arg in ("a", "sa", "b", "sb", "out"):
        assert "16-byte aligned" in _err(f(**{arg: FAKE + 8}))
    for kw in (dict(k=1 << 22), dict(n=1 << 20)):
        with pytest.raises(NotImplementedError, match="31-bit buffer range"):
            _lib.check(f(**kw))
    assert f(m=0, a=None, sa=None, out=None) == _lib.MI_OK


def test_grouped_product_refusals():
    assert "m_indptr is null" in _err(_gmm(ind=None))
    assert "batch_size must be in [1, 1024]" in _err(_gmm(e=0))
    assert "batch_size must be in [1, 1024]" in _err(_gmm(e=1025))


def _quant(**kw):
    return _call("mi_fp8_quantize", dict(x=FAKE, batch=1, rows=4, k=128, dt=_lib.MI_BF16, br=1,
                                         glu=0, codes=FAKE, scales=FAKE, stream=None), **kw)


def test_quantise_refusals():
    assert "x must be" in _err(_quant(dt=5))
    assert "block_rows must be 1 or 128" in _err(_quant(br=64))
    assert "swiglu needs block_rows == 1" in _err(_quant(br=128, glu=1))
    assert "K % 16 == 0" in _err(_quant(k=24))
    assert "K % 16 == 0" in _err(_quant(k=0))
    assert "out of range" in _err(_quant(rows=-1))
    assert "out of range" in _err(_quant(batch=1 << 30, rows=1 << 30, k=1 << 20))
    assert "null pointer" in _err(_quant(codes=None))
    assert "16-byte aligned" in _err(_quant(x=FAKE + 2))
    assert "too many blocks" in _err(_quant(batch=1 << 20, rows=1 << 14, k=1 << 14, br=128))
    assert _quant(rows=0, x=None) == _lib.MI_OK and _quant(batch=0, x=None) == _lib.MI_OK


def _norm(**kw):
    return _call("mi_add_rmsnorm_fp8", dict(x=FAKE, r=FAKE + (1 << 20), w=FAKE, dt=_lib.MI_BF16,
                                            wdt=_lib.MI_BF16, t=4, h=256, eps=1e-6,
                                            ro=FAKE + (2 << 20), no=None, codes=FAKE + (3 << 20),
                                            scales=FAKE + (4 << 20), stream=None), **kw)


def test_norm_refusals():
    assert "x must be" in _err(_norm(dt=9))
    assert "weight must be of x's type or fp32" in _err(_norm(wdt=_lib.MI_F16))
    assert "hidden_size % 16 == 0" in _err(_norm(h=250))
    assert "num_tokens out of range" in _err(_norm(t=-1))
    assert "eps must be >= 0" in _err(_norm(eps=-1.0))
    assert "eps must be >= 0" in _err(_norm(eps=float("nan")))
    assert "residual and residual_out go together" in _err(_norm(r=None))
    assert "residual and residual_out go together" in _err(_norm(ro=None))
    assert "null pointer" in _err(_norm(w=None))
    assert "16-byte aligned" in _err(_norm(no=FAKE + 4))
    # a stream written over rows that other workgroups still read
    assert "residual_out may be residual itself" in _err(_norm(ro=FAKE + (1 << 20) + 512))
    assert "residual_out may be x itself" in _err(_norm(ro=FAKE + 512))
    assert "norm_out may not overlap" in _err(_norm(no=FAKE))
    assert "norm_out may not overlap" in _err(_norm(no=FAKE + (2 << 20)))
    assert _norm(t=0, x=None) == _lib.MI_OK


def test_combine_refusals():
    f = lambda **kw: _call("mi_moe_combine_rows", dict(
        rows=FAKE, dt=_lib.MI_BF16, p=8, h=64, perm=FAKE, w=None, t=4, k=2, out=FAKE,
        odt=_lib.MI_BF16, stream=None), **kw)
    assert "rows and out must be" in _err(f(dt=4))
    assert "hidden_size % 8 == 0" in _err(f(h=60))
    assert "[0, 2^31)" in _err(f(k=0))
    assert "[0, 2^31)" in _err(f(t=1 << 30))
    assert "num_rows must be >= 0" in _err(f(p=-1))
    assert "null pointer" in _err(f(perm=None))
    assert "null pointer" in _err(f(rows=None))
    assert "16-byte aligned" in _err(f(out=FAKE + 4))
    assert f(t=0, out=None) == _lib.MI_OK
    b = lambda **kw: _call("mi_moe_combine_rows_backward", dict(
        go=FAKE, gdt=_lib.MI_BF16, rows=FAKE, dt=_lib.MI_BF16, p=8, h=64, perm=FAKE, inv=None,
        w=FAKE, t=4, k=2, gr=FAKE, gw=FAKE, stream=None), **kw)
    assert "grad_out and rows must be" in _err(b(gdt=4))
    assert "hidden_size % 8 == 0" in _err(b(h=60))
    assert "[0, 2^31)" in _err(b(k=0))
    assert "num_rows out of range" in _err(b(p=1 << 31))
    assert "is null" in _err(b(w=None))
    assert "grad_rows is null" in _err(b(gr=None))
    assert "grad_weights needs rows" in _err(b(rows=None))
    assert "16-byte aligned" in _err(b(gr=FAKE + 8))
    assert b(t=0, go=None) == _lib.MI_OK


def test_outputs_apart_from_the_inputs():
    """Every output against every tensor it may not share memory with: at its
    start, at its last bytes, and (no refusal for that reason) right behind it."""
    far = lambda i: FAKE + (i << 24)

    def each(fn, base, outs, size, allowed=()):
        for out in outs:
            for other in size:
                if other == out or (out, other) in allowed or (other, out) in allowed:
                    continue
                for at in (0, (size[other] - 1) // 16 * 16):
                    assert "overlap" in _err(_call(fn, base, **{out: base[other] + at})), (out, other)
                before = base[other] - -(-size[out] // 16) * 16 + 16
                assert "overlap" in _err(_call(fn, base, **{out: before})), (out, other)

    mm = dict(a=far(1), sa=far(2), m=5, k=128, b=far(3), sb=far(4), n=64, out=far(5),
              dt=_lib.MI_BF16, stream=None)
    sizes = dict(a=5 * 128, sa=5 * 16, b=64 * 128, sb=16, out=5 * 64 * 2)
    each("mi_mm_fp8_block", mm, ["out"], sizes)
    gmm = dict(a=far(1), sa=far(2), m=5, k=128, b=far(3), sb=far(4), e=4, n=64, ind=far(6), zero=0,
               out=far(5), dt=_lib.MI_F32, stream=None)
    each("mi_grouped_mm_fp8_block", gmm, ["out"],
         dict(a=5 * 128, sa=5 * 16, b=4 * 64 * 128, sb=4 * 16, ind=20, out=5 * 64 * 4))
    for glu in (0, 1):
        q = dict(x=far(1), batch=1, rows=4, k=128, dt=_lib.MI_BF16, br=1, glu=glu, codes=far(2),
                 scales=far(3), stream=None)
        each("mi_fp8_quantize", q, ["codes", "scales"],
             dict(x=4 * 128 * 2 * (1 + glu), codes=4 * 128, scales=4 * 16))
    norm = dict(x=far(1), r=far(2), w=far(3), dt=_lib.MI_BF16, wdt=_lib.MI_F32, t=4, h=256,
                eps=1e-6, ro=far(4), no=far(5), codes=far(6), scales=far(7), stream=None)
    sizes = dict(x=2048, r=2048, w=1024, ro=2048, no=2048, codes=1024, scales=64)
    each("mi_add_rmsnorm_fp8", norm, ["ro", "no", "codes", "scales"], sizes,
         allowed=[("ro", "x"), ("ro", "r")])
    comb = dict(rows=far(1), dt=_lib.MI_F16, p=8, h=64, perm=far(2), w=far(3), t=4, k=2, out=far(4),
                odt=_lib.MI_F32, stream=None)
    each("mi_moe_combine_rows", comb, ["out"], dict(rows=1024, perm=32, w=32, out=1024))
    back = dict(go=far(1), gdt=_lib.MI_F32, rows=far(2), dt=_lib.MI_BF16, p=8, h=64, perm=far(3),
                inv=far(4), w=far(5), t=4, k=2, gr=far(6), gw=far(7), stream=None)
    each("mi_moe_combine_rows_backward", back, ["gr", "gw"],
         dict(go=1024, rows=1024, perm=32, inv=32, w=32, gr=1024, gw=32))
    assert "num_rows out of range" in _err(_call("mi_moe_combine_rows", comb, p=1 << 31))


def test_python_refusals_before_the_gpu():
    """Shapes and types are checked first; then CPU tensors are refused."""
    f8 = torch.float8_e4m3fn
    a, b = torch.zeros(3, 144).to(f8), torch.zeros(130 // 2 * 2, 144).to(f8)
    sa, sb = torch.zeros(3, 4), torch.zeros(2, 4)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        mi.mm_fp8_block(a.float(), b, sa, sb)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        mi.mm_fp8_block(a, b[:, :128], sa, sb)
    with pytest.raises(ValueError, match=r"a_scale must be float32 \(M, fp8_scale_cols"):
        mi.mm_fp8_block(a, b, sa[:, :2], sb)
    with pytest.raises(ValueError, match="b_scale must be"):
        mi.mm_fp8_block(a, b, sa, sb[:1])
    with pytest.raises(ValueError, match="out_dtype"):
        mi.mm_fp8_block(a, b, sa, sb, out_dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        mi.mm_fp8_block(a, b, sa, sb)
    ind = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="m_indptr"):
        mi.grouped_mm_fp8_block(a, sa, b[None], sb[None], ind)
    with pytest.raises(ValueError, match="on the GPU"):
        mi.grouped_mm_fp8_block(a, sa, b[None], sb[None], ind[:2])
    with pytest.raises(ValueError, match="block_rows"):
        mi.fp8_quantize(torch.zeros(2, 16), block_rows=2)
    with pytest.raises(ValueError, match="on the GPU"):
        mi.fp8_quantize(torch.zeros(2, 16))
    x = torch.zeros(2, 16)
    with pytest.raises(ValueError, match="weight must be"):
        mi.add_rmsnorm_fp8(x, torch.zeros(15))
    with pytest.raises(ValueError, match="residual must have"):
        mi.add_rmsnorm_fp8(x, x[0], x.half())
    with pytest.raises(ValueError, match="needs a residual"):
        mi.add_rmsnorm_fp8(x, x[0], residual_out=x)
    perm, w = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 2)
    with pytest.raises(ValueError, match="topk_weights"):
        mi.moe_combine_rows(x, perm, w.double())
    with pytest.raises(ValueError, match="int32"):
        mi.moe_combine_rows(x, perm[:3], w)
    with pytest.raises(ValueError, match="num_tokens\\*top_k"):
        mi.moe_permute_rows_backward(x, perm, 3)
    with pytest.raises(ValueError, match="grad_out must be"):
        mi.moe_combine_rows_backward(x[:1], x, perm, w)
    with pytest.raises(ValueError, match="int32 \\[num_rows\\]"):
        mi.moe_combine_rows_backward(x, x, perm, w, permuted_idx_to_expanded_idx=perm)
    with pytest.raises(ValueError, match="needs with_weights"):
        mi.moe_combine_rows_backward(x, x, perm, w, with_weights=False, grad_weights=w)
