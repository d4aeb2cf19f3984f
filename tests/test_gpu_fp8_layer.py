"""The 8-bit operators and the combine run together as a routed MoE layer, in a
captured graph, on two streams at once, and at sizes whose offsets pass 32 bits.

Layer: residual + norm + quantisation -> routing -> permuted codes and scales ->
FC1 -> SwiGLU + quantisation -> FC2 -> combine.  Every stage is checked against
the fp64 oracle on the values the stage was given, with the tolerances of the
stage's own tests."""
import numpy as np
import pytest
import torch

import synth
from moe_expert_grouped_amd import (add_rmsnorm_fp8, fp8_quantize, fp8_scale_cols,
                                    grouped_mm_fp8_block, mm_fp8_block, moe_combine_rows,
                                    moe_combine_rows_backward, moe_permute_rows,
                                    moe_permute_rows_backward, moe_route_permutation,
                                    route_workspace_bytes)
from oracle import combine as C
from oracle import fp8 as F
from tests.test_gpu_fp8 import HALF, U, _check, _check_codes, _codes, _np, _scale_rows, _u8

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def _weights(E, n, k, g, gpu):
    w = torch.randn(E, n, k, generator=g) * k ** -0.5
    return fp8_quantize(w.to(gpu), block_rows=128)


def test_moe_layer_stage_by_stage(gpu):
    T, top, E, H, I = 133, 4, 9, 528, 272
    g = synth.gen(31)
    print("fp8 MoE layer", flush=True)
    x, res = (synth.bf16_normal((T, H), 1.0, g).to(gpu) for _ in range(2))
    nw = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).to(gpu)
    w1, s1 = _weights(E, 2 * I, H, g, gpu)
    w2, s2 = _weights(E, H, I, g, gpu)
    ids = synth.routing_ids(seed=32, T=T, top_k=top, E=E, invalid_frac=0.1, zipf_s=1.0).to(gpu)
    tw = synth.softmax_weights(T, top, synth.gen(33)).to(gpu)

    codes, sc, stream = add_rmsnorm_fp8(x, nw, res)
    m_indptr, perm, inv = moe_route_permutation(ids, E, with_inverse=True)
    a = moe_permute_rows(codes.view(torch.uint8), perm, top).view(F8)
    sa = moe_permute_rows(sc, perm, top)
    h = grouped_mm_fp8_block(a, sa, w1, s1, m_indptr)
    a2, sa2 = fp8_quantize(h, swiglu=True)
    y = grouped_mm_fp8_block(a2, sa2, w2, s2, m_indptr)
    out = moe_combine_rows(y, perm, tw)
    torch.cuda.synchronize()

    # norm and quantisation
    hr, yr = F.add_rmsnorm(_np(x), _np(nw), _np(res))
    assert (np.abs(_np(stream) - hr) <= (HALF[torch.bfloat16] + U) * np.abs(hr)).all()
    rel = (8 + 24) * U
    _check_codes(_u8(codes), _np(sc), yr, 1, "layer norm", rel)
    # the permuted copies are copies
    total, p = int(m_indptr[-1]), perm.cpu().numpy()
    for slot, row in enumerate(p):
        if row >= 0:
            assert (_u8(a)[row] == _u8(codes)[slot // top]).all()
            assert (_np(sa)[row] == _np(sc)[slot // top]).all()
    # FC1, and zeros behind the last group
    ind = m_indptr.cpu().numpy()
    ref, mag, tops, written = F.grouped_mm_fp8_block(_u8(a), _np(sa), _u8(w1), _np(s1), ind)
    assert written.sum() == total and total < T * top
    _check(h[:total], ref[:total], mag[:total], tops[:total], H, torch.bfloat16, "FC1")
    assert not h[total:].any()
    # SwiGLU and its quantisation
    act = F.swiglu(_np(h))
    srel = (np.abs(_np(h)).max() + 16) * U
    _check_codes(_u8(a2), _np(sa2), act, 1, "SwiGLU", srel)
    # FC2
    ref, mag, tops, _ = F.grouped_mm_fp8_block(_u8(a2), _np(sa2), _u8(w2), _np(s2), ind)
    _check(y[:total], ref[:total], mag[:total], tops[:total], I, torch.bfloat16, "FC2")
    # combine
    ref, mag = C.combine_rows(_np(y), perm.cpu(), tw.cpu(), T, top)
    tol = top * U * mag + HALF[torch.bfloat16] * np.abs(ref)
    assert (np.abs(_np(out) - ref) <= tol).all()


def test_layer_in_a_graph(gpu):
    """The layer and the combine's gradients captured once and replayed with
    other inputs, eager work and synchronisations between: every replay is bitwise
    the eager result."""
    T, top, E, H, I = 70, 3, 6, 256, 128
    g = synth.gen(41, gpu)
    print("fp8 MoE layer in a graph, 4 replays", flush=True)
    gc = synth.gen(42)
    w1, s1 = _weights(E, 2 * I, H, gc, gpu)
    w2, s2 = _weights(E, H, I, gc, gpu)
    nw = torch.ones(H, dtype=torch.bfloat16, device=gpu)
    x, res, go = (synth.bf16_normal((T, H), 1.0, g, gpu) for _ in range(3))
    ids = synth.routing_ids(seed=43, T=T, top_k=top, E=E, zipf_s=1.0).to(gpu)
    tw = synth.softmax_weights(T, top, synth.gen(44)).to(gpu)
    rws = torch.empty(route_workspace_bytes(T * top, E), dtype=torch.uint8, device=gpu)

    def layer():
        codes, sc, stream, norm = add_rmsnorm_fp8(x, nw, res, with_norm=True)
        m_indptr, perm, inv = moe_route_permutation(ids, E, with_inverse=True, workspace=rws)
        a = moe_permute_rows(codes.view(torch.uint8), perm, top).view(F8)
        h = grouped_mm_fp8_block(a, moe_permute_rows(sc, perm, top), w1, s1, m_indptr)
        a2, sa2 = fp8_quantize(h, swiglu=True)
        y = grouped_mm_fp8_block(a2, sa2, w2, s2, m_indptr, out_dtype=torch.float32)
        out = moe_combine_rows(y, perm, tw, out_dtype=torch.bfloat16)
        gy, gw = moe_combine_rows_backward(go, y, perm, tw, permuted_idx_to_expanded_idx=inv)
        gx = moe_permute_rows_backward(gy, perm, top)
        one = mm_fp8_block(codes, w1[0], sc, s1[0])
        return stream, norm, out, gy, gw, gx, one

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for rnd in range(4):
        for t in (x, res, go):
            t.copy_(synth.bf16_normal((T, H), 1.0 + rnd, g, gpu))
        ids.copy_(synth.routing_ids(seed=50 + rnd, T=T, top_k=top, E=E, zipf_s=0.5,
                                    invalid_frac=0.1 * rnd).to(gpu))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = layer()
        torch.cuda.synchronize()
        for i, (u, v) in enumerate(zip(kept, want)):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8)), (rnd, i)


def test_two_streams_at_once(gpu):
    """Calls that overlap on two streams share nothing."""
    g = synth.gen(61)
    m, n, k = 300, 1024, 1024
    cases = []
    for i in range(2):
        a, b = _codes(g, (m, k)).to(gpu).view(F8), _codes(g, (n, k)).to(gpu).view(F8)
        sa, sb = _scale_rows(g, (m,), k).to(gpu), _scale_rows(g, (n // 128,), k).to(gpu)
        x = synth.bf16_normal((m, k), 1.0 + i, g).to(gpu)
        cases.append((a, b, sa, sb, x))
    w = torch.ones(k, dtype=torch.bfloat16, device=gpu)

    def work(c):
        return mm_fp8_block(*c[:4]), *fp8_quantize(c[4]), *add_rmsnorm_fp8(c[4], w, c[4])

    print("fp8 calls on two streams", flush=True)
    want = [work(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append([work(c) for _ in range(4)])
        torch.cuda.synchronize()
        for one, ref in zip(got, want):
            for r in one:
                for u, v in zip(r, ref):
                    assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def _rand_codes(shape, gpu, g):
    """Finite codes of moderate size, drawn on the GPU."""
    c = torch.randint(0x20, 0x50, shape, generator=g, device=gpu, dtype=torch.uint8)
    return c | (torch.randint(0, 2, shape, generator=g, device=gpu, dtype=torch.uint8) << 7)


def test_offsets_past_32_bits(gpu):
    """More than 2^32 codes in a, in b and in the quantisers' outputs, more than
    2^31 values in the combine's rows: the last rows are the oracle's."""
    g = synth.gen(71, gpu)
    print("mm_fp8_block, a of 4.3 GB", flush=True)
    m, n, k = 525_000, 16, 8256
    assert m * k > 2 ** 32
    a, b = _rand_codes((m, k), gpu, g), _rand_codes((n, k), gpu, g)
    cols = fp8_scale_cols(k)
    sa = torch.rand(m, cols, generator=g, device=gpu) * 0.01
    sb = torch.rand(1, cols, generator=g, device=gpu) * 0.01
    got = mm_fp8_block(a.view(F8), b.view(F8), sa, sb, out_dtype=torch.float32)
    rows = [0, 1, m // 2, m - 130, m - 2, m - 1]
    ops = (_u8(a[rows]), _np(sa[rows]), _u8(b), _np(sb))
    ref, mag = F.mm_fp8_block(*ops)
    _check(got[rows], ref, mag, None, k, torch.float32, "a past 4 GB")
    del sa, got

    print("grouped_mm_fp8_block, b of 4.3 GB", flush=True)
    E, n = 525, 992
    bb = a.view(E, m // E, k)[:, :n].contiguous()
    assert E * n * k > 2 ** 32
    mm = 2 * E
    aa = _rand_codes((mm, k), gpu, g)
    s_a = torch.rand(mm, cols, generator=g, device=gpu) * 0.01
    s_b = torch.rand(E, -(-n // 128), cols, generator=g, device=gpu) * 0.01
    ind = torch.arange(E + 1, dtype=torch.int32, device=gpu) * 2
    got = grouped_mm_fp8_block(aa.view(F8), s_a, bb.view(F8), s_b, ind, out_dtype=torch.float32)
    for e in (0, E // 2, E - 1):
        r = slice(2 * e, 2 * e + 2)
        ref, mag = F.mm_fp8_block(_u8(aa[r]), _np(s_a[r]), _u8(bb[e]), _np(s_b[e]))
        _check(got[r], ref, mag, None, k, torch.float32, f"expert {e}")
    del a, b, bb, aa, s_a, s_b, got
    torch.cuda.empty_cache()

    print("quantisers of 4.3 G values", flush=True)
    x = torch.randn(m, k, generator=g, device=gpu, dtype=torch.bfloat16)
    codes, sc = fp8_quantize(x)
    y = x[rows].float().cpu().numpy()
    want = F.block_scales(y)
    assert np.array_equal(sc[rows].cpu().numpy(), want)
    _check_codes(_u8(codes[rows]), want, y.astype(np.float64), 1, "rows past 4 G")
    del codes, sc
    codes, sc = fp8_quantize(x, block_rows=128)
    last = m // 128 * 128
    y = x[last:].float().cpu().numpy()
    want = F.block_scales(y, 128)
    assert np.array_equal(sc[-1:].cpu().numpy(), want)
    _check_codes(_u8(codes[last:]), want, y.astype(np.float64), 128, "blocks past 4 G")
    del codes, sc
    w = torch.ones(k, dtype=torch.bfloat16, device=gpu)
    codes, sc, _, norm = add_rmsnorm_fp8(x, w, with_norm=True)
    _, yr = F.add_rmsnorm(_np(x[rows]), _np(w))
    rel = (-(-k // 2048) * 8 + 24) * U
    assert (np.abs(_np(norm[rows]) - yr) <= (HALF[torch.bfloat16] + rel) * np.abs(yr)).all()
    _check_codes(_u8(codes[rows]), _np(sc[rows]), yr, 1, "norm past 4 G", rel)
    del codes, sc, norm

    print("combine of 4.3 G values", flush=True)
    top, T = 4, m // 4
    perm = torch.arange(T * top, dtype=torch.int32, device=gpu).flip(0).contiguous()
    tw = torch.rand(T, top, generator=g, device=gpu)
    out = moe_combine_rows(x, perm, tw)
    pick = [0, 1, T - 1]
    slots = [perm.view(T, top)[t].tolist() for t in pick]
    for t, s in zip(pick, slots):
        ref, mag = C.combine_rows(_np(x[s]), np.arange(top), tw[t:t + 1].cpu(), 1, top)
        tol = top * U * mag + HALF[torch.bfloat16] * np.abs(ref)
        assert (np.abs(_np(out[t:t + 1]) - ref) <= tol).all(), t
    gr, gw = moe_combine_rows_backward(out, x, perm, tw)
    for t, s in zip(pick, slots):
        rr, rw, mag, _ = C.combine_rows_backward(_np(out[t:t + 1]), _np(x[s]), np.arange(top),
                                                 tw[t:t + 1].cpu())
        assert (np.abs(_np(gr[s]) - rr) <= (HALF[torch.bfloat16] + U) * np.abs(rr)).all(), t
        assert (np.abs(_np(gw[t:t + 1]) - rw) <= (k / 64 + 8) * U * mag + U * np.abs(rw)).all(), t


def test_more_rows_than_one_launch_dimension(gpu):
    """2^24 and a few rows, more than a launch has workgroups of 256 threads in one
    dimension: the first and the last rows are those of a small call."""
    t, h = 2 ** 24 + 5, 16
    g = synth.gen(72, gpu)
    x = torch.randn(t, h, generator=g, device=gpu, dtype=torch.bfloat16)
    w = torch.randn(h, generator=g, device=gpu, dtype=torch.bfloat16)
    parts = (slice(0, 300), slice(2 ** 20 - 40, 2 ** 20 + 40), slice(t - 300, t))
    print("add_rmsnorm_fp8", flush=True)
    codes, sc, ro = add_rmsnorm_fp8(x, w, x)
    for r in parts:
        c1, s1, r1 = add_rmsnorm_fp8(x[r], w, x[r])
        assert torch.equal(codes[r].view(torch.uint8), c1.view(torch.uint8))
        assert torch.equal(sc[r], s1) and torch.equal(ro[r], r1)
    print("fp8_quantize, blocks", flush=True)
    codes, sc = fp8_quantize(x[:, None], block_rows=128)
    for r in parts:
        c1, s1 = fp8_quantize(x[r][:, None], block_rows=128)
        assert torch.equal(codes[r].view(torch.uint8), c1.view(torch.uint8))
        assert torch.equal(sc[r], s1)
