"""A training step of a MoE layer with low-rank adapters around its experts, every operator
of the package in its place: projection and router with adapters, top_k, balance loss,
permutation, experts, combine, and all gradients back to the adapters.

Against torch's autograd in 64 bits with the step's own choices.  Between the input and any
result lie at most eight roundings to bf16 (2^-8 of a value each); the sums between them
are linear, and the router's weights have slopes below 1, so a result is off by at most
8 * 2^-8 of its norm if no error cancels, doubled for the products of two rounded factors."""
import pytest
import torch

import moe_expert_grouped_amd as mi
import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [48, 700])
def test_step_against_autograd(gpu, T):
    print(f"adapters and router, one training step T={T}", flush=True)
    H, E, k, L, R, coef = 256, 16, 2, 3, 16, 0.5
    g = synth.gen(T)
    bf = lambda *s, std: (torch.randn(s, generator=g) * std).to(torch.bfloat16)
    x, wp, wr, we = bf(T, H, std=1.0), bf(H, H, std=H ** -0.5), bf(E, H, std=H ** -0.5), bf(E, H, H, std=H ** -0.5)
    a1, b1 = bf(L, R, H, std=H ** -0.5), bf(L, H, R, std=0.2)
    a2, b2 = bf(L, R, H, std=H ** -0.5), bf(L, E, R, std=0.2)
    ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32)
    scale, go = torch.tensor([0.5, 1.0, 2.0]), bf(T, H, std=1.0)
    d = [t.to(gpu) for t in (x, wp, a1, b1, ids, scale, wr, a2, b2, we, go)]
    X, WP, A1, B1, IDS, S, WR, A2, B2, WE, GO = d

    h, act1 = mi.mm_lora(X, WP, A1, B1, IDS, S, with_act=True)
    logits, act2 = mi.mm_lora(h, WR, A2, B2, IDS, S, out_dtype=torch.float32, with_act=True)
    w, top = mi.moe_route_topk(logits, k)
    loss, counts, slopes = mi.moe_balance_loss(logits, top, coef=coef)
    m, perm, inverse = mi.moe_route_permutation(top, E, with_inverse=True)
    rows = mi.grouped_mm_bf16(mi.moe_permute_rows(h, perm, k), WE, m)
    out = mi.moe_combine_rows(rows, perm, w)
    assert torch.equal(torch.diff(m), counts)

    grad_rows, grad_w = mi.moe_combine_rows_backward(GO, rows, perm, w, permuted_idx_to_expanded_idx=inverse)
    grad_px = mi.grouped_mm_bf16(grad_rows, WE.transpose(1, 2).contiguous(), m)
    grad_z = mi.moe_route_backward(logits, topk_ids=top, topk_weights=w, grad_weights=grad_w, slopes=slopes,
                                   grad_loss=torch.ones((), device=gpu), grad_dtype=torch.bfloat16)
    gh2, ga2, gb2 = mi.mm_lora_backward(grad_z, h, WR, A2, B2, IDS, S, act=act2, grad_dtype=torch.float32)
    gh = mi.moe_permute_rows_backward(grad_px, perm, k) + gh2
    gx, ga1, gb1 = mi.mm_lora_backward(gh, X, WP, A1, B1, IDS, S, act=act1, grad_dtype=torch.float32)
    torch.cuda.synchronize()

    leaf = [t.double().requires_grad_() for t in (x, a1, b1, a2, b2)]
    rx, ra1, rb1, ra2, rb2 = leaf
    of = ((ids[:, None] == torch.arange(L)) * scale).double()  # a row's own adapter, scaled

    def project(x, w, a, b):
        return x @ w.double().t() + torch.einsum("tl,tlr,lnr->tn", of, torch.einsum("tk,lrk->tlr", x, a), b)

    rh = project(rx, wp, ra1, rb1)
    rz = project(rh, wr, ra2, rb2)
    t = top.cpu().long()
    p = torch.softmax(rz, 1)
    rw = p.gather(1, t)
    rw = rw / rw.sum(1, keepdim=True)
    f = torch.bincount(t.flatten(), minlength=E).double() / (T * k)
    rloss = coef * E * (f * p.mean(0)).sum()
    rout = sum(rw[:, j, None] * torch.einsum("th,tnh->tn", rh, we.double()[t[:, j]]) for j in range(k))
    (rout * go.double()).sum().add(rloss).backward()

    def near(got, ref, what, roundings=16):
        got, ref = got.cpu().double(), ref.detach()
        rel = ((got - ref).norm() / ref.norm()).item()
        assert rel <= roundings * 2.0 ** -8, (what, rel)

    near(out, rout, "out")
    near(logits, rz, "logits")
    near(loss, rloss, "loss")
    for got, ref, what in zip((gx, ga1, gb1, ga2, gb2), leaf, ("x", "a1", "b1", "a2", "b2")):
        near(got, ref.grad, what)
