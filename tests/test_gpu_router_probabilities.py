"""The choice's weights, the balance loss and the gradient have one probability for an expert:
the quotient of its exponential and the row's sum, rounded once.

With one token, choices all on one expert, and coef 1 / E for E a power of two, the slopes are
1 for that expert and 0 for the others, and the loss is its probability, bit by bit.
"""
import pytest
import torch

import moe_expert_grouped_amd as mi
import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("E", [4, 8, 16, 64])
def test_loss_holds_the_weights_probability(gpu, E, dtype):
    print(f"router one probability E={E} {dtype}", flush=True)
    g = synth.gen(E)
    k = min(E, 8)
    for _ in range(6):
        z = (torch.randn(1, E, generator=g) * 2).to(dtype).to(gpu)
        w, ids = mi.moe_route_topk(z, k, renormalize=False)
        for j in range(k):
            loss, _, slopes = mi.moe_balance_loss(z, ids[:, j : j + 1].contiguous(), coef=1 / E)
            assert slopes.sum() == 1 and slopes[ids[0, j]] == 1
            assert torch.equal(loss, w[0, j]), (j, loss.item(), w[0, j].item())


@pytest.mark.parametrize("E", [4, 8, 16, 64])
def test_gradient_holds_the_weights_probability(gpu, E):
    """With a slope of 1 for one expert, of probability p, the gradient of another is its own
    probability times -p, rounded once."""
    print(f"router gradient's probability E={E}", flush=True)
    g = synth.gen(E + 1)
    for _ in range(6):
        z = (torch.randn(1, E, generator=g) * 2).to(gpu)
        w, ids = mi.moe_route_topk(z, min(E, 8), renormalize=False)
        slopes = torch.zeros(E, device=gpu)
        slopes[ids[0, 0]] = 1.0
        got = mi.moe_route_backward(z, slopes=slopes, grad_loss=torch.ones((), device=gpu))[0]
        p = w[0, 0]
        for j in range(1, min(E, 8)):
            assert got[ids[0, j]] == -(w[0, j] * p), j
