"""The balance loss on both sides of the number of rows that one workgroup takes, for every number
of lanes that a row has."""
import numpy as np
import pytest
import torch

import moe_expert_grouped_amd as mi
import synth
from oracle import router as O

# experts, the most tokens of one workgroup
SIZES = [(3, 512), (8, 512), (64, 512), (65, 256), (128, 256), (256, 128), (257, 64), (1024, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("E,most", SIZES)
def test_both_sides(gpu, E, most):
    print(f"balance rounds E={E}", flush=True)
    k = min(E, 4)
    for T in (most - 1, most, most + 1, 4 * most + 3):
        g = synth.gen(T + E)
        z = torch.randn(T, E, generator=g)
        mask = torch.rand(T, generator=g) < 0.9
        w, ids = mi.moe_route_topk(z.to(gpu), k)
        loss, counts, slopes = mi.moe_balance_loss(z.to(gpu), ids, coef=0.5, token_mask=mask.to(gpu))
        rl, rc, rs = O.balance(z.double().numpy(), ids.cpu().numpy(), 0.5, mask)
        assert np.array_equal(counts.cpu().numpy(), rc), T
        # one rounding of the quotient of exact counts; sums of at most T / 8 rows and 32 parts
        assert np.allclose(slopes.cpu().double(), rs, rtol=2.0 ** -23, atol=0), T
        assert abs(loss.item() - rl) <= (E / 8 + T / 8 + 60) * 2.0 ** -24 * rl, T


@pytest.mark.parametrize("E,most", SIZES)
def test_more_rounds_go_to_several_workgroups(E, most):
    """Whose sums the query counts: one workgroup's are E sums, E counts and two totals."""
    one = (2 * E + 2 + (E + 63) // 64 + 1) * 4
    assert mi.balance_workspace_bytes(1, E) == mi.balance_workspace_bytes(most, E) == one
    assert mi.balance_workspace_bytes(most + 1, E) == one + most // 64 * (2 * E + 2) * 4
