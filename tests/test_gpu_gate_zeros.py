"""Logits of 0 with either sign are equal: ties, to the lower id."""
import numpy as np
import pytest
import torch

from oracle import step as os_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,k,groups,topk_groups,group_top", [(8, 3, 1, 1, 1), (40, 6, 1, 1, 1), (64, 16, 4, 2, 1), (64, 4, 8, 3, 2),
                                                              (300, 9, 1, 1, 1)])
def test_zeros_of_either_sign(E, k, groups, topk_groups, group_top, score):
    from combine_top_router_amd import Gate
    T = 40
    rng = np.random.default_rng(E)
    logits = torch.from_numpy(np.where(rng.random((T, E)) < 0.5, np.float32(-0.0), np.float32(0.0)))
    logits[::4] = torch.where(torch.from_numpy(rng.random((10, E)) < 0.9), logits[::4], -1e-44)   # below both
    op = Gate(T, E, k, score=score, groups=groups, topk_groups=topk_groups, group_top=group_top)
    op.forward(logits.cuda(), count=True)
    torch.cuda.synchronize()
    idx, _, counts = os_.gate_forward(logits.double().numpy(), None, None, k, score, groups=groups, topk_groups=topk_groups,
                                      group_top=group_top)
    assert np.array_equal(op.topk_idx.cpu().numpy(), idx) and np.array_equal(op.counts.cpu().numpy(), counts)
