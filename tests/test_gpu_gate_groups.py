"""Groups whose two best experts have biases of opposite sign: the group's score is far smaller than what it is the
sum of, and the choice of the groups hangs on bits that fp32 has lost in s + b."""
import numpy as np
import pytest
import torch

from oracle import step as os_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("big", [4.0, 16.0, 64.0, 1000.0])
@pytest.mark.parametrize("groups,per", [(2, 2), (8, 2), (16, 4), (32, 8)])
def test_groups_of_cancelling_scores(groups, per, big, score):
    """Sums of two scores about as far apart as fp32's numbers around b: fp64's own rounding of c = s + b, 2^-53 of b,
    is 2^-29 of that, so of the 16000 sums none is expected to lie as near to another."""
    from combine_top_router_amd import Gate
    T, E, top = 2000 if groups < 32 else 500, groups * per, max(1, groups // 2)
    rng = np.random.default_rng(groups + per)
    # scores 2^-23 big apart: a sigmoid's slope at 0 is 1/4, a softmax of E equal ones has 1 / E
    spread = (4.0 if score else E) * big * 2.0 ** -23
    logits = torch.from_numpy((rng.standard_normal((T, E)) * spread).astype(np.float32))
    bias = np.full(E, -4.0 * big, np.float32)
    sign = rng.integers(0, 2, groups)
    for g in range(groups):   # the two best of a group: one far up, one far down
        bias[g * per + sign[g]], bias[g * per + 1 - sign[g]] = big, -big
    k = min(4, top * per)
    op = Gate(T, E, k, score=score, groups=groups, topk_groups=top, group_top=2)
    op.forward(logits.cuda(), bias=torch.from_numpy(bias).cuda(), count=True)
    torch.cuda.synchronize()
    idx, _, counts = os_.gate_forward(logits.double().numpy(), bias, None, k, score, groups=groups, topk_groups=top, group_top=2)
    got = op.topk_idx.cpu().numpy()
    assert np.array_equal(got, idx), int((got != idx).any(axis=1).sum())
    assert np.array_equal(op.counts.cpu().numpy(), counts)
