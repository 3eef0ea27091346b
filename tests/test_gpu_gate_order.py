"""Routing by scores where the order hangs on the last bits: ids and counts against the fp64 oracle, to the bit."""
import numpy as np
import pytest
import torch

from oracle import step as os_

pytestmark = pytest.mark.gpu


def _check(logits, bias, k, score, groups, topk_groups, group_top):
    from combine_top_router_amd import Gate
    T, E = logits.shape
    op = Gate(T, E, k, score=score, groups=groups, topk_groups=topk_groups, group_top=group_top)
    op.forward(logits.cuda(), bias=None if bias is None else bias.cuda(), count=True)
    torch.cuda.synchronize()
    idx, _, counts = os_.gate_forward(logits.double().numpy(), None if bias is None else bias.numpy(), None, k, score,
                                      groups=groups, topk_groups=topk_groups, group_top=group_top)
    got = op.topk_idx.cpu().numpy()
    bad = np.flatnonzero((got != idx).any(axis=1))
    assert not len(bad), (len(bad), got[bad[0]], idx[bad[0]])
    assert np.array_equal(op.counts.cpu().numpy(), counts)


def _stepped(base, steps):
    """base moved up by that many fp32 numbers (down from a negative base by less)."""
    x = np.full(steps.shape, base, np.float32)
    for i in range(1, int(steps.max()) + 1):
        x = np.where(steps >= i, np.nextafter(x, np.float32(np.inf)), x)
    return torch.from_numpy(x)


SIZES = [(16, 3, 1, 1), (16, 3, 4, 4), (16, 3, 4, 2), (24, 12, 2, 2), (128, 8, 8, 8), (256, 8, 8, 4), (300, 5, 10, 10)]
BASES = (0.0, 1.0, 14.0, 27.5, 30.0, 40.0, -40.0, -800.0)


def _shut(logits, rng, groups, topk_groups):
    """All but topk_groups of the groups 200 lower: the groups' order is plain where their scores are."""
    T, E = logits.shape
    low = np.ones((T, groups), bool)
    for t in range(T):
        low[t, rng.choice(groups, topk_groups, replace=False)] = False
    return np.repeat(low, E // groups, axis=1)


@pytest.mark.parametrize("E,k,groups,topk_groups", SIZES)
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", [0, 1])
def test_two_logits_some_numbers_apart(score, group_top, E, k, groups, topk_groups):
    """Without a bias the logits order the experts, also where their scores are equal: two logits up to 7 fp32
    numbers apart, the larger at the higher or the lower id, on every pair of places of the order up to k + 1,
    around 0, where a score has risen to 1 and where it has sunk to 0.  The others lie 1/4 apart."""
    if groups == 1 and group_top == 2:
        pytest.skip("no groups")
    rng = np.random.default_rng(E + k + groups)
    T, per = 4 * (k + 1), E // groups
    for base in BASES:
        if base == -800.0 and topk_groups < groups and group_top == 2:
            continue   # all scores are 0: the groups tie, whatever lies in them
        logits = np.zeros((T, E), np.float32)
        shut = _shut(logits, rng, groups, topk_groups)
        for t in range(T):
            open_ = np.flatnonzero(~shut[t])
            rng.shuffle(open_)
            place = t % (k + 1)                       # the pair has the places `place` and the next
            if place + 1 >= len(open_):
                place = 0
            near = sorted(open_[place:place + 2])
            for j, e in enumerate(open_):
                logits[t, e] = base + 0.25 * (place - j)
            up = _stepped(base, np.array([0, 1 + t % 7])).numpy()
            logits[t, near] = up if t // (k + 1) % 4 else up[::-1]
        logits[shut] = base - 200.0
        _check(torch.from_numpy(logits), None, k, score, groups, topk_groups, group_top)
        if score == 0 and topk_groups == groups:   # one expert far above the rest, whose scores are 0
            logits[:, E // 2] = base + 1000.0
            _check(torch.from_numpy(logits), None, k, score, groups, topk_groups, group_top)


@pytest.mark.parametrize("E,k,groups,topk_groups", SIZES)
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", [0, 1])
def test_all_logits_some_numbers_apart(score, group_top, E, k, groups, topk_groups):
    """The same of all the open groups' logits at once, with ties among them."""
    if groups == 1 and group_top == 2:
        pytest.skip("no groups")
    rng = np.random.default_rng(E + k + groups)
    for base in BASES:
        if base == -800.0 and topk_groups < groups and group_top == 2:
            continue
        logits = _stepped(base, rng.integers(0, 8, (48, E))).numpy()
        logits[_shut(logits, rng, groups, topk_groups)] = base - 200.0
        _check(torch.from_numpy(logits), None, k, score, groups, topk_groups, group_top)
