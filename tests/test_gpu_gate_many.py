"""Routing by scores of more tokens than one launch has workgroups for at a token's lanes each (2^32 threads)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [1, 3])
def test_gate_of_many_tokens(E):
    from combine_top_router_amd import Gate, lib as L
    T = (1 << 28) + 37
    op = Gate(T, E, 1, score=L.MOE_SCORE_SIGMOID, renorm=0)
    logits = torch.zeros(T, E, device="cuda")
    logits[:, E - 1] = 1.0
    logits[-30:] = -1.0
    for count in (False, True):
        op.topk_idx.fill_(9)
        op.topk_w.fill_(9.0)
        op.forward(logits, count=count)
        assert (op.topk_idx[:-30] == E - 1).all() and (op.topk_idx[-30:] == 0).all()
        s = torch.sigmoid(torch.tensor([1.0, -1.0])).tolist()
        assert (op.topk_w[:-30] - s[0]).abs().max() < 1e-6 and (op.topk_w[-30:] - s[1]).abs().max() < 1e-6
    assert op.counts.sum() == T and op.counts[E - 1] == (T if E == 1 else T - 30)
    op.d_logits.fill_(9.0)
    d = op.backward(torch.ones(T, 1, device="cuda"))
    top = s[0] * (1 - s[0])
    assert (d[:-30, E - 1] - top).abs().max() < 1e-6 and (d[-30:, 0] - top).abs().max() < 1e-6   # of -1, too
    assert E == 1 or (not d[:-30, :E - 1].any() and not d[-30:, 1:].any())
