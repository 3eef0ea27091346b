"""The balance loss on the shares of an expert-parallel layer: d_logits is a sum over the
shares, in which the loss counts once."""
import numpy as np
import pytest
import torch

from oracle import train as ot

pytestmark = pytest.mark.gpu

T, H, I, E, K = 96, 128, 64, 8, 2
COEF = 40.0   # a gradient as large as the routing's


def _inputs():
    g = torch.Generator().manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    logits = (torch.randn(T, E, generator=g) + torch.arange(E) * 0.3).cuda()
    return logits, randn(T, H), randn(E, H, I) / 8, randn(E, H, I) / 8, randn(E, I, H) / 8, randn(T, H)


@pytest.mark.parametrize("bounds", [(0, 8), (0, 4, 8), (0, 2, 4, 6, 8), (0, 1, 8)])
@pytest.mark.parametrize("d_balance", [None, 0.5])
def test_the_loss_counts_once_over_the_shares(bounds, d_balance):
    from combine_top_router_amd import MoeLayer
    logits, x, wg, wu, wd, dy = _inputs()
    mask = (torch.arange(T) % 5 != 0).to(torch.uint8).cuda()
    up = None if d_balance is None else torch.full((1,), d_balance, device="cuda")
    total, routing, losses = np.zeros((T, E)), np.zeros((T, E)), []
    for b, e in zip(bounds, bounds[1:]):
        lay = MoeLayer(T, H, I, E, K, e_begin=b, e_local=e - b)
        w = [t[b:e].contiguous() for t in (wg, wu, wd)]
        lay.forward(logits, x, *w)
        routing += lay.backward(dy)["d_logits"].double().cpu().numpy()
        lay.forward(logits, x, *w)
        losses.append(float(lay.balance(COEF, mask=mask)))
        total += lay.backward(dy, d_balance=up)["d_logits"].double().cpu().numpy()
    n = logits.double().cpu().numpy()
    idx, m = lay.topk_idx.cpu().numpy(), mask.cpu().numpy()
    loss, counts, _ = ot.balance_forward(n, idx, m, COEF)
    want = ot.balance_backward(n, counts, K, m, COEF, 1.0 if d_balance is None else d_balance, routing)
    assert losses == [pytest.approx(loss, rel=1e-5)] * len(losses)   # the whole loss on each
    # the kernel's fp32 gradient (softmax and counts, a few 2^-24 of the largest each) and one rounded
    # sum with the routing's: well below 1e-5 of the largest
    assert np.abs(total - want).max() <= 1e-5 * np.abs(want).max()


def test_a_wrong_d_balance_is_refused_before_any_launch():
    from combine_top_router_amd import MoeLayer
    logits, x, wg, wu, wd, dy = _inputs()
    lay = MoeLayer(T, H, I, E, K)
    lay.forward(logits, x, wg, wu, wd)
    lay.balance(COEF)
    lay.dx.fill_(3.0)
    for bad in (torch.ones(2, device="cuda"), torch.ones(1), torch.ones(1, device="cuda", dtype=torch.float64)):
        with pytest.raises(ValueError):
            lay.backward(dy, d_balance=bad)
    torch.cuda.synchronize()
    assert (lay.dx == 3).all()
