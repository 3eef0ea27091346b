"""The router's balance loss, its counts and its gradient, against the fp64 oracle.

Counts are equal.  Bounds: exp of an fp32 difference l - m is within (|l - m| + 4) 2^-23 of
itself (the difference's rounding, and expf), the row's sum at most 16 values in sequence
and 6 levels of pairs; so p is within E_P = (2 span + 40) 2^-23 of itself, span the largest
|l - m|.  A mean adds the rows a lane group sees in sequence, at most T / 16 + 16."""
import numpy as np
import pytest
import torch

from oracle import train as ot

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SIZES = [(1, 1, 1), (1, 8, 2), (5, 3, 3), (64, 8, 2), (63, 16, 16), (100, 17, 4), (257, 64, 8), (1021, 37, 6),
         (300, 128, 8), (4096, 128, 8), (33, 130, 7), (77, 256, 16), (40, 257, 5), (50, 512, 8), (30, 1000, 3),
         (700, 1024, 16), (20000, 8, 1)]


def _inputs(T, E, k, seed, masked):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * 1.5 + torch.randn(E, generator=g)
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    mask = (torch.rand(T, generator=g) < 0.6).to(torch.uint8) if masked else None
    d_in = torch.randn(T, E, generator=g) * 1e-3 / T
    return logits, idx, mask, d_in


def _c(t):
    return None if t is None else t.cuda()


def _n(t):
    return None if t is None else t.cpu().numpy()


def _verify(logits, idx, mask, d_in, coef, d_loss, op, loss, d):
    T, E = logits.shape
    k = idx.shape[1]
    lg = logits.double().numpy()
    want, counts, prob = ot.balance_forward(lg, idx.numpy(), _n(mask), np.float32(coef))
    assert np.array_equal(_n(op.counts), counts)
    on = np.ones(T, bool) if mask is None else _n(mask) != 0
    live = lg[on]
    fin = live[np.isfinite(live)]
    span = float(fin.max() - fin.min()) if fin.size else 0.0
    ep = (2 * span + 40) * 2 * U
    es = ep + (T / 16 + 32) * U
    assert np.all(np.abs(_n(op.prob) - prob) <= es * prob + 1e-45)
    assert abs(float(loss) - want) <= (es + 8 * U) * abs(want)
    ref = ot.balance_backward(lg, counts, k, _n(mask), np.float32(coef), np.float32(d_loss), _n(d_in))
    n = int(counts[E])
    bound = 2 * U * np.abs(ref) + 1e-45
    if n:
        c = counts[:E] - k * n / E
        p = np.zeros((T, E))
        p[on] = ot._softmax(lg[on])
        size = abs(d_loss * coef) * E / (k * n * n) * p * (np.abs(c) + (p * np.abs(c)).sum(axis=1, keepdims=True))
        bound = bound + (3 * ep + 32 * U) * size
        # the oracle's own fp64: with every count equal, c - sum c p is 0 in exact arithmetic
        # and up to (E + 4) 2^-53 times the two terms as it is summed there
        bound = bound + (E + 4) * 2.0 ** -53 * abs(d_loss * coef) * E / (k * n * n) * p * 2 * counts[:E].max()
    bad = ~(np.abs(_n(d) - ref) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:3].tolist(), _n(d)[bad][:3], ref[bad][:3], bound[bad][:3])


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_balance_against_the_oracle(T, E, k, masked):
    from combine_top_router_amd import BalanceLoss
    logits, idx, mask, d_in = _inputs(T, E, k, T + E, masked)
    op = BalanceLoss(T, E, k)
    loss = op.forward(logits.cuda(), idx.cuda(), 0.02, mask=_c(mask))
    d = op.backward(torch.full((1,), 1.5, device="cuda"), d_logits_in=d_in.cuda())
    torch.cuda.synchronize()
    _verify(logits, idx, mask, d_in, 0.02, 1.5, op, loss, d)
    first = (loss.clone(), d.clone(), op.counts.clone())
    loss = op.forward(logits.cuda(), idx.cuda(), 0.02, mask=_c(mask))   # the same again, bit for bit; in place
    buf = d_in.cuda()
    d = op.backward(torch.full((1,), 1.5, device="cuda"), d_logits_in=buf, out=buf)
    assert torch.equal(loss, first[0]) and torch.equal(d, first[1]) and torch.equal(op.counts, first[2])
    d = op.backward()   # alone: upstream 1, nothing to add to
    torch.cuda.synchronize()
    _verify(logits, idx, mask, None, 0.02, 1.0, op, loss, d)


def test_balance_counts_nothing_that_is_masked():
    """Masked tokens may hold anything; with all masked the loss, counts and gradient are 0."""
    from combine_top_router_amd import BalanceLoss
    T, E, k = 70, 24, 3
    logits, idx, mask, d_in = _inputs(T, E, k, 9, True)
    op = BalanceLoss(T, E, k)
    loss = op.forward(logits.cuda(), idx.cuda(), 0.1, mask=mask.cuda()).clone()
    want = (loss, op.counts.clone(), op.prob.clone(), op.backward().clone())
    bad_l, bad_i = logits.clone(), idx.clone()
    bad_l[mask == 0] = float("nan")
    bad_i[mask == 0] = 1 << 30
    loss = op.forward(bad_l.cuda(), bad_i.cuda(), 0.1, mask=(mask * 200).cuda())   # any non-zero value counts
    for a, b in zip((loss, op.counts, op.prob, op.backward()), want):
        assert torch.equal(a, b)
    op.forward(bad_l.cuda(), idx.cuda(), 0.1, mask=torch.zeros(T, dtype=torch.uint8, device="cuda"))
    assert not op.loss.any() and not op.counts.any() and not op.prob.any()
    assert torch.equal(op.backward(d_logits_in=d_in.cuda()), d_in.cuda())


def test_balance_of_masked_experts():
    """Logits of -inf and of the type's lowest value have no probability; a row of nothing but
    -inf counts with none; NaN stays in its row."""
    from combine_top_router_amd import BalanceLoss
    T, E, k = 40, 20, 2
    logits, idx, _, d_in = _inputs(T, E, k, 10, False)
    logits[:, 5] = -float("inf")
    logits[:, 6] = torch.finfo(torch.float32).min
    logits[7] = -float("inf")
    op = BalanceLoss(T, E, k)
    loss = op.forward(logits.cuda(), idx.cuda(), 0.1)
    d = op.backward(d_logits_in=d_in.cuda())
    torch.cuda.synchronize()
    assert float(op.prob[5]) == 0 and float(op.prob[6]) == 0
    assert torch.equal(d[7].cpu(), d_in[7]) and torch.equal(d[:, 5].cpu(), d_in[:, 5])
    lg = logits.clone()
    lg[:, 6] = -float("inf")
    _verify(lg, idx, None, d_in, 0.1, 1.0, op, loss, d)
    logits[3, 2] = float("nan")
    op.forward(logits.cuda(), idx.cuda(), 0.1)
    d2 = op.backward(d_logits_in=d_in.cuda())
    keep = torch.arange(T) != 3
    assert torch.isnan(d2[3]).any() and torch.equal(d2[keep.cuda()], d[keep.cuda()])


def test_balance_ids_twice_and_outside():
    from combine_top_router_amd import BalanceLoss
    T, E, k = 9, 6, 3
    logits, idx, _, _ = _inputs(T, E, k, 11, False)
    idx[0] = 4
    idx[1] = torch.tensor([-1, 6, 2], dtype=torch.int32)
    op = BalanceLoss(T, E, k)
    loss = op.forward(logits.cuda(), idx.cuda(), 1.0)
    d = op.backward()
    torch.cuda.synchronize()
    _verify(logits, idx, None, None, 1.0, 1.0, op, loss, d)


def test_balance_without_tokens():
    lib = __import__("combine_top_router_amd").lib
    s = lib.MoeShape(0, 64, 64, 12, 2, 0, 12, lib.MOE_BF16, 0, 1, 0, 0, 0)
    loss, prob = torch.ones(1, device="cuda"), torch.ones(12, device="cuda")
    counts = torch.ones(13, dtype=torch.int32, device="cuda")
    ws = torch.empty(lib.moe_balance_scratch_bytes(s), dtype=torch.uint8, device="cuda")
    lib.moe_balance_fwd(s, 0, 0, 0, 1.0, loss.data_ptr(), counts.data_ptr(), prob.data_ptr(), ws.data_ptr(),
                        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert not loss.any() and not counts.any() and not prob.any()


def test_balance_refuses_other_tensors():
    from combine_top_router_amd import BalanceLoss
    op = BalanceLoss(4, 8, 2)
    lg, idx = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(RuntimeError):
        op.backward()
    for a in ((lg.bfloat16(), idx), (lg[:3], idx), (lg, idx.long()), (lg, idx[:, :1]), (lg.cpu(), idx)):
        with pytest.raises(ValueError):
            op.forward(*a, 1.0)
    with pytest.raises(ValueError):
        op.forward(lg, idx, 1.0, mask=torch.ones(4, device="cuda"))
