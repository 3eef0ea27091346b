"""Routing by scores against the fp64 oracle: ids and counts equal; weights and gradients to
their roundings.

Bounds: exp of an fp32 difference d is within (|d| + 4) 2^-23 of itself, a row's sum adds at
most 16 values in sequence and 6 levels of pairs, a division and a product one rounding each:
E = (2 span + 60) 2^-23 of a score or weight, span the largest |l| or |l - max l|."""
import numpy as np
import pytest
import torch

from oracle import step as os_

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# T, E, k, groups, topk_groups, group_top
SIZES = [(1, 1, 1, 1, 1, 1), (1, 128, 8, 1, 1, 1), (3, 5, 5, 1, 1, 1), (64, 8, 2, 2, 1, 2), (63, 64, 16, 1, 1, 1),
         (100, 63, 4, 7, 3, 2), (130, 65, 6, 13, 4, 1), (257, 128, 8, 8, 4, 2), (200, 84, 5, 7, 3, 1),
         (77, 256, 8, 8, 4, 2), (40, 256, 16, 64, 8, 2), (33, 257, 5, 1, 1, 1), (50, 512, 8, 8, 3, 2),
         (30, 1000, 3, 40, 2, 1), (20, 1024, 16, 64, 1, 2), (5000, 32, 4, 4, 2, 2)]


def _inputs(T, E, k, seed, biased, masked, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g)
    bias = torch.randn(E, generator=g) * (0.1 if biased == "sigmoid" else 0.5 / E) if biased else None
    mask = (torch.rand(T, generator=g) < 0.7).to(torch.uint8) if masked else None
    return logits, bias, mask, torch.randn(T, k, generator=g)


def _c(t):
    return None if t is None else t.cuda()


def _n(t):
    return None if t is None else t.cpu().numpy()


def _span(l):
    l = l[np.isfinite(l)]
    return float(max(np.abs(l).max(), l.max() - l.min())) if l.size else 0.0


def _gate(T, E, k, groups, topk_groups, group_top, score, renorm, scale):
    from combine_top_router_amd import Gate
    return Gate(T, E, k, score=score, groups=groups, topk_groups=topk_groups, group_top=group_top, renorm=renorm,
                scale=scale)


def _verify(op, logits, bias, mask, d, out):
    s = op.shape
    kw = dict(groups=s.groups, topk_groups=s.topk_groups, group_top=s.group_top, renorm=s.renorm, scale=s.scale)
    l = logits.double().numpy()
    idx, w, counts = os_.gate_forward(l, _n(bias), _n(mask), s.k, s.score, **kw)
    assert np.array_equal(_n(op.topk_idx), idx)
    assert np.array_equal(_n(op.counts), counts)
    E_ = (2 * _span(l) + 60) * 2 * U
    assert np.all(np.abs(_n(op.topk_w) - w) <= E_ * w + 1e-44)
    ref = os_.gate_backward(l, idx, _n(d), s.score, s.renorm, s.scale)
    # every term is a product of weights and d that carry E each, the sum over k another k U
    dd = np.where(idx >= 0, np.abs(_n(d)), 0.0)
    q = w / s.scale
    size = np.zeros_like(l)
    if s.score == 0 and not s.renorm:
        for t in range(len(l)):
            on = idx[t] >= 0
            p = os_._scores(l[t], 0)
            size[t] = s.scale * p * (q[t] * dd[t]).sum() if on.any() else 0.0
    for j in range(s.k):
        t = np.nonzero(idx[:, j] >= 0)[0]
        np.add.at(size, (t, idx[t, j]), w[t, j] * (dd[t, j] + (q * dd).sum(axis=1)[t]))
    bad = ~(np.abs(_n(out) - ref) <= (4 * E_ + 64 * U) * size + 1e-44)
    assert not bad.any(), (np.argwhere(bad)[:3].tolist(), _n(out)[bad][:3], ref[bad][:3])


@pytest.mark.parametrize("score,renorm,biased,masked", [(0, 1, False, False), (0, 0, True, True), (1, 1, True, False),
                                                        (1, 0, False, True), (0, 1, True, True), (1, 1, False, False)])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_gate_against_the_oracle(size, score, renorm, biased, masked):
    T, E, k = size[:3]
    logits, bias, mask, d = _inputs(T, E, k, T + E, biased and ("softmax", "sigmoid")[score], masked)
    op = _gate(*size, score, renorm, 2.5)
    idx, w = op.forward(logits.cuda(), bias=_c(bias), mask=_c(mask), count=True)
    assert idx is op.topk_idx and w is op.topk_w
    out = op.backward(d.cuda())
    torch.cuda.synchronize()
    _verify(op, logits, bias, mask, d, out)
    first = (idx.clone(), w.clone(), out.clone(), op.counts.clone())
    op.forward(logits.cuda(), bias=_c(bias), mask=_c(mask))   # without the counts; bit for bit
    buf = torch.empty_like(out)
    assert op.backward(d.cuda(), out=buf) is buf
    for a, b in zip((op.topk_idx, op.topk_w, buf, op.counts), first):
        assert torch.equal(a, b)


def test_gate_near_ties():
    """Scores that differ in the last bits of fp64 only, or not at all."""
    T, E, k = 300, 128, 8
    g = torch.Generator().manual_seed(3)
    logits = (torch.randint(0, 6, (T, E), generator=g) * 0.5 + 14.0)   # sigmoids a few fp32 steps below 1
    bias = torch.randint(-2, 3, (E,), generator=g) * 2.0 ** -24
    logits[7] = 30.0
    logits[8, ::2] = 40.0
    d = torch.randn(T, k, generator=g)
    for score in (0, 1):
        for groups, top, gt in ((1, 1, 1), (8, 3, 2), (8, 3, 1)):
            for b in (bias, None):
                op = _gate(T, E, k, groups, top, gt, score, 1, 1.0)
                op.forward(logits.cuda(), bias=_c(b), count=True)
                torch.cuda.synchronize()
                idx, _, counts = os_.gate_forward(logits.double().numpy(), _n(b), None, k, score, groups=groups,
                                                  topk_groups=top, group_top=gt)
                assert np.array_equal(_n(op.topk_idx), idx), (score, groups, gt, b is None)
                assert np.array_equal(_n(op.counts), counts)


@pytest.mark.parametrize("T", [1, 5, 16, 37])
@pytest.mark.parametrize("E,k,groups,top,gt", [(16, 16, 1, 1, 1), (24, 8, 3, 1, 2), (256, 16, 8, 2, 2), (600, 9, 1, 1, 1),
                                               (64, 4, 16, 1, 2), (8, 8, 2, 2, 1)])
def test_gate_of_equal_rows(T, E, k, groups, top, gt):
    """Nothing but ties, also in tokens that the mask leaves out and in a workgroup's places
    past the last token; and tokens of which the open groups are taken whole."""
    mask = (torch.arange(T) % 3 != 1).to(torch.uint8)
    for logits in (torch.zeros(T, E), torch.full((T, E), -float("inf")), torch.full((T, E), float("nan"))):
        for score in (0, 1):
            for biased in (False, True):
                op = _gate(T, E, k, groups, top, gt, score, 1, 1.0)
                bias = torch.zeros(E) if biased else None
                op.forward(logits.cuda(), bias=_c(bias), mask=mask.cuda(), count=True)
                torch.cuda.synchronize()
                idx, _, counts = os_.gate_forward(logits.double().numpy(), _n(bias), _n(mask), k, score, groups=groups,
                                                  topk_groups=top, group_top=gt)
                assert np.array_equal(_n(op.topk_idx), idx) and np.array_equal(_n(op.counts), counts)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("spread", [30.0, 300.0])
def test_gate_of_wide_logits(score, spread):
    """Scores that underflow in fp32 still share out a row's weights."""
    T, E, k = 64, 40, 6
    logits, bias, _, d = _inputs(T, E, k, 5, None, False, spread)
    logits[:8] -= 3 * spread   # whole rows far below 0
    op = _gate(T, E, k, 1, 1, 1, score, 1, 1.0)
    op.forward(logits.cuda(), count=True)
    out = op.backward(d.cuda())
    torch.cuda.synchronize()
    _verify(op, logits, None, None, d, out)
    assert np.abs(_n(op.topk_w).sum(axis=1) - 1).max() < 1e-5


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [0, 1])
def test_gate_of_masked_experts(score, biased, renorm):
    """-inf and the type's lowest value: a masked expert is taken only where others lack; a row
    of nothing but -inf has weights and gradients 0; NaN stays in its row, with valid ids."""
    T, E, k = 12, 24, 6
    logits, bias, _, d = _inputs(T, E, k, 6, biased and "sigmoid", False)
    inf = float("inf")
    logits[:, 5] = -inf
    logits[0] = -inf
    logits[1, 3:] = -inf             # three are left
    logits[2, 4:] = torch.finfo(torch.float32).min
    logits[3, 8:16] = -inf           # a whole group
    args = (T, E, k, 3, 2, 2, score, renorm, 1.0)
    op = _gate(*args)
    op.forward(logits.cuda(), bias=_c(bias), count=True)
    out = op.backward(d.cuda())
    torch.cuda.synchronize()
    _verify(op, logits, bias, None, d, out)
    assert not _n(op.topk_w)[0].any() and not _n(out)[0].any()
    keep = [t for t in range(T) if t not in (4, 5)]
    want = [x.clone() for x in (op.topk_idx[keep], op.topk_w[keep], out[keep])]
    logits[4, 2] = float("nan")
    logits[5] = float("nan")
    op.forward(logits.cuda(), bias=_c(bias), count=True)
    out = op.backward(d.cuda())
    idx = _n(op.topk_idx)
    assert ((idx >= 0) & (idx < E)).all() and all(len(set(r)) == k for r in idx.tolist())
    assert torch.isnan(op.topk_w[5]).all()
    for a, b in zip((op.topk_idx[keep], op.topk_w[keep], out[keep]), want):
        assert torch.equal(a, b)


def test_gate_padding_may_hold_anything():
    T, E, k = 70, 32, 4
    logits, bias, mask, d = _inputs(T, E, k, 8, "sigmoid", True)
    for score, renorm in ((0, 0), (1, 1)):
        op = _gate(T, E, k, 4, 2, 2, score, renorm, 1.0)
        op.forward(logits.cuda(), bias=bias.cuda(), mask=mask.cuda(), count=True)
        want = [x.clone() for x in (op.topk_idx, op.topk_w, op.counts, op.backward(d.cuda()))]
        bad, bd = logits.clone(), d.clone()
        bad[mask == 0], bd[mask == 0] = float("nan"), float("nan")
        op.forward(bad.cuda(), bias=bias.cuda(), mask=(mask * 200).cuda(), count=True)
        for a, b in zip((op.topk_idx, op.topk_w, op.counts, op.backward(bd.cuda())), want):
            assert torch.equal(a, b)
        op.forward(bad.cuda(), mask=torch.zeros(T, dtype=torch.uint8, device="cuda"), count=True)
        assert (op.topk_idx == -1).all() and not op.topk_w.any() and not op.counts.any() and not op.backward(bd.cuda()).any()


@pytest.mark.parametrize("score,renorm", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_gate_backward_of_ids_twice_and_outside(score, renorm):
    from combine_top_router_amd import lib as L
    T, E, k = 3, 10, 3
    logits, _, _, d = _inputs(T, E, k, 9, None, False)
    idx = torch.tensor([[4, 4, 1], [-1, 10, 2], [1 << 30, -5, -1]], dtype=torch.int32)
    out = torch.full((T, E), 7.0, device="cuda")
    lg, ic, dc = logits.cuda(), idx.cuda(), d.cuda()
    L.moe_gate_bwd(L.MoeGateShape(T, E, k, score, 1, 1, 1, renorm, 1.0), lg.data_ptr(), ic.data_ptr(), dc.data_ptr(),
                   out.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    ref = os_.gate_backward(logits.double().numpy(), idx.numpy(), d.numpy(), score, renorm)
    # (see the head) sums of three d of up to 3 in size
    assert np.abs(_n(out) - ref).max() <= (2 * _span(logits.numpy()) + 60) * 2 * U * 20
    assert not out[2].any()


def test_gate_gradient_against_differences():
    """The kernel's own weights, differenced in fp32: steps of 2^-8 leave 2^-16 of curvature
    times a third derivative of 2.5 at most, and 2^-22 of rounding over 2^-8."""
    T, E, k = 4, 12, 4
    for score in (0, 1):
        for renorm in (0, 1):
            logits, bias, _, d = _inputs(T, E, k, 10, "sigmoid", False)
            logits += 4.0 * torch.nn.functional.one_hot(torch.arange(T)[:, None] + torch.arange(k) * 2, E).sum(1)
            op = _gate(T, E, k, 1, 1, 1, score, renorm, 1.0)
            op.forward(logits.cuda(), bias=bias.cuda())
            g, idx = op.backward(d.cuda()).cpu(), op.topk_idx.clone()
            h = 2.0 ** -8
            for e in range(E):
                w = []
                for sign in (h, -h):
                    moved = logits.clone()
                    moved[:, e] += sign
                    _, out = op.forward(moved.cuda(), bias=bias.cuda())
                    assert torch.equal(op.topk_idx, idx)
                    w.append((out.double().cpu() * d).sum(1))
                assert ((w[0] - w[1]) / (2 * h) - g[:, e]).abs().max() < 3e-3, (score, renorm, e)


def test_gate_bias_step():
    from combine_top_router_amd import Gate
    for E in (1, 7, 128, 1024):
        g = torch.Generator().manual_seed(E)
        bias, counts = torch.randn(E, generator=g), torch.randint(0, 9, (E,), generator=g).to(torch.int32)
        if E == 128:
            counts[:] = 3
            counts *= 1 << 28   # sums past 32 bits
        op = Gate(4, E, 1)
        want = os_.gate_bias(bias.numpy(), counts.numpy(), 1e-3)
        b = bias.cuda()
        out = op.update_bias(b, 1e-3, counts=counts.cuda(), out=torch.empty(E, device="cuda"))
        assert np.array_equal(_n(out), want) and torch.equal(b.cpu(), bias)
        assert op.update_bias(b, 1e-3, counts=counts.cuda()) is b and np.array_equal(_n(b), want)


def test_gate_bias_evens_the_load():
    """With the bias stepped by the counts, a router that prefers some experts comes to an even load."""
    from combine_top_router_amd import Gate
    T, E, k = 4096, 16, 2
    g = torch.Generator().manual_seed(1)
    logits = (torch.randn(T, E, generator=g) + torch.linspace(-1, 1, E)).cuda()
    op, bias = Gate(T, E, k, score=1), torch.zeros(E, device="cuda")
    op.forward(logits, bias=bias, count=True)
    before = int(op.counts.max())
    for _ in range(200):
        op.forward(logits, bias=bias, count=True)
        op.update_bias(bias, 2e-3)
    op.forward(logits, bias=bias, count=True)
    assert int(op.counts.sum()) == T * k
    assert before > 2 * T * k / E > 1.2 * int(op.counts.max())


def test_gate_without_tokens():
    from combine_top_router_amd import lib as L
    s = L.MoeGateShape(0, 12, 2, 0, 1, 1, 1, 1, 1.0)
    counts = torch.ones(12, dtype=torch.int32, device="cuda")
    ws = torch.empty(L.moe_gate_scratch_bytes(s), dtype=torch.uint8, device="cuda")
    L.moe_gate_fwd(s, 0, 0, 0, 0, 0, counts.data_ptr(), ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert not counts.any()


def test_gate_refuses_other_tensors():
    from combine_top_router_amd import Gate
    op = Gate(4, 8, 2)
    lg = torch.zeros(4, 8, device="cuda")
    for bad in (lg.bfloat16(), lg[:3], lg.cpu(), torch.zeros(8, 4, device="cuda").t()):
        with pytest.raises(ValueError):
            op.forward(bad)
    for kw in (dict(bias=lg[0].double()), dict(bias=lg[0, :7]), dict(mask=torch.ones(4, device="cuda"))):
        with pytest.raises(ValueError):
            op.forward(lg, **kw)
    op.forward(lg)
    with pytest.raises(RuntimeError, match="counts"):
        op.update_bias(lg[0].clone(), 0.1)
    with pytest.raises(ValueError):
        op.backward(torch.zeros(4, 3, device="cuda"))


def test_gate_replayed():
    """Forward, backward and bias step as a graph: each replay goes on from the last bias."""
    from combine_top_router_amd import Gate
    T, E, k = 600, 64, 4
    logits, bias, mask, d = (_c(t) for t in _inputs(T, E, k, 12, "sigmoid", True))

    def step(op, b):
        op.forward(logits, bias=b, mask=mask, count=True)
        op.backward(d)
        op.update_bias(b, 0.05)

    eager, b0 = Gate(T, E, k, score=1, groups=4, topk_groups=2, group_top=2), bias.clone()
    op, b1 = Gate(T, E, k, score=1, groups=4, topk_groups=2, group_top=2), bias.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(op, b1)
    for _ in range(4):
        op.counts.fill_(-1)
        op.d_logits.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        step(eager, b0)
        torch.cuda.synchronize()
        for a, b in ((b0, b1), (eager.counts, op.counts), (eager.topk_idx, op.topk_idx), (eager.topk_w, op.topk_w),
                     (eager.d_logits, op.d_logits)):
            assert torch.equal(a, b)
