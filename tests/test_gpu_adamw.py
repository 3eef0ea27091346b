"""The AdamW step against the fp64 oracle, element by element.

Bounds, u = 2^-24: m = b1 m + (1 - b1) g and v likewise are two products and a sum of fp32
factors that are rounded themselves: 4 u of the sizes of the two terms (g^2, g times a scale:
2 u more each).  sqrt, its product, the sum with eps, the quotient and the rate are a rounding
each, and half of v's error: 10 u of the update, plus m's error through it.  8 bits: a code has to
be the oracle's for some value within m's (or sqrt v's) bound; all of the grid's steps are
monotone in it, so it lies between the codes of the bound's two ends.  Below 2^-126 fp32's
numbers lie 2^-149 apart: m and v have that much more (TINY, a few roundings), and a root of v the
root of it."""
import numpy as np
import pytest
import torch

from oracle import step as os_

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -147
HYPER = dict(lr=1e-2, b1=0.9, b2=0.95, eps=1e-8, wd=0.1)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _op(params, state="f32", **kw):
    from combine_top_router_amd import AdamW, lib as L
    h = HYPER
    return AdamW(params, state=L.MOE_STATE_8BIT if state == "8bit" else L.MOE_STATE_F32, betas=(h["b1"], h["b2"]),
                 eps=h["eps"], weight_decay=h["wd"], **kw)


def _tensors(sizes, dtypes, seed, scale=0.1):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale).to(DT[d]).cuda() for s, d in zip(sizes, dtypes)]


def _f(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def _hold(op, i, value, size, bound, r16, keep, codes, scales):
    """Tensor i's codes against the oracle's |value| +- bound."""
    n = value.size
    X = scales.astype(np.int64) - 127
    a = np.zeros(-(-n // 32) * 32)
    d = a.copy()
    a[:n], d[:n] = np.abs(value), bound
    blocks, room = a.reshape(-1, 32), d.reshape(-1, 32)
    for b in range(len(blocks)):
        lo = os_.scale_exponent(float((blocks[b] - room[b]).max()))
        hi = os_.scale_exponent(float((blocks[b] + room[b]).max()))
        assert X[b] in (lo, hi) or blocks[b].max() <= room[b].max(), (i, b, X[b], lo, hi)
    s = np.exp2(np.repeat(X, 32)[:n].astype(np.float64))
    got = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert not got[n:].any()
    got = got[:n] * s
    # ends past 448 (the exponent may be the lower of two) stay at it
    raw = [np.clip((a[:n] + sign * d[:n]) / s, 0, 448) for sign in (-1, 1)]
    ends = [os_.e4m3_grid(y, r16) * s for y in raw]
    if keep:
        ends = [np.where((y > 0) & (e == 0), 2.0 ** -9 * s, e) for y, e in zip(raw, ends)]
    ok = (np.abs(got) >= ends[0]) & (np.abs(got) <= ends[1])
    assert ok.all(), (i, np.flatnonzero(~ok)[:3], got[~ok][:3], ends[0][~ok][:3], ends[1][~ok][:3])
    assert (np.sign(got) * np.sign(value) >= 0).all() or (np.abs(value)[np.sign(got) * np.sign(value) < 0] <= d[:n][np.sign(got) * np.sign(value) < 0]).all()
    return got


def _verify(op, grads, before, grad_scale=1.0, lr=HYPER["lr"]):
    """`before`: (params, masters, moments) as fp64 arrays, of the step that op has just made."""
    h, t = HYPER, op.t
    torch.cuda.synchronize()
    stochastic, seed = bool(op.hyper.stochastic), int(op.hyper.seed)
    for i, g in enumerate(grads):
        p, master, (m, v) = before[0][i], before[1][i], before[2][i]
        now = op.params[i]
        if g is None:
            assert np.array_equal(_f(now), p)
            continue
        base = p if master is None else master
        gn = _f(g) * grad_scale
        q, m1, v1 = os_.adamw(base, _f(g), m, v, t, lr, h["b1"], h["b2"], h["eps"], h["wd"], grad_scale)
        dm = 6 * U * (np.abs(h["b1"] * m) + np.abs((1 - h["b1"]) * gn)) + TINY
        dv = 8 * U * v1 + TINY
        with np.errstate(divide="ignore", invalid="ignore"):
            step = lr * np.abs(m1) / (1 - h["b1"] ** t) / (np.sqrt(v1 / (1 - h["b2"] ** t)) + h["eps"])
            more = np.where(np.abs(m1) > 0, step / np.abs(m1) * dm, 0.0)
        dp = 4 * U * np.abs(base) + 16 * U * step + more + 1e-45
        r = os_.random_bits(seed, t, op._at[i] + np.arange(p.size)) if stochastic else None
        if op.master is not None and op.master[i] is not None:
            assert (np.abs(_f(op.master[i]) - q) <= dp).all()
            assert torch.equal(now, op.master[i].to(now.dtype))
        elif now.dtype == torch.float32:
            assert (np.abs(_f(now) - q) <= dp).all(), (i, np.abs(_f(now) - q).max())
        else:
            got = _f(now)
            lo, hi = (q - dp).astype(np.float32), (q + dp).astype(np.float32)
            if stochastic:
                ends = [os_.bf16_stochastic(e, os_.mix(r) & np.uint64(0xFFFF)).astype(np.float64) for e in (lo, hi)]
            else:
                ends = [torch.from_numpy(e).bfloat16().double().numpy() for e in (lo, hi)]
            low, high = np.minimum(*ends), np.maximum(*ends)
            assert ((got >= low) & (got <= high)).all(), (i, t)
        if op._eight:
            at, n = op._at[i], -(-p.size // 32) * 32
            part = lambda x, w: x[at // w:(at + n) // w].cpu().numpy()  # noqa: E731
            _hold(op, i, m1, m1, dm, None if r is None else r & np.uint64(0xFFFF), False, part(op.m, 1), part(op.m_scale, 32))
            _hold(op, i, np.sqrt(v1), v1, 6 * U * np.sqrt(v1) + TINY ** 0.5, None if r is None else r >> np.uint64(16), True, part(op.v, 1),
                  part(op.v_scale, 32))
        else:
            gm, gv = (_f(x) for x in op.moments(i))
            assert (np.abs(gm - m1) <= dm).all() and (np.abs(gv - v1) <= dv).all()


def _before(op):
    torch.cuda.synchronize()
    return ([_f(p) for p in op.params],
            [None if op.master is None or op.master[i] is None else _f(op.master[i]) for i in range(len(op.params))],
            [tuple(_f(x) for x in op.moments(i)) for i in range(len(op.params))])


SIZES = [1, 2, 7, 8, 31, 32, 33, 255, 0, 2048, 2049, 4095, 10001]


@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("dtype,g_dtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_adamw_against_the_oracle(dtype, g_dtype, state, master, stochastic):
    params = _tensors(SIZES, [dtype] * len(SIZES), 1)
    op = _op(params, state, master=master, stochastic=stochastic, seed=77 + (3 << 33))
    for t in range(1, 4):
        grads = _tensors(SIZES, [g_dtype] * len(SIZES), 10 + t, 1e-3)
        before = _before(op)
        op.step(grads, HYPER["lr"])
        assert op.t == t
        _verify(op, grads, before)


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_adamw_of_many_mixed_tensors(state):
    """More tensors than a launch takes, of mixed types, some without a gradient."""
    n = 131
    sizes = [1 + (i * 37) % 300 for i in range(n)]
    params = _tensors(sizes, ["f32" if i % 3 else "bf16" for i in range(n)], 2)
    op = _op(params, state, master=True)
    for t in range(2):
        grads = _tensors(sizes, ["bf16" if i % 2 else "f32" for i in range(n)], 20 + t, 1e-2)
        grads = [None if i % 11 == t else g for i, g in enumerate(grads)]
        before = _before(op)
        op.step(grads, HYPER["lr"])
        _verify(op, grads, before)


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_adamw_of_views(state):
    """Parameters and gradients that start at any element: their neighbours stay as they are."""
    buf, gbuf = torch.randn(4000).bfloat16().cuda(), (torch.randn(4000) * 1e-3).bfloat16().cuda()
    cuts = [(1, 700), (703, 704), (705, 1505), (1508, 3999)]
    params = [buf[a:b] for a, b in cuts]
    op = _op(params, state, stochastic=True, seed=5)
    before, whole = _before(op), buf.clone()
    grads = [gbuf[a:b] for a, b in cuts]
    op.step(grads, HYPER["lr"])
    _verify(op, grads, before)
    inside = torch.zeros(4000, dtype=torch.bool)
    for a, b in cuts:
        inside[a:b] = True
    assert torch.equal(buf.cpu()[~inside], whole.cpu()[~inside])


def test_adamw_large_places():
    """Random bits of elements past 2^32 of the numbering, through the C call's `at`."""
    from combine_top_router_amd import lib as L
    n, at = 5000, (1 << 32) - 2400
    p, g = _tensors([n, n], ["bf16", "f32"], 3)
    m, v = (torch.zeros(n, device="cuda") for _ in range(2))
    prm = L.MoeAdamwParams(1e-2, 0.9, 0.95, 1e-8, 0.0, 9, 1 << 40, L.MOE_STATE_F32, 1)
    tab = (L.MoeAdamwTensor * 1)(L.MoeAdamwTensor(p.data_ptr(), g.data_ptr(), 0, m.data_ptr(), v.data_ptr(), 0, 0, n, at,
                                                  L.MOE_BF16, L.MOE_F32))
    old = _f(p)
    L.moe_adamw(prm, tab, 1, 0, 0, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    q, _, _ = os_.adamw(old, _f(g), np.zeros(n), np.zeros(n), 9, 1e-2, 0.9, 0.95, 1e-8, 0.0)
    r = os_.mix(os_.random_bits(1 << 40, 9, at + np.arange(n))) & np.uint64(0xFFFF)
    d = 4 * U * np.abs(old) + 20 * U * np.abs(q - old)
    ends = [os_.bf16_stochastic((q + s * d).astype(np.float32), r).astype(np.float64) for s in (-1, 1)]
    got = _f(p)
    assert ((got >= np.minimum(*ends)) & (got <= np.maximum(*ends))).all()


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_adamw_grad_scale_and_device_rate(state):
    sizes = [100, 2000]
    a, b = (_op(_tensors(sizes, ["f32", "bf16"], 4), state, master=True) for _ in range(2))
    rate, scale = torch.tensor([3e-3], device="cuda"), torch.tensor([0.25], device="cuda")
    for t in range(2):
        grads = _tensors(sizes, ["bf16", "f32"], 40 + t)
        before = _before(a)
        a.step(grads, rate, grad_scale=scale)
        _verify(a, grads, before, 0.25, float(rate))
        # the powers of two of the scale leave nothing to round
        b.step([g * 0.25 for g in grads], rate)
        for x, y in zip(a.params, b.params):
            assert torch.equal(x, y)


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_adamw_replayed(state):
    """A captured step goes on counting: four replays are four eager steps."""
    sizes = [33, 4096, 999]
    grads = _tensors(sizes, ["bf16"] * 3, 50, 1e-2)
    kw = dict(stochastic=True, seed=9)
    eager = _op(_tensors(sizes, ["bf16"] * 3, 5), state, **kw)
    op = _op(_tensors(sizes, ["bf16"] * 3, 5), state, capturable=True, **kw)
    rate = torch.full((1,), 1e-2, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.step(grads, rate)
    assert op.t == 0
    for t in range(1, 5):
        rate.fill_(1e-2 / t)
        graph.replay()
        torch.cuda.synchronize()
        junk = torch.ones(1 << 16, device="cuda").sum()   # other work between
        before = _before(eager)
        eager.step(grads, rate)
        _verify(eager, grads, before, lr=float(rate))
        assert op.t == t and float(junk) == 1 << 16
        for i in range(3):
            # the factors of step t are rounded alike, pow of the device and of the host to 2^-50
            assert torch.equal(op.params[i], eager.params[i])
            assert all(torch.equal(x, y) for x, y in zip(op.moments(i), eager.moments(i)))
    op.t = 100
    assert op.t == 100


@pytest.mark.parametrize("stochastic", [False, True])
def test_adamw_8bit_extremes(stochastic):
    """Blocks of zeros, of one tiny value beside large ones, of the smallest and largest numbers."""
    n = 32 * 6
    g = torch.zeros(n)
    g[32:64] = torch.logspace(-12, 3, 32)
    g[64:96] = 1e-38
    g[96] = 1e18
    g[97:128] = 1e-3
    g[128:160] = torch.tensor([448.0, 449.0, 416.0, 1.0] * 8)
    op = _op([torch.ones(n, device="cuda")], "8bit", stochastic=stochastic, seed=1)
    g = g.cuda()
    for _ in range(3):
        before = _before(op)
        op.step([g], HYPER["lr"])
        _verify(op, [g], before)
    v = op.moments(0)[1].cpu()
    assert (v[32:128][g.cpu()[32:128] > 1e-6] > 0).all()   # what is above 0 stays
    assert not v[:32].any()
    assert torch.isfinite(op.params[0]).all()


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_adamw_what_is_not_finite_stays_where_it_is(state):
    n = 200
    a, b = (_op(_tensors([n], ["f32"], 6), state) for _ in range(2))
    g = _tensors([n], ["f32"], 60)[0]
    bad = g.clone()
    bad[3], bad[70], bad[71] = float("nan"), float("inf"), -float("inf")
    others = torch.ones(n, dtype=torch.bool)
    others[[3, 70, 71]] = False
    h = g.clone()
    h[[3, 70, 71]] = 0   # what the scales of the others' blocks go by
    for _ in range(2):
        a.step([bad], 1e-2)
        b.step([h], 1e-2)
    o = others.cuda()
    for x, y in zip((a.params[0], *a.moments(0)), (b.params[0], *b.moments(0))):
        assert torch.equal(x[o], y[o])
    assert not torch.isfinite(a.params[0][~o]).any()


def test_adamw_8bit_moves_on():
    """A second moment that decays by less than half a code each step reaches its goal when rounded
    stochastically."""
    n = 1 << 14
    op = _op([torch.zeros(n, device="cuda")], "8bit", stochastic=True, seed=3)
    big, small = torch.full((n,), 1.0, device="cuda"), torch.full((n,), 0.5, device="cuda")
    for _ in range(60):
        op.step([big], 0.0)
    for _ in range(120):
        op.step([small], 0.0)
    v = op.moments(0)[1].double().mean()
    # 0.25 + 0.75 0.95^120 = 0.2516; each step adds the rounding's spread, at most (1/16 / 2)^2 of
    # v a step in the mean of squares, which the decay of 1/20 a step holds below 20 times that
    assert 0.2516 * 0.98 < float(v) < 0.2516 * (1 + 20 / 1024)


def test_adamw_on_another_stream():
    sizes = [5000, 77]
    a, b = (_op(_tensors(sizes, ["bf16"] * 2, 7), "8bit") for _ in range(2))
    grads, side = _tensors(sizes, ["bf16"] * 2, 70, 1e-2), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        a.step(grads, 1e-2)
        b.step(grads, 1e-2, stream=side)
    torch.cuda.synchronize()
    for x, y in zip(a.params + [a.m, a.v], b.params + [b.m, b.v]):
        assert torch.equal(x, y)


def test_adamw_refuses_other_tensors():
    op = _op(_tensors([16], ["f32"], 8))
    g = torch.zeros(16, device="cuda")
    for bad in (g[:15], g.half(), g.cpu(), torch.zeros(32, device="cuda")[::2], g.view(4, 4)):
        with pytest.raises(ValueError, match=r"grads\[0\]"):
            op.step([bad], 0.1)
    with pytest.raises(ValueError, match="lr"):
        op.step([g], torch.zeros(1))
    with pytest.raises(ValueError, match="grad_scale"):
        op.step([g], 0.1, grad_scale=torch.ones(2, device="cuda"))
    op.params[0].data = torch.zeros(16, device="cuda")
    with pytest.raises(ValueError, match="other memory"):
        op.step([g], 0.1)
    assert op.t == 0


def test_adamw_captured_needs_its_clock():
    """A step number from the host would be the same at every replay."""
    from combine_top_router_amd import AdamW
    p = torch.zeros(64, device="cuda")
    op = AdamW([p])
    x = torch.ones(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.mul_(2.0)
        with pytest.raises(RuntimeError, match="capturable"):
            op.step([p], 0.1)
    graph.replay()
    torch.cuda.synchronize()
    assert op.t == 0 and not p.any() and (x == 2.0).all()


def test_adamw_of_few_bits_goes_by_the_formula_in_fp32():
    """Gradients of few bits put 0.9 m + 0.1 g halfway between two codes in fp32, each product and the sum
    rounded: the codes are those of that number, to the bit (a fused product would move it off)."""
    from combine_top_router_amd import AdamW, lib as L
    g = torch.Generator().manual_seed(6)
    n = 32 * 4096
    p = torch.zeros(n, device="cuda")
    op = AdamW([p], state=L.MOE_STATE_8BIT)
    m = torch.zeros(n)
    b, c = torch.tensor(0.9), torch.tensor(1.0 - 0.9)
    for _ in range(4):
        grad = (torch.randint(-64, 65, (n,), generator=g) / 16.0).bfloat16()
        op.step([grad.cuda()], 1e-3)
        m = b * m + c * grad.float()
        blocks = m.view(-1, 32)
        mant, e = torch.frexp(blocks.abs().amax(1))
        e = e - 9 + (mant > 0.875).to(e.dtype)
        codes = torch.ldexp(blocks, -e[:, None]).to(torch.float8_e4m3fn)
        assert torch.equal(op.m.cpu(), codes.view(torch.uint8).view(-1))
        assert torch.equal(op.m_scale.cpu(), (e + 127).to(torch.uint8))
        m = torch.ldexp(codes.float(), e[:, None]).view(-1)
