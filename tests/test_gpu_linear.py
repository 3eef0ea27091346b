"""The matrix product with bias, activation and residual, and its backward, against the fp64
oracle, element by element.

Bounds, u = 2^-24, h = half a step of the type (bf16 2^-8, fp32 2^-24): a sum of K products has an
error of (K + 8) u S, S the sum of their sizes; an activation's slope is at most 1.13 and its own
evaluation, from exp and erf of an argument z, is good to (|z| + 8) u z and 4 u (two hardware
functions of 1 to 2 ulp, and the argument's rounding); y is rounded once.  The backward
reads z with h and keeps dz with h: z h times the slope's own slope (at most 0.8), and dz h, enter
the products as errors of dz.  At relu's corner the sign of z is that of its rounding: where z is
within its error dz may be off by all of dy."""
import math

import numpy as np
import pytest
import torch

from oracle import step as os_

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ["none", "relu", "silu", "gelu"]


def _op(T, K, N, act, dtype, **kw):
    from combine_top_router_amd import Linear, lib as L
    code = {"f32": L.MOE_F32, "bf16": L.MOE_BF16}[dtype]
    return Linear(T, K, N, act=ACTS.index(act), dtype=code, **kw)


def _inputs(T, K, N, dtype, seed, bias=True, res=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = DT[dtype]
    x, w = rnd(T, K).to(dt), (rnd(K, N) / K ** 0.5).to(dt)
    b = (0.3 * rnd(N)).to(dt) if bias else None
    r = rnd(T, N).to(dt) if res else None
    return x.cuda(), w.cuda(), None if b is None else b.cuda(), None if r is None else r.cuda(), rnd(T, N).to(dt).cuda()


def _f(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _near(got, want, bound):
    bad = ~(np.abs(_f(got) - want) <= bound + 1e-40)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), _f(got)[bad][:3], want[bad][:3], bound[bad][:3])


def _forward_bound(x, w, b, res, act, dtype):
    K = x.shape[1]
    y, z = os_.linear_forward(x, w, b, res, act)
    dz = (K + 8) * U * (np.abs(x) @ np.abs(w) + (0 if b is None else np.abs(b)))
    err = 1.13 * dz
    if act in ("silu", "gelu"):
        err = err + (np.abs(z) + 8) * U * np.abs(z) + 4 * U
    return y, z, dz, HALF[dtype] * np.abs(y) + (1 + HALF[dtype]) * err + 2 * U * np.abs(y)


def _verify(op, t, out, grads=None, dx_in=None):
    x, w, b, res, dy = (_f(v) for v in t)
    dtype = "bf16" if op.dtype == torch.bfloat16 else "f32"
    act = ACTS[op.shape.act]
    y, z, dzerr, bound = _forward_bound(x, w, b, res, act, dtype)
    _near(out, y, bound)
    if grads is None:
        return
    T, K, N, h = *x.shape, w.shape[1], HALF[dtype]
    dx, dw, db, dz = os_.linear_backward(dy, x, w, z, _f(dx_in), act)
    if act == "none":
        e = np.zeros_like(dz)
        held = e
    else:
        e = np.abs(dy) * (0.8 * (h * np.abs(z) + (1 + h) * dzerr) + (np.abs(z) + 12) * U) if act != "relu" else np.where(
            np.abs(z) <= dzerr, np.abs(dy), 0.0) + 2 * U * np.abs(dz)
        held = h * (np.abs(dz) + e)
    a = np.abs(dz) + e + held
    size = np.abs(dx)
    _near(grads["dx"], dx, h * size + (1 + h) * ((e + held) @ np.abs(w).T + (N + 8) * U * (a @ np.abs(w).T)
                                              + (0 if dx_in is None else 2 * U * np.abs(_f(dx_in)))))
    _near(grads["dw"], dw, h * np.abs(dw) + (1 + h) * (np.abs(x).T @ (e + held) + (T + 8) * U * (np.abs(x).T @ a)))
    if b is not None:
        _near(grads["db"], db, h * np.abs(db) + (1 + h) * (e.sum(axis=0) + (T + 8) * U * a.sum(axis=0)))
    else:
        assert grads["db"] is None


# T, K, N: single rows and columns, tiles and their edges, sizes that no wide load divides, long sums
SIZES = [(1, 1, 1), (1, 64, 64), (1, 2048, 768), (2, 8, 1000), (3, 100, 7), (16, 512, 256), (17, 520, 264), (33, 72, 40),
         (64, 64, 64), (65, 63, 129), (127, 256, 384), (128, 128, 128), (129, 192, 136), (250, 333, 77), (256, 512, 256),
         (300, 1000, 520), (513, 264, 1032), (1000, 8, 8), (1030, 96, 200), (40, 4096, 64), (2500, 64, 128),
         (1024, 1024, 512)]


@pytest.mark.parametrize("act,bias,res", [("none", True, True), ("relu", True, False), ("silu", False, True),
                                          ("gelu", True, True), ("none", False, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_linear_against_the_oracle(size, dtype, act, bias, res):
    T, K, N = size
    t = _inputs(T, K, N, dtype, T + K + N, bias, res)
    x, w, b, r, dy = t
    op = _op(T, K, N, act, dtype)
    y = op.forward(x, w, b, res=r)
    grads = op.backward(dy)
    torch.cuda.synchronize()
    _verify(op, t, y, grads)
    first = [v.clone() for v in (y, *[g for g in grads.values() if g is not None])]
    op.forward(x, w, b, res=r)   # the same again, bit for bit
    again = op.backward(dy)
    for a, c in zip(first, (op.y, *[g for g in again.values() if g is not None])):
        assert torch.equal(a, c)
    dx_in = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).to(x.dtype).cuda()
    grads = op.backward(dy, dx_in=dx_in)
    torch.cuda.synchronize()
    _verify(op, t, y, grads, dx_in)
    infer = _op(T, K, N, act, dtype, train=False)
    assert torch.equal(infer.forward(x, w, b, res=r), y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(5, 64, 128), (130, 256, 264), (300, 77, 130), (512, 512, 512)])
def test_linear_in_place(size, dtype):
    """y in the place of res, and dx in that of dx_in, through the C calls; dx not wanted."""
    from combine_top_router_amd import lib as L
    T, K, N = size
    x, w, b, r, dy = _inputs(T, K, N, dtype, 3)
    op = _op(T, K, N, "silu", dtype)
    want = op.forward(x, w, b, res=r).clone()
    dx_in = torch.randn(T, K, generator=torch.Generator().manual_seed(2)).to(x.dtype).cuda()
    g = {n: v.clone() for n, v in op.backward(dy, dx_in=dx_in).items()}
    st, buf, dx = torch.cuda.current_stream().cuda_stream, r.clone(), dx_in.clone()
    L.moe_linear_fwd(op.shape, x.data_ptr(), w.data_ptr(), b.data_ptr(), buf.data_ptr(), 0, buf.data_ptr(),
                     op.scratch.data_ptr(), st)
    L.moe_linear_bwd(op.shape, dy.data_ptr(), x.data_ptr(), w.data_ptr(), op.z.data_ptr(), dx.data_ptr(), dx.data_ptr(),
                     op.dw.data_ptr(), op.db.data_ptr(), op.scratch.data_ptr(), st)
    torch.cuda.synchronize()
    assert torch.equal(buf, want) and torch.equal(dx, g["dx"])
    op.dw.fill_(7)
    L.moe_linear_bwd(op.shape, dy.data_ptr(), x.data_ptr(), w.data_ptr(), op.z.data_ptr(), 0, 0, op.dw.data_ptr(), 0,
                     op.scratch.data_ptr(), st)
    torch.cuda.synchronize()
    assert torch.equal(op.dw, g["dw"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off", [1, 3, 4])
def test_linear_of_views(dtype, off):
    """Matrices that start anywhere in their memory (no 16-byte address): nothing around them is
    read into the result or written."""
    T, K, N = 70, 128, 72
    t = _inputs(T, K, N, dtype, 4)

    def moved(v):
        if v is None:
            return None
        buf = torch.full((v.numel() + 16,), float("nan"), dtype=v.dtype, device="cuda")
        buf[off:off + v.numel()] = v.reshape(-1)
        return buf[off:off + v.numel()].view(v.shape)

    x, w, b, r, dy = (moved(v) for v in t)
    op = _op(T, K, N, "gelu", dtype)
    y = op.forward(x, w, b, res=r)
    grads = op.backward(dy, dx_in=moved(torch.zeros(T, K, dtype=x.dtype, device="cuda")))
    torch.cuda.synchronize()
    _verify(op, t, y, grads)
    from combine_top_router_amd import lib as L
    bufs = {n: torch.full((s + 16,), 7.0, dtype=x.dtype, device="cuda") for n, s in
            (("y", T * N), ("dx", T * K), ("dw", K * N), ("db", N))}
    at = {n: v[off:].data_ptr() for n, v in bufs.items()}
    st = torch.cuda.current_stream().cuda_stream
    L.moe_linear_fwd(op.shape, x.data_ptr(), w.data_ptr(), b.data_ptr(), r.data_ptr(), op.z.data_ptr(), at["y"],
                     op.scratch.data_ptr(), st)
    L.moe_linear_bwd(op.shape, dy.data_ptr(), x.data_ptr(), w.data_ptr(), op.z.data_ptr(), 0, at["dx"], at["dw"], at["db"],
                     op.scratch.data_ptr(), st)
    torch.cuda.synchronize()
    for n, want in (("y", y), ("dx", grads["dx"]), ("dw", grads["dw"]), ("db", grads["db"])):
        v = bufs[n]
        assert (v[:off] == 7).all() and (v[off + want.numel():] == 7).all(), n
    _verify(op, t, bufs["y"][off:off + T * N].view(T, N),
            {n: bufs[n][off:off + v.numel()].view(v.shape) for n, v in grads.items()})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_keeps_nan_in_its_row_and_column(dtype):
    T, K, N = 200, 256, 264
    x, w, b, r, dy = _inputs(T, K, N, dtype, 5)
    op = _op(T, K, N, "relu", dtype)
    want = op.forward(x, w, b, res=r).clone()
    g = {n: v.clone() for n, v in op.backward(dy).items()}
    x2 = x.clone()
    x2[77, 5] = float("nan")
    y = op.forward(x2, w, b, res=r)
    keep = torch.arange(T) != 77
    assert torch.equal(y[keep.cuda()], want[keep.cuda()]) and torch.isnan(y[77]).all()
    got = op.backward(dy)
    assert torch.equal(got["dx"][keep.cuda()], g["dx"][keep.cuda()]) and torch.isnan(got["dw"]).any()
    dy2 = dy.clone()
    dy2[:, 9] = float("inf")
    op.forward(x, w, b, res=r)
    got = op.backward(dy2)
    cols = torch.arange(N) != 9
    assert torch.equal(got["dw"][:, cols.cuda()], g["dw"][:, cols.cuda()])
    assert torch.equal(got["db"][cols.cuda()], g["db"][cols.cuda()])


def test_linear_of_masked_activations():
    """Far out on the activations: large negative and positive z, infinities in the residual."""
    T, K, N = 8, 64, 64
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.tensor([-3e38, -1e5, -90.0, -20.0, 20.0, 90.0, 1e5, 3e38])
    w = torch.zeros(K, N, dtype=torch.bfloat16, device="cuda")
    w[0] = 1.0
    for act in ACTS:
        y = _op(T, K, N, act, "bf16").forward(x, w).float().cpu()
        z = x[:, :1].float().cpu().expand(T, N)
        if act == "none":
            assert torch.equal(y, z)
        else:
            assert torch.equal(y[4:], z[4:].clone()) and (y[:3].abs() < 1e-30).all() and (y[3].abs() < 1e-6).all()
    res = torch.full((T, N), -float("inf"), dtype=torch.bfloat16, device="cuda")
    assert (_op(T, K, N, "silu", "bf16").forward(x, w, res=res) == -float("inf")).all()


def test_linear_without_rows():
    from combine_top_router_amd import lib as L
    for dtype, dt in ((L.MOE_BF16, torch.bfloat16), (L.MOE_F32, torch.float32)):
        for K, N in ((64, 128), (33, 7)):
            s = L.MoeLinearShape(0, K, N, dtype, L.MOE_ACT_GELU)
            dw, db = torch.ones(K, N, dtype=dt, device="cuda"), torch.ones(N, dtype=dt, device="cuda")
            ws = torch.empty(L.moe_linear_scratch_bytes(s), dtype=torch.uint8, device="cuda")
            L.moe_linear_bwd(s, 0, 0, 0, 0, 0, 0, dw.data_ptr(), db.data_ptr(), ws.data_ptr(),
                             torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert not dw.any() and not db.any()


def test_linear_gradient_against_differences():
    """The kernel's own fp32 outputs, differenced: steps of 2^-6 leave 2^-12 of curvature / 6 times
    a third derivative below 2, and 2^-21 of rounding over 2^-6, summed over 24 outputs."""
    T, K, N = 3, 6, 8
    for act in ("silu", "gelu", "none"):
        x, w, b, r, dy = _inputs(T, K, N, "f32", 7)
        op = _op(T, K, N, act, "f32")
        op.forward(x, w, b, res=r)
        g = {n: v.double().cpu() for n, v in op.backward(dy).items()}
        loss = lambda *a: float((op.forward(*a, res=r).double() * dy.double()).sum())  # noqa: E731
        h = 2.0 ** -6
        for which, name in ((0, "dx"), (1, "dw"), (2, "db")):
            for i in np.ndindex(tuple(g[name].shape)):
                ends = []
                for s in (h, -h):
                    a = [x.clone(), w.clone(), b.clone()]
                    a[which][i] += s
                    ends.append(loss(*a))
                assert abs((ends[0] - ends[1]) / (2 * h) - float(g[name][i])) < 5e-3, (act, name, i)


def test_linear_replayed_and_shared():
    """Two products as graphs that run in turn with the program's own work between."""
    t = _inputs(300, 256, 512, "bf16", 8)
    x, w, b, r, dy = t
    ops = [_op(300, 256, 512, "silu", "bf16") for _ in range(2)]
    want = []
    y = ops[0].forward(x, w, b, res=r)
    want = [v.clone() for v in (y, *ops[0].backward(dy).values())]
    torch.cuda.synchronize()
    graphs = []
    for op in ops:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op.forward(x, w, b, res=r)
            op.backward(dy)
        graphs.append(graph)
    for _ in range(3):
        for op, graph in zip(ops, graphs):
            for v in (op.y, op.dx, op.dw, op.db):
                v.fill_(3)
            op.scratch.fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            for a, c in zip((op.y, op.dx, op.dw, op.db), want):
                assert torch.equal(a, c)


def test_linear_on_another_stream():
    t = _inputs(700, 512, 256, "bf16", 9)
    x, w, b, r, dy = t
    a, c, side = _op(700, 512, 256, "gelu", "bf16"), _op(700, 512, 256, "gelu", "bf16"), torch.cuda.Stream()
    want = [a.forward(x, w, b, res=r).clone()] + [v.clone() for v in a.backward(dy).values()]
    side.wait_stream(torch.cuda.current_stream())
    y = c.forward(x, w, b, res=r, stream=side)
    g = c.backward(dy, stream=side)
    torch.cuda.synchronize()
    for p, q in zip((y, *g.values()), want):
        assert torch.equal(p, q)


def test_linear_refuses_other_tensors():
    op = _op(8, 64, 32, "none", "bf16")
    x, w, b, r, dy = _inputs(8, 64, 32, "bf16", 10)
    for a in ((x.float(), w), (x[:7], w), (x, w.t()), (x, w.t().contiguous()), (x.cpu(), w), (x, w, b[:31]),
              (x, w.t().contiguous().t())):
        with pytest.raises(ValueError):
            op.forward(*a)
    with pytest.raises(ValueError):
        op.forward(x, w, res=r[:, :31])
    op.forward(x, w)
    for kw in (dict(dy=dy.float()), dict(dy=dy[:7]), dict(dy=dy, dx_in=dy)):
        with pytest.raises(ValueError):
            op.backward(**kw)


@pytest.mark.parametrize("T", [2, 193])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gelu_far_out(dtype, T):
    """gelu and its slope relative to their own values, down the negative side: z itself is exact (one product
    with 1, of multiples of 1/16 below 2^8 of them).  The value is good to 1.1e-5 (the polynomial's fit), z^2 u
    (the exponent's two roundings, times it) and 16 u (reciprocal, exponential, eight steps); the slope is
    Q + z phi, each of them so.  Roundings to the type: y once, dx twice."""
    z = torch.arange(-192, 1).double()[:T] / 16 if T > 4 else torch.tensor([-9.0, -5.5]).double()
    x, w = torch.zeros(T, 8, dtype=DT[dtype], device="cuda"), torch.zeros(8, 8, dtype=DT[dtype], device="cuda")
    x[:, 0], w[0, 0] = z.to(DT[dtype]).cuda(), 1.0
    dy = torch.zeros(T, 8, dtype=DT[dtype], device="cuda")
    dy[:, 0] = 1.0
    op = _op(T, 8, 8, "gelu", dtype)
    y = _f(op.forward(x, w))[:, 0]
    dx = _f(op.backward(dy)["dx"])[:, 0]
    z = z.numpy()
    q = 0.5 * np.array([math.erfc(-v / math.sqrt(2.0)) for v in z])
    phi = z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    rel = 1.1e-5 + (z * z + 16) * U
    assert (np.abs(y - z * q) <= (rel * (1 + HALF[dtype]) + HALF[dtype]) * np.abs(z * q)).all()
    err = rel * (q + np.abs(phi))
    assert (np.abs(dx - (q + phi)) <= 2.1 * HALF[dtype] * np.abs(q + phi) + (1 + HALF[dtype]) ** 2 * err).all()


# widths that no 16 bytes divide, large enough for the copies with padded rows, of one operand or of both;
# 8185 rows: the general kernel's larger tiles; one and three rows of 7, 8 and 9 columns
ODD = [(300, 777, 1555), (1000, 1001, 520), (1000, 520, 1001), (4100, 1001, 100), (8185, 261, 1021), (1, 300, 9), (3, 70, 7),
       (3, 4100, 17), (4, 1, 8)]


@pytest.mark.parametrize("act,bias,res", [("none", False, False), ("silu", True, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", ODD, ids=lambda s: "x".join(map(str, s)))
def test_linear_of_odd_widths(size, dtype, act, bias, res):
    T, K, N = size
    t = _inputs(T, K, N, dtype, T + K, bias, res)
    x, w, b, r, dy = t
    op = _op(T, K, N, act, dtype)
    op.scratch.fill_(0xFF)   # NaN wherever it is read before it is written
    y = op.forward(x, w, b, res=r)
    op.scratch.fill_(0xFF)
    dx_in = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).to(x.dtype).cuda()
    grads = op.backward(dy, dx_in=dx_in)
    torch.cuda.synchronize()
    _verify(op, t, y, grads, dx_in)


@pytest.mark.parametrize("size", [(300, 777, 1555), (1000, 1001, 520), (1000, 520, 1001)])
@pytest.mark.parametrize("off", [1, 8])
def test_linear_of_odd_widths_anywhere(size, off):
    """The same from any address, and nothing around the results is written."""
    from combine_top_router_amd import lib as L
    T, K, N = size
    t = _inputs(T, K, N, "bf16", 4)

    def moved(v):
        buf = torch.full((v.numel() + 16,), float("nan"), dtype=v.dtype, device="cuda")
        buf[off:off + v.numel()] = v.reshape(-1)
        return buf[off:off + v.numel()].view(v.shape)

    x, w, b, r, dy = t = tuple(moved(v) for v in t)
    op = _op(T, K, N, "silu", "bf16")
    bufs = {n: torch.full((s + 16,), 7.0, dtype=x.dtype, device="cuda") for n, s in
            (("y", T * N), ("z", T * N), ("dx", T * K), ("dw", K * N), ("db", N))}
    at = {n: v[off:].data_ptr() for n, v in bufs.items()}
    st = torch.cuda.current_stream().cuda_stream
    L.moe_linear_fwd(op.shape, x.data_ptr(), w.data_ptr(), b.data_ptr(), r.data_ptr(), at["z"], at["y"],
                     op.scratch.data_ptr(), st)
    L.moe_linear_bwd(op.shape, dy.data_ptr(), x.data_ptr(), w.data_ptr(), at["z"], 0, at["dx"], at["dw"], at["db"],
                     op.scratch.data_ptr(), st)
    torch.cuda.synchronize()
    size_of = {"y": (T, N), "z": (T, N), "dx": (T, K), "dw": (K, N), "db": (N,)}
    for n, s in size_of.items():
        assert (bufs[n][:off] == 7).all() and (bufs[n][off + math.prod(s):] == 7).all(), n
    got = {n: bufs[n][off:off + math.prod(s)].view(s) for n, s in size_of.items()}
    _verify(op, t, got["y"], got)
