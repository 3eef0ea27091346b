"""relu's corner in fp32: the gradient goes by the sign of z = x W + b itself, not by that of its fp32 sum.

z is compared with fp64's, whose own sums (1e-16 of 30) are far below the smallest z here.  The gradients' bounds are
those of their own sums alone (u = 2^-24): dz = dy or 0 is exact."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _op(T, K, N, **kw):
    from combine_top_router_amd import Linear, lib as L
    return Linear(T, K, N, act=L.MOE_ACT_RELU, dtype=L.MOE_F32, **kw)


def _inputs(T, K, N, bias, share, seed=0):
    """Ordinary data, in which a part of W's columns was turned until z of one of the rows is 0 but for what the
    column's rounding to fp32 leaves."""
    g = torch.Generator().manual_seed(seed + T + K + N)
    x, w = torch.randn(T, K, generator=g).float(), torch.randn(K, N, generator=g) / K ** 0.5
    b = 0.3 * torch.randn(N, generator=g) if bias else None
    x64, w64 = x.double(), w.double()
    for n in range(0, N, share):
        r = x64[(7 * n) % T]
        z = r @ w64[:, n] + (b[n].double() if bias else 0.0)
        w64[:, n] -= r * z / (r @ r)
    return x.cuda(), w64.float().cuda(), None if b is None else b.cuda(), torch.randn(T, N, generator=g).cuda()


def _check(op, x, w, b, dy, y, g):
    xd, wd, dyd = x.double(), w.double(), dy.double()
    z = xd @ wd
    if b is not None:
        z = z + b.double()
    K = x.shape[1]
    room = (K + 8) * U * (xd.abs() @ wd.abs() + (0 if b is None else b.double().abs()))
    assert (z != 0).all()
    wrong = (op.z > 0) != (z > 0)
    assert not wrong.any(), (int(wrong.sum()), z[wrong][:4].tolist())
    assert ((op.z.double() - z).abs() <= room).all() and ((y.double() - z.clamp(min=0)).abs() <= room).all()
    dz = torch.where(z > 0, dyd, 0.0)
    T, N = z.shape
    assert ((g["dx"].double() - dz @ wd.t().contiguous()).abs() <= (N + 8) * U * (dz.abs() @ wd.abs().t().contiguous()) + 1e-40).all()
    assert ((g["dw"].double() - xd.t().contiguous() @ dz).abs() <= (T + 8) * U * (xd.abs().t().contiguous() @ dz.abs()) + 1e-40).all()
    if b is not None:
        assert ((g["db"].double() - dz.sum(0)).abs() <= (T + 8) * U * dz.abs().sum(0) + 1e-40).all()


# up to four rows, single columns and rows, the general kernel's two tiles, with and without shares, long sums
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("size", [(1, 300, 64), (2, 64, 1000), (3, 2049, 33), (4, 769, 128), (3, 100, 7), (40, 100, 1), (33, 300, 50),
                                  (1003, 769, 333), (300, 4000, 64), (1000, 64, 2000), (8185, 261, 1021)],
                         ids=lambda s: "x".join(map(str, s)))
def test_sign_of_z(size, bias):
    T, K, N = size
    x, w, b, dy = _inputs(T, K, N, bias, 1 if N < 100 else 5)
    op = _op(T, K, N)
    op.scratch.fill_(0xFF)
    y = op.forward(x, w, b)
    g = op.backward(dy)
    torch.cuda.synchronize()
    _check(op, x, w, b, dy, y, g)
    first = [v.clone() for v in (op.z, y, *(v for v in g.values() if v is not None))]
    op.scratch.fill_(0xFF)
    op.forward(x, w, b)
    again = op.backward(dy)
    for p, q in zip(first, (op.z, op.y, *(v for v in again.values() if v is not None))):
        assert torch.equal(p, q)
    # what is not trained has the same y, to the bit
    assert torch.equal(_op(T, K, N, train=False).forward(x, w, b), y)


def test_sign_of_z_anywhere():
    """The same where the matrices start at any element."""
    T, K, N = 130, 200, 77
    t = _inputs(T, K, N, True, 1)

    def moved(v):
        buf = torch.full((v.numel() + 16,), float("nan"), device="cuda")
        buf[3:3 + v.numel()] = v.reshape(-1)
        return buf[3:3 + v.numel()].view(v.shape)

    x, w, b, dy = (moved(v) for v in t)
    op = _op(T, K, N)
    y = op.forward(x, w, b)
    _check(op, x, w, b, dy, y, op.backward(dy))


@pytest.mark.parametrize("T", [2, 4, 500])
def test_sums_that_are_zero(T):
    """z = 0 by the data's structure, or of rows and columns of zeros, infinities and NaN: relu'(0) = 0, NaN stays in
    its row."""
    K, N = 96, 130
    g = torch.Generator().manual_seed(T)
    x, w = torch.zeros(T, K), torch.randn(K, N, generator=g)
    x[torch.arange(T), torch.randint(0, K, (T,), generator=g)] = 1.0
    w[torch.rand(K, N, generator=g) < 0.5] = 0.0
    w[:, 3] = 0.0
    x[0] = 0.0
    dy = torch.randn(T, N, generator=g).cuda()
    op = _op(T, K, N)
    x, w = x.cuda(), w.cuda()
    y = op.forward(x, w)
    z = x.double() @ w.double()
    assert torch.equal(op.z.double(), z) and torch.equal(y.double(), z.clamp(min=0))
    dw = op.backward(dy)["dw"]
    dz = torch.where(z > 0, dy.double(), 0.0)
    want, size = x.double().t().contiguous() @ dz, x.double().t().contiguous() @ dz.abs()
    assert ((dw.double() - want).abs() <= (T + 8) * U * size).all()
    x[1, 5] = float("nan")
    y = op.forward(x, w)
    assert torch.isnan(op.z[1]).all() and torch.equal(op.z[0].double(), z[0])
    x[1, 5] = 3e38   # squares beyond fp32: the sum stays as it is
    op.forward(x, w)
    assert torch.equal(op.z[0].double(), z[0])


def test_sign_of_z_replayed():
    T, K, N = 300, 769, 70
    x, w, b, dy = _inputs(T, K, N, True, 1)
    op = _op(T, K, N)
    want = [v.clone() for v in (op.forward(x, w, b), op.z, *op.backward(dy).values())]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(x, w, b)
        op.backward(dy)
    for _ in range(3):
        for v in (op.y, op.z, op.dx, op.dw, op.db):
            v.fill_(3.0)
        op.scratch.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(want, (op.y, op.z, op.dx, op.dw, op.db)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("kind", ["offset", "one-hot"])
@pytest.mark.parametrize("size", [(2, 96, 130), (4, 1000, 40), (3, 70, 7), (64, 2048, 200), (40, 100, 1), (1003, 769, 333), (8185, 261, 1021)],
                         ids=lambda s: "x".join(map(str, s)))
def test_sums_that_cancel_in_bulk(size, kind):
    """Rows far off 0 against columns without a mean, all of whose sums lie within the rounding, and rows with
    two entries of W that differ by less than that: the matrices' other way to fp64."""
    T, K, N = size
    g = torch.Generator().manual_seed(T + K)
    w = torch.randn(K, N, generator=g) / K ** 0.5
    if kind == "offset":
        x, w = 1000.0 + torch.randn(T, K, generator=g), w - w.mean(0, keepdim=True)
    else:
        w[1::2] = w[0:K - K % 2:2] + 1e-7 * torch.randn(K // 2, N, generator=g)
        x = torch.zeros(T, K)
        at = 2 * torch.randint(0, K // 2, (T,), generator=g)
        x[torch.arange(T), at], x[torch.arange(T), at + 1] = 1.1, -1.1
    x, w, dy = x.cuda(), w.cuda(), torch.randn(T, N, generator=g).cuda()
    op = _op(T, K, N)
    y = op.forward(x, w)
    grads = op.backward(dy)
    z = x.double() @ w.double()
    assert torch.equal(op.z > 0, z > 0)
    dz = torch.where(z > 0, dy.double(), 0.0)
    xt = x.double().t().contiguous()
    assert ((grads["dw"].double() - xt @ dz).abs() <= (T + 8) * U * (xt.abs() @ dz.abs()) + 1e-40).all()
    assert ((y.double() - z.clamp(min=0)).abs() <= (K + 8) * U * (x.double().abs() @ w.double().abs())).all()
    assert torch.equal(_op(T, K, N, train=False).forward(x, w), y)


@pytest.mark.parametrize("size", [(2, 96, 130), (64, 2048, 200), (1003, 769, 333)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("sx,sw", [(2.0 ** -50, 2.0 ** -50), (2.0 ** 50, 2.0 ** 50), (2.0 ** -40, 2.0 ** 60)])
def test_sign_of_z_of_other_sizes(size, sx, sw):
    """The same data times powers of two, of which the products of the squares leave fp32's range: the same signs."""
    T, K, N = size
    x, w, _, dy = _inputs(T, K, N, False, 5)
    op = _op(T, K, N)
    op.forward(x * sx, w * sw)
    z = x.double() @ w.double()
    assert torch.equal(op.z > 0, z > 0)
