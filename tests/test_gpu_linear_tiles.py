"""The matrix product on its larger tiles, element by element against fp64 on the card, at sizes that leave ragged
edges on each of them.

On a card of 256 CUs the plans are, forward / dx / dw: 16392 x 1544 x 4104 tiles of 256 / 256 / 256 in 2 shares;
1544 x 4104 x 16392 256 / 256 in 2 shares / 256; 1544 x 16392 x 4104 256 in 2 shares / 256 / 256; 8200 x 1032 x 2056
128 / 256 / 128 in 3 shares; 1032 x 16400 x 2056 128 in 3 shares / 128 / 256; 8185 x 1029 x 2051 (element by
element) 128 / 128 / 128 in 3 shares; 16400 x 1029 x 2056 (x with padded rows) 128 / 128 element by element / 128 in
3 shares; 2056 cubed in fp32 128 in 3 shares throughout.  From odd addresses the bf16 ones take the general kernel's
tiles of 128, with shares where the tiles have them.

Bounds as in test_gpu_linear.py: u = 2^-24, h half a step of the type; sums of K products (K + 8) u S; an
activation's slope at most 1.13, the slope's own 0.8, their evaluation (|z| + 12) u and 4 u; z, dz and the results
rounded to the type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACTS = ["none", "relu", "silu", "gelu"]


def _act(z, act):
    """The activation and its slope."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    c = 0.5 * torch.erfc(-z / math.sqrt(2.0))
    return z * c, c + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _t(x):
    return x.t().contiguous()


def _near(got, want, bound, name):
    bad = ~((got.double() - want).abs() <= bound + 1e-40)
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist())


def _run(size, act, dtype, off=0, bias=True, res=True, dx_in=True):
    from combine_top_router_amd import Linear, lib as L
    T, K, N = size
    dt, h = (torch.bfloat16, 2.0 ** -8) if dtype == "bf16" else (torch.float32, U)
    g = torch.Generator(device="cuda").manual_seed(T + K + N)

    def rnd(scale, *d):
        n = math.prod(d)
        buf = torch.full((n + 16,), float("nan"), dtype=dt, device="cuda")
        buf[off:off + n] = torch.randn(n, generator=g, device="cuda") * scale
        return buf[off:off + n].view(d)

    x, w, dy = rnd(1, T, K), rnd(K ** -0.5, K, N), rnd(1, T, N)
    b, r, di = rnd(0.3, N) if bias else None, rnd(1, T, N) if res else None, rnd(1, T, K) if dx_in else None
    op = Linear(T, K, N, act=ACTS.index(act), dtype=L.MOE_BF16 if dtype == "bf16" else L.MOE_F32)
    op.scratch.fill_(0xFF)
    for v in (op.y, op.z, op.dx, op.dw, op.db):
        if v is not None:
            v.fill_(float("nan"))
    y = op.forward(x, w, b, res=r)
    op.scratch.fill_(0xFF)
    out = op.backward(dy, dx_in=di)
    torch.cuda.synchronize()
    xd, wd, d = x.double(), w.double(), dy.double()
    z = xd @ wd
    size_z = xd.abs() @ wd.abs()
    if b is not None:
        z, size_z = z + b.double(), size_z + b.double().abs()
    err_z = (K + 8) * U * size_z
    a, slope = _act(z, act)
    want = a if r is None else a + r.double()
    err = 1.13 * err_z + (((z.abs() + 8) * U * z.abs() + 4 * U) if act in ("silu", "gelu") else 0.0)
    _near(y, want, h * want.abs() + (1 + h) * err + 2 * U * want.abs(), "y")
    dz = d * slope
    if act == "none":
        e, held = torch.zeros_like(dz), torch.zeros_like(dz)
    else:
        if act == "relu":
            e = torch.where(z.abs() <= err_z, d.abs(), 0.0) + 2 * U * dz.abs()
        else:
            e = d.abs() * (0.8 * (h * z.abs() + (1 + h) * err_z) + (z.abs() + 12) * U)
        held = h * (dz.abs() + e)
    s = dz.abs() + e + held
    del z, size_z, err_z, a, slope, err, want
    wt, xt = _t(wd), _t(xd)
    want = dz @ wt
    bound = (1 + h) * ((e + held) @ wt.abs() + (N + 8) * U * (s @ wt.abs()))
    if di is not None:
        want, bound = want + di.double(), bound + 2 * U * di.double().abs()
    _near(out["dx"], want, h * want.abs() + bound, "dx")
    want = xt @ dz
    _near(out["dw"], want, h * want.abs() + (1 + h) * (xt.abs() @ (e + held) + (T + 8) * U * (xt.abs() @ s)), "dw")
    if b is not None:
        want = dz.sum(0)
        _near(out["db"], want, h * want.abs() + (1 + h) * (e.sum(0) + (T + 8) * U * s.sum(0)), "db")
    first = [v.clone() for v in (y, *[v for v in out.values() if v is not None])]
    op.forward(x, w, b, res=r)   # the same again, bit for bit
    again = op.backward(dy, dx_in=di)
    for p, q in zip(first, (op.y, *[v for v in again.values() if v is not None])):
        assert torch.equal(p, q)


LARGE = [(16392, 1544, 4104), (1544, 4104, 16392), (1544, 16392, 4104), (8200, 1032, 2056), (1032, 16400, 2056),
         (8185, 1029, 2051), (16400, 1029, 2056)]


@pytest.mark.parametrize("act,bias,res,dx_in", [("silu", True, True, True), ("none", False, False, False)])
@pytest.mark.parametrize("size", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_large_products(size, act, bias, res, dx_in):
    _run(size, act, "bf16", bias=bias, res=res, dx_in=dx_in)


@pytest.mark.parametrize("act", ["relu", "gelu"])
def test_other_activations_on_large_tiles(act):
    _run((16392, 1544, 4104), act, "bf16")


@pytest.mark.parametrize("size", [(8200, 1032, 2056), (1032, 16400, 2056)], ids=lambda s: "x".join(map(str, s)))
def test_large_products_from_odd_addresses(size):
    _run(size, "silu", "bf16", off=1)


@pytest.mark.parametrize("size,act", [((2056, 2056, 2056), "gelu"), ((2055, 2049, 2051), "relu"), ((8192, 1024, 2048), "relu")],
                         ids=lambda s: s if isinstance(s, str) else "x".join(map(str, s)))
def test_large_products_in_fp32(size, act):
    _run(size, act, "f32")
