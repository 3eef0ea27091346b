"""Routing by scores and the matrix product on matrices of more than 2^31 elements: what lies past that is as what
lies before it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


@pytest.mark.parametrize("score,renorm", [(1, 1), (0, 0)])
def test_gate_past_32_bits(score, renorm):
    """The same 4096 tokens over and over."""
    from combine_top_router_amd import Gate
    _room(40)
    B, E, k, n = 4096, 130, 6, 4100
    T = B * n
    assert T * E > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    logits, d = torch.randn(B, E, generator=g, device="cuda"), torch.randn(B, k, generator=g, device="cuda")
    kw = dict(score=score, groups=10, topk_groups=4, group_top=2, renorm=renorm)
    one, all_ = Gate(B, E, k, **kw), Gate(T, E, k, **kw)
    one.forward(logits, count=True)
    want = one.backward(d)
    all_.d_logits.fill_(7.0)
    all_.forward(logits.repeat(n, 1), count=True)
    got = all_.backward(d.repeat(n, 1))
    for a, b in ((one.topk_idx, all_.topk_idx), (one.topk_w, all_.topk_w), (want, got)):
        for part in b.view(n, *a.shape).split(100):
            assert (part == a).all()
    assert torch.equal(one.counts.long() * n, all_.counts.long())
    del all_, got, part, b
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,T,K,N", [("bf16", 140000, 64, 16384), ("bf16", 140001, 65, 16391), ("f32", 70003, 40, 32771)],
                         ids=lambda v: str(v))
def test_linear_past_32_bits(dtype, T, K, N):
    """Blocks of rows of y, z and dx against fp64 (bounds as in test_gpu_linear.py), dw and db against fp64's sums."""
    from combine_top_router_amd import Linear, lib as L
    _room(120)
    assert T * N > 1 << 31
    dt, h = (torch.bfloat16, 2.0 ** -8) if dtype == "bf16" else (torch.float32, U)
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda s, *d: (torch.randn(*d, generator=g, device="cuda") * s).to(dt)  # noqa: E731
    x, w, b, res, dy = rnd(1, T, K), rnd(K ** -0.5, K, N), rnd(0.3, N), rnd(1, T, N), rnd(1, T, N)
    op = Linear(T, K, N, act=L.MOE_ACT_RELU, dtype=L.MOE_BF16 if dtype == "bf16" else L.MOE_F32)
    for v in (op.y, op.z, op.dx, op.dw, op.db):
        v.fill_(float("nan"))
    y = op.forward(x, w, b, res=res)
    out = op.backward(dy)
    torch.cuda.synchronize()
    wd, bd = w.double(), b.double()
    wt = wd.t().contiguous()
    dw, db, dw_room, db_room = (torch.zeros(s, dtype=torch.float64, device="cuda") for s in ((K, N), (N,), (K, N), (N,)))
    for r in range(0, T, 8192):
        s = slice(r, min(T, r + 8192))
        xd, d = x[s].double(), dy[s].double()
        z = xd @ wd + bd
        err = (K + 8) * U * (xd.abs() @ wd.abs() + bd.abs())
        want = z.clamp(min=0) + res[s].double()
        assert ((y[s].double() - want).abs() <= h * want.abs() + 1.1 * err + 2 * U * want.abs()).all(), r
        assert ((op.z[s].double() - z).abs() <= h * z.abs() + 1.1 * err).all(), r
        dz = torch.where(z > 0, d, 0.0)
        e = torch.where(z.abs() <= err, d.abs(), 0.0) + h * dz.abs()
        size = dz.abs() + e
        want = dz @ wt
        assert ((out["dx"][s].double() - want).abs() <= h * want.abs() + (1 + h) * ((e + (N + 8) * U * size) @ wt.abs())).all(), r
        xt = xd.t().contiguous()
        dw += xt @ dz
        db += dz.sum(0)
        dw_room += xt.abs() @ (e + (T + 8) * U * size)
        db_room += (e + (T + 8) * U * size).sum(0)
    assert ((out["dw"].double() - dw).abs() <= h * dw.abs() + (1 + h) * dw_room).all()
    assert ((out["db"].double() - db).abs() <= h * db.abs() + (1 + h) * db_room).all()
    del op, y, out, res, dy
    torch.cuda.empty_cache()
