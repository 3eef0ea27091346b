"""The norm in front of the layer, forward and backward, against the fp64 oracle.

Bounds, element by element: half a step of the output's type at its value (one rounding),
plus fp32 arithmetic.  A row's sums run at most 16 values in sequence, then 6 + 4 levels of
pairs, so a sum is within 32 * 2^-24 of the sum of its terms' magnitudes; the mean's error
counts times rstd in the normalised value, and every further factor adds one 2^-24."""
import numpy as np
import pytest
import torch

from oracle import train as ot

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SIZES = [(1, 1), (3, 7), (40, 3), (5, 8), (6, 9), (1, 64), (2, 511), (2, 1023), (700, 1001), (2, 2047), (3, 2049), (2, 8191), (2, 16383), (5, 100), (64, 128), (7, 512), (9, 513), (33, 769), (6, 1000), (5, 1024), (5, 1032),
         (300, 2048), (3, 2056), (4, 4095), (4, 4096), (3, 5000), (3, 8192), (2, 8200), (2, 16384), (2, 16385),
         (3, 20000), (1030, 96)]


def L():
    from combine_top_router_amd import lib
    return lib


def _half(dt):
    return torch.finfo(dt).eps / 2


def _inputs(T, H, dt, seed, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (r(T, H) * (1 + 10 * (torch.rand(H, generator=g) < 0.01)) + mean).to(dt)
    return dict(x=x, res=r(T, H).to(dt), w=(1 + 0.3 * r(H)).to(dt), b=(0.2 * r(H)).to(dt), dy=r(T, H).to(dt),
                ds=r(T, H).to(dt))


def _n(t):
    return None if t is None else t.double().cpu().numpy()


def _near(got, want, slack, dt, name):
    got = _n(got)
    bound = _half(dt) * (np.abs(want) + slack) + slack + 2.0 ** -140
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (name, np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3], bound[bad][:3])


def _run(T, H, dt, rms, with_res, with_b, seed=0, stream=None, mean=0.3):
    from combine_top_router_amd import MoeNorm
    lib = L()
    c = {k: v.cuda() for k, v in _inputs(T, H, dt, seed, mean).items()}
    op = MoeNorm(T, H, kind=lib.MOE_NORM_RMS if rms else lib.MOE_NORM_LAYER,
                 dtype=lib.MOE_BF16 if dt == torch.bfloat16 else lib.MOE_F32, eps=1e-5)
    y = op.forward(c["x"], c["w"], c["b"] if with_b else None, res=c["res"] if with_res else None)
    g = op.backward(c["dy"], ds_in=c["ds"] if with_res else None)
    torch.cuda.synchronize()
    return op, c, y, g


def _verify(T, H, dt, rms, with_res, with_b, op, c, y, g):
    x, res = _n(c["x"]), _n(c["res"]) if with_res else None
    w, b = _n(c["w"]), _n(c["b"]) if with_b else None
    want, s, mu, rs = ot.norm_forward(x, res, w, b, np.float32(1e-5), rms)
    mag = np.abs(s).mean(axis=1)
    e_mu = 0.0 if rms else 40 * U * mag
    top = np.abs(s).max(axis=1)
    # relative error of rstd: its sum of squares, and the mean's error in each square
    e_rs = 40 * U + 2 * (e_mu + 4 * U * top) * rs
    if not rms:
        _near(op.mean, mu, e_mu + 0 * mu, torch.float32, "mean")
    _near(op.rstd, rs, e_rs * rs, torch.float32, "rstd")
    xh = (s - mu[:, None]) * rs[:, None]
    e_xh = ((e_mu + 0 * mu)[:, None] + 4 * U * np.abs(s)) * rs[:, None] + (e_rs[:, None] + 4 * U) * np.abs(xh)
    _near(y, want, e_xh * np.abs(w) + 4 * U * (np.abs(xh * w) + (0 if b is None else np.abs(b))), dt, "y")
    if with_res:
        _near(op.sum, s, 2 * U * np.abs(s), dt, "sum")
    # the backward from the forward's own statistics
    s_in = s
    mean = _n(op.mean) if not rms else np.zeros(T)
    rstd = _n(op.rstd)
    dx, dw, db = ot.norm_backward(_n(c["dy"]), s_in, w, mean, rstd, _n(c["ds"]) if with_res else None, rms)
    xh = (s_in - mean[:, None]) * rstd[:, None]
    big = (2 * U * np.abs(s_in) + U * np.abs(mean[:, None])) * rstd[:, None]   # xh's own error
    gg = np.abs(_n(c["dy"]) * w)
    gx = np.abs(_n(c["dy"]) * w * xh)
    e = 48 * U * rstd[:, None] * (gg + gg.mean(axis=1, keepdims=True) + np.abs(xh) * gx.mean(axis=1, keepdims=True))
    e = e + rstd[:, None] * (big * gx.mean(axis=1, keepdims=True) + np.abs(xh) * (gg * big).mean(axis=1, keepdims=True))
    _near(g["dx"], dx, e + 2 * U * np.abs(dx), dt, "dx")
    # a column's sum: at most T / 16 rows in sequence in a share, then the shares
    seq = 16 + T // 4
    dyx = np.abs(_n(c["dy"]) * xh).sum(axis=0)
    _near(g["dw"], dw, (seq + 8) * U * dyx + (np.abs(_n(c["dy"])) * big).sum(axis=0), dt, "dw")
    if with_b:
        _near(g["db"], db, (seq + 8) * U * np.abs(_n(c["dy"])).sum(axis=0), dt, "db")
    else:
        assert g["db"] is None


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm_against_the_oracle(T, H, dt):
    rms = (T + H) % 2 == 0
    for flip in (False, True):
        args = (T, H, dt, rms != flip, flip, (T % 3 == 0) != flip)
        _verify(*args, *_run(*args, seed=T + H))


def test_norm_of_views_off_a_16_byte_boundary():
    """Rows that start at an odd element (a slice of a larger buffer)."""
    from combine_top_router_amd import MoeNorm
    T, H = 5, 200
    c = _inputs(T, H, torch.bfloat16, 3)
    op, base = MoeNorm(T, H), MoeNorm(T, H)
    want = base.forward(c["x"].cuda(), c["w"].cuda(), c["b"].cuda(), res=c["res"].cuda()).clone()
    gw = {k: v.clone() for k, v in base.backward(c["dy"].cuda()).items()}

    def off(t):
        big = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        big[1:] = t.reshape(-1).cuda()
        return big[1:].view(t.shape)

    assert torch.equal(op.forward(off(c["x"]), off(c["w"]), off(c["b"]), res=off(c["res"])), want)
    g = op.backward(off(c["dy"]))
    for k in gw:
        assert torch.equal(g[k], gw[k]), k


def test_norm_in_place_sum_and_gradient():
    lib = L()
    T, H = 6, 300
    c = {k: v.cuda() for k, v in _inputs(T, H, torch.bfloat16, 4).items()}
    from combine_top_router_amd import MoeNorm
    op = MoeNorm(T, H)
    y = op.forward(c["x"], c["w"], None, res=c["res"]).clone()
    g = {k: v.clone() for k, v in op.backward(c["dy"], ds_in=c["ds"]).items() if v is not None}
    s = lib.MoeNormShape(T, H, lib.MOE_BF16, lib.MOE_NORM_LAYER, 1e-5)
    st = torch.cuda.current_stream().cuda_stream
    y2, mean, rstd = torch.empty_like(y), torch.empty_like(op.mean), torch.empty_like(op.rstd)
    x, dx = c["x"].clone(), c["ds"].clone()
    p = lambda t: t.data_ptr()  # noqa: E731
    lib.moe_norm_fwd(s, p(x), p(c["res"]), p(c["w"]), 0, p(x), p(y2), p(mean), p(rstd), st)      # sum is x
    dw = torch.empty_like(c["w"])
    lib.moe_norm_bwd(s, p(c["dy"]), p(c["x"]), p(c["res"]), p(c["w"]), p(mean), p(rstd), p(dx), p(dx), p(dw), 0,
                     p(op.scratch), st)
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(x, op.sum)
    assert torch.equal(dx, g["dx"]) and torch.equal(dw, g["dw"])
    # from the stored sum: what the oracle gives for that
    lib.moe_norm_bwd(s, p(c["dy"]), p(x), 0, p(c["w"]), p(mean), p(rstd), 0, p(dx), p(dw), 0, p(op.scratch), st)
    torch.cuda.synchronize()
    dx64, dw64, _ = ot.norm_backward(_n(c["dy"]), _n(x), _n(c["w"]), _n(mean), _n(rstd), None, False)
    assert np.linalg.norm(_n(dx) - dx64) < 2.0 ** -8 * np.linalg.norm(dx64)
    assert np.linalg.norm(_n(dw) - dw64) < 2.0 ** -8 * np.linalg.norm(dw64)


def test_norm_rows_apart():
    """A row of NaN or infinities spoils no other row; a constant row gives its bias."""
    from combine_top_router_amd import MoeNorm
    T, H = 6, 130
    c = {k: v.cuda() for k, v in _inputs(T, H, torch.float32, 5).items()}
    op = MoeNorm(T, H, dtype=L().MOE_F32, eps=1e-5)
    clean = op.forward(c["x"], c["w"], c["b"]).clone()
    x = c["x"].clone()
    x[1, 3] = float("nan")
    x[2, 0] = float("inf")
    x[4] = 2.0
    y = op.forward(x, c["w"], c["b"])
    for t in (0, 3, 5):
        assert torch.equal(y[t], clean[t])
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).any()
    assert torch.equal(y[4], c["b"])


def test_norm_far_from_zero():
    """A mean a thousand times the spread: the variance is taken about the mean."""
    args = (4, 1000, torch.float32, False, False, False)
    op, c, y, g = _run(*args, seed=6, mean=1000.0)
    _verify(*args, op, c, y, g)


def test_norm_without_rows():
    lib = L()
    s = lib.MoeNormShape(0, 70, lib.MOE_F32, lib.MOE_NORM_LAYER, 1e-5)
    dw = torch.full((70,), 3.0, device="cuda")
    db = torch.full((70,), 3.0, device="cuda")
    ws = torch.empty(lib.moe_norm_scratch_bytes(s), dtype=torch.uint8, device="cuda")
    lib.moe_norm_bwd(s, 0, 0, 0, 0, 0, 0, 0, 0, dw.data_ptr(), db.data_ptr(), ws.data_ptr(),
                     torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


def test_norm_writes_nothing_past_its_outputs():
    lib = L()
    T, H = 3, 77
    s = lib.MoeNormShape(T, H, lib.MOE_BF16, lib.MOE_NORM_LAYER, 1e-5)
    c = {k: v.cuda() for k, v in _inputs(T, H, torch.bfloat16, 7).items()}
    p = lambda t: t.data_ptr()  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    buf = {n: torch.full((T * H + 64,), 9.0, dtype=torch.bfloat16, device="cuda") for n in ("sum", "y", "dx")}
    vec = {n: torch.full((H + 64,), 9.0, dtype=torch.bfloat16, device="cuda") for n in ("dw", "db")}
    stat = {n: torch.full((T + 64,), 9.0, device="cuda") for n in ("mean", "rstd")}
    nb = lib.moe_norm_scratch_bytes(s)
    ws = torch.full((nb + 256,), 7, dtype=torch.uint8, device="cuda")
    lib.moe_norm_fwd(s, p(c["x"]), p(c["res"]), p(c["w"]), p(c["b"]), p(buf["sum"]), p(buf["y"]), p(stat["mean"]),
                     p(stat["rstd"]), st)
    lib.moe_norm_bwd(s, p(c["dy"]), p(buf["sum"]), 0, p(c["w"]), p(stat["mean"]), p(stat["rstd"]), 0, p(buf["dx"]),
                     p(vec["dw"]), p(vec["db"]), p(ws), st)
    torch.cuda.synchronize()
    for t in buf.values():
        assert (t[T * H:] == 9).all()
    for t in vec.values():
        assert (t[H:] == 9).all()
    for t in stat.values():
        assert (t[T:] == 9).all()
    assert (ws[nb:] == 7).all()


def test_norm_refuses_other_tensors():
    from combine_top_router_amd import MoeNorm
    op = MoeNorm(4, 8)
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda"), torch.ones(8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError):
        op.backward(x)
    for bad in (x.float(), x[:3], x.t().contiguous().t(), x.cpu()):
        with pytest.raises(ValueError):
            op.forward(bad, w)
    with pytest.raises(ValueError):
        op.forward(x, w[:7])
    with pytest.raises(ValueError):
        op.forward(x, w, res=x.float())
