"""Orthogonalised updates against the fp64 oracle.

Bound: the oracle with the iterates held as the kernels hold them is within 2e-3 of the exact
one for five steps over these spectra (test_oracle_train.py); fp32 sums in another order move
some of its roundings to the other side, which at most doubles it in the worst case seen as
independent errors, sqrt(2) 2e-3 = 2.9e-3; the output's own rounding adds at most half a step,
2^-8 of each value, so of the norm.  Together 2^-8 + 3e-3 of the norm."""
import numpy as np
import pytest
import torch

from oracle import train as ot

from test_oracle_train import spectra

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -8 + 3e-3
SIZES = [(100, 200), (128, 150), (60, 320), (40, 500), (64, 700), (700, 64), (130, 1100), (1, 1), (1, 9), (9, 1), (2, 2), (17, 33), (64, 64), (65, 64), (63, 130), (128, 64), (130, 257), (257, 130),
         (256, 256), (300, 700), (768, 256), (520, 520), (333, 1000), (1000, 333)]


def _op(n, rows, cols, dt, steps=5):
    from combine_top_router_amd import Orthogonalizer
    import combine_top_router_amd.lib as L
    return Orthogonalizer(n, rows, cols, dtype=L.MOE_BF16 if dt == torch.bfloat16 else L.MOE_F32, steps=steps)


def _off(got, want):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_orth_against_the_oracle(rows, cols, dt):
    kinds = ["flat", "low_rank", "power"]
    g = torch.stack([torch.from_numpy(spectra(k, rows, cols, i)) for i, k in enumerate(kinds)])
    g = (g * torch.tensor([1e-3, 5.0, 1.0]).double()[:, None, None]).to(dt)
    o = _op(3, rows, cols, dt).update(g.cuda(), scale=0.7)
    torch.cuda.synchronize()
    for i, k in enumerate(kinds):
        assert _off(o[i], ot.orthogonalize(g[i].double().numpy(), 5, 0.7)) < TOL, k


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_orth_steps(steps, dt):
    g = torch.from_numpy(spectra("flat", 90, 200, steps)).to(dt)[None]
    o = _op(1, 90, 200, dt, steps).update(g.cuda())
    torch.cuda.synchronize()
    assert _off(o[0], ot.orthogonalize(g[0].double().numpy(), steps)) < TOL


@pytest.mark.parametrize("size", [1e-30, 1e-9, 1e20, 1e30])
def test_orth_of_any_magnitude(size):
    """The norm is summed in fp64: squares of 1e30 or 1e-30 leave fp32's range."""
    g = (torch.from_numpy(spectra("flat", 70, 96, 3)) * size).float()[None]
    o = _op(1, 70, 96, torch.float32).update(g.cuda())
    torch.cuda.synchronize()
    want = ot.orthogonalize(g[0].double().numpy(), 5)
    if size < 1e-20:   # far below the 1e-7 in the divisor: as good as zero
        assert torch.isfinite(o).all() and float(o.float().abs().max()) < 1e-9
    else:
        assert _off(o[0], want) < TOL


def test_orth_matrices_apart():
    """A zero matrix gives zeros; one with a NaN or an infinity gives NaN; the others are as
    they are alone, bit for bit, and as before from run to run."""
    g = torch.stack([torch.from_numpy(spectra("flat", 80, 72, i)) for i in range(5)]).to(torch.bfloat16).cuda()
    clean = _op(5, 80, 72, torch.bfloat16).update(g).clone()
    bad = g.clone()
    bad[1] = 0
    bad[2, 3, 4] = float("nan")
    bad[3, 0, 0] = float("inf")
    op = _op(5, 80, 72, torch.bfloat16)
    o = op.update(bad)
    assert not o[1].any() and torch.isnan(o[2]).all() and torch.isnan(o[3]).all()
    assert torch.equal(o[0], clean[0]) and torch.equal(o[4], clean[4])
    assert torch.equal(op.update(g), clean)
    alone = _op(1, 80, 72, torch.bfloat16).update(g[2:3].contiguous())
    assert torch.equal(alone[0], clean[2])


# one launch; step by step on small tiles; two steps merged; 256-row tiles (40 matrices)
@pytest.mark.parametrize("n,rows,cols", [(2, 70, 33), (2, 260, 250), (2, 70, 700), (2, 700, 70), (40, 500, 610)])
def test_orth_in_place_and_within_bounds(n, rows, cols):
    import combine_top_router_amd.lib as L
    s = L.MoeOrthShape(n, rows, cols, L.MOE_BF16, 5)
    g = torch.randn(n, rows, cols, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
    want = _op(n, rows, cols, torch.bfloat16).update(g)
    count = g.numel()
    buf = torch.full((count + 128,), 9.0, dtype=torch.bfloat16, device="cuda")
    buf[:count] = g.reshape(-1)
    nb = L.moe_orth_scratch_bytes(s)
    ws = torch.full((nb + 256,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN in every type: all of it is written first
    L.moe_orthogonalize(s, buf.data_ptr(), buf.data_ptr(), 1.0, ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(buf[:count].view(n, rows, cols), want)
    assert (buf[count:] == 9).all() and (ws[nb:] == 0xFF).all()


@pytest.mark.parametrize("n,rows,cols", [(40, 512, 640), (40, 640, 512), (36, 300, 1500), (36, 1500, 300), (48, 260, 520)])
@pytest.mark.parametrize("steps", [2, 3, 5])
def test_orth_of_many_matrices(n, rows, cols, steps):
    """Enough of them for the larger tiles, step by step and merged; three of them looked at."""
    gen = torch.Generator().manual_seed(rows)
    g = torch.randn(n, rows, cols, generator=gen).to(torch.bfloat16)
    for i, k in enumerate(("flat", "low_rank", "power")):
        g[i * (n // 3)] = torch.from_numpy(spectra(k, rows, cols, i)).to(torch.bfloat16)
    o = _op(n, rows, cols, torch.bfloat16, steps).update(g.cuda())
    torch.cuda.synchronize()
    for i in (0, n // 3, 2 * (n // 3), n - 1):
        assert _off(o[i], ot.orthogonalize(g[i].double().numpy(), steps)) < TOL, i


@pytest.mark.parametrize("rows,cols,steps", [(1536, 768, 3), (768, 1536, 3), (1500, 700, 5), (700, 1500, 1), (1500, 700, 1)])
def test_orth_on_the_largest_tiles(rows, cols, steps):
    """64 of them go to the 256-row tiles: both orientations, the lo part read by the last step
    (three steps), sizes off the tiles, and a NaN that stays in its matrix."""
    n = 64
    g = torch.randn(n, rows, cols, generator=torch.Generator().manual_seed(rows)).to(torch.bfloat16)
    g[1] = torch.from_numpy(spectra("low_rank", rows, cols, 1)).to(torch.bfloat16)
    g[2, 5, 7] = float("nan")
    g[3] = 0
    o = _op(n, rows, cols, torch.bfloat16, steps).update(g.cuda(), scale=2.0)
    torch.cuda.synchronize()
    for i in (0, 1, n - 1):
        assert _off(o[i], ot.orthogonalize(g[i].double().numpy(), steps, 2.0)) < TOL, i
    assert torch.isnan(o[2]).all() and not o[3].any()
    assert torch.isfinite(torch.cat([o[:2], o[3:]])).all()


@pytest.mark.parametrize("rows,cols", [(64, 640), (33, 1999), (100, 600), (700, 128), (1100, 97)])
@pytest.mark.parametrize("steps,dt", [(1, torch.bfloat16), (2, torch.float32), (3, torch.bfloat16), (4, torch.float32),
                                      (6, torch.bfloat16)])
def test_orth_of_few_rows(rows, cols, steps, dt):
    """A step's squares in one launch: zero, NaN and ordinary matrices side by side, each as it
    is alone, bit for bit."""
    g = torch.stack([torch.from_numpy(spectra(k, rows, cols, i)) for i, k in enumerate(("flat", "low_rank", "power", "flat"))])
    g = g.to(dt)
    g[3, 1, 2] = float("nan")
    g = torch.cat([g, torch.zeros_like(g[:1])])
    o = _op(5, rows, cols, dt, steps).update(g.cuda(), scale=1.5)
    alone = _op(1, rows, cols, dt, steps).update(g[2:3].cuda(), scale=1.5)
    torch.cuda.synchronize()
    for i in range(3):
        assert _off(o[i], ot.orthogonalize(g[i].double().numpy(), steps, 1.5)) < TOL, i
    assert torch.isnan(o[3]).all() and not o[4].any()
    assert torch.equal(o[2], alone[0])


# one launch; squares in one launch a step; small tiles; the largest tiles
@pytest.mark.parametrize("n,rows,cols", [(8, 128, 64), (5, 600, 100), (3, 300, 520), (64, 520, 1100)])
def test_orth_as_graphs_that_share_an_operator(n, rows, cols):
    """Two graphs on one operator's scratch, replayed in turn with eager calls in between."""
    gen = torch.Generator().manual_seed(n)
    op = _op(n, rows, cols, torch.bfloat16)
    g = [torch.randn(n, rows, cols, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [op.update(x).clone() for x in g]
    out = [torch.empty_like(x) for x in g]
    graphs = []
    for x, o in zip(g, out):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op.update(x, out=o)
        graphs.append(graph)
    for _ in range(3):
        for o in out:
            o.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert torch.equal(op.update(g[1]), want[1])


def test_orth_two_at_once():
    """Two operators on two streams, over several calls each."""
    a, b = _op(3, 300, 520, torch.bfloat16), _op(8, 128, 64, torch.bfloat16)
    ga = torch.randn(3, 300, 520, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    gb = torch.randn(8, 128, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    wa, wb = a.update(ga).clone(), b.update(gb).clone()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        oa = a.update(ga, stream=sa)
        ob = b.update(gb, stream=sb)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_orth_refuses_other_tensors():
    op = _op(2, 8, 16, torch.bfloat16)
    g = torch.zeros(2, 8, 16, dtype=torch.bfloat16, device="cuda")
    for bad in (g.float(), g[:1], g.transpose(1, 2), g.cpu()):
        with pytest.raises(ValueError):
            op.update(bad)
    with pytest.raises(ValueError):
        op.update(g, out=g.float())
