"""How exact the orthogonalised updates are on the gradients of experts that saw few tokens: of
rank 1 to 64, a few rows or columns (outlier features) far above the rest.  What is lost early
in a strong direction lands beside the weak ones, which the steps multiply.

On the CPU the oracle with the kernels' roundings; on the GPU each matrix is held to what the
oracle says of that matrix: fp32 sums in another order move some roundings to the other side,
as independent errors of the same size sqrt(2) in all; the output's own rounding adds at most
half a step, 2^-8 of each value, so of the norm."""
import numpy as np
import pytest
import torch

from oracle import train as ot


def few_tokens(m, l, rank, rows, cols, boost, floor, seed, dt=torch.bfloat16):
    """Rank `rank`, `rows` rows and `cols` columns `boost` times the others, over a floor."""
    r = np.random.default_rng(seed)
    g = r.normal(size=(m, rank)) @ r.normal(size=(rank, l))
    g[r.choice(m, rows, replace=False)] *= boost
    g[:, r.choice(l, cols, replace=False)] *= boost
    g += floor * r.normal(size=(m, l)) * np.linalg.norm(g) / np.sqrt(m * l)
    return torch.from_numpy(g).to(dt)


KINDS = [(1, 0, 0, 1, 0), (1, 3, 0, 100, 0), (2, 1, 0, 1000, 0), (2, 3, 0, 100, 1e-3), (3, 3, 0, 100, 0), (4, 4, 0, 100, 1e-3),
         (4, 0, 0, 1, 0), (8, 0, 4, 100, 0), (8, 8, 0, 30, 3e-2), (24, 8, 0, 30, 0), (32, 0, 0, 1, 1e-3), (64, 2, 2, 100, 1e-3)]


def _off(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,l", [(70, 96), (100, 500), (192, 400)])
def test_precision_of_few_tokens(m, l, kind, fp32):
    """bf16 matrices enter exactly.  fp32 ones in 15 bits: errors of 2^-16 / sqrt(3) of each value
    (half a step of lo, spread evenly), 8.8e-6 of the norm, which the five steps multiply by up
    to 3.4445^5 = 485 where nothing else lies, 4.3e-3 beside a single singular value that they
    take to 0.7 or more: 6.1e-3, and with the 5e-3 of the iterates 8e-3."""
    g = few_tokens(m, l, *kind, seed=m, dt=torch.float32 if fp32 else torch.bfloat16).double().numpy()
    for steps in (3, 5):
        assert _off(ot.orthogonalize_rounded(g, steps, fp32=fp32), ot.orthogonalize(g, steps)) < (8e-3 if fp32 else 5e-3), steps


@pytest.mark.parametrize("size", [1e-7, 1e-9, 1e-12, 1e-15, 1e-18, 1e-24, 1e-30])
@pytest.mark.parametrize("m,l,steps", [(100, 200, 5), (200, 100, 3), (60, 90, 6)])
def test_precision_of_small_norms(m, l, steps, size):
    """Far below the 1e-7 in the divisor the iterates are as small, X_i = a^i X_0, and each
    rounding is one to fp16, 2^-12 of a value at most; five stored iterates stay
    below 5 * 2^-12 = 1.3e-3, and next to 1e-7 below the 2e-3 of ordinary norms."""
    g = few_tokens(m, l, m // 3, 0, 0, 1, 0.1, 1, dt=torch.float32).double().numpy()
    g *= size / np.linalg.norm(g)
    assert _off(ot.orthogonalize_rounded(g, steps), ot.orthogonalize(g, steps)) < 2e-3
    assert _off(ot.orthogonalize_rounded(g, steps, fp32=True), ot.orthogonalize(g, steps)) < 2e-3


# in one CU; squares in one launch a step; small tiles; a tall one; the largest tiles, padded with
# other matrices to the number that takes them there
@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,n", [(96, 70, 12), (70, 96, 12), (100, 700, 12), (64, 1024, 12), (192, 768, 12),
                                         (768, 192, 12), (384, 1024, 40), (1024, 384, 40)])
def test_orth_of_few_tokens(rows, cols, n, dt):
    from combine_top_router_amd import Orthogonalizer
    import combine_top_router_amd.lib as L
    m, l = min(rows, cols), max(rows, cols)
    g = torch.randn(n, rows, cols, generator=torch.Generator().manual_seed(rows)).to(dt)
    for i, kind in enumerate(KINDS):
        a = few_tokens(m, l, *kind, seed=i, dt=dt)
        g[i] = a if rows <= cols else a.T
    op = Orthogonalizer(n, rows, cols, dtype=L.MOE_BF16 if dt == torch.bfloat16 else L.MOE_F32)
    o = op.update(g.cuda()).double().cpu().numpy()
    for i, kind in enumerate(KINDS):
        a = g[i].double().numpy()
        want = ot.orthogonalize(a, 5)
        tol = 2.0 ** -8 + 2 ** 0.5 * _off(ot.orthogonalize_rounded(a, 5, fp32=dt == torch.float32), want)
        assert np.isfinite(o[i]).all() and _off(o[i], want) < tol, kind


@pytest.mark.gpu
def test_orth_does_not_depend_on_the_others():
    """A matrix's update is as exact alone as among many, where other tiles are taken."""
    from combine_top_router_amd import Orthogonalizer
    a = few_tokens(384, 1024, 2, 3, 0, 100, 0, 7)
    want = ot.orthogonalize(a.double().numpy(), 5)
    tol = 2.0 ** -8 + 2 ** 0.5 * _off(ot.orthogonalize_rounded(a.double().numpy(), 5), want)
    for n in (1, 8, 16, 64, 128):
        g = torch.randn(n, 384, 1024, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16)
        g[n // 2] = a
        o = Orthogonalizer(n, 384, 1024).update(g.cuda())
        assert _off(o[n // 2].double().cpu().numpy(), want) < tol, n


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,n", [(96, 70, 8), (64, 1024, 8), (192, 500, 8), (500, 192, 8), (320, 600, 64)])
@pytest.mark.parametrize("steps", [1, 2, 5])
def test_orth_of_small_norms(rows, cols, n, steps, dt):
    """Matrices of norms from 1e-6 to 1e-30 side by side."""
    from combine_top_router_amd import Orthogonalizer
    import combine_top_router_amd.lib as L
    sizes = [1e-6, 1e-7, 1e-9, 1e-12, 1e-15, 1e-18, 1e-24, 1e-30]
    g = torch.randn(n, rows, cols, generator=torch.Generator().manual_seed(steps)).to(dt)
    for i, size in enumerate(sizes):
        a = few_tokens(rows, cols, min(rows, cols) // 3, 0, 0, 1, 0.1, i, dt=torch.float64)
        g[i] = (a * (size / a.norm())).to(dt)
    op = Orthogonalizer(n, rows, cols, dtype=L.MOE_BF16 if dt == torch.bfloat16 else L.MOE_F32, steps=steps)
    o = op.update(g.cuda()).double().cpu().numpy()
    for i, size in enumerate(sizes):
        a = g[i].double().numpy()
        want = ot.orthogonalize(a, steps)
        tol = 2.0 ** -8 + 2 ** 0.5 * _off(ot.orthogonalize_rounded(a, steps, fp32=dt == torch.float32), want)
        assert np.isfinite(o[i]).all() and _off(o[i], want) < tol, size
