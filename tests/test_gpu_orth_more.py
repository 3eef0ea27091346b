"""Orthogonalised updates: fp32 matrices on the largest tiles."""
import numpy as np
import pytest
import torch

from oracle import train as ot

from test_oracle_train import spectra

pytestmark = pytest.mark.gpu


def _off(got, want):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("rows,cols,steps", [(1536, 768, 3), (768, 1536, 2), (1500, 700, 5), (700, 1500, 1), (1500, 700, 1)])
def test_fp32_on_the_largest_tiles(rows, cols, steps):
    """64 of them go to the 256-row tiles; g enters with its lo part, which the first product
    (and, of one step, the last) reads."""
    from combine_top_router_amd import Orthogonalizer
    import combine_top_router_amd.lib as L
    n = 64
    g = torch.randn(n, rows, cols, generator=torch.Generator().manual_seed(rows))
    g[1] = torch.from_numpy(spectra("low_rank", rows, cols, 1))
    g[2, 5, 7] = float("nan")
    g[3] = 0
    o = Orthogonalizer(n, rows, cols, dtype=L.MOE_F32, steps=steps).update(g.cuda(), scale=2.0)
    torch.cuda.synchronize()
    for i in (0, 1, n - 1):
        a = g[i].double().numpy()
        want = ot.orthogonalize(a, steps, 2.0)
        # fp32 sums in another order: sqrt(2) of what the roundings cost; the output's half step
        tol = 2.0 ** -8 + 2 ** 0.5 * _off(2.0 * torch.from_numpy(ot.orthogonalize_rounded(a, steps, fp32=True)), want)
        assert _off(o[i], want) < tol, i
    assert torch.isnan(o[2]).all() and not o[3].any()
    assert torch.isfinite(torch.cat([o[:2], o[3:]])).all()
