"""Orthogonalised updates: fp32 matrices on the largest tiles, and operators that share scratch."""
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


def test_operators_that_share_scratch():
    from combine_top_router_amd import Orthogonalizer
    gen = torch.Generator().manual_seed(1)
    a = Orthogonalizer(4, 300, 520)
    b = Orthogonalizer(4, 520, 300, steps=3, scratch=a.scratch)
    assert b.scratch is a.scratch
    ga = torch.randn(4, 300, 520, generator=gen).bfloat16().cuda()
    gb = torch.randn(4, 520, 300, generator=gen).bfloat16().cuda()
    wa, wb = Orthogonalizer(4, 300, 520).update(ga), Orthogonalizer(4, 520, 300, steps=3).update(gb)
    for _ in range(2):
        assert torch.equal(a.update(ga), wa) and torch.equal(b.update(gb), wb)
    for bad in (a.scratch[:-300], a.scratch[1:], a.scratch.cpu(), a.scratch.view(torch.int32), a.scratch[::2]):
        with pytest.raises(ValueError):
            Orthogonalizer(4, 300, 520, scratch=bad)


def test_the_layers_updates_share_scratch():
    """Also those of other numbers of steps: the memory does not grow with them."""
    from combine_top_router_amd import MoeLayer, Orthogonalizer
    gen = torch.Generator().manual_seed(2)
    T, H, I, E, k = 128, 256, 512, 8, 2
    randn = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()  # noqa: E731
    lay = MoeLayer(T, H, I, E, k)
    lay.forward(torch.randn(T, E, generator=gen).cuda(), randn(T, H), randn(E, H, I) / 16, randn(E, H, I) / 16,
                randn(E, I, H) / 16)
    lay.backward(randn(T, H))
    for steps in (5, 3):
        up = lay.orthogonalize(steps=steps)
        for name, g in (("gate", lay.dw_gate), ("up", lay.dw_up), ("down", lay.dw_down)):
            assert torch.equal(up[name], Orthogonalizer(E, *g.shape[1:], steps=steps).update(g)), (steps, name)
    assert len({o.scratch.data_ptr() for o in lay._orth.values()}) == 1 and len(lay._orth) == 4
