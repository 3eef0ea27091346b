"""What the matrix product writes lies apart from what it reads behind it: the bias, which every row reads, and db,
which is written before both products (no GPU needed; the pointers are never read)."""
import os

import pytest

P = 4096


def _lib():
    from combine_top_router_amd import lib as L
    if not os.path.exists(L.lib_path()):
        pytest.skip("libmoe.so not built")
    return L


def test_bias_apart_from_the_outputs():
    L = _lib()
    s = L.MoeLinearShape(4, 8, 16, L.MOE_BF16, L.MOE_ACT_SILU)
    for b in (4 * P, 5 * P):
        with pytest.raises(L.MoeError) as e:
            L.moe_linear_fwd(s, P, 2 * P, b, 0, 4 * P, 5 * P, P)
        assert e.value.code == L.MOE_EINVAL


@pytest.mark.parametrize("which", range(7))
def test_db_apart_from_the_rest(which):
    L = _lib()
    s = L.MoeLinearShape(4, 8, 16, L.MOE_BF16, L.MOE_ACT_SILU)
    dy, x, w, z, dx_in, dx, dw = others = [P * (i + 1) for i in range(7)]
    with pytest.raises(L.MoeError) as e:
        L.moe_linear_bwd(s, dy, x, w, z, dx_in, dx, dw, others[which], P)
    assert e.value.code == L.MOE_EINVAL
