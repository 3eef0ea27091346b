"""Calls that would take a launch of 2^32 threads or more along an axis, which the runtime cuts off without an error:
refused before the launch (no GPU needed; the pointers are never read)."""
import os

import pytest

P = 4096


def _lib():
    from combine_top_router_amd import lib as L
    if not os.path.exists(L.lib_path()):
        pytest.skip("libmoe.so not built")
    return L


@pytest.mark.parametrize("dtype,K,N", [(0, 1, 1), (0, 8, 8), (1, 1, 1), (1, 8, 8)])
def test_products_of_too_many_rows(dtype, K, N):
    """2^31 - 1 rows are 2^32 threads on tiles of any height."""
    L = _lib()
    T = 2 ** 31 - 1
    s = L.MoeLinearShape(T, K, N, dtype, L.MOE_ACT_NONE)
    for _ in range(2):   # a refusal leaves nothing behind
        with pytest.raises(L.MoeError) as e:
            L.moe_linear_fwd(s, P, 2 * P, 0, 0, 0, 3 * P, P)
        assert e.value.code == L.MOE_EUNSUPPORTED and "2^32" in str(e.value)
    L.moe_linear_fwd(L.MoeLinearShape(0, K, N, dtype, L.MOE_ACT_NONE), 0, 0, 0, 0, 0, 0, 0)
