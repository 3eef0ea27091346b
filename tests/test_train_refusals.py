"""Calls out of order: refused on the host (no GPU needed; nothing is launched)."""
import os

import pytest


def _layer(**kw):
    from combine_top_router_amd import lib as L
    if not os.path.exists(L.lib_path()):
        pytest.skip("libmoe.so not built")
    from combine_top_router_amd import MoeLayer
    return MoeLayer(16, 64, 64, 8, 2, device="cpu", **kw)


@pytest.mark.parametrize("recompute", [0, 1])
def test_updates_need_gradients(recompute):
    """The gradients' buffers hold whatever was in the memory until a backward has run."""
    lay = _layer(recompute=recompute)
    with pytest.raises(RuntimeError, match="without a backward"):
        lay.orthogonalize()
    assert not lay._updates and not lay._orth   # nothing allocated either


def test_a_balance_loss_needs_a_forward():
    with pytest.raises(RuntimeError, match="without a forward"):
        _layer().balance(0.1)
