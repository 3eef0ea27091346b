"""The smallest eps of AdamW: what is below fp32's smallest normal number has no finite reciprocal there, and an
element without moments would become 0 inf = NaN where the formula has 0 / eps = 0."""
import os

import pytest
import torch


def _lib():
    from combine_top_router_amd import lib as L
    if not os.path.exists(L.lib_path()):
        pytest.skip("libmoe.so not built")
    return L


@pytest.mark.parametrize("eps", [1e-40, 2.0 ** -127, 1.0e-45])
def test_eps_without_a_reciprocal_is_refused(eps):
    L = _lib()
    from combine_top_router_amd import AdamW
    with pytest.raises(L.MoeError) as e:
        AdamW([torch.zeros(8)], eps=eps)
    assert e.value.code == L.MOE_EINVAL
    AdamW([torch.zeros(8)], eps=2.0 ** -126)


@pytest.mark.gpu
@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_elements_without_moments_decay(state):
    from combine_top_router_amd import AdamW, lib as L
    p = torch.ones(100, device="cuda")
    op = AdamW([p], state=L.MOE_STATE_8BIT if state == "8bit" else L.MOE_STATE_F32, eps=2.0 ** -126, weight_decay=0.5)
    op.step([torch.zeros(100, device="cuda")], 0.5)
    assert (p == 0.75).all()
