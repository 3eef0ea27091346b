"""AdamW over more elements than one launch takes (2^32 threads of 8)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def _same(t, value):
    """Every element of a flat tensor, by parts."""
    return all(float(c.min()) == value == float(c.max()) for c in t.split(1 << 30))


@pytest.mark.parametrize("tensors", [1, 3])
def test_adamw_of_many_elements(tensors):
    """2^35 elements and some in bf16 with 8-bit moments; the gradient of ones is the parameter itself."""
    from combine_top_router_amd import AdamW, lib as L
    _room(150)
    n = (1 << 35) + 5000
    buf = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    cuts = [n * i // tensors for i in range(tensors + 1)]
    params = [buf[a:b] for a, b in zip(cuts, cuts[1:])]
    op = AdamW(params, state=L.MOE_STATE_8BIT, weight_decay=0.0, betas=(0.5, 0.5))
    op.step(params, 0.25)
    torch.cuda.synchronize()
    # m = v = 1/2, unbiased 1: a step of 0.25; codes of 1/2 and sqrt(1/2), scales by the blocks' largest
    assert _same(buf, 0.75)
    first = [x[:32].view(torch.uint8)[0].item() for x in (op.m, op.v)]
    for codes, want, scale in ((op.m, first[0], op.m_scale), (op.v, first[1], op.v_scale)):
        for i, (a, b) in enumerate(zip(cuts, cuts[1:])):
            at = op._at[i]
            assert all(int(c.min()) == want == int(c.max()) for c in codes[at:at + b - a].split(1 << 30))
        assert int(scale.min()) == int(scale.max())
    del op, params, buf
    torch.cuda.empty_cache()
