"""AdamW called in ways of a user's program: states from elsewhere, a clock read beside other streams, captured
steps on a given stream."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _op(p, state="8bit", **kw):
    from combine_top_router_amd import AdamW, lib as L
    return AdamW([p], state=L.MOE_STATE_8BIT if state == "8bit" else L.MOE_STATE_F32, **kw)


@pytest.mark.parametrize("scale", [0, 1, 127, 254, 255])
def test_zeroed_codes_with_any_scale(scale):
    """Zeroed codes are zero moments, with any scale."""
    g = torch.randn(1000, generator=torch.Generator().manual_seed(1)).cuda()
    a, b = (_op(torch.ones(1000, device="cuda")) for _ in range(2))
    for s in (b.m_scale, b.v_scale):
        s.fill_(scale)
    for x in b.moments(0):
        assert not x.any() and torch.isfinite(x).all()
    for _ in range(2):
        a.step([g], 1e-2)
        b.step([g], 1e-2)
    for x, y in ((a.params[0], b.params[0]), (a.m, b.m), (a.v, b.v), (a.m_scale, b.m_scale), (a.v_scale, b.v_scale)):
        assert torch.equal(x, y)


def test_moments_are_what_the_codes_stand_for():
    """moments() to the bit over fp32's exponents, against fp64 on the CPU (codes of 4 bits, squares of 8: exact)."""
    n = 32 * 120
    g = (torch.randn(n, generator=torch.Generator().manual_seed(2)).view(-1, 32) * torch.exp2(torch.arange(-60, 60.0))[:, None]).view(-1)
    op = _op(torch.zeros(n, device="cuda"))
    op.step([g.cuda()], 0.0)
    for x, codes, scale, square in zip(op.moments(0), (op.m, op.v), (op.m_scale, op.v_scale), (False, True)):
        want = codes.cpu().view(torch.float8_e4m3fn).double().view(-1, 32).numpy()
        want = np.ldexp(want, scale.cpu().numpy().astype(np.int64)[:, None] - 127).reshape(-1)
        want = want * want if square else want
        assert np.array_equal(x.double().cpu().numpy(), want.astype(np.float32).astype(np.float64))


def test_steps_taken_on_another_stream_are_counted():
    """`t` read while the step's stream is still at work."""
    op, side = _op(torch.ones(64, device="cuda"), capturable=True), torch.cuda.Stream()
    g = torch.ones(64, device="cuda")
    rate = torch.ones(1, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            big = (big @ big) * 1e-4
    op.step([g], rate, stream=side)
    assert op.t == 1
    side.synchronize()


def test_clock_set_beside_another_stream():
    """`t` set while the step's stream is still at work: the step before it counts from the old number, the next
    from the new one."""
    op, side = _op(torch.ones(64, device="cuda"), capturable=True), torch.cuda.Stream()
    g, rate = torch.ones(64, device="cuda"), torch.ones(1, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            big = (big @ big) * 1e-4
    op.step([g], rate, stream=side)
    op.t = 10
    op.step([g], rate, stream=side)
    assert op.t == 11


def test_captured_on_a_given_stream_needs_the_clock():
    """The step's own stream decides, not the current one."""
    op = _op(torch.ones(64, device="cuda"))
    g = torch.ones(64, device="cuda")
    with_clock = _op(torch.ones(64, device="cuda"), capturable=True)
    rate = torch.full((1,), 1e-2, device="cuda")
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = torch.cuda.current_stream()
        with torch.cuda.stream(other):
            with pytest.raises(RuntimeError, match="capturable"):
                op.step([g], 1e-2, stream=captured)
            with_clock.step([g], rate, stream=captured)
    assert op.t == 0
    for n in range(3):
        graph.replay()
        torch.cuda.synchronize()
        op.step([g], 1e-2)
        assert op.t == n + 1 == with_clock.t
        assert torch.equal(op.params[0], with_clock.params[0])
