"""The operators around the layer on another stream than the one that their memory comes from:
that memory may still be in use by the latter's queued work, so the first call waits for it."""
import pytest
import torch


class _Fake:
    """Stands for a stream, and for the event that it records."""

    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def record_event(self):
        self.log.append(("record", self.cuda_stream))
        return ("event", self.cuda_stream)

    def wait_event(self, event):
        self.log.append(("wait", self.cuda_stream, event))


class _Nothing:
    def __init__(self, *a):
        pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        return False


def _operator(monkeypatch, state):
    from combine_top_router_amd import layer
    monkeypatch.setattr(layer.torch.cuda, "current_stream", lambda *a: state["current"])
    monkeypatch.setattr(layer.torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(layer.torch.cuda, "device", _Nothing)
    monkeypatch.setattr(layer.torch.cuda, "stream", _Nothing)
    monkeypatch.setattr(layer, "_raw_stream", lambda i: state["current"].cuda_stream)
    monkeypatch.setattr(layer, "_current_device", lambda: 0)
    op = layer._OnDevice()
    op.device, op._index = torch.device("cuda", 0), 0
    return op


@pytest.mark.parametrize("capturing", [False, True])
def test_the_first_call_on_another_stream_waits(monkeypatch, capturing):
    log = []
    home, side = _Fake(1, log), _Fake(2, log)
    state = {"capturing": False, "current": home}
    op = _operator(monkeypatch, state)
    op._allocated()
    call = lambda stream: op._call(lambda s: log.append(("launch", s)), stream)  # noqa: E731
    call(None)
    state["capturing"] = capturing
    call(side)
    call(side)
    waits = [] if capturing else [("wait", 2, ("event", 1))]   # a capture takes no wait for work outside it
    assert log == [("record", 1), ("launch", 1)] + waits + [("launch", 2), ("launch", 2)]
    state["capturing"] = False
    call(side)
    assert log[-2:] == [("wait", 2, ("event", 1)) if capturing else ("launch", 2), ("launch", 2)]


@pytest.mark.parametrize("capturing", [False, True])
def test_buffers_made_on_two_streams(monkeypatch, capturing):
    """A later buffer of another stream: what runs there, and elsewhere, waits for both."""
    log = []
    one, two, three = (_Fake(i, log) for i in (1, 2, 3))
    state = {"capturing": False, "current": one}
    op = _operator(monkeypatch, state)
    op._allocated()
    state.update(current=two, capturing=capturing)
    op._allocated()
    later = [] if capturing else [("wait", 2, ("event", 1)), ("record", 2)]
    assert log == [("record", 1)] + later
    state["capturing"] = False
    op._call(lambda s: log.append(("launch", s)), three)
    assert log[-2:] == [("wait", 3, ("event", 1 if capturing else 2)), ("launch", 3)]


# ---- on the GPU: the blocks that the operators get are ones that the current stream has freed
# while work that writes NaN into them is still queued on it ----
def _busy(sizes):
    """Frees blocks of these many bytes with such work pending; their addresses."""
    a = torch.ones(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    for _ in range(60):
        a = (a @ a).clamp(max=1.0)
    for b in blocks:
        b.fill_(0xFF)
    return {b.data_ptr() for b in blocks}


@pytest.mark.gpu
@pytest.mark.parametrize("n,rows,cols", [(16, 256, 384), (64, 128, 64)])
def test_orth_first_used_on_another_stream(n, rows, cols):
    from combine_top_router_amd import Orthogonalizer
    g = torch.randn(n, rows, cols, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want = Orthogonalizer(n, rows, cols).update(g).clone()
    op, side = Orthogonalizer(n, rows, cols), torch.cuda.Stream()
    torch.cuda.synchronize()
    ptrs = _busy([g.numel() * 2])
    got = op.update(g, stream=side)
    torch.cuda.synchronize()
    assert got.data_ptr() in ptrs and torch.equal(got, want)
    # made while the memory is busy, first called on the other stream
    ptrs = _busy([op.scratch.numel()])
    op = Orthogonalizer(n, rows, cols)
    got = op.update(g, out=got, stream=side)
    torch.cuda.synchronize()
    assert op.scratch.data_ptr() in ptrs and torch.equal(got, want)


@pytest.mark.gpu
def test_norm_and_balance_first_used_on_another_stream():
    from combine_top_router_amd import BalanceLoss, MoeNorm
    gen = torch.Generator().manual_seed(2)
    T, H, E, k = 2048, 1024, 64, 4
    x, w = torch.randn(T, H, generator=gen).bfloat16().cuda(), torch.ones(H).bfloat16().cuda()
    logits = torch.randn(T, E, generator=gen).cuda()
    idx = torch.topk(logits, k, dim=1).indices.int()
    want_y = MoeNorm(T, H).forward(x, w).clone()
    b = BalanceLoss(T, E, k)
    want_loss, want_counts = b.forward(logits, idx, 0.1).clone(), b.counts.clone()
    want_d = b.backward().clone()
    side = torch.cuda.Stream()
    ptrs = _busy([T * H * 2] * 3)
    op = MoeNorm(T, H)
    y = op.forward(x, w, stream=side)
    torch.cuda.synchronize()
    assert y.data_ptr() in ptrs and torch.equal(y, want_y)
    ptrs = _busy([512] * 3 + [T * E * 4, b.scratch.numel()])   # in the order of the operator's own
    op = BalanceLoss(T, E, k)
    loss = op.forward(logits, idx, 0.1, stream=side)
    d = op.backward(stream=side)
    torch.cuda.synchronize()
    assert {loss.data_ptr(), d.data_ptr()} & ptrs
    assert torch.equal(loss, want_loss) and torch.equal(op.counts, want_counts) and torch.equal(d, want_d)


@pytest.mark.gpu
def test_layer_balance_and_orthogonalize_first_used_on_another_stream():
    from combine_top_router_amd import MoeLayer
    gen = torch.Generator().manual_seed(3)
    T, H, I, E, k = 256, 256, 512, 8, 2
    randn = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()  # noqa: E731
    logits = torch.randn(T, E, generator=gen).cuda()
    x, dy = randn(T, H), randn(T, H)
    wg, wu, wd = randn(E, H, I) / 16, randn(E, H, I) / 16, randn(E, I, H) / 16

    def step(lay, side, busy):
        lay.forward(logits, x, wg, wu, wd, stream=side)
        ptrs = busy([512] * 3 + [T * E * 4])
        loss = lay.balance(0.1, stream=side)
        g = lay.backward(dy, stream=side)
        if ptrs:
            assert loss.data_ptr() in ptrs
        ptrs = busy([E * H * I * 2] * 3)
        up = lay.orthogonalize(stream=side)
        torch.cuda.synchronize()
        if ptrs:
            assert up["gate"].data_ptr() in ptrs
        return {"loss": loss, "counts": lay.balance_counts, "d_logits": g["d_logits"], **up}

    want = {n: v.clone() for n, v in step(MoeLayer(T, H, I, E, k), None, lambda sizes: None).items()}
    lay, side = MoeLayer(T, H, I, E, k), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = step(lay, side, _busy)
    for n, v in got.items():
        assert torch.equal(v, want[n]), n


@pytest.mark.gpu
def test_orth_first_used_in_a_capture():
    """The operator is made, and its result allocated, inside a capture; then used on other streams."""
    from combine_top_router_amd import Orthogonalizer
    g = torch.randn(4, 96, 200, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    want = Orthogonalizer(4, 96, 200).update(g).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op = Orthogonalizer(4, 96, 200)
        out = op.update(g)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_()
        assert torch.equal(op.update(g), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    op.update(g, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
