"""The norm, the router, the layer, the balance loss, the backward and the orthogonalised
updates run together, as a training step runs them: the results are those of the parts, also
on another stream and as a captured graph replayed with eager work in between."""
import numpy as np
import pytest
import torch

import workloads as wl
from oracle import train as ot
from gpu_util import BF16_TOL, rel, to_dev

pytestmark = pytest.mark.gpu

T, H, I, E, K = 200, 128, 64, 8, 2
COEF = 0.05


class Step:
    def __init__(self, seed=0):
        import combine_top_router_amd as moe
        self.moe = moe
        cfg = wl.CONFIGS["tiny_bf16"].replace(T=T, H=H, I=I, E=E, k=K, e_local=E, seed=seed)
        self.inp = wl.make_inputs(cfg)
        g = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16
        self.h = to_dev(self.inp["x"], bf)
        self.attn = torch.randn(T, H, generator=g).to(bf).cuda()
        self.w = (1 + 0.1 * torch.randn(H, generator=g)).to(bf).cuda()
        self.ds = torch.randn(T, H, generator=g).to(bf).cuda()
        self.w_r = (torch.randn(H, E, generator=g) / H ** 0.5).to(bf).cuda()
        self.wg, self.wu, self.wd = (to_dev(self.inp[n], bf) for n in ("w_gate", "w_up", "w_down"))
        self.dy = to_dev(self.inp["dy"], bf)
        self.mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8).cuda()
        self.norm = moe.MoeNorm(T, H, kind=moe.MOE_NORM_RMS, eps=1e-6)
        self.layer = moe.MoeLayer(T, H, I, E, K)
        self.logits = torch.empty(T, E, device="cuda")
        self.idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
        self.wk = torch.empty(T, K, device="cuda")
        self.dx = torch.empty(T, H, dtype=bf, device="cuda")
        self.dw_r = torch.empty(H, E, dtype=bf, device="cuda")

    def __call__(self):
        L, lay = self.moe.lib, self.layer
        st = torch.cuda.current_stream().cuda_stream
        p = lambda t: t.data_ptr()  # noqa: E731
        x = self.norm.forward(self.h, self.w, res=self.attn)
        L.moe_router_fwd(lay.shape, p(x), p(self.w_r), p(self.logits), p(self.idx), p(self.wk), p(lay.scratch), st)
        y = lay.forward(self.logits, x, self.wg, self.wu, self.wd)
        loss = lay.balance(COEF, mask=self.mask)
        g = lay.backward(self.dy)
        L.moe_router_bwd(lay.shape, p(x), p(self.w_r), p(g["d_logits"]), p(g["dx"]), p(self.dx), p(self.dw_r),
                         p(lay.scratch), st)
        n = self.norm.backward(self.dx, ds_in=self.ds)
        up = lay.orthogonalize()
        return {"y": y, "loss": loss, "counts": lay.balance_counts, "d_logits": g["d_logits"], "dw_r": self.dw_r,
                "dh": n["dx"], "dw": n["dw"], "o_gate": up["gate"], "o_up": up["up"], "o_down": up["down"]}


def _copy(out):
    torch.cuda.synchronize()
    return {k: v.clone() for k, v in out.items()}


def test_step_is_its_parts():
    s = Step()
    out = _copy(s())
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    lay = s.layer
    # the balance loss of the routing that ran, and its gradient on top of the routing's own
    loss, counts, _ = ot.balance_forward(n(s.logits), lay.topk_idx.cpu().numpy(), s.mask.cpu().numpy(), COEF)
    assert np.array_equal(out["counts"].cpu().numpy(), counts)
    assert float(out["loss"]) == pytest.approx(loss, rel=1e-5)
    routing = om_route_bwd(n(s.logits), lay)
    want = ot.balance_backward(n(s.logits), counts, K, s.mask.cpu().numpy(), COEF, 1.0, routing)
    assert rel(n(out["d_logits"]), want) < 1e-4
    # the norm's backward of what the router's backward gave
    dx, dw, _ = ot.norm_backward(n(s.dx), n(s.h) + n(s.attn), n(s.w), np.zeros(T), n(s.norm.rstd), n(s.ds), True)
    assert rel(n(out["dh"]), dx) < BF16_TOL and rel(n(out["dw"]), dw) < BF16_TOL
    for name, g in (("o_gate", lay.dw_gate), ("o_up", lay.dw_up), ("o_down", lay.dw_down)):
        for e in (0, E - 1):
            assert rel(n(out[name][e]), ot.orthogonalize(n(g[e]), 5)) < BF16_TOL, name


def om_route_bwd(logits, lay):
    """d_logits of the routing weights alone (softmax over the selected)."""
    idx = lay.topk_idx.cpu().numpy()
    w, dw = lay.topk_w.double().cpu().numpy(), lay.d_topk_w.double().cpu().numpy()
    d = np.zeros_like(logits)
    g = w * (dw - (w * dw).sum(axis=1, keepdims=True))
    np.put_along_axis(d, idx.astype(np.int64), g, axis=1)
    return d


def test_step_without_a_balance_loss_is_as_before():
    s = Step()
    s()
    lay = s.layer
    lay.forward(s.logits, s.norm.y, s.wg, s.wu, s.wd)
    g = lay.backward(s.dy)
    torch.cuda.synchronize()
    assert rel(g["d_logits"].double().cpu().numpy(), om_route_bwd(s.logits.double().cpu().numpy(), lay)) < 1e-5


def test_step_on_another_stream():
    s = Step()
    want = _copy(s())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = s()
    torch.cuda.current_stream().wait_stream(side)
    for k, v in _copy(got).items():
        assert torch.equal(v, want[k]), k


def test_step_as_a_graph():
    s = Step()
    want = _copy(s())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s()
    other = Step(seed=5)
    for i in range(3):
        for v in out.values():
            v.zero_()
        graph.replay()
        for k, v in _copy(out).items():
            assert torch.equal(v, want[k]), (i, k)
        other()   # eager work of the same kinds, with buffers of its own
        s()       # and on the graph's own buffers
        torch.cuda.synchronize()
