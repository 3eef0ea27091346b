"""A block's training step with the operators together: projection with bias and residual, norm,
router GEMM, routing by scores in the layer, all the backward, the AdamW step of what is no
expert, the orthogonalised update of the experts and the step of the routing's bias.

Each stage's result is one or two roundings to bf16 (2.3e-3 of its norm each at most: 2^-8 / sqrt 3)
on top of its input's; the longest chain, to the projection's gradients, has ten: 7.2e-3, and three
times that is the bound."""
import numpy as np
import pytest
import torch

from oracle import moe as om, step as os_, train as ot

pytestmark = pytest.mark.gpu

T, D, H, I, E, K = 192, 256, 128, 64, 16, 4
TOL = 2.2e-2
GATE = dict(groups=4, topk_groups=2, group_top=2, renorm=1, scale=2.0)


def _f(t):
    return t.detach().double().cpu().numpy()


def _rel(got, want):
    return np.linalg.norm(_f(got) - want) / np.linalg.norm(want)


class Block:
    """What a user's program holds of the block."""

    def __init__(self, seed=0):
        import combine_top_router_amd as moe
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        bf = lambda t: t.bfloat16().cuda()  # noqa: E731
        self.a, self.s0, self.dy = bf(rnd(T, D)), bf(rnd(T, H)), bf(rnd(T, H))
        self.mask = (torch.arange(T) % 12 != 0).to(torch.uint8).cuda()   # a padded batch
        self.p = {"w_o": bf(rnd(D, H) / 16), "b_o": bf(0.1 * rnd(H)), "w_n": bf(1 + 0.1 * rnd(H)),
                  "w_r": bf(rnd(H, E) / 11)}
        self.w = {"gate": bf(rnd(E, H, I) / 11), "up": bf(rnd(E, H, I) / 11), "down": bf(rnd(E, I, H) / 8)}
        self.bias = (0.05 * rnd(E)).cuda()
        self.linear = moe.Linear(T, D, H)
        self.norm = moe.MoeNorm(T, H, kind=moe.MOE_NORM_RMS, eps=1e-6)
        self.gate = moe.Gate(T, E, K, score=moe.MOE_SCORE_SIGMOID, **GATE)
        self.layer = moe.MoeLayer(T, H, I, E, K, gate=self.gate)
        self.logits = torch.empty(T, E, device="cuda")
        self.ids, self.tw = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
        self.dw_r = torch.empty_like(self.p["w_r"])
        self.adamw = moe.AdamW(list(self.p.values()), state=moe.MOE_STATE_8BIT, master=True, weight_decay=0.1,
                               stochastic=True, seed=4, capturable=True)

    def step(self):
        import combine_top_router_amd as moe
        lay, p, s = self.layer, self.p, torch.cuda.current_stream().cuda_stream
        s1 = self.linear.forward(self.a, p["w_o"], p["b_o"], res=self.s0)
        n = self.norm.forward(s1, p["w_n"])
        moe.moe_router_fwd(lay.shape, n.data_ptr(), p["w_r"].data_ptr(), self.logits.data_ptr(), self.ids.data_ptr(),
                           self.tw.data_ptr(), lay.scratch.data_ptr(), s)
        y = lay.forward(self.logits, n, self.w["gate"], self.w["up"], self.w["down"], bias=self.bias, mask=self.mask,
                        count=True)
        g = lay.backward(self.dy)
        moe.moe_router_bwd(lay.shape, n.data_ptr(), p["w_r"].data_ptr(), g["d_logits"].data_ptr(), g["dx"].data_ptr(),
                           g["dx"].data_ptr(), self.dw_r.data_ptr(), lay.scratch.data_ptr(), s)
        gn = self.norm.backward(g["dx"], ds_in=self.dy)   # the residual stream goes on past the layer
        gl = self.linear.backward(gn["dx"])
        self.adamw.step([gl["dw"], gl["db"], gn["dw"], self.dw_r], 1e-2)
        up = lay.orthogonalize()
        self.gate.update_bias(self.bias, 1e-2)
        return {"y": y, "s1": s1, "n": n, "logits": self.logits, "ids": self.gate.topk_idx, "tw": self.gate.topk_w,
                "counts": self.gate.counts, "d_logits": g["d_logits"], "dn": g["dx"], "dw_r": self.dw_r, "dw_n": gn["dw"],
                "dw_o": gl["dw"], "db_o": gl["db"], "da": gl["dx"], "ds0": gn["dx"], "up_gate": up["gate"],
                **{"dw_" + k: g["dw_" + k] for k in ("gate", "up", "down")}}


def test_block_step_against_the_oracle():
    b = Block()
    p = {k: _f(v) for k, v in b.p.items()}
    bias = b.bias.cpu().numpy().copy()
    mask = b.mask.cpu().numpy()
    out = b.step()
    torch.cuda.synchronize()
    # forward
    s1, _ = os_.linear_forward(_f(b.a), p["w_o"], p["b_o"], _f(b.s0), "none")
    n, s, mean, rstd = ot.norm_forward(s1, None, p["w_n"], None, 1e-6, True)
    assert _rel(out["s1"], s1) < TOL and _rel(out["n"], n) < TOL
    logits = out["logits"].cpu().numpy()
    assert _rel(out["logits"], om.router_logits(n, p["w_r"])) < TOL
    idx, tw, counts = os_.gate_forward(logits, bias, mask, K, os_.SIGMOID, **GATE)   # of the logits there are
    assert np.array_equal(out["ids"].cpu().numpy(), idx) and np.array_equal(out["counts"].cpu().numpy(), counts)
    assert (idx[mask == 0] == -1).all() and counts.sum() == K * mask.sum()
    inp = {"x": n, "dy": _f(b.dy), **{"w_" + k: _f(v) for k, v in b.w.items()}}
    y, saved = om.layer_forward(inp, K, 0, E, idx, tw)
    assert _rel(out["y"], y) < TOL and not out["y"][b.mask == 0].any()
    # backward
    ref = om.layer_backward(inp, K, 0, E, idx, tw, saved)
    for k in ("gate", "up", "down"):
        assert _rel(out["dw_" + k], ref["dw_" + k]) < TOL, k
    dl = os_.gate_backward(logits, idx, ref["d_topk_w"], os_.SIGMOID, GATE["renorm"], GATE["scale"])
    assert _rel(out["d_logits"], dl) < TOL
    dx, dw_r = om.router_gemm_backward(n, p["w_r"], dl)
    dn = ref["dx"] + dx
    assert _rel(out["dn"], dn) < TOL and _rel(out["dw_r"], dw_r) < TOL
    ds, dw_n, _ = ot.norm_backward(dn, s, p["w_n"], mean, rstd, _f(b.dy), True)
    assert _rel(out["ds0"], ds) < TOL and _rel(out["dw_n"], dw_n) < TOL
    da, dw_o, db_o, _ = os_.linear_backward(ds, _f(b.a), p["w_o"], s1, None, "none")
    assert _rel(out["da"], da) < TOL and _rel(out["dw_o"], dw_o) < TOL and _rel(out["db_o"], db_o) < TOL
    # the updates, of the gradients there are
    for i, (name, grad) in enumerate(zip(b.p, (out["dw_o"], out["db_o"], out["dw_n"], out["dw_r"]))):
        q, _, _ = os_.adamw(p[name], _f(grad), np.zeros(grad.shape), np.zeros(grad.shape), 1, 1e-2, 0.9, 0.999, 1e-8, 0.1)
        assert np.abs(_f(b.adamw.master[i]) - q).max() < 1e-6   # 20 u of values around 1
        assert torch.equal(b.p[name], b.adamw.master[i].bfloat16())
    assert np.array_equal(b.bias.cpu().numpy(), os_.gate_bias(bias, counts, 1e-2))
    up = np.stack([ot.orthogonalize(m, 5) for m in _f(out["dw_gate"])])
    assert _rel(out["up_gate"], up) < 1e-2 and b.adamw.t == 1


def test_block_steps_replayed():
    """The whole step as a graph: three replays are three eager steps, to the bit."""
    eager, captured = Block(), Block()
    for b in (eager, captured):   # first calls allocate
        b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = eager.step()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), k
        for x, y in zip(captured.adamw.params + [captured.adamw.m, captured.adamw.v, captured.bias],
                        eager.adamw.params + [eager.adamw.m, eager.adamw.v, eager.bias]):
            assert torch.equal(x, y)
    assert eager.adamw.t == captured.adamw.t == 4


@pytest.mark.parametrize("bounds", [(0, 16), (0, 5, 16)])
def test_gate_in_the_shares_of_a_layer(bounds):
    """Each share routes alike; y and d_logits are sums over the shares."""
    from combine_top_router_amd import Gate, MoeLayer
    b = Block(3)
    g = torch.Generator().manual_seed(5)
    logits, x = torch.randn(T, E, generator=g).cuda(), torch.randn(T, H, generator=g).bfloat16().cuda()
    y, dl = np.zeros((T, H)), np.zeros((T, E))
    for lo, hi in zip(bounds, bounds[1:]):
        lay = MoeLayer(T, H, I, E, K, e_begin=lo, e_local=hi - lo, gate=Gate(T, E, K, score=1, **GATE))
        w = [b.w[n][lo:hi].contiguous() for n in ("gate", "up", "down")]
        y += _f(lay.forward(logits, x, *w, bias=b.bias, mask=b.mask))
        lay.balance(0.0, mask=b.mask)   # counts the padded tokens out, and their ids of -1
        dl += _f(lay.backward(b.dy)["d_logits"])
        assert int(lay.balance_counts[E]) == int(b.mask.sum())
    idx, tw, _ = os_.gate_forward(logits.double().cpu().numpy(), b.bias.cpu().numpy(), b.mask.cpu().numpy(), K, 1, **GATE)
    inp = {"x": _f(x), "dy": _f(b.dy), **{"w_" + k: _f(v) for k, v in b.w.items()}}
    want, saved = om.layer_forward(inp, K, 0, E, idx, tw)
    ref = om.layer_backward(inp, K, 0, E, idx, tw, saved)
    d = os_.gate_backward(logits.double().cpu().numpy(), idx, ref["d_topk_w"], 1, 1, GATE["scale"])
    assert np.linalg.norm(y - want) < 1e-2 * np.linalg.norm(want)
    assert np.linalg.norm(dl - d) < 1e-2 * np.linalg.norm(d)
