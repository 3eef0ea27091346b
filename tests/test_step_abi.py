"""Refusals of the routing by scores, the matrix product and AdamW: checked on the host before
any launch (no GPU needed; the pointers are never read)."""
import ctypes
import math
import os

import pytest
import torch

P = 4096  # a pointer that is not NULL


def _lib():
    from combine_top_router_amd import lib as L
    if not os.path.exists(L.lib_path()):
        pytest.skip("libmoe.so not built")
    return L


def _code(call):
    with pytest.raises(Exception) as e:
        call()
    return e.value.code


def _gate(L, **kw):
    base = dict(T=4, E=12, k=3, score=L.MOE_SCORE_SOFTMAX, groups=3, topk_groups=2, group_top=2, renorm=1, scale=1.0)
    base.update(kw)
    return L.MoeGateShape(**base)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17, E=96), dict(k=9),
                                 dict(score=2), dict(groups=0), dict(groups=5), dict(groups=65, E=130),
                                 dict(topk_groups=0), dict(topk_groups=4), dict(group_top=0), dict(group_top=3),
                                 dict(groups=12, group_top=2), dict(renorm=2), dict(scale=0.0), dict(scale=-1.0),
                                 dict(scale=math.nan), dict(scale=math.inf), dict(T=1 << 30)])
def test_gate_shapes(bad):
    L = _lib()
    s = _gate(L, **bad)
    assert _code(lambda: L.moe_gate_scratch_bytes(s)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_gate_fwd(s, P, 0, 0, P, P, 0, 0)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_gate_bwd(s, P, P, P, 2 * P)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_gate_update_bias(s, P, P, 0.1, P)) == L.MOE_EINVAL


def test_gate_pointers():
    L = _lib()
    s = _gate(L)
    assert L.moe_gate_scratch_bytes(s) > 0 and L.moe_gate_scratch_bytes(_gate(L, T=0)) > 0
    good = dict(logits=P, bias=0, mask=0, topk_idx=P, topk_w=P, counts=0, scratch=0)
    for name in ("logits", "topk_idx", "topk_w"):
        assert _code(lambda: L.moe_gate_fwd(s, *dict(good, **{name: 0}).values())) == L.MOE_EINVAL, name
    assert _code(lambda: L.moe_gate_fwd(s, *dict(good, counts=P).values())) == L.MOE_EWORKSPACE
    good = dict(logits=P, topk_idx=P, d_topk_w=P, d_logits=2 * P)
    for name in good:
        assert _code(lambda: L.moe_gate_bwd(s, *dict(good, **{name: 0}).values())) == L.MOE_EINVAL, name
    assert _code(lambda: L.moe_gate_bwd(s, *dict(good, d_logits=P).values())) == L.MOE_EINVAL   # is logits
    good = dict(counts=P, bias=P, rate=0.1, out=P)
    for name in ("counts", "bias", "out"):
        assert _code(lambda: L.moe_gate_update_bias(s, *dict(good, **{name: 0}).values())) == L.MOE_EINVAL, name
    for rate in (math.nan, math.inf):
        assert _code(lambda: L.moe_gate_update_bias(s, *dict(good, rate=rate).values())) == L.MOE_EINVAL
    L.moe_gate_fwd(_gate(L, T=0), 0, 0, 0, 0, 0, 0, 0)   # no tokens: nothing to do
    L.moe_gate_bwd(_gate(L, T=0), 0, 0, 0, 0)


def _linear(L, **kw):
    base = dict(T=4, K=8, N=16, dtype=L.MOE_BF16, act=L.MOE_ACT_SILU)
    base.update(kw)
    return L.MoeLinearShape(**base)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(K=0), dict(N=0), dict(K=(1 << 20) + 1), dict(N=(1 << 20) + 1),
                                 dict(dtype=2), dict(act=-1), dict(act=4)])
def test_linear_shapes(bad):
    L = _lib()
    s = _linear(L, **bad)
    assert _code(lambda: L.moe_linear_scratch_bytes(s)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_linear_fwd(s, P, P, 0, 0, 0, 2 * P, P)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_linear_bwd(s, P, P, P, P, 0, 2 * P, P, 0, P)) == L.MOE_EINVAL


def test_linear_pointers():
    L = _lib()
    s = _linear(L)
    assert L.moe_linear_scratch_bytes(s) > 0 and L.moe_linear_scratch_bytes(_linear(L, T=0, act=0)) > 0
    good = dict(x=P, w=P, b=0, res=0, z=0, y=2 * P, scratch=P)
    for name in ("x", "w", "y"):
        assert _code(lambda: L.moe_linear_fwd(s, *dict(good, **{name: 0}).values())) == L.MOE_EINVAL, name
    assert _code(lambda: L.moe_linear_fwd(s, *dict(good, scratch=0).values())) == L.MOE_EWORKSPACE
    for same in (dict(y=P), dict(z=2 * P), dict(z=P), dict(z=3 * P, res=3 * P)):
        assert _code(lambda: L.moe_linear_fwd(s, *dict(good, **same).values())) == L.MOE_EINVAL, same
    good = dict(dy=P, x=2 * P, w=3 * P, z=4 * P, dx_in=0, dx=5 * P, dw=6 * P, db=0, scratch=P)
    for name in ("dy", "x", "w", "z", "dw"):
        assert _code(lambda: L.moe_linear_bwd(s, *dict(good, **{name: 0}).values())) == L.MOE_EINVAL, name
    assert _code(lambda: L.moe_linear_bwd(s, *dict(good, scratch=0).values())) == L.MOE_EWORKSPACE
    for name in ("dy", "x", "z"):
        assert _code(lambda: L.moe_linear_bwd(s, *dict(good, dx=good[name]).values())) == L.MOE_EINVAL, name
    assert _code(lambda: L.moe_linear_bwd(s, *dict(good, dx=0, dx_in=P).values())) == L.MOE_EINVAL
    L.moe_linear_fwd(_linear(L, T=0), 0, 0, 0, 0, 0, 0, 0)


def _params(L, **kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=1, seed=0, state=L.MOE_STATE_F32,
                stochastic=0)
    base.update(kw)
    return L.MoeAdamwParams(**base)


def _tensor(L, **kw):
    base = dict(p=P, g=P, master=0, m=P, v=P, m_scale=0, v_scale=0, n=4, at=0, p_dtype=L.MOE_BF16, g_dtype=L.MOE_F32)
    base.update(kw)
    return (L.MoeAdamwTensor * 1)(L.MoeAdamwTensor(**base))


@pytest.mark.parametrize("bad", [dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1),
                                 dict(beta2=1.0), dict(beta2=math.nan), dict(eps=0.0), dict(eps=-1.0),
                                 dict(eps=math.inf), dict(eps=1e-60), dict(eps=1e60), dict(weight_decay=math.nan),
                                 dict(step=0), dict(state=2), dict(stochastic=2)])
def test_adamw_params(bad):
    L = _lib()
    assert _code(lambda: L.moe_adamw(_params(L, **bad), _tensor(L), 1, 0, 0, 0)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_adamw(_params(L, **bad), None, 0, 0, 0, 0)) == L.MOE_EINVAL


@pytest.mark.parametrize("bad", [dict(n=-1), dict(at=-1), dict(p_dtype=2), dict(g_dtype=-1), dict(p=0), dict(m=0),
                                 dict(v=0), dict(m=P + 16), dict(v=P + 4), dict(p=P + 1), dict(g=P + 2),
                                 dict(master=P + 2), dict(p=P + 2, p_dtype=0)])
def test_adamw_tensors(bad):
    L = _lib()
    assert _code(lambda: L.moe_adamw(_params(L), _tensor(L, **bad), 1, 0, 0, 0)) == L.MOE_EINVAL


def test_adamw_arguments():
    L = _lib()
    for scales in (dict(), dict(m_scale=P), dict(v_scale=P)):
        assert _code(lambda: L.moe_adamw(_params(L, state=L.MOE_STATE_8BIT), _tensor(L, **scales), 1, 0, 0, 0)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_adamw(_params(L), _tensor(L), -1, 0, 0, 0)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_adamw(_params(L), None, 1, 0, 0, 0)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_adamw(_params(L), _tensor(L), 1, 0, 0, P + 4)) == L.MOE_EINVAL   # the clock's place
    # nothing to do: no tensors, no gradient, no elements
    L.moe_adamw(_params(L), None, 0, 0, 0, 0)
    L.moe_adamw(_params(L), _tensor(L, g=0), 1, 0, 0, 0)
    L.moe_adamw(_params(L), _tensor(L, n=0), 1, 0, 0, 0)


def test_null_shapes():
    raw = ctypes.CDLL(_lib().lib_path())
    n = ctypes.c_size_t(0)
    for f in ("moe_gate_scratch_bytes", "moe_linear_scratch_bytes"):
        assert getattr(raw, f)(None, ctypes.byref(n)) == -1
        assert getattr(raw, f)(None, None) == -1
    assert raw.moe_adamw(None, None, 0, None, None, None, None) == -1


# ---- the classes ----
def test_classes_refuse_calls_out_of_order():
    L = _lib()
    from combine_top_router_amd import Gate, Linear, MoeLayer
    g = Gate(4, 8, 2, device="cpu")
    with pytest.raises(RuntimeError):
        g.backward(torch.zeros(4, 2))
    with pytest.raises(RuntimeError):
        g.update_bias(torch.zeros(8), 0.1)
    lin = Linear(4, 8, 16, device="cpu")
    with pytest.raises(RuntimeError):
        lin.backward(torch.zeros(4, 16, dtype=torch.bfloat16))
    with pytest.raises(RuntimeError):
        Linear(4, 8, 16, train=False, device="cpu").backward(torch.zeros(4, 16, dtype=torch.bfloat16))
    for other in (Gate(5, 8, 2, device="cpu"), Gate(4, 16, 2, device="cpu"), Gate(4, 8, 1, device="cpu")):
        with pytest.raises(ValueError, match="gate"):
            MoeLayer(4, 64, 64, 8, 2, device="cpu", gate=other)
    lay = MoeLayer(4, 64, 64, 8, 2, device="cpu", gate=g)
    assert lay.topk_idx is g.topk_idx and lay.topk_w is g.topk_w
    plain = MoeLayer(4, 64, 64, 8, 2, device="cpu")
    for kw in (dict(bias=torch.zeros(8)), dict(mask=torch.zeros(4, dtype=torch.uint8)), dict(count=True)):
        with pytest.raises(ValueError, match="gate"):
            plain.route(torch.zeros(4, 8), **kw)
    with pytest.raises(L.MoeError):
        Gate(4, 8, 9, device="cpu")


def test_adamw_refuses_parameters():
    L = _lib()
    from combine_top_router_amd import AdamW
    a = torch.zeros(64)
    for bad in ([], [a.double()], [torch.zeros(4, 4).t()[1:]], [a, a], [a[:40], a[32:]], [a, a[:1]]):
        with pytest.raises(ValueError):
            AdamW(bad)
    for kw in (dict(betas=(1.0, 0.9)), dict(eps=0.0), dict(state=3), dict(weight_decay=math.nan)):
        with pytest.raises(L.MoeError):
            AdamW([a], **kw)
    op = AdamW([a[:32], a[32:], torch.zeros(0)], master=True)
    assert op.master == [None, None, None] and op.t == 0
    for grads in ([a], [a[:32], a[32:], None, None]):
        with pytest.raises(ValueError, match="expected 3"):
            op.step(grads, 0.1)
    for g in (a[:31], a[:32].half(), a[:32].view(4, 8)):
        with pytest.raises(ValueError, match=r"grads\[0\]"):
            op.step([g, None, None], 0.1)
    assert op.t == 0


@pytest.mark.parametrize("K,N", [(64, 128), (33, 7), (1 << 20, 1 << 20)])
@pytest.mark.parametrize("T", [0, 1, 2 ** 31 - 1])
@pytest.mark.parametrize("act", [0, 3])
def test_linear_scratch_of_the_extremes(T, K, N, act):
    """No division by what may be 0, no size that wraps."""
    L = _lib()
    for dtype in (L.MOE_BF16, L.MOE_F32):
        n = L.moe_linear_scratch_bytes(_linear(L, T=T, K=K, N=N, dtype=dtype, act=act))
        assert n >= (T * N * (2 if dtype else 4) if act else 1)


def test_linear_outputs_apart():
    """What is written lies apart from what the call reads after it."""
    L = _lib()
    s = _linear(L)
    fwd = dict(x=P, w=2 * P, b=0, res=0, z=0, y=3 * P, scratch=P)
    for same in (dict(y=2 * P), dict(z=2 * P)):
        assert _code(lambda: L.moe_linear_fwd(s, *dict(fwd, **same).values())) == L.MOE_EINVAL, same
    bwd = dict(dy=P, x=2 * P, w=3 * P, z=4 * P, dx_in=0, dx=5 * P, dw=6 * P, db=0, scratch=P)
    assert _code(lambda: L.moe_linear_bwd(s, *dict(bwd, dx=3 * P).values())) == L.MOE_EINVAL
    for name in ("dy", "x", "w", "z", "dx"):
        assert _code(lambda: L.moe_linear_bwd(s, *dict(bwd, dw=bwd[name]).values())) == L.MOE_EINVAL, name


def test_a_gate_is_one_layers():
    _lib()
    from combine_top_router_amd import Gate, MoeLayer
    g = Gate(4, 8, 2, device="cpu")
    lay = MoeLayer(4, 64, 64, 8, 2, device="cpu", gate=g)
    with pytest.raises(ValueError, match="another layer"):
        MoeLayer(4, 64, 64, 8, 2, device="cpu", gate=g)
    del lay
    MoeLayer(4, 64, 64, 8, 2, device="cpu", gate=g)
