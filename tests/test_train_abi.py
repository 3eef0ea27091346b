"""Refusals of the norm, the balance loss and the orthogonalised update: checked on the host
before any launch (no GPU needed; the pointers are never read)."""
import ctypes
import math
import os

import pytest

P = 4096  # a pointer that is not NULL


def _lib():
    from combine_top_router_amd import lib as L
    if not os.path.exists(L.lib_path()):
        pytest.skip("libmoe.so not built")
    return L


def _norm(L, **kw):
    base = dict(T=4, H=64, dtype=L.MOE_BF16, kind=L.MOE_NORM_LAYER, eps=1e-5)
    base.update(kw)
    return L.MoeNormShape(**base)


def _orth(L, **kw):
    base = dict(n=2, rows=64, cols=32, dtype=L.MOE_BF16, steps=5)
    base.update(kw)
    return L.MoeOrthShape(**base)


def _route(L, **kw):
    base = dict(T=4, H=64, I=64, E=8, k=2, e_begin=0, e_local=8, dtype=L.MOE_BF16, bwd=0, renorm=1)
    base.update(kw)
    return L.MoeShape(**base)


def _code(call):
    with pytest.raises(Exception) as e:
        call()
    return e.value.code


@pytest.mark.parametrize("bad", [dict(T=-1), dict(H=0), dict(H=(1 << 20) + 1), dict(dtype=2), dict(kind=2),
                                 dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf)])
def test_norm_shapes(bad):
    L = _lib()
    s = _norm(L, **bad)
    assert _code(lambda: L.moe_norm_scratch_bytes(s)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_norm_fwd(s, P, 0, P, 0, 0, P, P, P)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_norm_bwd(s, P, P, 0, P, P, P, 0, P, P, 0, P)) == L.MOE_EINVAL


def test_norm_pointers():
    L = _lib()
    s = _norm(L)
    good = dict(x=P, res=0, w=P, b=0, sum=0, y=2 * P, mean=P, rstd=P)
    for name in ("x", "w", "y", "mean", "rstd"):
        a = dict(good, **{name: 0})
        assert _code(lambda: L.moe_norm_fwd(s, *a.values())) == L.MOE_EINVAL, name
    assert _code(lambda: L.moe_norm_fwd(s, *dict(good, res=P).values())) == L.MOE_EINVAL      # res without sum
    assert _code(lambda: L.moe_norm_fwd(s, *dict(good, sum=P).values())) == L.MOE_EINVAL      # sum without res
    assert _code(lambda: L.moe_norm_fwd(s, *dict(good, res=P, sum=2 * P).values())) == L.MOE_EINVAL   # y is sum
    good = dict(dy=P, s=2 * P, res=0, w=P, mean=P, rstd=P, ds_in=0, dx=3 * P, dw=P, db=0, scratch=P)
    for name in ("dy", "s", "w", "mean", "rstd", "dx", "dw"):
        a = dict(good, **{name: 0})
        assert _code(lambda: L.moe_norm_bwd(s, *a.values())) == L.MOE_EINVAL, name
    assert _code(lambda: L.moe_norm_bwd(s, *dict(good, scratch=0).values())) == L.MOE_EWORKSPACE
    for name in ("dy", "s", "res"):
        a = dict(good, res=4 * P)
        a["dx"] = a[name]
        assert _code(lambda: L.moe_norm_bwd(s, *a.values())) == L.MOE_EINVAL
    L.moe_norm_fwd(_norm(L, T=0), 0, 0, 0, 0, 0, 0, 0, 0)   # no rows: nothing to do


@pytest.mark.parametrize("bad", [dict(n=-1), dict(n=65536), dict(rows=0), dict(cols=0), dict(rows=16385),
                                 dict(cols=16385), dict(dtype=3), dict(steps=0), dict(steps=7)])
def test_orth_shapes(bad):
    L = _lib()
    s = _orth(L, **bad)
    assert _code(lambda: L.moe_orth_scratch_bytes(s)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_orthogonalize(s, P, P, 1.0, P)) == L.MOE_EINVAL


def test_orth_arguments():
    L = _lib()
    s = _orth(L)
    assert L.moe_orth_scratch_bytes(s) > 0
    assert _code(lambda: L.moe_orthogonalize(s, 0, P, 1.0, P)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_orthogonalize(s, P, 0, 1.0, P)) == L.MOE_EINVAL
    assert _code(lambda: L.moe_orthogonalize(s, P, P, 1.0, 0)) == L.MOE_EWORKSPACE
    for v in (math.nan, math.inf):
        assert _code(lambda: L.moe_orthogonalize(s, P, 2 * P, v, P)) == L.MOE_EINVAL
    f = _orth(L, dtype=L.MOE_F32)
    assert _code(lambda: L.moe_orthogonalize(f, P, P, 1.0, P)) == L.MOE_EINVAL   # o is g, of another type
    L.moe_orthogonalize(_orth(L, n=0), 0, 0, 1.0, 0)


def test_balance_arguments():
    L = _lib()
    s = _route(L)
    assert L.moe_balance_scratch_bytes(s) > 0
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9)):
        b = _route(L, **bad)
        assert _code(lambda: L.moe_balance_scratch_bytes(b)) == L.MOE_EINVAL
        assert _code(lambda: L.moe_balance_fwd(b, P, P, 0, 1.0, P, P, P, P)) == L.MOE_EINVAL
        assert _code(lambda: L.moe_balance_bwd(b, P, P, 0, 1.0, 0, 0, 2 * P)) == L.MOE_EINVAL
    good = dict(logits=P, topk_idx=P, mask=0, coef=1.0, loss=P, counts=P, prob=P, scratch=P)
    for name in ("logits", "topk_idx", "loss", "counts", "prob"):
        a = dict(good, **{name: 0})
        assert _code(lambda: L.moe_balance_fwd(s, *a.values())) == L.MOE_EINVAL, name
    assert _code(lambda: L.moe_balance_fwd(s, *dict(good, scratch=0).values())) == L.MOE_EWORKSPACE
    assert _code(lambda: L.moe_balance_fwd(s, *dict(good, coef=math.nan).values())) == L.MOE_EINVAL
    good = dict(logits=P, counts=P, mask=0, coef=1.0, d_loss=0, d_in=0, d_logits=2 * P)
    for name in ("logits", "counts", "d_logits"):
        a = dict(good, **{name: 0})
        assert _code(lambda: L.moe_balance_bwd(s, *a.values())) == L.MOE_EINVAL, name
    assert _code(lambda: L.moe_balance_bwd(s, *dict(good, d_logits=P).values())) == L.MOE_EINVAL   # is logits
    assert _code(lambda: L.moe_balance_bwd(s, *dict(good, coef=math.inf).values())) == L.MOE_EINVAL
    L.moe_balance_bwd(_route(L, T=0), 0, 0, 0, 1.0, 0, 0, 0)


def test_null_shapes_and_sizes():
    raw = ctypes.CDLL(_lib().lib_path())
    n = ctypes.c_size_t(0)
    for f in ("moe_norm_scratch_bytes", "moe_orth_scratch_bytes", "moe_balance_scratch_bytes"):
        assert getattr(raw, f)(None, ctypes.byref(n)) == -1
        assert getattr(raw, f)(None, None) == -1
