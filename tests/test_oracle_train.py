"""The fp64 oracle of the norm, the balance loss and the orthogonalised update, pinned by
differences, closed forms and invariants."""
import numpy as np
import pytest

from oracle import train as ot


def _diff(f, a, pos, h=1e-6):
    up, dn = a.copy(), a.copy()
    up[pos] += h
    dn[pos] -= h
    return (f(up) - f(dn)) / (2 * h)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients_against_differences(rms):
    r = np.random.default_rng(1)
    T, H = 4, 7
    x, res, w, b = r.normal(size=(T, H)), r.normal(size=(T, H)), r.normal(size=H), r.normal(size=H)
    dy, ds = r.normal(size=(T, H)), r.normal(size=(T, H))

    def goal(x_, res_, w_, b_):
        y, s, _, _ = ot.norm_forward(x_, res_, w_, b_, 1e-3, rms)
        return float((y * dy).sum() + (s * ds).sum())

    _, s, mean, rstd = ot.norm_forward(x, res, w, b, 1e-3, rms)
    dx, dw, db = ot.norm_backward(dy, s, w, mean, rstd, ds, rms)
    for pos in [(0, 0), (1, 3), (3, 6)]:
        assert dx[pos] == pytest.approx(_diff(lambda a: goal(a, res, w, b), x, pos), rel=1e-6, abs=1e-8)
        assert dx[pos] == pytest.approx(_diff(lambda a: goal(x, a, w, b), res, pos), rel=1e-6, abs=1e-8)
    for j in (0, 4, 6):
        assert dw[j] == pytest.approx(_diff(lambda a: goal(x, res, a, b), w, j), rel=1e-6, abs=1e-8)
        assert db[j] == pytest.approx(_diff(lambda a: goal(x, res, w, a), b, j), rel=1e-6, abs=1e-8)


def test_norm_rows_are_normalised():
    r = np.random.default_rng(2)
    x = r.normal(size=(5, 64)) * 3 + 1
    y, _, _, _ = ot.norm_forward(x, None, np.ones(64), None, 0.0, False)
    assert np.allclose(y.mean(axis=1), 0) and np.allclose(y.std(axis=1), 1)
    y, _, _, _ = ot.norm_forward(x, None, np.ones(64), None, 0.0, True)
    assert np.allclose((y * y).mean(axis=1), 1)


def test_balance_gradient_against_differences():
    r = np.random.default_rng(3)
    T, E, k = 6, 5, 2
    logits = r.normal(size=(T, E))
    idx = np.argsort(-logits, axis=1)[:, :k].astype(np.int32)
    mask = np.array([1, 1, 0, 1, 1, 0], np.uint8)
    _, counts, _ = ot.balance_forward(logits, idx, mask, 0.3)
    d = ot.balance_backward(logits, counts, k, mask, 0.3, 1.7, None)
    for pos in [(0, 0), (1, 4), (2, 1), (4, 3)]:   # the counts are constants
        want = 1.7 * _diff(lambda a: ot.balance_forward(a, idx, mask, 0.3)[0], logits, pos)
        assert d[pos] == pytest.approx(want, rel=1e-6, abs=1e-9)
    assert np.all(d[mask == 0] == 0)
    assert np.allclose(d.sum(axis=1), 0)


def test_balance_of_an_even_load_is_coef():
    T, E = 8, 4
    idx = (np.arange(T * 2).reshape(T, 2) % E).astype(np.int32)
    loss, counts, prob = ot.balance_forward(np.zeros((T, E)), idx, None, 0.25)
    assert loss == pytest.approx(0.25) and list(counts) == [4, 4, 4, 4, 8] and np.allclose(prob, 0.25)
    loss, counts, prob = ot.balance_forward(np.zeros((T, E)), idx, np.zeros(T), 0.25)
    assert loss == 0 and not counts.any() and not prob.any()


def test_orthogonalize_maps_singular_values():
    r = np.random.default_rng(4)
    g = r.normal(size=(6, 11))
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    p = s / (np.linalg.norm(g) + 1e-7)
    for _ in range(5):
        p = 3.4445 * p - 4.7750 * p ** 3 + 2.0315 * p ** 5
    assert np.allclose(ot.orthogonalize(g, 5), (u * p) @ vt)
    assert np.allclose(ot.orthogonalize(g.T, 5), ((u * p) @ vt).T)
    assert not ot.orthogonalize(np.zeros((3, 4)), 5).any()


def spectra(kind, m, l, seed):
    """Matrices as gradients come: flat spectra, a few strong directions, a power law."""
    r = np.random.default_rng(seed)
    if kind == "flat":
        return r.normal(size=(m, l))
    if kind == "low_rank":
        q = max(1, min(m, l) // 8)
        return r.normal(size=(m, q)) @ r.normal(size=(q, l)) + 0.1 * r.normal(size=(m, l))
    u = np.linalg.qr(r.normal(size=(m, min(m, l))))[0]
    v = np.linalg.qr(r.normal(size=(l, min(m, l))))[0]
    return (u * np.arange(1, min(m, l) + 1.0) ** -1) @ v.T


@pytest.mark.parametrize("merged", [False, True])
@pytest.mark.parametrize("kind", ["flat", "low_rank", "power"])
@pytest.mark.parametrize("m,l", [(64, 64), (96, 200), (200, 96), (64, 512)])
def test_the_precision_of_the_iterates_costs_little(kind, m, l, merged):
    g = spectra(kind, m, l, 5)
    want = ot.orthogonalize(g, 5)
    off = np.linalg.norm(ot.orthogonalize_rounded(g, 5, merged) - want) / np.linalg.norm(want)
    assert off < 2e-3
