"""The fp64 oracle of the routing by scores, the matrix product and AdamW: gradients against
differences, and the rules that its discrete parts follow."""
import numpy as np
import pytest

from oracle import step as os_


def _difference(f, x, i, h=1e-6):
    a, b = x.copy(), x.copy()
    a[i] += h
    b[i] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [0, 1])
def test_gate_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(1)
    T, E, k = 3, 12, 4
    l, d = rng.standard_normal((T, E)) * 2, rng.standard_normal((T, k))
    kw = dict(groups=3, topk_groups=2, group_top=2)
    bias = rng.standard_normal(E) * 0.05
    idx, _, _ = os_.gate_forward(l, bias, None, k, score, renorm=renorm, scale=2.5, **kw)

    def loss(x):
        i, w, _ = os_.gate_forward(x, bias, None, k, score, renorm=renorm, scale=2.5, **kw)
        assert np.array_equal(i, idx)
        return float((w * d).sum())

    g = os_.gate_backward(l, idx, d, score, renorm, 2.5)
    for t in range(T):
        for e in range(E):
            # central differences: 1e-12 of truncation, 1e-16 / 1e-6 of rounding
            assert abs(_difference(loss, l, (t, e)) - g[t, e]) < 1e-8


def test_gate_choice():
    l = np.array([[0.5, 3.0, 3.0, -np.inf, 1.0, 2.0]], np.float32)
    idx, w, counts = os_.gate_forward(l, None, None, 3, 0)
    assert idx.tolist() == [[1, 2, 5]] and counts.tolist() == [0, 1, 1, 0, 0, 1]
    assert np.isclose(w.sum(), 1)
    # a bias chooses and does not weigh
    idx, w, _ = os_.gate_forward(l, np.array([9, 0, 0, 9, 0, 0.0]), None, 2, 1, renorm=0)
    assert idx.tolist() == [[0, 1]]   # the masked expert ranks behind all, whatever its bias
    assert np.allclose(w, 1 / (1 + np.exp([[-0.5, -3.0]])))
    # groups: {0, 1}, {2, 3}, {4, 5} by the sum of two: sigmoid sums 1.57, 0.95, 1.61
    idx, _, _ = os_.gate_forward(l, None, None, 2, 1, groups=3, topk_groups=1, group_top=2)
    assert idx.tolist() == [[5, 4]]
    idx, w, counts = os_.gate_forward(l, None, np.zeros(1, np.uint8), 2, 0)
    assert idx.tolist() == [[-1, -1]] and not w.any() and not counts.any()
    assert os_.gate_bias(np.zeros(3), np.array([2, 5, 5]), 0.5).tolist() == [0.5, -0.5, -0.5]
    assert os_.gate_bias(np.zeros(2), np.array([4, 4]), 0.5).tolist() == [0, 0]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_linear_gradient_against_differences(act):
    rng = np.random.default_rng(2)
    x, w, b = rng.standard_normal((4, 5)), rng.standard_normal((5, 3)), rng.standard_normal(3)
    res, dy = rng.standard_normal((4, 3)), rng.standard_normal((4, 3))
    _, z = os_.linear_forward(x, w, b, res, act)
    dx, dw, db, _ = os_.linear_backward(dy, x, w, z, None, act)
    assert np.abs(z).min() > 1e-4   # away from relu's corner
    for i in np.ndindex(x.shape):
        assert abs(_difference(lambda a: float((os_.linear_forward(a, w, b, res, act)[0] * dy).sum()), x, i) - dx[i]) < 1e-7
    for i in np.ndindex(w.shape):
        assert abs(_difference(lambda a: float((os_.linear_forward(x, a, b, res, act)[0] * dy).sum()), w, i) - dw[i]) < 1e-7
    for i in np.ndindex(b.shape):
        assert abs(_difference(lambda a: float((os_.linear_forward(x, w, a, res, act)[0] * dy).sum()), b, i) - db[i]) < 1e-7


def test_grids_of_eight_bits():
    # every finite E4M3 value stays, halves go to even, and the scale takes the largest to 448 at most
    vals = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    vals = np.array([v for v in vals if v <= 448])
    assert np.array_equal(os_.e4m3_grid(vals), vals)
    mids = (vals[1:] + vals[:-1]) / 2
    near = os_.e4m3_grid(mids)
    assert all(n in (a, b) for n, a, b in zip(near, vals, vals[1:]))
    assert near[0] == 0 and near[1] == vals[2]
    assert np.array_equal(os_.e4m3_grid(mids, np.full(len(mids), 32767)), vals[1:])
    assert np.array_equal(os_.e4m3_grid(mids, np.full(len(mids), 32768)), vals[:-1])
    for a in (1.0, 448.0, 448.5, 1e-30, 3e38, 5.0):
        X = os_.scale_exponent(a)
        assert a <= 448 * 2.0 ** X and a > 448 * 2.0 ** (X - 1)


def test_stochastic_rounding_has_the_mean():
    """Over all places of many steps the rounded value's mean is the value."""
    n = 1 << 16
    r = np.concatenate([os_.random_bits(123 + (5 << 32), t, np.arange(n)) for t in (1, 2, 3, 4)])
    for half in (r & np.uint64(0xFFFF), r >> np.uint64(16), os_.mix(r) & np.uint64(0xFFFF)):
        assert abs(float(half.mean()) / 65535 - 0.5) < 5 * 0.289 / 2 ** 9   # five standard errors of 2^18 uniform ones
        q = os_.e4m3_grid(np.full(4 * n, 1.03), half)
        assert abs(q.mean() - 1.03) < 5 * 0.0625 / 2 ** 9
    x = np.full(n, 1.001, np.float32)
    assert abs(os_.bf16_stochastic(x, r[:n] & np.uint64(0xFFFF)).mean() - 1.001) < 5 * 0.004 / 2 ** 8


def test_adamw_first_step():
    """After one step from zero moments the update is the gradient's sign."""
    p, g = np.array([1.0, -2.0, 0.0]), np.array([0.5, -1e-3, 0.0])
    q, m, v = os_.adamw(p, g, np.zeros(3), np.zeros(3), 1, 0.1, 0.9, 0.99, 1e-12, 0.0)
    assert np.allclose(q, [0.9, -1.9, 0.0]) and np.allclose(m, 0.1 * g) and np.allclose(v, 0.01 * g * g)
