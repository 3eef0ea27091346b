"""Routing by scores, the AdamW step and the matrix product with its epilogue, in plain numpy
fp64.  Shares no code with the HIP path."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["gate_forward", "gate_backward", "gate_bias", "linear_forward", "linear_backward", "activation", "adamw",
           "mix", "random_bits", "e4m3_grid", "scale_exponent", "bf16_stochastic"]

SOFTMAX, SIGMOID = 0, 1


# ---- routing by scores ----
def _scores(l, score):
    with np.errstate(invalid="ignore", over="ignore"):
        if score == SIGMOID:
            e = np.exp(-np.abs(l))
            return np.where(l >= 0, 1.0, e) / (1.0 + e)
        m = np.fmax.reduce(l)
        if m == -np.inf:
            return np.zeros_like(l)
        e = np.exp(l - m)
        return e / e.sum()


def _order(c):
    """Indices by c descending, ties to the lower; NaN behind all, as -inf."""
    c = np.where(np.isnan(c), -np.inf, c)
    return np.argsort(-c, kind="stable")


def _weights(l, s, ids, score, renorm, scale):
    if not renorm:
        return scale * s[ids]
    x = l[ids]
    if np.all(x == -np.inf):
        return np.zeros(len(ids))
    with np.errstate(invalid="ignore"):
        if score == SOFTMAX:
            q = np.exp(x - np.fmax.reduce(x)) + 0.0 * np.where(np.isnan(x), np.nan, 0.0)
        else:   # sigmoid(x) exp(-min(max x, 0))
            m = min(np.fmax.reduce(x), 0.0)
            q = np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(np.minimum(x, 0.0) - m) / (1.0 + np.exp(-np.abs(x))))
        return scale * q / q.sum()


def gate_forward(logits, bias, mask, k, score, groups=1, topk_groups=1, group_top=1, renorm=1, scale=1.0):
    """(topk_idx, topk_w, counts)."""
    T, E = logits.shape
    idx, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    per = E // groups
    for t in range(T):
        if mask is not None and mask[t] == 0:
            continue
        l = logits[t].astype(np.float64)
        s = _scores(l, score)
        c = s if bias is None else s + bias.astype(np.float64)
        c = np.where(np.isnan(l) | (l == -np.inf) | np.isnan(c), -np.inf, c)
        if bias is None:
            by = np.where(np.isnan(l), -np.inf, l)   # the scores rise with the logits
        else:
            by = c
        shown = np.arange(E)
        if groups > 1:
            if group_top == 1:
                g = by.reshape(groups, per).max(axis=1)
            else:
                with np.errstate(invalid="ignore"):
                    g = np.sort(c.reshape(groups, per), axis=1)[:, -2:].sum(axis=1)
            best = np.sort(_order(g)[:topk_groups])
            shown = np.concatenate([np.arange(b * per, (b + 1) * per) for b in best])
        ids = shown[_order(by[shown])[:k]]
        idx[t] = ids
        w[t] = _weights(l, s, ids, score, renorm, scale)
    live = idx[idx >= 0]
    return idx, w, np.bincount(live, minlength=E).astype(np.int32)


def gate_backward(logits, idx, d_w, score, renorm=1, scale=1.0):
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        on = (idx[t] >= 0) & (idx[t] < E)
        ids, d = idx[t][on], d_w[t][on].astype(np.float64)
        if not len(ids):
            continue
        l = logits[t].astype(np.float64)
        s = _scores(l, score)
        q = _weights(l, s, ids, score, renorm, 1.0)
        if renorm:
            g = scale * q * (d - (q * d).sum())
            if score == SIGMOID:
                g = g * _scores(-l[ids], SIGMOID)
            np.add.at(out[t], ids, g)
        elif score == SIGMOID:
            np.add.at(out[t], ids, scale * s[ids] * _scores(-l[ids], SIGMOID) * d)
        else:
            g = np.zeros(E)
            np.add.at(g, ids, d)
            out[t] = scale * s * (g - (s[ids] * d).sum())
    return out


def gate_bias(bias, counts, rate):
    n, E = int(counts.sum()), len(counts)
    return np.array([np.float32(b) + np.float32(rate) * np.float32(np.sign(n - E * int(c)))
                     for b, c in zip(bias, counts)], np.float32)


# ---- the matrix product ----
_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(z, act):
    """(act(z), act'(z)); act: "none", "relu", "silu", "gelu"."""
    if act == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return z * s, s + z * s * (1.0 - s)
    if act == "gelu":
        c = 0.5 * (1.0 + _erf(z / math.sqrt(2.0)))
        return z * c, c + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return z, np.ones_like(z)


def linear_forward(x, w, b, res, act):
    """(y, z)."""
    z = x.astype(np.float64) @ w.astype(np.float64)
    if b is not None:
        z = z + b
    y = activation(z, act)[0]
    return (y if res is None else y + res), z


def linear_backward(dy, x, w, z, dx_in, act):
    """(dx, dw, db, dz)."""
    dz = dy.astype(np.float64) * activation(z.astype(np.float64), act)[1]
    dx = dz @ w.astype(np.float64).T
    return (dx if dx_in is None else dx + dx_in), x.astype(np.float64).T @ dz, dz.sum(axis=0), dz


# ---- AdamW ----
def mix(v):
    """The output permutation of PCG (O'Neill 2014) on 32 bits, elementwise."""
    v = np.asarray(v, np.uint64) & np.uint64(0xFFFFFFFF)
    low = np.uint64(0xFFFFFFFF)
    s = (v * np.uint64(747796405) + np.uint64(2891336453)) & low
    w = (((s >> ((s >> np.uint64(28)) + np.uint64(4))) ^ s) * np.uint64(277803737)) & low
    return (w >> np.uint64(22)) ^ w


def random_bits(seed, t, at):
    """32 bits for each place `at` (an array of whole numbers) of step t."""
    low = 0xFFFFFFFF
    k = int(mix((t & low) + int(mix((seed & low) + int(mix(seed >> 32))))))
    at = np.asarray(at, np.uint64)
    return mix((at & np.uint64(low)) ^ mix((at >> np.uint64(32)) + np.uint64(k)))


def scale_exponent(amax):
    """Smallest X with amax <= 448 2^X, in -127..127; 0 for amax = 0."""
    if not amax > 0:
        return 0
    X = math.frexp(amax)[1] - 10
    while amax > math.ldexp(448.0, X):
        X += 1
    return max(-127, min(127, X))


def e4m3_grid(y, r16=None):
    """y >= 0 on E4M3's grid: to nearest, ties to even, or up where r16 / 2^16 is below the rest."""
    y = np.asarray(y, np.float64)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(y, 2.0 ** -20))), -6.0) - 3.0)
    n = y / step
    if r16 is None:
        return np.round(n) * step
    low = np.floor(n)
    return (low + (np.asarray(r16, np.float64) < (n - low) * 65536.0)) * step


def bf16_stochastic(x, r16):
    """fp32 x as bf16 values, after r16 was added below the 16 bits that stay."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    up = ((u + np.asarray(r16, np.uint64)) >> np.uint64(16)) << np.uint64(16)
    return up.astype(np.uint32).view(np.float32)


def adamw(p, g, m, v, t, lr, b1, b2, eps, wd, grad_scale=1.0):
    """(p, m, v) after step t."""
    g = g.astype(np.float64) * grad_scale
    m = b1 * m.astype(np.float64) + (1 - b1) * g
    v = b2 * v.astype(np.float64) + (1 - b2) * g * g
    step = (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p.astype(np.float64) * (1 - lr * wd) - lr * step, m, v
