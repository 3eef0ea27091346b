"""The operators around the layer in a training step, in plain numpy fp64: the norm with its
backward, the router's balance loss with its gradient, and the Newton-Schulz
orthogonalisation of an update.  Shares no code with the HIP path."""
from __future__ import annotations

import numpy as np

from . import mx

__all__ = ["norm_forward", "norm_backward", "balance_forward", "balance_backward", "orthogonalize",
           "orthogonalize_rounded"]


def norm_forward(x, res, w, b, eps, rms):
    """(y, s, mean, rstd): s = x + res; y = (s - mean) rstd w + b, mean = 0 for rms."""
    s = np.asarray(x, np.float64) + (0.0 if res is None else np.asarray(res, np.float64))
    mean = np.zeros(s.shape[0]) if rms else s.mean(axis=1)
    c = s - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    y = c * rstd[:, None] * np.asarray(w, np.float64)
    return y + (0.0 if b is None else np.asarray(b, np.float64)), s, mean, rstd


def norm_backward(dy, s, w, mean, rstd, ds_in, rms):
    """(dx, dw, db) from the forward's s, mean and rstd."""
    dy, s = np.asarray(dy, np.float64), np.asarray(s, np.float64)
    xh = (s - mean[:, None]) * rstd[:, None]
    g = dy * np.asarray(w, np.float64)
    dx = g - xh * (g * xh).mean(axis=1, keepdims=True)
    if not rms:
        dx = dx - g.mean(axis=1, keepdims=True)
    dx = dx * rstd[:, None]
    if ds_in is not None:
        dx = dx + np.asarray(ds_in, np.float64)
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def _softmax(logits):
    m = logits.max(axis=1, keepdims=True)
    e = np.exp(logits - np.where(np.isneginf(m), 0.0, m))
    z = e.sum(axis=1, keepdims=True)
    return np.divide(e, z, out=np.zeros_like(e), where=z != 0)


def balance_forward(logits, topk_idx, mask, coef):
    """(loss, counts [E + 1], prob [E]) over the tokens with mask != 0 (None: all)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    k = topk_idx.shape[1]
    on = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    n = int(on.sum())
    counts = np.zeros(E + 1, np.int64)
    for e in np.asarray(topk_idx)[on].reshape(-1):
        if 0 <= e < E:
            counts[e] += 1
    counts[E] = n
    if n == 0:
        return 0.0, counts, np.zeros(E)
    prob = _softmax(logits[on]).sum(axis=0) / n
    return coef * E / (k * n) * float((counts[:E] * prob).sum()), counts, prob


def balance_backward(logits, counts, k, mask, coef, d_loss, d_in):
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    d = np.zeros((T, E)) if d_in is None else np.asarray(d_in, np.float64).copy()
    on = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    n = int(counts[E])
    if n > 0 and on.any():
        c = np.asarray(counts[:E], np.float64)
        p = _softmax(logits[on])
        d[on] += d_loss * coef * E / (k * float(n) ** 2) * p * (c - (p * c).sum(axis=1, keepdims=True))
    return d


NS = (3.4445, -4.7750, 2.0315)


def orthogonalize(g, steps, scale=1.0):
    """One matrix."""
    a, b, c = NS
    x = np.asarray(g, np.float64)
    x = x / (np.sqrt((x * x).sum()) + 1e-7)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for _ in range(steps):
        q = x @ x.T
        x = a * x + (b * q + c * (q @ q)) @ x
    return scale * (x.T if tall else x)


def orthogonalize_rounded(g, steps, merged=False, fp32=False):
    """The same with the iterates held in fp16: the first two as pairs hi + lo, lo in E4M3
    times 16 (hi in the products, both in a X), A - I in place of A from the fourth step on,
    scales 2^15 (X; times 2^s where the norm is so far below 1e-7 that the iterates stay below
    2^-s) and 2^14.  fp32: g, too, enters as such a pair (bf16 values are fp16
    numbers times a power of two).  What this is off is what such a precision costs.  merged:
    the first two steps as one, in the square matrices, which saves products but costs more
    on matrices of a few strong rows (up to 2e-2, where step by step stays below 5e-3); the
    kernels go step by step."""
    def half(v, s):
        return (v * s).astype(np.float16).astype(np.float64) / s

    def pair(v):
        hi = half(v, more * 2.0 ** 15)
        lo = mx.e4m3_decode(mx.e4m3_encode((v - hi) * (more * 2.0 ** 19))) / (more * 2.0 ** 19)
        return hi, hi + lo

    a, b, c = NS
    x = np.asarray(g, np.float64)
    norm = np.sqrt((x * x).sum())
    hi = x
    if fp32 and norm > 0:   # as it enters, its norm in [2^14, 2^15)
        more = 2.0 ** -np.frexp(norm)[1]
        hi, x = pair(x)
    hi, x = hi / (norm + 1e-7), x / (norm + 1e-7)
    most = norm / (norm + 1e-7) * a ** (steps - 1)
    more = 2.0 ** max(0, -np.frexp(most)[1]) if most > 0 else 1.0
    tall = x.shape[0] > x.shape[1]
    if tall:
        hi, x = hi.T, x.T
    first, los = 0, 2
    if merged:
        r = half(hi @ hi.T, 2.0 ** 14)
        b0 = half(b * r + c * (r @ r), 2.0 ** 14)
        s = half(b0 @ r, 2.0 ** 14)
        a1 = half(a * a * r + 2 * a * s + b0 @ s, 2.0 ** 14)
        b1 = half(b * a1 + c * (a1 @ a1), 2.0 ** 14)
        p = half(a * b0 + a * b1 + b1 @ b0, 2.0 ** 12)
        x = a * a * x + p @ hi
        if steps > 2:
            hi, x = pair(x)
        first, los = 2, 1
    for i in range(first, steps):
        t = 1.0 if i >= 3 else 0.0
        d = half(hi @ hi.T - t * np.eye(len(x)), 2.0 ** 14)
        p = half((b + 2 * c * t) * d + c * (d @ d), 2.0 ** 14)
        x = (a + b * t + c * t * t) * x + p @ hi
        if i < steps - 1:
            if i - first < los - (1 if merged else 0):
                hi, x = pair(x)
            else:
                hi = x = half(x, more * 2.0 ** 15)
    return x.T if tall else x
