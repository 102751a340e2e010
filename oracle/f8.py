"""The operators of an expert layer in 8-bit floating point in fp64: routing,
quantisers, products with block scales, the experts' weighted sum (numpy only)."""
from __future__ import annotations

import numpy as np

TOP, B = 448.0, 128


def e4m3(v):
    """v rounded to the nearest e4m3 number (ties to even), +-448 past the ends."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    step = 2.0 ** (np.maximum(e, -6) - 3)   # 3 bits behind the leading one; 2^-9 below 2^-6
    return np.sign(v) * np.minimum(np.rint(a / step) * step, TOP)   # rint: halves to even


def blocks(n):
    return (n + B - 1) // B


def quotients(x, rows=1):
    """(x * 448 / max of its block, scales): blocks of `rows` rows x 128 columns."""
    x = np.asarray(x, np.float64)
    T, K = x.shape
    p = np.zeros((-(-T // rows) * rows, blocks(K) * B))
    p[:T, :K] = x
    p = p.reshape(-1, rows, blocks(K), B)
    top = np.abs(p).max(axis=(1, 3), keepdims=True)
    v = np.divide(p * TOP, top, out=np.zeros_like(p), where=top > 0)
    return v.reshape(-1, blocks(K) * B)[:T, :K], top[:, 0, :, 0] / TOP


def silu_up(x):
    """silu(gate) * up of rows [gate | up]."""
    x = np.asarray(x, np.float64)
    g, u = np.split(x, 2, axis=1)
    return g / (1 + np.exp(-g)) * u


def spread(s, rows, N, K):
    """Scales of blocks of `rows` x 128 at every element of [N][K]."""
    return np.repeat(np.repeat(np.asarray(s, np.float64), rows, axis=0)[:N], B, axis=1)[:, :K]


def linear(x, xs, w, ws, bias=None):
    """(out, sum of the absolute products): x [T][K], w [N][K] as numbers."""
    a = np.asarray(x, np.float64) * spread(xs, 1, *x.shape)
    b = np.asarray(w, np.float64) * spread(ws, B, *w.shape)
    out = a @ b.T
    return (out if bias is None else out + np.asarray(bias, np.float64)), np.abs(a) @ np.abs(b).T


def route(logits, k, renorm):
    """dict of idx, weight, offsets, perm, inv.  A NaN counts as -inf; rows of -inf
    alone have weights 0; +inf shares the weight among its like."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    T, E = x.shape
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    m = x.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.where(x == m, 1.0, np.exp(x - m))
    p = np.where(np.isneginf(m), 0.0, p)
    w = np.take_along_axis(p, order, axis=1)
    s = (w if renorm else p).sum(axis=1, keepdims=True)
    w = np.divide(w, s, out=np.zeros_like(w), where=s > 0)
    flat = order.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(T * k)
    off = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    return dict(idx=order, weight=w, offsets=off, perm=perm, inv=inv)


def combine(y, weight, inv, residual=None):
    """(out, sum of the absolute terms)."""
    y, w = np.asarray(y, np.float64), np.asarray(weight, np.float64)
    inv = np.asarray(inv).reshape(w.shape)
    out = np.zeros((w.shape[0], y.shape[1]))
    size = np.zeros_like(out)
    for j in range(w.shape[1]):
        ok = (inv[:, j] >= 0) & (inv[:, j] < len(y)) & (w[:, j] != 0)
        out[ok] += w[ok, j:j + 1] * y[inv[ok, j]]
        size[ok] += np.abs(w[ok, j:j + 1] * y[inv[ok, j]])
    if residual is not None:
        out, size = out + np.asarray(residual, np.float64), size + np.abs(np.asarray(residual, np.float64))
    return out, size
