"""The operators around the expert layer in fp64: norm with the residual's
addition, row quantiser, int8 product, log probabilities (numpy only)."""
from __future__ import annotations

import numpy as np


def rms_norm(x, weight, eps, residual=None):
    """(s, y): s = x + residual, y = s * weight / sqrt(mean(s^2) + eps)."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    r = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return s, s * r * np.asarray(weight, np.float64)


def quant_i8(y):
    """(steps, scale): y in units of its row's scale max|y| / 127, unrounded."""
    y = np.asarray(y, np.float64)
    scale = np.abs(y).max(axis=1) / 127.0
    return np.divide(y, scale[:, None], out=np.zeros_like(y), where=scale[:, None] > 0), scale


def linear_i8(x, x_scale, w, w_scale, bias=None):
    """(sums, out): the whole-number sums and the scaled product."""
    acc = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T     # below 2^53: exact
    out = acc * np.asarray(x_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)[None, :]
    return acc, out if bias is None else out + np.asarray(bias, np.float64)[None, :]


def logprobs(logits, ids=None, top=0):
    """dict of logprob, rank, entropy, top_ids, top_logprobs; a row of -inf
    alone has entropy 0 and log probabilities -inf; ids outside [0, V) give
    logprob 0 and rank -1.  Rows hold no NaN and no +inf."""
    x = np.asarray(logits, np.float64)
    T, V = x.shape
    m = x.max(axis=1, keepdims=True)
    empty = np.isneginf(m)
    d = np.where(np.isneginf(x), -np.inf, x - np.where(empty, 0.0, m))
    e = np.exp(d)
    s = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        ls = np.log(s)
        l = np.where(empty, -np.inf, d - ls)
        ent = np.where(empty[:, 0], 0.0, -np.where(e > 0, e / s * l, 0.0).sum(axis=1))
    out = {"entropy": ent}
    order = np.argsort(-x, axis=1, kind="stable")
    out["top_ids"] = order[:, :top]
    out["top_logprobs"] = np.take_along_axis(l, order[:, :top], axis=1)
    if ids is not None:
        ids = np.asarray(ids, np.int64)
        lp, rank = np.zeros(T), np.full(T, -1, np.int64)
        for t, i in enumerate(ids):
            if 0 <= i < V:
                lp[t] = l[t, i]
                rank[t] = (x[t] > x[t, i]).sum() + (x[t, :i] == x[t, i]).sum()
        out["logprob"], out["rank"] = lp, rank
    return out
