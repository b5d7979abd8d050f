"""Plain fp64 form of the router by scores: scores, choice with a bias and groups, gates, and the
gradient of the logits."""
from __future__ import annotations

import numpy as np

from .dense_oracle import sigmoid


def scores(logits, kind):
    x = np.asarray(logits, np.float64)
    if kind == "sigmoid":
        return sigmoid(x)
    m = x.max(1, keepdims=True)
    e = np.exp(x - np.where(np.isinf(m), 0.0, m))
    den = e.sum(1, keepdims=True)
    return e / np.where(den == 0, 1.0, den)


def choose(logits, bias, k, kind, groups=1, keep=1, top=1):
    """(scores [T][E], ids [T][k]): larger value first, lower id on equal ones."""
    s = scores(logits, kind)
    T, E = s.shape
    rank = np.asarray(logits, np.float64) if bias is None else s + np.asarray(bias, np.float64)
    value = s if bias is None else rank
    ids = np.empty((T, k), np.int64)
    size = E // groups
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-rank[t, e], e))
        if groups > 1:
            v = [sum(sorted(value[t, g * size:(g + 1) * size], reverse=True)[:top]) for g in range(groups)]
            kept = set(sorted(range(groups), key=lambda g: (-v[g], g))[:keep])
            order = [e for e in order if e // size in kept]
        ids[t] = order[:k]
    return s, ids


def gates(s, ids, renorm, scale):
    p = np.take_along_axis(s, ids, 1)
    if renorm:
        total = p.sum(1, keepdims=True)
        p = p / np.where(total == 0, 1.0, total)
    return scale * p


def shares(logits, ids, kind):
    """The chosen scores over their sum, 0 where that is 0; softmax: that of the chosen logits, however far they lie
    below the row's largest."""
    if kind == "softmax":
        return scores(np.take_along_axis(np.asarray(logits, np.float64), ids, 1), kind)
    p = np.take_along_axis(scores(logits, kind), ids, 1)
    total = p.sum(1, keepdims=True)
    return p / np.where(total == 0, 1.0, total)


def gates_of(logits, ids, kind, renorm, scale):
    if renorm:
        return scale * shares(logits, ids, kind)
    return gates(scores(logits, kind), ids, 0, scale)


def backward(logits, ids, dw, kind, renorm, scale):
    """dL/dlogits of the gates of fixed ids."""
    d = scale * np.asarray(dw, np.float64)
    s = scores(logits, kind)
    if renorm:
        # (products of shares, which are 1 at most: a sum of scores can be the least of 64-bit numbers)
        a = shares(logits, ids, kind)
        d = (d - (d * a).sum(1, keepdims=True)) * a
        if kind == "sigmoid":
            d = d * sigmoid(-np.take_along_axis(np.asarray(logits, np.float64), ids, 1))
        out = np.zeros_like(s)
        np.put_along_axis(out, ids, d, 1)
        return out
    full = np.zeros_like(s)
    np.put_along_axis(full, ids, d, 1)
    if kind == "sigmoid":
        return full * s * sigmoid(-np.asarray(logits, np.float64))
    return s * (full - (d * np.take_along_axis(s, ids, 1)).sum(1, keepdims=True))


def group_pairs(ids, E):
    """counts, offsets, perm, inv of the pairs of ids, grouped by expert, in order within one."""
    flat = np.asarray(ids).ravel()
    counts = np.bincount(flat, minlength=E)
    perm = np.argsort(flat, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(flat.size)
    return counts, np.concatenate([[0], np.cumsum(counts)]), perm, inv
