"""fp64 oracle of routing by scores (sigmoid or softmax, balancing bias, group
limit, renormalised and scaled gates) and of its gradient.

TEST INFRASTRUCTURE ONLY, plain numpy, no code shared with the HIP library.
"""
from __future__ import annotations

import numpy as np


def scores(logits, kind):
    l = np.asarray(logits, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(axis=1, keepdims=True)
        e = np.where(np.isneginf(l), 0.0, np.exp(l - np.where(np.isneginf(m), 0.0, m)))
        s = e.sum(axis=1, keepdims=True)
        return e / np.where(s > 0, s, 1.0)


def select(logits, bias, top_k, kind, n_groups=1, top_groups=1, group_top=2):
    """[T, k] ids by key = score + bias: keys descending, equal keys by lower
    index, among the top_groups groups with the largest sums of their
    group_top largest keys (equal sums: lower group)."""
    s = scores(logits, kind)
    key = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    T, E = key.shape
    out = np.empty((T, top_k), dtype=np.int64)
    gs = E // n_groups
    for t in range(T):
        allowed = range(E)
        if n_groups > 1 and top_groups < n_groups:
            def group_score(g):
                v = sorted(key[t, g * gs:(g + 1) * gs], reverse=True)
                return v[0] + v[1] if group_top == 2 and gs > 1 else v[0]
            best = sorted(range(n_groups), key=lambda g: (-group_score(g), g))[:top_groups]
            allowed = [e for g in sorted(best) for e in range(g * gs, (g + 1) * gs)]
        out[t] = sorted(allowed, key=lambda e: (-key[t, e], e))[:top_k]
    return out


def gates(logits, topk_idx, kind, renormalise=True, scale=1.0):
    s = np.take_along_axis(scores(logits, kind), topk_idx, axis=1)
    if renormalise:
        s = s / (s.sum(axis=1, keepdims=True) + 1e-20)
    return s * scale


def backward(logits, topk_idx, d_gates, kind, renormalise=True, scale=1.0):
    """(d_logits [T, E], the same formula on magnitudes).  An id outside
    [0, E) has score 0 and no gradient."""
    p = scores(logits, kind)
    T, E = p.shape
    ids = np.asarray(topk_idx)
    on = (ids >= 0) & (ids < E)
    s = np.where(on, np.take_along_axis(p, np.where(on, ids, 0), axis=1), 0.0)
    dg = np.where(on, np.asarray(d_gates, dtype=np.float64) * scale, 0.0)
    ds, mag = dg, np.abs(dg)
    if renormalise:
        S = s.sum(axis=1, keepdims=True) + 1e-20
        ds = np.where(on, (dg - (dg * s).sum(axis=1, keepdims=True) / S) / S, 0.0)
        mag = np.where(on, (np.abs(dg) + np.abs(dg * s).sum(axis=1, keepdims=True) / S) / S, 0.0)
    rows = np.repeat(np.arange(T), ids.shape[1])
    sel = np.where(on, ids, 0).ravel()
    out, bound = np.zeros((T, E)), np.zeros((T, E))
    if kind == "sigmoid":
        # 1 - s as the score of -l: the difference would lose what is below 2^-53
        rest = np.take_along_axis(scores(-np.asarray(logits, dtype=np.float64), kind), np.where(on, ids, 0), axis=1)
        np.add.at(out, (rows, sel), (ds * s * rest).ravel())
        np.add.at(bound, (rows, sel), (mag * s * rest).ravel())
        return out, bound
    np.add.at(out, (rows, sel), ds.ravel())
    np.add.at(bound, (rows, sel), mag.ravel())
    return (p * (out - (ds * s).sum(axis=1, keepdims=True)),
            p * (bound + (mag * s).sum(axis=1, keepdims=True)))
