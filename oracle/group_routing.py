"""Routing with expert groups, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

s = softmax(l) over all experts or sigmoid(l); the selection score is c = s +
bias, or the logit itself without a bias (both scores rise with it). A group's
score is its largest c, or the sum of its two largest s + bias. The best
groups are kept, then the k best experts in them; equal scores go to the lower
index. The weights are s of the chosen, renormalised if asked, times a factor.
Non-finite logits as in ``oracle.routing``.

Parity: pinned (closed forms and brute force in tests/test_oracle_block.py).
"""
import numpy as np

from .routing import _nan_as_neg_inf, _topk_desc


def _softmax(l):
    m = l.max(axis=1, keepdims=True)
    finite = np.isfinite(m)
    with np.errstate(invalid="ignore"):
        e = np.where(finite, np.exp(np.where(finite, l - m, 0.0)), (l == m).astype(np.float64))
    return e / e.sum(axis=1, keepdims=True)


def route_grouped(logits, bias, k, score="softmax", n_group=1, topk_group=1, group_score="max",
                  renormalize=True, scale=1.0):
    """logits [T, E] -> (ids int32 [T, k], weights float64 [T, k])."""
    l = _nan_as_neg_inf(logits)
    T, E = l.shape
    with np.errstate(over="ignore"):
        s = _softmax(l) if score == "softmax" else 1.0 / (1.0 + np.exp(-l))
    sb = s if bias is None else _nan_as_neg_inf(s + np.asarray(bias, dtype=np.float64))
    c = l if bias is None else sb
    if topk_group < n_group:
        if group_score == "top2":
            g = np.sort(sb.reshape(T, n_group, -1), axis=2)[:, :, -2:].sum(axis=2)
        else:
            g = c.reshape(T, n_group, -1).max(axis=2)
        keep = np.zeros((T, n_group), dtype=bool)
        np.put_along_axis(keep, _topk_desc(g, topk_group), True, axis=1)
        keep = np.repeat(keep, E // n_group, axis=1)
    else:
        keep = np.ones((T, E), dtype=bool)
    ids = np.empty((T, k), dtype=np.int32)
    for t in range(T):
        at = np.flatnonzero(keep[t])
        ids[t] = at[_topk_desc(c[t:t + 1, at], k)[0]]
    w = np.take_along_axis(s, ids, axis=1)
    if renormalize:
        if score == "softmax":
            w = _softmax(np.take_along_axis(l, ids, axis=1))
        else:
            # ratios of sigmoids, also where each is 0 in float64
            ls = np.take_along_axis(l, ids, axis=1)
            low = ls.max(axis=1) < -500.0
            w[low] = _softmax(ls[low])
            w = w / w.sum(axis=1, keepdims=True)
    return ids, w * scale
