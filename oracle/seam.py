"""The seam between two blocks, in float64: h = residual + alpha * gate *
post(z), y = pre(h).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Parity: pinned (closed forms in tests/test_oracle_block.py).
"""
import numpy as np


def norm(x, kind, weight=None, bias=None, eps=1e-5, offset=0.0):
    """(normalised x [T, H], 1 / sqrt(. + eps) [T, 1])."""
    x = np.asarray(x, dtype=np.float64)
    if kind == "layer":
        x = x - x.mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)
    y = x * r
    if weight is not None:
        y = y * (np.asarray(weight, dtype=np.float64) + offset)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    return y, r


def residual_norm(z, residual, gate, post, alpha, pre):
    """post, pre: None or the keyword arguments of norm. Returns (h, y or None)."""
    h = 0.0 if residual is None else np.asarray(residual, dtype=np.float64)
    if z is not None:
        u = np.asarray(z, dtype=np.float64)
        if post is not None:
            u = norm(u, **post)[0]
        h = h + alpha * (1.0 if gate is None else np.asarray(gate, dtype=np.float64)) * u
    return h, None if pre is None else norm(h, **pre)[0]
