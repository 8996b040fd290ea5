"""Rotary positions in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``). Angles are taken modulo a turn in exact rational arithmetic where a
frequency is given as a fraction of 2^64 of a turn, else from the definition.

Parity: pinned (closed forms in tests/test_oracle_plan_rope.py).
"""
import math

import numpy as np


def frequencies(R, base=10000.0, scaling="none", factor=1.0, original_len=4096, truncate=True, low=1.0, high=None):
    """(frequencies [R / 2] in radians a position, amplitude)."""
    high = (32.0 if scaling == "yarn" else 4.0) if high is None else high
    out, amp = [], 1.0
    for i in range(R // 2):
        f = base ** (-2.0 * i / R)
        if scaling == "linear":
            f /= factor
        elif scaling == "ntk":
            f = (base * factor ** (R / (R - 2))) ** (-2.0 * i / R)
        elif scaling == "yarn":
            lo, hi = (R * math.log(original_len / (2 * math.pi * x)) / (2 * math.log(base)) for x in (high, low))
            if truncate:
                lo, hi = math.floor(lo), math.ceil(hi)
            lo, hi = max(lo, 0), min(hi, R - 1)
            stretched = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f / factor * stretched + f * (1 - stretched)
            amp = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        elif scaling == "llama3":
            turns = original_len * f / (2 * math.pi)
            kept = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = f / factor * (1 - kept) + f * kept
        out.append(f)
    return np.array(out), amp


def angles(positions, turns):
    """[T, R / 2] radians of positions under 64-bit fractions of a turn, exact before the last rounding."""
    return np.array([[(int(p) * int(t) % 2 ** 64) * (2 * math.pi / 2 ** 64) for t in turns] for p in positions])


def rotate(x, a, layout="half", amplitude=1.0):
    """x [T, heads, D] rotated by angles a [T, R / 2]."""
    x = np.array(x, dtype=np.float64)
    R = 2 * a.shape[1]
    c, s = amplitude * np.cos(a)[:, None], amplitude * np.sin(a)[:, None]
    one = slice(0, R // 2) if layout == "half" else slice(0, R, 2)
    two = slice(R // 2, R) if layout == "half" else slice(1, R, 2)
    u, v = x[..., one].copy(), x[..., two].copy()
    x[..., one], x[..., two] = u * c - v * s, v * c + u * s
    return x
