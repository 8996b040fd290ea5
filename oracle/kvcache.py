"""The quantised paged key-value cache and attention over it, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

A record holds 16 tokens of one head: K codes [16][R], V codes [16][R], for
NVFP4 the K and V block scales [D / 16][16] (E4M3), for FP8 and NVFP4 the K and
V row exponents [16] (biased by 127; 255 marks a row with a NaN or infinity).
Byte p of token i's codes lies at (i R + p) ^ 16 f(i).

Parity: pinned (round trips and closed forms in tests/test_oracle_block.py).
"""
import numpy as np

from .formats import E2M1_VALUES

_E4M3 = np.array([(c & 7) * 2.0 ** -9 if (c >> 3) == 0 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10)
                  for c in range(127)])
_E2M1 = E2M1_VALUES[:8]


def row_bytes(fmt, D):
    return {"bf16": 2 * D, "fp16": 2 * D, "fp8": D, "nvfp4": D // 2}[fmt]


def record_bytes(fmt, D):
    return 32 * row_bytes(fmt, D) + {"bf16": 0, "fp16": 0, "fp8": 32, "nvfp4": 2 * D + 32}[fmt]


def place(fmt, D):
    """[16, R]: where each byte of the codes lies."""
    R = row_bytes(fmt, D)
    i = np.arange(16)
    f = i & 7 if R >= 128 else i & 6 if R == 64 else (i >> 1) & 2
    return (i[:, None] * R + np.arange(R)) ^ (16 * f[:, None])


def nearest_code(x, grid):
    """Index into the rising grid of the nearest value to x >= 0, ties to the even index, past the end the last."""
    hi = np.minimum(np.searchsorted(grid, x), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - x, x - grid[lo]
    return np.where(x >= grid[-1], len(grid) - 1, np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo))


def quantise(x, fmt):
    """x [..., D] float64 -> (codes uint8 [..., D] one a value, block scales uint8 [..., D / 16] or None,
    exponents uint8 [...])."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(axis=-1)
    x = np.where(bad[..., None], 0.0, x)
    amax = np.abs(x).max(axis=-1)
    pow2 = 2.0 ** np.arange(-127, 128)
    e = np.minimum(np.searchsorted(pow2 * (448.0 if fmt == "fp8" else 2688.0), amax), 254)
    x = x / pow2[e][..., None]
    sign = np.signbit(x).astype(np.uint8)
    e = np.where(bad, 255, e).astype(np.uint8)
    if fmt == "fp8":
        return (nearest_code(np.abs(x), _E4M3) | (sign << 7)).astype(np.uint8), None, e
    b = x.reshape(*x.shape[:-1], -1, 16)
    sc = nearest_code(np.abs(b).max(axis=-1) / 6.0, _E4M3)
    s = _E4M3[sc][..., None]
    c = nearest_code(np.abs(np.where(s > 0, b / np.where(s > 0, s, 1.0), 0.0)), _E2M1)
    c = np.where(s > 0, c | (sign.reshape(b.shape) << 3), 0).astype(np.uint8)
    return c.reshape(x.shape), sc.astype(np.uint8), e


def decode(codes, scales, exps, fmt):
    """The values of quantise's answer (NaN rows where the exponent is 255)."""
    if fmt == "fp8":
        v = _E4M3[np.minimum(codes & 127, 126)] * np.where(codes >> 7, -1.0, 1.0)
    else:
        v = _E2M1[codes & 7] * np.where(codes >> 3, -1.0, 1.0)
        v = v * np.repeat(_E4M3[np.minimum(scales & 127, 126)], 16, axis=-1)
    v = v * (2.0 ** (exps.astype(np.float64) - 127.0))[..., None]
    return np.where((exps == 255)[..., None], np.nan, v)


def unpack_record(rec, fmt, D):
    """rec uint8 [record bytes] -> (K codes, K scales, K exponents), (V ...): codes one a value (uint8), or raw
    uint16 words for 16-bit formats."""
    R = row_bytes(fmt, D)
    out = []
    for part in (0, 1):
        raw = rec[part * 16 * R:(part + 1) * 16 * R][place(fmt, D)]
        if fmt in ("bf16", "fp16"):
            out.append((np.ascontiguousarray(raw).view(np.uint16), None, None))
            continue
        exps = rec[-32 + 16 * part:][:16]
        if fmt == "fp8":
            out.append((raw, None, exps))
        else:
            codes = np.stack([raw & 15, raw >> 4], axis=2).reshape(16, D)
            sc = rec[32 * R + part * D:32 * R + (part + 1) * D].reshape(D // 16, 16).T
            out.append((codes, sc, exps))
    return out


def values(data, fmt, D):
    """Keys and values [num_pages, kv_heads, page_size, D] float64 of a whole cache (uint8, 4-D)."""
    P, H, N, _ = data.shape
    kv = np.empty((2, P, H, N, 16, D))
    for at in np.ndindex(P, H, N):
        for part, (codes, sc, ex) in enumerate(unpack_record(data[at], fmt, D)):
            if fmt == "bf16":
                v = (codes.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
            elif fmt == "fp16":
                v = codes.view(np.float16).astype(np.float64)
            else:
                v = decode(codes, sc, ex, fmt)
            kv[(part,) + at] = v
    return kv[0].reshape(P, H, N * 16, D), kv[1].reshape(P, H, N * 16, D)


def attend(q, keys, vals, table, lens, scale, window=0, sinks=None):
    """q [B, heads, D]; keys, vals as from ``values``; page numbers outside the cache leave their tokens out.
    Returns out [B, heads, D], lse [B, heads], and for error bounds sum_i p_i |v_i|, the largest scale * sum |q||k|
    and n times the largest p_i max |v_i|."""
    q = np.asarray(q, dtype=np.float64)
    B, heads, D = q.shape
    P, H, page, _ = keys.shape
    G = heads // H
    out, mag = np.zeros((B, heads, D)), np.zeros((B, heads, D))
    lse, size, peak = np.full((B, heads), -np.inf), np.zeros((B, heads)), np.zeros((B, heads))
    for b in range(B):
        n = int(min(max(lens[b], 0), table.shape[1] * page))
        at = [i for i in range(max(0, n - window) if window else 0, n) if 0 <= table[b, i // page] < P]
        pages, offs = table[b, [i // page for i in at]], [i % page for i in at]
        for h in range(heads):
            k, v = keys[pages, h // G, offs], vals[pages, h // G, offs]
            s = scale * (k @ q[b, h]) if at else np.empty(0)
            top = max([s.max()] if at else [], default=-np.inf)
            if sinks is not None:
                top = max(top, float(sinks[h]))
            if top == -np.inf:
                continue
            p = np.exp(s - top)
            tot = p.sum() + (np.exp(float(sinks[h]) - top) if sinks is not None else 0.0)
            lse[b, h] = top + np.log(tot)
            if at:
                out[b, h] = (p / tot) @ v
                mag[b, h] = (p / tot) @ np.abs(v)
                size[b, h] = abs(scale) * (np.abs(k) @ np.abs(q[b, h])).max()
                peak[b, h] = len(at) * (p / tot * np.abs(v).max(axis=1)).max()
    return out, lse, mag, size, peak
