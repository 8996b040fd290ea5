"""Rows quantised to NVFP4 or MXFP4, the tiles their block scales lie in, and the product of two such matrices, in
float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

NVFP4: row scale the least power of two r with amax / r <= 6 * 448, block scales E4M3(amax16 / r / 6), codes
E2M1(x / r / s). MXFP4: block scale the least power of two s with amax32 / s <= 6, codes E2M1(x / s).

Parity: pinned (closed forms and brute force in tests/test_oracle_fp4.py).
"""
import numpy as np

from .formats import E2M1_VALUES, E4M3_VALUES, E8M0_VALUES, unpack_nibbles
from .kvcache import nearest_code, quantise

BLOCK = {"nvfp4": 16, "mxfp4": 32}


def quantise_rows(x, fmt):
    """x [T, K] -> (q uint8 [T, K / 2], block scales uint8 [T, K / BLOCK], row scales float64 [T] or None)."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "nvfp4":
        codes, scales, e = quantise(x, "nvfp4")
        r = np.where(e == 255, np.nan, 2.0 ** (e.astype(np.float64) - 127))
        codes, scales = np.where((e == 255)[:, None], 0, codes), np.where((e == 255)[:, None], 0, scales)
    else:
        b = x.reshape(x.shape[0], -1, 32)
        bad = ~np.isfinite(b).all(axis=-1)
        b = np.where(bad[..., None], 0.0, b)
        pow2 = 2.0 ** np.arange(-127, 128)
        e = np.minimum(np.searchsorted(pow2 * 6.0, np.abs(b).max(axis=-1)), 254)
        b = b / pow2[e][..., None]
        codes = nearest_code(np.abs(b), E2M1_VALUES[:8]) | (np.signbit(b).astype(np.uint8) << 3)
        codes = np.where(bad[..., None], 0, codes).reshape(x.shape)
        scales, r = np.where(bad, 255, e), None
    codes = codes.astype(np.uint8)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales.astype(np.uint8), r


def tile(scales):
    """Plain block scales [rows, blocks] -> the bytes of their tiles (0 where no block is)."""
    rows, blocks = scales.shape
    tr, tk = -(-rows // 128), -(-blocks // 4)
    out = np.zeros((tr, tk, 32, 4, 4), dtype=np.uint8)
    for r in range(rows):
        for b in range(blocks):
            out[r // 128, b // 4, r % 32, r % 128 // 32, b % 4] = scales[r, b]
    return out.reshape(-1)


def untile(tiles, rows, blocks):
    t = np.asarray(tiles).reshape(-1, -(-blocks // 4), 32, 4, 4)  # [row tile, block tile, row % 32, row % 128 / 32, block % 4]
    return t.transpose(0, 3, 2, 1, 4).reshape(-1, t.shape[1] * 4)[:rows, :blocks]


def values(q, scales, row_scale, fmt):
    """The numbers that codes q, plain block scales and row scales stand for."""
    s = (E4M3_VALUES if fmt == "nvfp4" else E8M0_VALUES)[scales]
    v = E2M1_VALUES[unpack_nibbles(q)] * np.repeat(s, BLOCK[fmt], axis=1)
    return v if row_scale is None else v * np.asarray(row_scale, dtype=np.float64).reshape(-1, 1)


def linear(x, w, bias=None):
    """(x w^T + bias, the sum of the products' magnitudes) of two matrices of values."""
    out = x @ w.T
    return out if bias is None else out + np.asarray(bias, dtype=np.float64), np.abs(x) @ np.abs(w).T
