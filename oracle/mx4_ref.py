"""Plain fp64 forms of the microscaled 4-bit layer and of the heads' norm and
rotation, written from the formulas of the C header, with numpy alone."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks(v: np.ndarray) -> np.ndarray:
    """Rows in blocks of 32, the last filled up with zeros."""
    B, K = v.shape
    out = np.zeros((B, -(-K // 32) * 32))
    out[:, :K] = v
    return out.reshape(B, -1, 32)


def exponents(v: np.ndarray) -> np.ndarray:
    """The exponents (rows, blocks) of the scales of rows of finite values."""
    m = np.abs(blocks(v)).max(axis=2)
    e = np.frexp(np.where(m > 0, m, 1.0))[1] - 3        # frexp's fraction is below 1
    return np.where(m > 0, np.maximum(e, -127), -127)


def quantise(v: np.ndarray):
    """(codes (rows, 32 blocks), scale bytes (rows, blocks)) of rows v, in
    fp64: the quotient by a power of two is exact."""
    b = blocks(np.asarray(v, dtype=np.float64))
    good = np.isfinite(b).all(axis=2)
    b = np.where(good[:, :, None], b, 0.0)
    e = exponents(b.reshape(b.shape[0], -1))
    a = np.ldexp(np.abs(b), -e[:, :, None])
    mid = (GRID[1:] + GRID[:-1]) / 2                    # a tie lies between the codes i and i + 1
    low, high = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    code = np.where(low % 2 == 0, low, high).astype(np.uint8)
    code |= np.where(np.signbit(b), 8, 0).astype(np.uint8)
    return code.reshape(b.shape[0], -1), np.where(good, e + 127, 255).astype(np.uint8)


def decode(code: np.ndarray, scale: np.ndarray, K: int) -> np.ndarray:
    """The values that codes and scale bytes stand for (NaN for byte 255)."""
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return (v.reshape(v.shape[0], -1, 32) * s[:, :, None]).reshape(v.shape[0], -1)[:, :K]


def pack(code: np.ndarray) -> np.ndarray:
    """Two codes a byte, the even one in the low half."""
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(data: np.ndarray) -> np.ndarray:
    out = np.empty((data.shape[0], 2 * data.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = data & 15, data >> 4
    return out


def scale_places(rows: int, K: int) -> np.ndarray:
    """Where the scale byte of row n's block j lies, (rows, whole blocks of 8)."""
    units = -(-K // 256)
    n, j = np.arange(rows)[:, None], np.arange(8 * units)[None, :]
    return ((n // 16) * units + j // 8) * 128 + 8 * (n % 16) + 2 * (j % 4) + j // 4 % 2


def panels(scale: np.ndarray, K: int, fill: int = 0) -> np.ndarray:
    """Scale bytes (rows, blocks) in the library's order, the others `fill`."""
    rows = scale.shape[0]
    out = np.full(-(-rows // 16) * -(-K // 256) * 128, fill, dtype=np.uint8)
    out[scale_places(rows, K)[:, :scale.shape[1]]] = scale
    return out


def product(q: np.ndarray, w: np.ndarray, row_scale=None, bias=None):
    """(y, the sums of the magnitudes of its terms) of decoded rows."""
    y, size = q @ w.T, np.abs(q) @ np.abs(w).T
    if row_scale is not None:
        r = np.asarray(row_scale, dtype=np.float64)
        y, size = y * r, size * np.abs(r)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    return y, size


def norm_rope(x, pos, freq, w=None, norm=True, one_plus=False, eps=1e-5, interleaved=False):
    """Heads x (tokens, heads, dim) normed and rotated."""
    x = np.array(x, dtype=np.float64)
    if norm:
        x = x / np.sqrt(np.mean(x * x, axis=2, keepdims=True) + float(np.float32(eps)))
        if w is not None:
            x = x * (np.asarray(w, dtype=np.float64) + (1.0 if one_plus else 0.0))
    half = len(freq)
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    t = np.asarray(pos, dtype=np.float64)[:, None, None] * np.asarray(freq, dtype=np.float64)
    a, b = x[:, :, first], x[:, :, second]
    out = x.copy()
    out[:, :, first], out[:, :, second] = a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)
    return out
