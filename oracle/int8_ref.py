"""Plain fp64 forms of the 8-bit layer and of the norms around a block,
written from the formulas of the C header, with numpy alone."""
from __future__ import annotations

import numpy as np

from .liftquant_ref import whiten

ACTS = ("none", "silu", "gelu", "sigmoid", "tanh")


def act(name: str, g: np.ndarray) -> np.ndarray:
    g = np.asarray(g, dtype=np.float64)
    if name == "none":
        return g
    if name == "tanh":
        return np.tanh(g)
    with np.errstate(over="ignore"):
        if name == "gelu":
            return 0.5 * g * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)))
        s = 1.0 / (1.0 + np.exp(-g))
    return g * s if name == "silu" else s


def transform(x, gate=None, act_name="none", hb=1, c=None) -> np.ndarray:
    """v = T (act(gate) * x) in fp64."""
    v = np.asarray(x, dtype=np.float64)
    if gate is not None:
        v = v * act(act_name, gate)
    if c is None:
        c = np.ones(v.shape[1])
    return whiten(v, np.asarray(c, dtype=np.float64), hb) if hb > 1 else v * c


def quotients(v: np.ndarray) -> np.ndarray:
    """127 v / max|v| of every row (0 for a row of zeros)."""
    top = np.abs(v).max(axis=1, keepdims=True)
    return np.divide(127.0 * v, top, out=np.zeros_like(v), where=top > 0)


def codes(v: np.ndarray):
    """8-bit codes and fp64 scales of the rows of v (fp32 values held in
    fp64: the products by 127 are exact and no quotient that is not a tie
    rounds to one)."""
    return np.rint(quotients(v)).astype(np.int64), np.abs(v).max(axis=1) / 127.0


def product(q, scale, w, row_scale, bias=None) -> np.ndarray:
    """scale row_scale (q w^T) + bias; the sums of byte products are exact."""
    acc = np.asarray(q, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    y = acc * np.asarray(scale, dtype=np.float64)[:, None] * np.asarray(row_scale, dtype=np.float64)
    return y if bias is None else y + np.asarray(bias, dtype=np.float64)


def rms_norm(v, w, one_plus, eps):
    n = np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)
    w = 1.0 if w is None else np.asarray(w, dtype=np.float64) + (1.0 if one_plus else 0.0)
    return v / n * w


def norm_block(y=None, gate=None, act_name="none", gate_first=False, post=False, w_post=None,
               h=None, alpha=1.0, pre=False, w_pre=None, one_plus=False, eps=1e-5):
    """(u, h', a) in fp64."""
    u = None
    if y is not None:
        u = np.asarray(y, dtype=np.float64)
        g = None if gate is None else act(act_name, gate)
        if g is not None and gate_first:
            u = u * g
        if post:
            u = rms_norm(u, w_post, one_plus, eps)
        if g is not None and not gate_first:
            u = u * g
    hn = np.zeros_like(u) if h is None else np.asarray(h, dtype=np.float64)
    if u is not None:
        hn = hn + float(np.float32(alpha)) * u
    return u, hn, rms_norm(hn, w_pre, one_plus, eps) if pre else hn
