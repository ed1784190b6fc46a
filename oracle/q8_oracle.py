"""The 8-bit cache and the norm with rotation, from their definitions.

Plain NumPy: quantisation in float32 exactly as the definition has it (every
operation rounded once, which NumPy's float32 does), everything else in
float64.  Shares no code with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 64
TOP = {"int8": 127.0, "e4m3": 448.0}


def round_e4m3(y: np.ndarray) -> np.ndarray:
    """Nearest value with 4 exponent and 3 mantissa bits (ties to even, largest
    448, smallest normal 2^-6, spacing 2^-9 below it)."""
    y = np.asarray(y, dtype=np.float64)
    _, e = np.frexp(np.where(y == 0, 1.0, np.abs(y)))          # |y| = f 2^e, f in [1/2, 1)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.round(y / step) * step, -448.0, 448.0)


def quantise_block(x: np.ndarray, fmt: str):
    """x [..., 64, d] -> (codes' values float64, scales float32 [...])."""
    x = np.asarray(x, dtype=np.float32)
    top = np.float32(TOP[fmt])
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        a = np.abs(x).max(axis=(-1, -2))
        bad = ~np.isfinite(x).all(axis=(-1, -2))
        live = (a >= np.float32(2.0 ** -100)) & ~bad
        inv = np.where(live, top / np.where(live, a, np.float32(1)), np.float32(0)).astype(np.float32)
        scale = np.where(bad, np.float32(np.nan), np.where(live, (a / top).astype(np.float32), np.float32(1)))
        y = (np.where(live[..., None, None], x, np.float32(0)) * inv[..., None, None]).astype(np.float32)
    codes = np.round(y.astype(np.float64)) if fmt == "int8" else round_e4m3(y)
    return codes, scale.astype(np.float32)


def held(x: np.ndarray, length: int, fmt: str):
    """The first `length` tokens of one (row, kv head) stream x [>= length, d]
    as the cache holds them: (codes' values, per-token scales), the open
    block's tokens as themselves with scale 1; float64."""
    whole = length // BLOCK
    d = x.shape[-1]
    codes, scales = quantise_block(np.asarray(x[:whole * BLOCK], dtype=np.float64).reshape(whole, BLOCK, d), fmt)
    c = np.concatenate([codes.reshape(whole * BLOCK, d), np.asarray(x[whole * BLOCK:length], dtype=np.float64)])
    s = np.concatenate([np.repeat(scales.astype(np.float64), BLOCK), np.ones(length - whole * BLOCK)])
    return c, s


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, sigma: float | None = None):
    """q [n, G, d] of the newest n tokens, k, v [L, d] -> (o [n, G, d], weights
    [n, G, L]).  Query i attends to positions below L - n + 1 + i; a query that
    has none gives zeros, one that meets a value that is no number NaN."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, g, d = q.shape
    length = k.shape[0]
    sigma = 1.0 / math.sqrt(d) if not sigma else sigma
    bad = ~(np.isfinite(k).all(-1) & np.isfinite(v).all(-1)) if length else np.zeros(0, bool)
    k, v = np.where(bad[:, None], 0.0, k), np.where(bad[:, None], 0.0, v)
    o, w = np.zeros((n, g, d)), np.zeros((n, g, length))
    for i in range(n):
        end = length - n + 1 + i
        if end <= 0:
            continue
        a = sigma * (q[i] @ k[:end].T)
        e = np.exp(a - a.max(-1, keepdims=True))
        w[i, :, :end] = e / e.sum(-1, keepdims=True)
        o[i] = np.nan if bad[:end].any() else w[i, :, :end] @ v[:end]
    return o, w


def norm_rope(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray, weight=None, eps: float = 1e-6,
              interleaved: bool = False) -> np.ndarray:
    """x [..., heads, d] with positions [...]: norm of each head, then the
    rotation of its pairs."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    ang = np.asarray(positions, dtype=np.float64)[..., None, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang), np.sin(ang)
    y = np.empty(np.broadcast_shapes(x.shape, ang.shape[:-1] + (d,)))
    first, second = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y
