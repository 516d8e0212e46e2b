"""Block-scaled 8-bit values and products in fp64 (test infrastructure).

A value is e4m3 code * scale; a token's scale covers 128 consecutive values of
its row, a weight's 128 x 128.  encode(): per block s = max(amax / 448, 2^-126),
code = nearest e4m3 of v / s, ties to the even code.  Codes are handled as the
values they stand for.
"""

from __future__ import annotations

import numpy as np

from .ffn import silu

BLOCK = 128


def _per_value(scale: np.ndarray, n: int, axis: int) -> np.ndarray:
    return np.take(scale, np.arange(n) // BLOCK, axis=axis)


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value of |v| <= 464 (ties to even); steps of 2^-3 of the power of two below, at least 2^-9."""
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    return np.rint(v / step) * step


def scales(v: np.ndarray) -> np.ndarray:
    """[T, K] -> [T, ceil(K/128)]; infinities and NaN have no part."""
    T, K = v.shape
    a = np.abs(np.where(np.isfinite(v), v, 0.0))
    return np.stack([np.maximum(a[:, b:b + BLOCK].max(axis=1) / 448.0, 2.0 ** -126) for b in range(0, K, BLOCK)], axis=1)


def encode(v: np.ndarray):
    """(code values, scales); the code of an infinity or NaN is NaN."""
    s = scales(v)
    ratio = v / _per_value(s, v.shape[1], 1)
    return np.where(np.isfinite(v), round_e4m3(np.where(np.isfinite(v), ratio, 0.0)), np.nan), s


def tokens(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    return q * _per_value(np.asarray(s, np.float64), q.shape[1], 1)


def weight(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    """[..., N, K] code values and [..., N/128, K/128] scales -> fp64 weights."""
    s = np.asarray(s, np.float64)
    return q * _per_value(_per_value(s, q.shape[-2], -2), q.shape[-1], -1)


def norm(x: np.ndarray, residual, weight: np.ndarray, offset: float, eps: float, rounded):
    """(y, x + residual before its rounding): RMS norm of r = rounded(x + residual)."""
    total = x if residual is None else x + residual
    r = total if residual is None else rounded(total)
    return r / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps) * (weight + offset), total


def block_linear(x: np.ndarray, w: np.ndarray, bias=0.0):
    """(y, magnitudes) of fp64 x [T, K], w [N, K]."""
    return x @ w.T + bias, np.abs(x) @ np.abs(w).T + np.abs(bias)


def block_expert_ffn(x: np.ndarray, gate: np.ndarray, up: np.ndarray, down: np.ndarray, idx, w) -> np.ndarray:
    """[T, H]: fp64 x [T, H], gate, up [E, I, H], down [E, H, I], ids and gate weights [T, k]."""
    y = np.zeros(x.shape)
    for t in range(x.shape[0]):
        for j in range(idx.shape[1]):
            e = idx[t, j]
            h = silu(gate[e] @ x[t]) * (up[e] @ x[t])
            q, s = encode(h[None])
            y[t] += w[t, j] * (down[e] @ tokens(q, s)[0])
    return y
