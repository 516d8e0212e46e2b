"""Dense 4-bit products in fp64 (test infrastructure).

A weight is e2m1(code) * scale * global; NVFP4 has an e4m3 scale per 16
weights, MXFP4 a scale 2^(byte - 127) per 32.  Each function also returns what
its tolerance needs: the sum of the products' magnitudes.
"""

from __future__ import annotations

import numpy as np

from .ffn import silu
from .formats import E2M1_VALUES, bf16_bits_to_f64, e4m3_table, unpack_nibbles


def dequant(codes: np.ndarray, scales: np.ndarray, g, fmt: str) -> np.ndarray:
    """[N, K] fp64 weights."""
    v = np.asarray(E2M1_VALUES, dtype=np.float64)[unpack_nibbles(codes)]
    if fmt == "nvfp4":
        s, group = np.asarray(e4m3_table(), dtype=np.float64)[scales], 16
    else:
        s, group = np.ldexp(1.0, scales.astype(np.int64) - 127), 32
    return v * np.repeat(s, group, axis=1) * (1.0 if g is None else float(g))


def quant_linear(x_bf16: np.ndarray, weight: tuple, fmt: str, bias_bf16=None):
    """(y, magnitudes): x W^T + bias and |x| |W|^T + |bias|, [T, N] fp64."""
    x, w = bf16_bits_to_f64(x_bf16), dequant(*weight, fmt)
    b = 0.0 if bias_bf16 is None else bf16_bits_to_f64(bias_bf16)
    return x @ w.T + b, np.abs(x) @ np.abs(w).T + np.abs(b)


def quant_shared_expert(x_bf16, gate, up, down, fmt: str, token_gate_bf16=None, add_bf16=None) -> np.ndarray:
    """[T, H] fp64: add + sigmoid(x . token_gate) * W_down (SiLU(W_gate x) * (W_up x))."""
    x = bf16_bits_to_f64(x_bf16)
    h = silu(x @ dequant(*gate, fmt).T) * (x @ dequant(*up, fmt).T)
    y = h @ dequant(*down, fmt).T
    if token_gate_bf16 is not None:
        y = y / (1.0 + np.exp(-(x @ bf16_bits_to_f64(token_gate_bf16))))[:, None]
    return y if add_bf16 is None else y + bf16_bits_to_f64(add_bf16)
