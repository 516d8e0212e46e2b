"""Inputs and tolerances of the GPU tests of grouped routing and the 4-bit
dense products."""

import numpy as np
import torch

import oracle
import sparse_moe_expert_amd as sme
from gpu_harness import DEV, to_dev
from moe_inputs.generate import f64_to_bf16_bits
from nvfp4_testlib import pack_codes

BF16_HALF = 2.0 ** -8                        # half a step of bf16, relative
ADD = 2.0 ** -23                             # one fp32 addition, rounded or truncated


def bits(a):
    return f64_to_bf16_bits(np.asarray(a, dtype=np.float64))


def dev_bf16(b):
    return to_dev(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16)


def weight(rng, N, K, fmt):
    """Random codes, and scales that make the weights' size about K^-1/2."""
    codes = pack_codes(rng.integers(0, 16, (N, K), dtype=np.uint8))
    if fmt == "nvfp4":
        scales = rng.integers(0x20, 0x50, (N, K // 16)).astype(np.uint8)
        return codes, scales, np.float32(0.2 / np.sqrt(K))
    return codes, rng.integers(118, 125, (N, K // 32)).astype(np.uint8), None


def handle(w, fmt):
    codes, scales, g = w
    return sme.QuantWeight(to_dev(codes), to_dev(scales), None if g is None else to_dev(np.array([g], np.float32)), fmt)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def linear_tolerance(ref, mag, K):
    """K products and additions and K/16 scalings, each off by at most ADD of
    a partial sum, which the magnitudes bound; the global scale and the bias;
    the output's rounding."""
    return BF16_HALF * np.abs(ref) + (K + K // 16 + 8) * ADD * (1 + BF16_HALF) * mag


def shared_reference(x, gate, up, down, fmt, v=None, add=None):
    """(y, tolerance) of the shared expert.  The products' errors as in
    linear_tolerance; |d SiLU| <= 1.1; the exponential of e^-g is off by
    |g| ulp and a few, the quotient and the product by a few more; h is
    rounded to bf16; the token gate's slope is at most 1/4."""
    H, Is = x.shape[1], gate[0].shape[0]
    terms = lambda K: (K + K // 16 + 8) * ADD  # noqa: E731
    g, gm = oracle.quant_linear(x, gate, fmt)
    u, um = oracle.quant_linear(x, up, fmt)
    a = oracle.ffn.silu(g)
    h = a * u
    eh = 1.1 * terms(H) * gm * np.abs(u) + (np.abs(a) + 1.1 * terms(H) * gm) * terms(H) * um
    eh += (np.abs(g) + 16) * ADD * np.abs(h)
    eh += BF16_HALF * (np.abs(h) + eh)
    wd = np.abs(oracle.quant.dequant(*down, fmt))
    y = oracle.quant_shared_expert(x, gate, up, down, fmt, v, add)
    mag = (np.abs(h) + eh) @ wd.T
    e = eh @ wd.T + terms(Is) * mag
    if v is not None:
        xf, vf = oracle.bf16_bits_to_f64(x), oracle.bf16_bits_to_f64(v)
        dot = xf @ vf
        s = 1.0 / (1.0 + np.exp(-dot))
        es = 0.25 * (H + 8) * ADD * (np.abs(xf) @ np.abs(vf)) + (np.abs(dot) + 16) * ADD * s
        e = e * s[:, None] + (mag + e) * es[:, None] + 2 * ADD * mag
    if add is not None:
        e = e + 2 * ADD * (mag + np.abs(oracle.bf16_bits_to_f64(add)))
    return y, e + BF16_HALF * (np.abs(y) + e)


def assert_near(got, ref, tol, what):
    assert got.shape == ref.shape
    off = np.abs(got - ref)
    bad = ~(off <= tol)                      # NaN is bad
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(off / np.maximum(tol, 1e-300)):.3g} " \
                          f"of its tolerance at {np.argwhere(bad)[0]}"


def assert_weights(got, ref, what):
    """fp64 arithmetic, then one rounding to fp32 (half a step, or half the
    smallest subnormal)."""
    tol = np.abs(ref) * 2.0 ** -24 * (1 + 1e-6) + 2.0 ** -150
    assert_near(got.astype(np.float64), ref, tol, what)
