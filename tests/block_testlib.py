"""Inputs and tolerances of the tests of the block-scaled 8-bit operators."""

import numpy as np
import torch

import oracle
import sparse_moe_expert_amd as sme
from gpu_harness import DEV
from layer_testlib import ADD, BF16_HALF

E4M3 = torch.float8_e4m3fn
FP32_HALF = 2.0 ** -24


def blocks(n):
    return -(-n // 128)


def codes(rng, *shape):
    """Random finite e4m3 codes, as values: every exponent, mostly the upper ones."""
    b = rng.integers(0x20, 0x7F, shape).astype(np.uint8) | (rng.integers(0, 2, shape).astype(np.uint8) << 7)
    small = rng.random(shape) < 0.05
    b = np.where(small, b & 0x8F, b)                                   # subnormals and zeros
    return oracle.e4m3_table()[b]


def random_tokens(rng, T, K):
    return codes(rng, T, K), (rng.uniform(0.5, 2.0, (T, blocks(K))) / 256).astype(np.float32)


def random_weight(rng, *shape):
    *lead, N, K = shape
    return codes(rng, *shape), (rng.uniform(0.5, 2.0, (*lead, blocks(N), blocks(K))) / (128 * np.sqrt(K))).astype(np.float32)


def dev_codes(v):
    """Code values -> float8 on the device (exact)."""
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(E4M3).to(DEV)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def dev_tokens(t):
    return sme.Fp8Tokens(dev_codes(t[0]), dev(t[1]))


def dev_weight(w):
    return sme.Fp8Weight(dev_codes(w[0]), dev(w[1]))


def dev_experts(gate, up, down):
    return sme.Fp8Experts(*(t for q, s in (gate, up, down) for t in (dev_codes(q), dev(s))))


def as_f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def terms(K):
    """Relative to the sum of magnitudes: the additions inside a block (each product is exact) and, per block, the scales'
    product, its multiplication and an addition, each off by at most ADD of a partial sum; sums of parts of the blocks may
    be added once more."""
    return (min(K, 128) + 4 * blocks(K) + 8) * ADD


KEPT = 2.0 ** -13


def group_squares(x, w):
    """[T, N]: sum over groups of 8 neighbouring reduction indices of (max |x| * max |w|)^2."""
    top = lambda a: np.abs(a).reshape(a.shape[0], -1, 8).max(axis=2) ** 2  # noqa: E731
    return top(x) @ top(w).T


def product_error(x, w, mag):
    """Bound of the error of x w^T from the matrix instruction and the sums behind it.  The instruction adds the products of
    8 neighbouring indices at the weight of the largest, M, and drops what lies more than 13 bits below its leading one
    (measured with powers of two: 2^16 - 2^3 is kept, 2^16 - 2^2 is 2^16; with any other index of the block, or C, all 24
    bits count).  So 7 of the 8 are cut, towards zero, by less than 2^-13 M each.  The inputs' signs are independent, so are
    the cuts': by Hoeffding's inequality their sum exceeds 8 sqrt(sum of the squared bounds) with probability
    2 exp(-32) = 3e-14, over the 2e8 outputs compared in all 5e-6."""
    return terms(x.shape[1]) * mag + 8 * KEPT * np.sqrt(7 * group_squares(x, w))


def linear_reference(x, w, bias=0.0):
    """(y, tolerance) of fp64 x [T, K], w [N, K]."""
    ref, mag = oracle.block.block_linear(x, w, bias)
    e = product_error(x, w, mag)
    return ref, e + BF16_HALF * (np.abs(ref) + e)


def code_reach(v, ev):
    """Largest distance from round(v) that a ratio within ev of v can be rounded to (rounding is monotone)."""
    q = oracle.block.round_e4m3(v)
    lim = lambda a: oracle.block.round_e4m3(np.clip(a, -448.0, 448.0))  # noqa: E731
    return np.maximum(np.abs(lim(v + ev) - q), np.abs(lim(v - ev) - q))


def encode_error(h, eh):
    """Bound of |decoded encoding of h' - decoded encoding of h| for any h' within eh of h, computed in fp32: the scale
    is off by at most the largest error in its block and the division's, the ratio by that, its own and the reciprocal's."""
    T, K = h.shape
    q, s = oracle.block.encode(h)
    es = oracle.block.scales(eh) + 2 * ADD * s                        # |amax' - amax| <= max eh
    per = lambda a: np.repeat(a, 128, axis=1)[:, :K]  # noqa: E731
    s_, es_ = per(s), per(es)
    v = h / s_
    ev = (eh + np.abs(v) * es_) / np.maximum(s_ - es_, 2.0 ** -126) + 4 * ADD * np.abs(v)
    dq = code_reach(v, ev)
    return s_ * dq + es_ * (np.abs(q) + dq)


def ffn_reference(x, gate, up, down, idx, w):
    """(y, tolerance): the products' errors as in product_error, through SiLU (slope at most 1.1; e^-g off by |g| ulp and
    a few), the product and the encoding; then the down product, a route's sum being kept to half a step of fp16 (2^-11), and
    the weighted sum."""
    T, H = x.shape
    E, I, _ = gate.shape  # noqa: E741
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        g, gm = oracle.block.block_linear(x[t], gate[e])
        u, um = oracle.block.block_linear(x[t], up[e])
        eg, eu = product_error(x[t], gate[e], gm), product_error(x[t], up[e], um)
        a = oracle.ffn.silu(g)
        h = a * u
        ea = 1.1 * eg + (np.abs(g) + 16) * ADD * np.abs(a)
        eh = ea * np.abs(u) + (np.abs(a) + ea) * eu + 2 * ADD * np.abs(h)
        q, s = oracle.block.encode(h)
        d = oracle.block.tokens(q, s)
        dh = encode_error(h, eh)
        o, om = oracle.block.block_linear(d, down[e])
        wide = 8 * np.sqrt(dh ** 2 @ (down[e] ** 2).T)            # the weights' signs are independent of dh: as in product_error
        eo = wide + product_error(d + dh * np.sign(d), down[e], om + wide)
        eo = eo + 2.0 ** -11 * (np.abs(o) + eo)
        wt = w[t, j].astype(np.float64)[:, None]
        np.add.at(y, t, wt * o)
        np.add.at(tol, t, np.abs(wt) * (eo + (idx.shape[1] + 2) * ADD * (np.abs(o) + eo)))
    return y, tol + BF16_HALF * (np.abs(y) + tol)


def routes(rng, T, E, k, skew=0.0):
    """Ids, gate weights and the buckets' route lists on the device."""
    z = rng.standard_normal((T, E)) + skew * rng.standard_normal(E)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    w = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    return idx, w, sme.moe_bucket_routes(dev(idx), E)


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))
