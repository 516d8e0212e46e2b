"""Pins of the oracle's block-scaled 8-bit values: hand-worked encodings, brute force over every code, torch's own
conversion, exactly rounded sums; and mistakes planted in it, which these catch."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import block


def check_rounding():
    finite = np.array([v for v in oracle.e4m3_table() if not np.isnan(v)])
    values = np.unique(finite)
    mid = (values[1:] + values[:-1]) / 2
    v = np.concatenate([values, mid, np.nextafter(mid, np.inf), np.nextafter(mid, -np.inf),
                        np.random.default_rng(0).standard_normal(2000) * 100])
    v = v[np.abs(v) <= 448.0]
    got = block.round_e4m3(v)
    even = {float(b): i % 2 == 0 for i, b in enumerate(oracle.e4m3_table()[:127])}
    for a, r in zip(v, got):
        d = np.abs(values - a)
        near = values[d == d.min()]
        want = near[0] if len(near) == 1 else next(n for n in near if even[abs(float(n))])
        assert r == want, (a, r, want)


def test_rounding():
    check_rounding()
    v = np.float32(np.random.default_rng(1).standard_normal(5000) * 60)
    v = v[np.abs(v) <= 448]
    assert np.array_equal(block.round_e4m3(v.astype(np.float64)), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def check_encode():
    v = np.zeros((2, 130))
    v[0, 3], v[0, 4], v[0, 129] = 896.0, 3.3, -56.0
    v[1, 0], v[1, 1], v[1, 2] = np.nan, np.inf, 7.0
    q, s = block.encode(v)
    assert s.tolist() == [[2.0, 0.125], [0.015625, 2.0 ** -126]]
    assert q[0, 3] == 448 and q[0, 4] == 1.625 and q[0, 129] == -448     # 3.3 / 2 = 1.65
    assert np.isnan(q[1, :2]).all() and q[1, 2] == 448 and not q[1, 3:].any()


def test_encode():
    check_encode()


def check_weight():
    q = np.ones((3, 130, 260))
    s = np.arange(1, 19, dtype=np.float32).reshape(3, 2, 3)
    w = block.weight(q, s)
    assert w[1, 129, 259] == 12 and w[0, 0, 128] == 2 and w[2, 127, 0] == 13


def test_weight():
    check_weight()


def test_linear_exact():
    rng = np.random.default_rng(2)
    x, w = rng.integers(-8, 9, (3, 40)) / 16, rng.integers(-8, 9, (5, 40)) / 8
    y, mag = block.block_linear(x, w, np.arange(5.0))
    for t in range(3):
        for n in range(5):
            assert y[t, n] == float(sum(Fraction(a) * Fraction(b) for a, b in zip(x[t], w[n])) + n)
    assert (mag >= np.abs(y)).all()


def test_norm():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    y, total = block.norm(x, None, np.full(4, 2.0), 1.0, 0.0, None)
    assert np.allclose(y, [[3.6, 4.8, 0, 0]])                     # rms 2.5, factor 3
    y, total = block.norm(x, -x + 1.25, np.ones(4), 0.0, 0.0, lambda v: np.full_like(v, 2.0))
    assert np.array_equal(total, np.full((1, 4), 1.25)) and np.array_equal(y, np.ones((1, 4)))


def check_ffn():
    """Values that every encoding holds exactly: the plain mixture."""
    x = np.array([[1.0, 2.0]])
    gate = np.array([[[50.0, 0.0], [0.0, 50.0]]] * 2)             # SiLU(g) = g to 1e-20
    up = np.array([[[0.01, 0.0], [0.0, 0.01]], [[0.02, 0.0], [0.0, 0.02]]])
    down = np.array([[[1.0, 0.0], [0.0, 1.0]], [[0.0, 1.0], [1.0, 0.0]]])
    y = block.block_expert_ffn(x, gate, up, down, np.array([[1, 0]]), np.array([[0.25, 0.75]]))
    # expert 0: h = (.5, 2), expert 1: (1, 4), swapped
    assert np.allclose(y, [[0.25 * 4 + 0.75 * 0.5, 0.25 * 1 + 0.75 * 2]], rtol=1e-12)


def test_ffn():
    check_ffn()


def test_ffn_is_the_mixture():
    """h in 8 bits is h to half a step (2^-4): the mixture with h itself lies that near."""
    rng = np.random.default_rng(3)
    T, H, I, E = 4, 32, 160, 5  # noqa: E741
    x, gate, up, down = rng.standard_normal((T, H)), *(rng.standard_normal(s) for s in ((E, I, H), (E, I, H), (E, H, I)))
    idx = np.array([[0, 3], [1, 2], [4, 0], [2, 3]])
    w = rng.uniform(0, 1, (T, 2))
    y = block.block_expert_ffn(x, gate, up, down, idx, w)
    for t in range(T):
        ref, reach = np.zeros(H), np.zeros(H)
        for e, g in zip(idx[t], w[t]):
            h = oracle.ffn.silu(gate[e] @ x[t]) * (up[e] @ x[t])
            ref += g * (down[e] @ h)
            reach += g * (np.abs(down[e]) @ np.maximum(2.0 ** -4 * np.abs(h), 2.0 ** -10 * block.scales(h[None])[0].max()))
        assert (np.abs(y[t] - ref) <= reach + 1e-12).all()


@pytest.mark.parametrize("mistake,check", [
    ("ties away", check_rounding), ("no subnormals", check_rounding), ("nan in amax", check_encode),
    ("one scale a row", check_encode), ("scale by column", check_weight), ("weights swapped", check_ffn)])
def test_planted_mistakes(monkeypatch, mistake, check):
    if mistake == "ties away":
        def wrong(v):
            _, e = np.frexp(v)
            step = np.ldexp(1.0, np.maximum(e - 4, -9))
            return np.sign(v) * np.floor(np.abs(v) / step + 0.5) * step
        monkeypatch.setattr(block, "round_e4m3", wrong)
    elif mistake == "no subnormals":
        right = block.round_e4m3
        monkeypatch.setattr(block, "round_e4m3", lambda v: np.where(np.abs(v) < 2.0 ** -6, 0.0, right(v)))
    elif mistake == "nan in amax":
        monkeypatch.setattr(block, "scales", lambda v: np.stack(
            [np.maximum(np.abs(v[:, b:b + 128]).max(axis=1) / 448.0, 2.0 ** -126) for b in range(0, v.shape[1], 128)], axis=1))
    elif mistake == "one scale a row":
        monkeypatch.setattr(block, "scales", lambda v: np.repeat(
            np.abs(np.nan_to_num(v, posinf=0)).max(axis=1, keepdims=True) / 448.0, -(-v.shape[1] // 128), axis=1))
    elif mistake == "scale by column":
        right = block._per_value
        monkeypatch.setattr(block, "_per_value", lambda s, n, axis: right(s[..., ::-1] if axis == -1 else s, n, axis))
    elif mistake == "weights swapped":
        right = block.block_expert_ffn
        monkeypatch.setattr(block, "block_expert_ffn", lambda x, g, u, d, i, w: right(x, g, u, d, i, w[:, ::-1]))
    with np.errstate(all="ignore"), pytest.raises(AssertionError):
        check()
