"""Pins of the oracle's grouped routing and 4-bit products: hand-worked cases,
the softmax rule it generalises, brute force over sets, exactly rounded dot
products with closed-form decoders; and mistakes planted in it, which the
hand-worked cases catch."""

import itertools
import math

import numpy as np
import pytest

import oracle
from oracle import grouped
from nvfp4_testlib import bf16_values, e2m1_closed_form, e4m3_closed_form, pack_codes

INF, NAN = float("inf"), float("nan")


def _logit(p):
    return math.log(p / (1 - p))


# sigmoid scores .9 .1 | .6 .5 | .55 .52 | .2 .1: the group sums are 1.0, 1.1, 1.07, .3, the maxima .9, .6, .55, .2
ROW = np.array([[_logit(p) for p in (0.9, 0.1, 0.6, 0.5, 0.55, 0.52, 0.2, 0.1)]])


def check_hand_worked():
    idx, w = oracle.route_grouped(ROW, None, 3, "sigmoid", 4, 2, 2, False, 2.0)
    assert idx.tolist() == [[2, 4, 5]]                        # groups 1 and 2; expert 0 is left out
    assert np.allclose(w, [[1.2, 1.1, 1.04]], rtol=1e-14)
    idx, w = oracle.route_grouped(ROW, None, 3, "sigmoid", 4, 2, 1, True, 1.0)
    assert idx.tolist() == [[0, 2, 3]]                        # groups 0 and 1
    assert np.allclose(w, [[0.45, 0.3, 0.25]], rtol=1e-14)
    bias = np.array([0, 0, 0, 0, 0, 0, 0, 0.95])              # the bias selects, it does not weigh
    idx, w = oracle.route_grouped(ROW, bias, 2, "sigmoid", 1, 1, 1, True, 1.0)
    assert idx.tolist() == [[7, 0]]
    assert np.allclose(w, [[0.1, 0.9]], rtol=1e-14)
    # masks: expert 0 by -inf, 2 by NaN; group 1 keeps .5 alone
    row = ROW.copy()
    row[0, 0], row[0, 2] = -INF, NAN
    idx, w = oracle.route_grouped(row, None, 4, "sigmoid", 4, 2, 2, False, 1.0)
    assert idx.tolist() == [[4, 5, 3, 2]]                     # groups 2 (1.07) and 1 (.5); the masked one last
    assert np.allclose(w, [[0.55, 0.52, 0.5, 0.0]], rtol=1e-14)
    # nothing left: lowest groups, lowest ids, no weight
    idx, w = oracle.route_grouped(np.full((1, 8), -3.4e38), None, 3, "softmax", 4, 2, 2, True, 1.0)
    assert idx.tolist() == [[0, 1, 2]] and not w.any()
    # ties go to the lower group and the lower expert
    idx, w = oracle.route_grouped(np.zeros((1, 8)), None, 4, "sigmoid", 4, 2, 2, True, 1.0)
    assert idx.tolist() == [[0, 1, 2, 3]] and np.allclose(w, 0.25)


def test_hand_worked():
    check_hand_worked()


def test_reduces_to_softmax_topk():
    rng = np.random.default_rng(1)
    logits = rng.standard_normal((5, 24)).astype(np.float32)
    ref = oracle.route_topk(logits, None, 6)
    idx, w = oracle.route_grouped(logits, None, 6, "softmax")
    assert np.array_equal(idx, ref[0]) and np.allclose(w, ref[1], rtol=1e-13)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_best_of_every_set(score):
    """The choice is the best of all sets of experts inside all sets of groups."""
    rng = np.random.default_rng(2)
    E, G, kept, k = 12, 4, 2, 3
    for _ in range(20):
        logits, bias = rng.standard_normal((1, E)), rng.standard_normal(E) * 0.2
        e = np.exp(logits[0])
        s = e / e.sum() if score == "softmax" else e / (1 + e)
        c = s + bias
        pair = lambda g: max(a + b for a, b in itertools.combinations(c[3 * g:3 * g + 3], 2))  # noqa: E731
        gs = max(itertools.combinations(range(G), kept), key=lambda q: sum(pair(g) for g in q))
        best = max(itertools.combinations([e for e in range(E) if e // 3 in gs], k), key=lambda q: sum(c[e] for e in q))
        idx, w = oracle.route_grouped(logits, bias, k, score, G, kept, 2, False, 1.0)
        assert sorted(idx[0].tolist()) == sorted(best)
        assert np.allclose(w[0], s[idx[0]], rtol=1e-12)


def _random_weight(rng, N, K, fmt):
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    if fmt == "nvfp4":
        scales, g = rng.integers(0, 0x7F, (N, K // 16)).astype(np.uint8), np.float32(0.037)
        dense = [[e2m1_closed_form(int(codes[n, k])) * e4m3_closed_form(int(scales[n, k // 16])) * float(g) for k in range(K)]
                 for n in range(N)]
    else:
        scales, g = rng.integers(2, 253, (N, K // 32)).astype(np.uint8), None
        dense = [[e2m1_closed_form(int(codes[n, k])) * 2.0 ** (int(scales[n, k // 32]) - 127) for k in range(K)]
                 for n in range(N)]
    return (pack_codes(codes), scales, g), np.array(dense)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_linear_exactly_rounded(fmt):
    rng = np.random.default_rng(3)
    weight, dense = _random_weight(rng, 5, 64, fmt)
    x = rng.integers(0x3E00, 0x4100, (3, 64)).astype(np.uint16) | (rng.integers(0, 2, (3, 64)) << 15).astype(np.uint16)
    bias = rng.integers(0x3E00, 0x4100, 5).astype(np.uint16)
    y, mag = oracle.quant_linear(x, weight, fmt, bias)
    ref = [[math.fsum([a * b for a, b in zip(xr, wr)] + [bv]) for wr, bv in zip(dense, bf16_values(bias))]
           for xr in bf16_values(x)]
    assert np.all(np.abs(y - ref) <= 1e-14 * mag)


def test_shared_expert_is_the_linear_chain():
    rng = np.random.default_rng(4)
    T, H, Is = 3, 64, 32
    gate, up, down = (_random_weight(rng, n, k, "nvfp4")[0] for n, k in ((Is, H), (Is, H), (H, Is)))
    x = rng.integers(0x3C00, 0x3E00, (T, H)).astype(np.uint16)
    v = rng.integers(0x3C00, 0x3E00, H).astype(np.uint16)
    add = rng.integers(0x3C00, 0x4000, (T, H)).astype(np.uint16)
    y = oracle.quant_shared_expert(x, gate, up, down, "nvfp4", v, add)
    dense = [oracle.quant.dequant(*m, "nvfp4") for m in (gate, up, down)]
    for t in range(T):
        xt = bf16_values(x[t])
        g, u = dense[0] @ xt, dense[1] @ xt
        ref = dense[2] @ (g / (1 + np.exp(-g)) * u) / (1 + math.exp(-float(xt @ bf16_values(v)))) + bf16_values(add[t])
        assert np.allclose(y[t], ref, rtol=1e-12)


@pytest.mark.parametrize("slip", ["bias_in_weight", "max_for_sum", "masked_scores", "ties_up"])
def test_planted_mistakes_fail(slip, monkeypatch):
    right = grouped.route_grouped

    def wrong(logits, bias, k, score="sigmoid", groups=1, kept=1, top=2, renorm=True, scale=1.0):
        if slip == "max_for_sum":
            top = 1
        if slip == "ties_up":
            idx, w = right(logits[:, ::-1], None if bias is None else bias[::-1], k, score, groups, kept, top, renorm, scale)
            return logits.shape[1] - 1 - idx, w
        if slip == "masked_scores":
            logits = np.where(np.isnan(logits), 0.0, logits)
        idx, w = right(logits, bias, k, score, groups, kept, top, renorm, scale)
        if slip == "bias_in_weight" and bias is not None:
            w = w + bias[idx]
        return idx, w

    monkeypatch.setattr(oracle, "route_grouped", wrong)
    with pytest.raises(AssertionError):
        check_hand_worked()
