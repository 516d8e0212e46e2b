"""Grouped routing over the documented range of the bias: values down to just
above -3.3e38 are live, and the sum of two of them lies outside fp32."""

import numpy as np
import pytest
import torch

import sparse_moe_expert_amd as sme
from gpu_harness import to_dev
from test_gpu_route_grouped import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_hand_worked_overflows(score):
    """Two groups of two experts, zero logits: an empty group against a live one whose fp32 sum is -inf; two such sums
    of different size; and their like above."""
    logits = np.zeros((1, 4), np.float32)
    for bias, chosen in (((-np.inf, -np.inf, -2.4e38, -2.4e38), [2, 3]), ((-2.9e38, -2.9e38, -2.0e38, -2.0e38), [2, 3]),
                         ((-2.0e38, -2.0e38, -2.9e38, -2.9e38), [0, 1]), ((2.0e38, 2.0e38, 2.9e38, 2.9e38), [2, 3]),
                         ((np.nan, -3.4e38, -3.2e38, -1.0e38), [3, 2]), ((1.6e38, 1.6e38, 1.8e38, 1.8e38), [2, 3]),
                         ((np.inf, -3.2e38, 3.2e38, 3.2e38), [0, 1])):
        b = np.array(bias, np.float32)
        idx, w = sme.moe_route_grouped(to_dev(logits), to_dev(b), sme.RouteRule(2, score, 2, 1, 2))
        torch.cuda.synchronize()
        assert idx.tolist() == [chosen], bias
        assert w.tolist() == [[0.5, 0.5]], bias
        args = (2, score, 2, 1, 2, True, 1.0)
        _check(logits, to_dev(logits), b, sme.RouteRule(*args), args, bias)


# tokens either side of one launch; few and many experts a lane; groups of two, and not a power of two of them
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,kept", [(1, 8, 3, 4, 2), (7, 64, 8, 8, 3), (40, 512, 10, 16, 5), (65, 60, 5, 12, 4),
                                               (33, 1024, 16, 32, 9), (9, 128, 4, 64, 3)])
def test_large_biases(score, T, E, k, groups, kept):
    """Whole groups of biases of either sign near the range's ends, masked ones and ordinary ones, in rows that keep
    few of them."""
    rng = np.random.default_rng(E + T)
    logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    logits[rng.random((T, E)) < 0.1] = -np.inf
    size = E // groups
    for kind in ("low", "high", "both"):
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
        for g in range(groups):
            part = slice(g * size, (g + 1) * size)
            draw = rng.integers(0, 8) if g < groups - 1 else 7
            far = rng.uniform(1.0e38, 3.29e38, size).astype(np.float32)
            if 1 <= draw <= 2:
                bias[part] = -np.inf
            elif draw > 2:
                bias[part] = far if kind == "high" else -far if kind == "low" else far * rng.choice([-1, 1], size)
        for top in (1, 2):
            args = (k, score, groups, kept, top, True, 1.0)
            _check(logits, to_dev(logits), bias, sme.RouteRule(*args), args, (score, kind, top))
