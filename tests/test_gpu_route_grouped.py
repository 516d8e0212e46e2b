"""moe_route_grouped and moe_route_grouped_bucket against the fp64 oracle: ids
and buckets exact, weights to fp32's rounding."""

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_expert_amd as sme
from gpu_harness import DEV, to_dev
from layer_testlib import assert_weights, bits, dev_bf16

pytestmark = pytest.mark.gpu

# (T, E, k, groups, kept, group_top): one token to thousands; one expert; group sizes of one, odd, and not a divisor of
# the lanes' share; all slots taken; the largest k; E below, at and above multiples of 64; tokens and routes either side
# of 8, 16, 64 tokens and of 256, 1024 and 131072 routes; few tokens of many experts
SHAPES = [
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 8, 8, 4, 4, 2), (2, 64, 4, 64, 8, 2), (5, 60, 6, 12, 5, 1),
    (4, 512, 10, 1, 1, 1), (8, 512, 32, 16, 3, 2), (9, 96, 5, 3, 2, 2), (16, 160, 16, 8, 5, 1), (17, 65, 7, 5, 3, 2),
    (33, 1024, 32, 32, 7, 2), (40, 1000, 13, 1, 1, 1), (64, 63, 3, 7, 2, 2), (65, 768, 6, 6, 2, 1), (129, 128, 8, 8, 4, 2),
    (300, 320, 10, 5, 2, 2), (2049, 32, 32, 1, 1, 1), (4097, 16, 2, 4, 2, 2), (8200, 40, 32, 5, 5, 1),
    (13, 1000, 9, 8, 3, 2), (12, 512, 10, 1, 1, 1), (2047, 48, 32, 6, 6, 1), (4095, 100, 32, 4, 3, 2), (4096, 64, 32, 8, 5, 2),
]


def _inputs(T, E, dtype, seed):
    rng = np.random.default_rng(seed)
    logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    if dtype == "bf16":
        b = bits(logits)
        return oracle.bf16_bits_to_f64(b).astype(np.float32), dev_bf16(b), bias
    return logits, to_dev(logits), bias


def _check(logits, dev_logits, bias, rule, ref_args, what):
    T, E = logits.shape
    k = rule.k
    idx, w, b = sme.moe_route_grouped_bucket(dev_logits, None if bias is None else to_dev(bias), rule)
    idx2, w2 = sme.moe_route_grouped(dev_logits, None if bias is None else to_dev(bias), rule)
    torch.cuda.synchronize()
    assert torch.equal(idx, idx2) and torch.equal(w.view(torch.int32), w2.view(torch.int32))
    ref_idx, ref_w = oracle.route_grouped(logits, bias, *ref_args)
    assert np.array_equal(idx.cpu().numpy(), ref_idx), what
    assert_weights(w.cpu().numpy(), ref_w, what)
    ref_b = oracle.bucket_routes(ref_idx, E)
    for name, t in zip(sme.Buckets._fields, b):
        assert np.array_equal(t.cpu().numpy().reshape(np.shape(ref_b[name]) or (1,)), np.atleast_1d(ref_b[name])), name


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "T%d_E%d_k%d_g%d_%d_%d" % s)
@pytest.mark.parametrize("score,dtype,renorm,scale", [("sigmoid", "fp32", True, 2.5), ("softmax", "fp32", False, 16.0),
                                                      ("sigmoid", "bf16", False, 1.0), ("softmax", "bf16", True, 1.0)])
def test_route(shape, score, dtype, renorm, scale):
    T, E, k, groups, kept, top = shape
    logits, dev_logits, bias = _inputs(T, E, dtype, T + 7 * E)
    args = (k, score, groups, kept, top, renorm, scale)
    _check(logits, dev_logits, bias if T % 2 else None, sme.RouteRule(*args), args, shape)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,kept,top", [(9, 64, 8, 8, 4, 2), (37, 512, 10, 1, 1, 1), (20, 24, 6, 4, 2, 1)])
def test_masks(score, T, E, k, groups, kept, top):
    """Masked logits (-inf, NaN, the lowest values of fp32 and bf16), +inf, rows with nothing left and with fewer than
    k experts left; biases that mask, force and outweigh."""
    rng = np.random.default_rng(E)
    logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    for v, share in ((-np.inf, 0.2), (np.nan, 0.1), (np.finfo(np.float32).min, 0.1), (-3.3895313892515355e38, 0.1)):
        logits[rng.random((T, E)) < share] = v
    logits[0] = -np.inf
    logits[1] = np.nan
    logits[2, : E - 2] = np.finfo(np.float32).min          # two left, in the last group
    logits[3, 5] = np.inf
    logits[4, 3:6] = np.inf
    logits[5] = -200.0                                     # scores near zero, all alive
    logits[6] = 88.0
    logits[7] = -3.2e38                                    # the lowest that does not mask
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    bias[[1, E - 1]] = -np.inf
    bias[2] = np.nan
    bias[E // 2] = np.inf
    bias[E // 2 + 1] = -1e30
    for b in (None, bias):
        for renorm in (True, False):
            args = (k, score, groups, kept, top, renorm, 1.5)
            _check(logits, to_dev(logits), b, sme.RouteRule(*args), args, (score, b is None, renorm))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_near_ties(score):
    """Scores that agree in fp32 and differ in fp64 (large logits, a common bias), and exact ties."""
    E, k = 256, 8
    rng = np.random.default_rng(5)
    base = np.float32(12.0)
    logits = np.full((8, E), base, np.float32)
    for t in range(8):
        logits[t] += rng.integers(0, 4, E) * np.spacing(base) * np.float32(t)
    bias = np.full(E, 0.25, np.float32)
    for b in (None, bias):
        args = (k, score, 8, 3, 2, True, 1.0)
        _check(logits, to_dev(logits), b, sme.RouteRule(*args), args, score)


def test_no_tokens():
    idx, w, b = sme.moe_route_grouped_bucket(torch.empty((0, 64), device=DEV), None, sme.RouteRule(4, groups=8, groups_kept=2))
    assert idx.shape == (0, 4) and w.shape == (0, 4)


def test_refusals():
    logits = torch.zeros((2, 64), device=DEV)
    with pytest.raises(sme.MoeError) as e:
        sme.moe_route_grouped(logits, None, sme.RouteRule(9, groups=8, groups_kept=1))
    assert e.value.status == 2
    with pytest.raises(sme.MoeError):
        sme.moe_route_grouped(logits, None, sme.RouteRule(0))
    with pytest.raises(ValueError, match="contiguous"):
        sme.moe_route_grouped(torch.zeros((64, 2), device=DEV).t(), None, sme.RouteRule(4))
    with pytest.raises(ValueError, match="bias"):
        sme.moe_route_grouped(logits, torch.zeros(63, device=DEV), sme.RouteRule(4))
    with pytest.raises(TypeError, match="bias"):
        sme.moe_route_grouped(logits, torch.zeros(64, device=DEV, dtype=torch.bfloat16), sme.RouteRule(4))
    with pytest.raises(ValueError, match="topk_idx"):
        sme.moe_route_grouped(logits, None, sme.RouteRule(4), torch.empty((2, 3), dtype=torch.int32, device=DEV))


def test_graph_replays():
    """Two captured calls of different sizes, replayed with new logits and eager calls between."""
    rules = [(sme.RouteRule(8, "sigmoid", 8, 4), (8, "sigmoid", 8, 4, 2, True, 1.0), 4, 256),
             (sme.RouteRule(6, "softmax", 4, 2, 1, False), (6, "softmax", 4, 2, 1, False, 1.0), 700, 64)]
    state = []
    for rule, args, T, E in rules:
        logits = torch.empty((T, E), device=DEV)
        logits.normal_()
        out = sme.moe_route_grouped_bucket(logits, None, rule)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sme.moe_route_grouped_bucket(logits, None, rule, *out)
        state.append((graph, logits, out, args, E))
    rng = np.random.default_rng(1)
    for _ in range(3):
        for graph, logits, (idx, w, b), args, E in state:
            new = rng.standard_normal(tuple(logits.shape)).astype(np.float32)
            logits.copy_(to_dev(new))
            graph.replay()
            torch.cuda.synchronize()
            ref_idx, ref_w = oracle.route_grouped(new, None, *args)
            assert np.array_equal(idx.cpu().numpy(), ref_idx)
            assert_weights(w.cpu().numpy(), ref_w, "replay")
            ref_b = oracle.bucket_routes(ref_idx, E)
            assert np.array_equal(b.route_src.cpu().numpy(), ref_b["route_src"])
            assert np.array_equal(b.active_experts.cpu().numpy(), ref_b["active_experts"])
