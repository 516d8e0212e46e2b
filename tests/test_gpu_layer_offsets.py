"""Operands of more than 2^31 elements: the rows at their start, about the
places where 32-bit offsets end, and at their end, against the oracle."""

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_expert_amd as sme
from gpu_harness import DEV
from layer_testlib import assert_near, assert_weights, f64, linear_tolerance

pytestmark = pytest.mark.gpu


def _normal(*shape):
    """bf16 normal values, made in pieces (no fp32 tensor of the whole size)."""
    t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(1)
    for piece in t.split(max(1, (1 << 26) // shape[1])):
        piece.copy_(torch.randn(piece.shape, generator=gen, device=DEV))
    return t


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def _rows(n, width):
    """Rows either side of every multiple of 2^31 elements, the first and the last."""
    at = [r + d for r in range(0, n, -(-(1 << 31) // width)) for d in (-1, 0, 1)] + [n - 2, n - 1]
    return sorted({min(max(r, 0), n - 1) for r in at})


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
# tokens, outputs, and codes (2^32 bytes of them) beyond
@pytest.mark.parametrize("T,N,K", [(70001, 33, 32768), (70001, 700, 32768), (1 << 20, 2051, 32), (2, 270001, 32768), (40, 270001, 32768)])
def test_linear(T, N, K, fmt):
    gen = torch.Generator(device=DEV).manual_seed(N)
    group, lo, hi = (16, 0x20, 0x50) if fmt == "nvfp4" else (32, 118, 125)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=gen)
    scales = torch.randint(lo, hi, (N, K // group), dtype=torch.uint8, device=DEV, generator=gen)
    g = np.float32(0.2 / np.sqrt(K)) if fmt == "nvfp4" else None
    x = _normal(T, K)
    y = sme.moe_quant_linear(x, sme.QuantWeight(codes, scales, None if g is None else torch.full((1,), float(g), device=DEV), fmt))
    ts, ns = _rows(T, max(N, K)), _rows(N, K // 2)
    if N * K >= 1 << 32:
        ns = sorted({*ns, *(n + d for n in range(0, N, (1 << 32) // (K // 2)) for d in (-1, 0, 1) if 0 <= n + d < N)})
    elif N < 4096:
        ns = list(range(N))
    it, io = torch.tensor(ts, device=DEV), torch.tensor(ns, device=DEV)
    ref, mag = oracle.quant_linear(_bits(x[it]), (codes[io].cpu().numpy(), scales[io].cpu().numpy(), g), fmt)
    assert_near(f64(y[it][:, io]), ref, linear_tolerance(ref, mag, K), (T, N, K, fmt))


def test_route():
    """2^22 tokens of 1024 experts, 2^24 routes: rows against the oracle, and buckets against a stable sort."""
    T, E, k = 1 << 22, 1024, 4
    logits = _normal(T, E)
    args = (k, "softmax", 8, 3, 2, True, 1.0)
    idx, w, b = sme.moe_route_grouped_bucket(logits, None, sme.RouteRule(*args))
    ts = _rows(T, E)
    it = torch.tensor(ts, device=DEV)
    ref_idx, ref_w = oracle.route_grouped(oracle.bf16_bits_to_f64(_bits(logits[it])).astype(np.float32), None, *args)
    assert np.array_equal(idx[it].cpu().numpy(), ref_idx)
    assert_weights(w[it].cpu().numpy(), ref_w, "weights")
    flat = idx.flatten()
    assert int(flat.min()) >= 0 and int(flat.max()) < E
    order = torch.sort(flat, stable=True).indices.int()
    assert torch.equal(b.route_src, order)
    assert torch.equal(b.route_pos[order.long()], torch.arange(T * k, dtype=torch.int32, device=DEV))
    assert torch.equal(b.expert_count, torch.bincount(flat, minlength=E).int())
