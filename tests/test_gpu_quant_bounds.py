"""The 4-bit products on operands that lie inside larger buffers: what follows
an operand has no part in the result, and what follows an output, or the
workspace of the size asked for, stays as it was."""

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_expert_amd as sme
from gpu_harness import DEV, to_dev
from layer_testlib import assert_near, bits, dev_bf16, f64, linear_tolerance, shared_reference, weight

pytestmark = pytest.mark.gpu

GUARD = 256


def _followed(a: np.ndarray, fill: int) -> torch.Tensor:
    """The array on the device, with bytes `fill` right behind it."""
    raw = np.ascontiguousarray(a).view(np.uint8).reshape(-1)
    t = to_dev(np.concatenate([raw, np.full(GUARD, fill, np.uint8)]))
    dtype = {np.dtype(np.uint8): torch.uint8, np.dtype(np.uint16): torch.bfloat16}[a.dtype]
    return t[:raw.size].view(dtype).view(a.shape)


def _handle(w, fmt):
    """Scales followed by 0xFF, which is NaN as e4m3 and as e8m0."""
    codes, scales, g = w
    return sme.QuantWeight(_followed(codes, 0xFF), _followed(scales, 0xFF),
                           None if g is None else to_dev(np.array([g], np.float32)), fmt)


def _guarded(shape, dtype):
    """A tensor of 7s, and the whole buffer whose head it is."""
    n = int(np.prod(shape))
    whole = torch.full((n + GUARD,), 7, dtype=dtype, device=DEV)
    return whole[:n].view(shape), whole[n:]


# (T, N, K): odd outputs a token and token counts on every kernel; N * K/16 and N * K/32 of every remainder by 4 with K
# an odd multiple of 32 (the last row's scales end inside a dword); split reductions of aligned and other scale rows
LINEAR = [
    (1, 7, 32), (3, 101, 160), (5, 17, 32), (7, 301, 672), (12, 33, 96), (15, 65, 4064), (17, 31, 224), (65, 257, 128),
    (31, 999, 1056), (33, 899, 8224), (63, 71, 96), (127, 1, 64), (129, 385, 1088), (33, 4097, 4096), (20, 33, 16384),
    (700, 11001, 96), (700, 11002, 96), (2501, 11003, 32), (300, 1001, 2080), (701, 11000, 160), (1301, 4091, 1184), (641, 8193, 608),
    (300, 22001, 64), (2049, 2561, 224), (900, 10241, 128),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear_in_larger_buffers(T, N, K, fmt):
    rng = np.random.default_rng(T + 3 * N + K)
    w = weight(rng, N, K, fmt)
    x, bias = bits(rng.standard_normal((T, K))), bits(rng.standard_normal(N)) if N % 3 else None
    y, behind = _guarded((T, N), torch.bfloat16)
    ws, past = _guarded((sme.moe_quant_linear_workspace_size(T, N, K),), torch.uint8)
    sme.moe_quant_linear(_followed(x, 0xFF), _handle(w, fmt), None if bias is None else _followed(bias, 0xFF), y, ws)
    torch.cuda.synchronize()
    assert torch.all(behind == 7) and torch.all(past == 7)
    ref, mag = oracle.quant_linear(x, w, fmt, bias)
    assert_near(f64(y), ref, linear_tolerance(ref, mag, K), (T, N, K, fmt))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,H,Is", [(3, 96, 160), (21, 416, 352), (100, 2080, 672), (1301, 96, 3040), (4100, 1056, 1056),
                                    (90, 544, 5216)])
def test_shared_in_larger_buffers(T, H, Is, fmt):
    rng = np.random.default_rng(T + H + Is)
    gate, up, down = weight(rng, Is, H, fmt), weight(rng, Is, H, fmt), weight(rng, H, Is, fmt)
    x, v, a = bits(rng.standard_normal((T, H))), bits(rng.standard_normal(H) / np.sqrt(H)), bits(rng.standard_normal((T, H)))
    y, behind = _guarded((T, H), torch.bfloat16)
    ws, past = _guarded((sme.moe_quant_shared_expert_workspace_size(T, H, Is),), torch.uint8)
    sme.moe_quant_shared_expert(_followed(x, 0xFF), *(_handle(m, fmt) for m in (gate, up, down)), _followed(v, 0xFF),
                                _followed(a, 0xFF), y, ws)
    torch.cuda.synchronize()
    assert torch.all(behind == 7) and torch.all(past == 7)
    ref, tol = shared_reference(x, gate, up, down, fmt, v, a)
    assert_near(f64(y), ref, tol, (T, H, Is, fmt))


# tokens on every kernel (the fewest, more of small weights, a split reduction, whole tiles), and the weight's sizes
RANGE = [(1, 20, 32), (3, 20, 64), (8, 70, 608), (40, 70, 96), (40, 300, 8224), (600, 300, 2048), (700, 11000, 96)]


@pytest.mark.parametrize("T,N,K", RANGE)
def test_linear_large_tokens(T, N, K):
    """Tokens of up to 2^124 with NVFP4 scales of 2^-6 .. 2^-9: every product and every sum of them lies inside fp32,
    sums of unscaled codes (16 of up to 6) would not."""
    rng = np.random.default_rng(K)
    codes, _, _ = weight(rng, N, K, "nvfp4")
    codes = codes & 0x77                                     # no signs: nothing cancels
    scales = np.array([1, 2, 4, 8], np.uint8)[rng.integers(0, 4, (N, K // 16))]
    w = (codes, scales, np.float32(2.0 ** -14))
    x = np.full((T, K), 2.0 ** -20)
    # 16 of every row: at most 16 * 6 * 2^124 * 2^-6 < 2^125
    x[:, 16:32] = 2.0 ** 124
    y = sme.moe_quant_linear(dev_bf16(bits(x)), sme.QuantWeight(to_dev(codes), to_dev(scales), to_dev(w[2].reshape(1))))
    ref, mag = oracle.quant_linear(bits(x), w, "nvfp4")
    assert_near(f64(y), ref, linear_tolerance(ref, mag, K), (T, N, K))


@pytest.mark.parametrize("T,N,K", RANGE)
def test_linear_small_tokens(T, N, K):
    """Tokens of the smallest normal numbers: products with small codes lie below fp32's normal range, the outputs by
    a large global scale do not."""
    rng = np.random.default_rng(K + 1)
    codes = weight(rng, N, K, "nvfp4")[0]
    scales = rng.integers(0x70, 0x7F, (N, K // 16)).astype(np.uint8)
    w = (codes, scales, np.float32(2.0 ** 60))
    x = bits(rng.choice([-1.5, -1.0, 1.0, 1.9921875], (T, K)) * 2.0 ** -126)
    y = sme.moe_quant_linear(dev_bf16(x), sme.QuantWeight(to_dev(codes), to_dev(scales), to_dev(w[2].reshape(1))))
    ref, mag = oracle.quant_linear(x, w, "nvfp4")
    assert_near(f64(y), ref, linear_tolerance(ref, mag, K), (T, N, K))


@pytest.mark.parametrize("T,N,K", RANGE)
def test_linear_mxfp4_scale_range(T, N, K):
    """Every code under the smallest and largest e8m0 scales: weights down to 2^-128, which bf16 has as subnormal numbers,
    and up to 6 * 2^125.  One weight and one token value a row that are not zero: the product is exact."""
    rng = np.random.default_rng(N)
    for lo, hi, size in ((0, 3, 100), (250, 253, -30)):
        codes = np.zeros((N, K // 2), np.uint8)
        codes[:, 3] = np.arange(N) % 16 * 0x11
        scales = rng.integers(lo, hi, (N, K // 32)).astype(np.uint8)
        x = np.zeros((T, K))
        x[np.arange(T), 6 + np.arange(T) % 2] = 2.0 ** size
        y = sme.moe_quant_linear(dev_bf16(bits(x)), sme.QuantWeight(to_dev(codes), to_dev(scales), None, "mxfp4"))
        ref, _ = oracle.quant_linear(bits(x), (codes, scales, None), "mxfp4")
        assert np.array_equal(f64(y), ref), (lo, size)


def test_refuses_tokens_beyond_32_bits():
    """2^32 + 1 tokens are not one (a tensor without memory: refused by its size, before anything else)."""
    w = sme.QuantWeight(torch.zeros((64, 16), dtype=torch.uint8, device=DEV),
                        torch.zeros((64, 1), dtype=torch.uint8, device=DEV), format="mxfp4")
    x = torch.empty(((1 << 32) + 1, 32), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="tokens"):
        sme.moe_quant_linear(x, w)
    with pytest.raises(ValueError, match="tokens"):
        sme.moe_quant_shared_expert(x, w, w, w)


def test_refuses_a_workspace_that_is_no_tensor():
    w = sme.QuantWeight(torch.zeros((32, 16), dtype=torch.uint8, device=DEV),
                        torch.zeros((32, 1), dtype=torch.uint8, device=DEV), format="mxfp4")
    x = torch.zeros((2, 32), dtype=torch.bfloat16, device=DEV)
    for workspace in (bytearray(1024), 1024):
        with pytest.raises(TypeError, match="workspace"):
            sme.moe_quant_linear(x, w, workspace=workspace)
        with pytest.raises(TypeError, match="workspace"):
            sme.moe_quant_shared_expert(x, w, w, w, workspace=workspace)
    with pytest.raises(ValueError, match="contiguous"):
        sme.moe_quant_linear(x, w, workspace=torch.zeros((64, 32), dtype=torch.uint8, device=DEV).t())
