"""The block-scaled 8-bit operators against the fp64 oracle, with tolerances counted from the arithmetic
(block_testlib)."""

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_expert_amd as sme
from block_testlib import (E4M3, FP32_HALF, as_f64, blocks, code_reach, codes, dev, dev_codes, dev_experts, dev_tokens,
                           dev_weight, ffn_reference, linear_reference, terms, random_tokens, random_weight, routes, same_bits)
from gpu_harness import DEV
from layer_testlib import ADD, BF16_HALF, assert_near, bits, dev_bf16

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def bf16_values(a):
    return oracle.bf16_bits_to_f64(bits(a))


# ------------------------------------------------------------------ encoding

def check_encoded(tokens, v, ev, what):
    """Codes and scales of fp64 values v that the kernel holds to within ev (relative)."""
    q, s = as_f64(tokens.q), tokens.scale.cpu().numpy().astype(np.float64)
    ref = oracle.block.scales(v)
    assert_near(s, ref, ref * (ev + FP32_HALF) * (1 + 1e-6), f"{what}: scales")
    ratio = v / np.repeat(ref, 128, axis=1)[:, :v.shape[1]]
    finite = np.isfinite(v)
    assert np.array_equal(np.isnan(q), ~finite), f"{what}: NaN codes"
    ratio, got = np.where(finite, ratio, 0.0), np.where(finite, q, 0.0)
    # the value's error, the largest's (in the scale), and the scale's, the reciprocal's and the product's roundings
    reach = code_reach(ratio, np.abs(ratio) * (2 * ev + 4 * FP32_HALF))
    assert_near(got, oracle.block.round_e4m3(ratio), reach, f"{what}: codes")


QUANT = [(1, 16), (1, 128), (2, 144), (3, 48), (33, 720), (5, 2048), (2, 32768), (257, 144), (1000, 528), (64, 4096), (7, 5120)]


@pytest.mark.parametrize("T,K", QUANT)
def test_quantize(T, K):
    rng = np.random.default_rng(T + K)
    x = bf16_values(rng.standard_normal((T, K)) * np.exp(rng.standard_normal((T, 1)) * 4))
    x[rng.random((T, K)) < 0.1] = 0.0
    out = sme.empty_fp8_tokens(T + 1, K, DEV)
    out.q.view(torch.uint8).fill_(0x55)
    out.scale.fill_(7.0)
    got = sme.moe_block_quantize(dev_bf16(bits(x)), sme.Fp8Tokens(out.q[:T], out.scale[:T]))
    torch.cuda.synchronize()
    check_encoded(got, x, 0.0, (T, K))
    assert (out.q[T:].view(torch.uint8) == 0x55).all() and (out.scale[T:] == 7.0).all()    # behind the last row


def test_quantize_edges():
    """Zeros, one value, ties, the smallest and largest numbers, infinities and NaN in one block only."""
    x = np.zeros((9, 272))
    x[1, 130] = -3.0
    x[2, :128] = np.arange(128) / 128 * 448                        # many ties: the scale is 447.. / 448
    x[3, :16] = 448.0 - np.arange(16) * 17.0                       # scale 1: halves between codes
    x[4] = 2.0 ** -133                                             # below every scale
    x[5, 0], x[5, 1] = 3.3e38, 1e30
    x[6, 5], x[6, 7] = INF, 2.0
    x[7, 140], x[7, 141] = NAN, -INF
    x[8, 256:] = -INF
    x = bf16_values(x)
    check_encoded(sme.moe_block_quantize(dev_bf16(bits(x))), x, 0.0, "edges")


NORM = [(1, 16), (1, 2048), (2, 144), (3, 2064), (33, 720), (5, 4112), (300, 2560), (2, 8208), (3, 16400), (2, 32768), (1000, 528),
        (4100, 640)]


@pytest.mark.parametrize("stream", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", NORM)
def test_norm(T, H, stream):
    rng = np.random.default_rng(T + H)
    x = bf16_values(rng.standard_normal((T, H)))
    offset, eps = float((T + H) % 32 // 16), 1e-5
    w = bf16_values(1.0 - offset + 0.1 * rng.standard_normal(H))
    res = None
    if stream is torch.bfloat16:
        res = bf16_values(3 * rng.standard_normal((T, H)))
    elif stream is torch.float32:
        res = np.float32(3 * rng.standard_normal((T, H))).astype(np.float64)
    held = None if res is None else dev(res.astype(np.float32)).to(stream)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    tokens, r = sme.moe_norm_quantize(dev_bf16(bits(x)), dev_bf16(bits(w)), held, eps, offset, y=y)
    torch.cuda.synchronize()
    # a sum rounded to fp32, then to its type
    single = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731
    rounded = single if stream is torch.float32 else lambda a: bf16_values(single(a))
    ref, total = oracle.block.norm(x, res, w, offset, eps, rounded)
    if res is None:
        assert r is None
    else:
        assert np.array_equal(as_f64(r) if stream is torch.bfloat16 else r.double().cpu().numpy(), rounded(total))
    # the reciprocal root and weight + offset rounded to fp32, two products
    ev = 4.1 * FP32_HALF
    check_encoded(tokens, ref, ev, (T, H, stream))
    assert_near(as_f64(y), ref, BF16_HALF * np.abs(ref) * (1 + ev) + ev * np.abs(ref), "y")
    # without y, and with the residual updated in place: the same bits
    again, r2 = sme.moe_norm_quantize(dev_bf16(bits(x)), dev_bf16(bits(w)), held, eps, offset, residual_out=held)
    torch.cuda.synchronize()
    assert same_bits(again.q, tokens.q) and torch.equal(again.scale, tokens.scale)
    if res is not None:
        assert r2 is held and torch.equal(held, r)


def test_norm_range():
    """Rows of zeros, of numbers whose squares leave fp32, of tiny ones; a row with a NaN or an infinity is its own matter."""
    T, H = 7, 640
    rng = np.random.default_rng(5)
    x = bf16_values(rng.standard_normal((T, H)))
    x[0] = 0.0
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -110
    x[3, 1:] = 0.0
    x[5, 9] = INF
    x[6, 639] = NAN
    w = bf16_values(np.ones(H))
    y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    tokens, _ = sme.moe_norm_quantize(dev_bf16(bits(x)), dev_bf16(bits(w)), eps=1e-30, y=y)
    torch.cuda.synchronize()
    ref, _ = oracle.block.norm(x[:5], None, w, 0.0, 1e-30, None)
    ev = 4.1 * FP32_HALF
    check_encoded(sme.Fp8Tokens(tokens.q[:5], tokens.scale[:5]), ref, ev, "range")
    assert_near(as_f64(y[:5]), ref, BF16_HALF * np.abs(ref) * (1 + ev) + ev * np.abs(ref), "y")
    assert not torch.isfinite(y[5].float()).all() and torch.isnan(y[6].float()).all()
    assert torch.isnan(tokens.q[6].float()).all()


# ------------------------------------------------------------------ dense layer

# (T, N, K): one token to hundreds, either side of 1, 16, 32, 64, 128, 256; N of one, odd, of whole tiles and blocks; K of one
# piece, of part of a block, of whole blocks, and long
LINEAR = [
    (1, 1, 16), (1, 7, 64), (1, 2048, 2048), (2, 33, 96), (3, 100, 176), (4, 130, 2560), (5, 17, 32), (7, 300, 672),
    (8, 64, 1056), (9, 129, 288), (15, 65, 4096), (16, 256, 512), (17, 31, 224), (31, 127, 640), (32, 999, 1024),
    (33, 128, 2080), (63, 72, 96), (64, 512, 256), (65, 257, 128), (100, 640, 320), (127, 1, 64), (128, 128, 48),
    (129, 385, 1104), (255, 200, 16), (257, 512, 512), (1, 20, 32768), (40, 20, 16400), (600, 300, 2048),
    (4, 40, 12288), (4, 30, 32768), (600, 6500, 80), (513, 8200, 144), (300, 16390, 64), (20, 33, 16384), (17, 1000, 4128),
    (60, 700, 8192), (130, 2600, 4160), (24, 130, 32752), (512, 640, 640), (16, 30, 32768), (700, 11000, 96),
    (1025, 4100, 160), (33000, 260, 32), (650, 5000, 640), (1300, 4090, 1152), (256, 4096, 384), (2050, 2049, 272),
    # each kind of tile with odd sizes and a long reduction, whole and in parts
    (1, 9999, 4096), (12, 8200, 656), (16, 16385, 2064), (821, 9429, 1680), (2212, 1982, 1584), (69, 9536, 5600),
    (93, 9870, 1520), (451, 2055, 1504), (1725, 74, 7552), (40, 8235, 1632), (2872, 681, 1680), (419, 527, 7808), (2132, 8, 7008),
]


@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear(T, N, K):
    rng = np.random.default_rng(T * 1000 + N + K)
    x, w = random_tokens(rng, T, K), random_weight(rng, N, K)
    bias = bits(rng.standard_normal(N)) if (T + N) % 2 else None
    hx, hw, hb = dev_tokens(x), dev_weight(w), None if bias is None else dev_bf16(bias)
    out = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((max(sme.moe_block_linear_workspace_size(T, N, K), 16),), 0xFF, dtype=torch.uint8, device=DEV)
    y = sme.moe_block_linear(hx, hw, hb, out[:T], ws)
    y2 = sme.moe_block_linear(hx, hw, hb)
    torch.cuda.synchronize()
    assert same_bits(y, y2)                                            # reproducible
    assert torch.all(out[T:] == 7.0)                                   # rows behind the last token
    b = 0.0 if bias is None else oracle.bf16_bits_to_f64(bias)
    ref, tol = linear_reference(oracle.block.tokens(*x), oracle.block.weight(*w), b)
    assert_near(as_f64(y), ref, tol, (T, N, K))
    if N * T >= 64:
        assert np.linalg.norm(as_f64(y) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)


@pytest.mark.parametrize("T", [1, 5, 40, 200, 300])
def test_linear_every_code(T):
    """Each finite e4m3 weight code against unit tokens in each place of a block and a half: the products are exact."""
    K = 192
    table = oracle.e4m3_table()
    w = np.stack([np.roll(np.resize(table[~np.isnan(table)], K), n) for n in range(254)])
    x = np.zeros((T, K))
    x[np.arange(T), np.arange(T) % K] = 1.0
    tokens = (x, np.full((T, 2), 2.0, np.float32))
    y = sme.moe_block_linear(dev_tokens(tokens), dev_weight((w, np.full((2, 2), 0.25, np.float32))))
    assert np.array_equal(as_f64(y), 0.5 * w[:, np.arange(T) % K].T)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_linear_sums_keep_small_products(T):
    """Products of 2^-4 and more beside two of 448^2 that cancel, in another group of 8 indices: what fp32 sums keep is kept."""
    N, K = 40, 256
    rng = np.random.default_rng(T)
    x, w = np.where(np.arange(K) % 2, 0.5, 1.0) * np.ones((T, 1)), rng.integers(1, 9, (N, K)) / 8
    x[:, :8] = 0.0
    x[:, 1], w[:, 1], x[:, 3], w[:, 3] = 448.0, 448.0, -448.0, 448.0
    y = sme.moe_block_linear(dev_tokens((x, np.ones((T, 2), np.float32))), dev_weight((w, np.ones((1, 2), np.float32))))
    ref, mag = oracle.block.block_linear(x, w)
    e = terms(K) * mag                                             # nothing is cut: each group's products lie within 13 bits
    assert_near(as_f64(y), ref, e + BF16_HALF * (np.abs(ref) + e), T)


@pytest.mark.parametrize("T,N,K", [(4, 70, 96), (12, 70, 608), (40, 300, 8208), (130, 2600, 4160), (700, 5000, 80)])
def test_linear_nonfinite(T, N, K):
    """A token's NaN codes or scale are its own row's matter, a weight's its own output's: the others keep their bits."""
    rng = np.random.default_rng(T)
    x, w = dev_tokens(random_tokens(rng, T, K)), dev_weight(random_weight(rng, N, K))
    clean = sme.moe_block_linear(x, w)
    q, s = x.q.clone(), x.scale.clone()
    bad = [1, T // 2, T - 1]
    q.view(torch.uint8)[bad[0], 0] = 0x7F
    q.view(torch.uint8)[bad[1]] = 0xFF
    s[bad[2], -1] = INF
    y = sme.moe_block_linear(sme.Fp8Tokens(q, s), w)
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[bad] = False
    assert same_bits(y[rest], clean[rest])
    assert torch.isnan(y[bad[:2]].float()).all() and not torch.isfinite(y[bad[2]].float()).any()
    wq = w.q.clone()
    wq.view(torch.uint8)[[0, N - 1], K - 1] = 0x7F
    y = sme.moe_block_linear(x, sme.Fp8Weight(wq, w.scale))
    assert same_bits(y[:, 1:N - 1].contiguous(), clean[:, 1:N - 1].contiguous())
    assert torch.isnan(y[:, [0, N - 1]].float()).all()


# ------------------------------------------------------------------ routed experts

# (T, H, I, E, k, skew)
FFN = [
    (1, 16, 16, 1, 1, 0), (1, 256, 128, 8, 2, 0), (4, 2048, 512, 40, 10, 0), (2, 144, 80, 3, 3, 0), (5, 640, 272, 17, 4, 0),
    (16, 512, 256, 4, 1, 0), (33, 272, 400, 6, 2, 1.0), (64, 128, 640, 2, 2, 0), (100, 640, 160, 64, 10, 0),
    (129, 384, 128, 3, 2, 2.0), (200, 144, 144, 5, 5, 0), (257, 256, 384, 1, 1, 0), (300, 512, 256, 40, 6, 1.0),
    (1000, 160, 96, 7, 3, 2.0), (2000, 128, 256, 300, 8, 0), (40, 4112, 112, 4, 2, 0), (24, 96, 4112, 4, 2, 0),
    (70, 2048, 512, 8, 2, 0.5), (3, 8208, 32, 2, 1, 0), (3, 32, 8208, 2, 2, 0), (4, 2560, 640, 16, 10, 0),
    (7, 48, 16, 1024, 32, 0), (1500, 1040, 528, 4, 2, 0.5),
]


def ffn_case(rng, T, H, I, E, k, skew):  # noqa: E741
    # scales that make g and u about 1, so that SiLU bends, and h's values spread
    x = random_tokens(rng, T, H)
    gate, up, down = random_weight(rng, E, I, H), random_weight(rng, E, I, H), random_weight(rng, E, H, I)
    return x, gate, up, down, *routes(rng, T, E, k, skew)


@pytest.mark.parametrize("T,H,I,E,k,skew", FFN)
def test_ffn(T, H, I, E, k, skew):  # noqa: E741
    rng = np.random.default_rng(T + H + I + E)
    x, gate, up, down, idx, w, b = ffn_case(rng, T, H, I, E, k, skew)
    experts, hx, hw = dev_experts(gate, up, down), dev_tokens(x), dev(w)
    out = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = sme.make_block_ffn_workspace(T, H, I, E, k, DEV)
    ws.fill_(0xFF)
    y = sme.moe_block_expert_ffn(hx, experts, hw, b, ws, out[:T])
    y2 = sme.moe_block_expert_ffn(hx, experts, hw, b)
    torch.cuda.synchronize()
    assert same_bits(y, y2)
    assert torch.all(out[T:] == 7.0)
    deq = oracle.block.weight
    ref, tol = ffn_reference(oracle.block.tokens(*x), deq(*gate), deq(*up), deq(*down), idx, w)
    assert_near(as_f64(y), ref, tol, (T, H, I, E, k))
    # far off on the whole: each output's rounding (2^-8 at most) and as much again for the sums and codes
    assert np.linalg.norm(as_f64(y) - ref) <= 2.0 ** -7 * np.linalg.norm(ref)


@pytest.mark.parametrize("T,H,I,E,k", [(5, 256, 144, 6, 2), (90, 272, 256, 4, 2), (700, 256, 272, 3, 1)])
def test_ffn_nonfinite(T, H, I, E, k):  # noqa: E741
    """A token with a NaN is its own row's matter."""
    rng = np.random.default_rng(T)
    x, gate, up, down, idx, w, b = ffn_case(rng, T, H, I, E, k, 0)
    experts, hx, hw = dev_experts(gate, up, down), dev_tokens(x), dev(w)
    clean = sme.moe_block_expert_ffn(hx, experts, hw, b)
    q, s = hx.q.clone(), hx.scale.clone()
    bad = [0, T // 2, T - 1]
    q.view(torch.uint8)[bad[0], H - 1] = 0x7F
    s[bad[1], 0] = NAN
    s[bad[2], -1] = INF
    y = sme.moe_block_expert_ffn(sme.Fp8Tokens(q, s), experts, hw, b)
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[bad] = False
    assert same_bits(y[rest], clean[rest])
    assert torch.isnan(y[bad].float()).any(dim=1).all()


@pytest.mark.parametrize("T,H,I,E,k,top", [(3, 256, 144, 8, 8, 1), (16, 144, 272, 32, 32, 2), (16, 512, 128, 5, 4, 3), (20, 256, 256, 4, 4, 1),
                                           (60, 272, 144, 16, 9, 2), (128, 128, 640, 8, 5, 1), (128, 640, 128, 70, 32, 64),
                                           (129, 256, 144, 3, 3, 1), (300, 272, 256, 6, 5, 2)])
def test_ffn_expert_twice(T, H, I, E, k, top):  # noqa: E741
    """Tokens that name an expert more than once: up to T * k routes of one expert."""
    rng = np.random.default_rng(T + top)
    x, gate, up, down, _, w, _ = ffn_case(rng, T, H, I, E, k, 0)
    idx = (rng.integers(0, top, (T, k)) * (E // top)).astype(np.int32)
    out = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = sme.make_block_ffn_workspace(T, H, I, E, k, DEV)
    ws.fill_(0xFF)
    y = sme.moe_block_expert_ffn(dev_tokens(x), dev_experts(gate, up, down), dev(w), sme.moe_bucket_routes(dev(idx), E), ws, out[:T])
    deq = oracle.block.weight
    ref, tol = ffn_reference(oracle.block.tokens(*x), deq(*gate), deq(*up), deq(*down), idx, w)
    assert_near(as_f64(y), ref, tol, (T, H, I, E, k, top))
    assert torch.all(out[T:] == 7.0)


def test_ffn_zero_weights():
    """Routes of weight zero and tokens of zeros: exactly zero."""
    rng = np.random.default_rng(3)
    T, H, I, E, k = 6, 128, 64, 4, 2  # noqa: E741
    x, gate, up, down, idx, w, b = ffn_case(rng, T, H, I, E, k, 0)
    x[0][2] = 0.0
    w[4] = 0.0
    y = as_f64(sme.moe_block_expert_ffn(dev_tokens(x), dev_experts(gate, up, down), dev(w), b))
    assert not y[2].any() and not y[4].any() and y[[0, 1, 3, 5]].any(axis=1).all()


def test_no_tokens():
    rng = np.random.default_rng(0)
    w = dev_weight(random_weight(rng, 64, 64))
    x = sme.moe_block_quantize(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV))
    assert x.q.shape == (0, 64) and x.scale.shape == (0, 1)
    assert sme.moe_block_linear(x, w).shape == (0, 64)
    t, r = sme.moe_norm_quantize(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV),
                                 torch.ones(64, dtype=torch.bfloat16, device=DEV))
    assert t.q.shape == (0, 64) and r is None


def test_refusals():
    rng = np.random.default_rng(0)
    w, x = dev_weight(random_weight(rng, 40, 32)), dev_tokens(random_tokens(rng, 2, 32))
    xb = torch.zeros((2, 32), dtype=torch.bfloat16, device=DEV)
    wb = torch.zeros(32, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="q"):
        sme.moe_block_linear(dev_tokens(random_tokens(rng, 2, 48)), w)
    with pytest.raises(TypeError, match="q"):
        sme.moe_block_linear(sme.Fp8Tokens(xb, x.scale), w)
    with pytest.raises(ValueError, match="scale"):
        sme.moe_block_linear(sme.Fp8Tokens(x.q, x.scale[:1]), w)
    with pytest.raises(ValueError, match="bias"):
        sme.moe_block_linear(x, w, wb)
    with pytest.raises(ValueError, match="contiguous"):
        sme.moe_block_quantize(torch.zeros((32, 2), dtype=torch.bfloat16, device=DEV).t())
    with pytest.raises(TypeError, match="x"):
        sme.moe_block_quantize(xb.float())
    with pytest.raises(sme.MoeError) as e:                       # K not a multiple of 16
        sme.moe_block_quantize(xb[:, :24].contiguous())
    assert e.value.status == 2
    with pytest.raises(sme.MoeError) as e:                       # a misaligned view
        sme.moe_block_quantize(torch.zeros(65, dtype=torch.bfloat16, device=DEV)[1:].view(2, 32))
    assert e.value.status == 4
    with pytest.raises(sme.MoeError) as e:
        sme.moe_norm_quantize(xb, wb, eps=0.0)
    assert e.value.status == 2
    with pytest.raises(TypeError, match="residual"):
        sme.moe_norm_quantize(xb, wb, xb.half())
    with pytest.raises(TypeError, match="residual_out"):
        sme.moe_norm_quantize(xb, wb, xb.float(), residual_out=xb)
    with pytest.raises(ValueError, match="residual_out"):
        sme.moe_norm_quantize(xb, wb, residual_out=xb)
    with pytest.raises(ValueError, match="scale"):
        sme.Fp8Weight(w.q, w.scale[:0])
    with pytest.raises(ValueError, match="multiple of 16"):
        sme.Fp8Weight(dev_codes(np.zeros((4, 24))), torch.zeros((1, 1), device=DEV))
    with pytest.raises(AttributeError, match="Fp8Weight"):
        w.q = w.q
    T, H, I, E, k = 5, 64, 32, 3, 2  # noqa: E741
    x, gate, up, down, idx, tw, b = ffn_case(rng, T, H, I, E, k, 0)
    experts, hx, hw = dev_experts(gate, up, down), dev_tokens(x), dev(tw)
    with pytest.raises(ValueError, match="w_down"):
        dev_experts(gate, up, up)
    with pytest.raises(ValueError, match="topk_w"):
        sme.moe_block_expert_ffn(hx, experts, hw[:4], b)
    with pytest.raises(sme.MoeError) as e:
        sme.moe_block_expert_ffn(hx, experts, hw, b, torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5


# ------------------------------------------------------------------ as programs call them

def test_graph_replays():
    """Norm, linear and experts captured on one stream, replayed with new activations, eager calls between."""
    rng = np.random.default_rng(9)
    T, H, I, E, k = 6, 256, 144, 5, 2  # noqa: E741
    _, gate, up, down, idx, w, b = ffn_case(rng, T, H, I, E, k, 0)
    experts, lin, hw = dev_experts(gate, up, down), dev_weight(random_weight(rng, 75, H)), dev(w)
    norm_w = dev_bf16(bits(1 + 0.1 * rng.standard_normal(H)))
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    res, res_out = torch.zeros_like(x), torch.zeros_like(x)
    tokens, p, y = sme.empty_fp8_tokens(T, H, DEV), torch.empty((T, 75), dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    ws = sme.make_block_ffn_workspace(T, H, I, E, k, DEV)

    def run(tokens, res_out, p, y, ws=None):
        sme.moe_norm_quantize(x, norm_w, res, out=tokens, residual_out=res_out)
        sme.moe_block_linear(tokens, lin, None, p)
        sme.moe_block_expert_ffn(tokens, experts, hw, b, ws, y)

    run(tokens, res_out, p, y, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(tokens, res_out, p, y, ws)
    for _ in range(4):
        x.copy_(torch.from_numpy(rng.standard_normal((T, H))).to(DEV, torch.bfloat16))
        res.copy_(torch.from_numpy(rng.standard_normal((T, H))).to(DEV, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        t2, r2, p2, y2 = sme.empty_fp8_tokens(T, H, DEV), torch.empty_like(x), torch.empty_like(p), torch.empty_like(y)
        run(t2, r2, p2, y2, ws)
        torch.cuda.synchronize()
        assert same_bits(t2.q, tokens.q) and torch.equal(t2.scale, tokens.scale)
        assert same_bits(r2, res_out) and same_bits(p2, p) and same_bits(y2, y)


def test_graphs_share_workspaces():
    """Graphs of different sizes with one pair of workspaces, of the largest's size, replayed in turn."""
    rng = np.random.default_rng(10)
    H, I, E, k, sizes = 2048, 144, 12, 3, (300, 4, 40, 130)  # noqa: E741
    gate, up, down = random_weight(rng, E, I, H), random_weight(rng, E, I, H), random_weight(rng, E, H, I)
    experts, lin = dev_experts(gate, up, down), dev_weight(random_weight(rng, 70, H))
    ws, lws = sme.make_block_ffn_workspace(max(sizes), H, I, E, k, DEV), sme.make_block_linear_workspace(DEV)
    ws.fill_(0xFF)
    lws.fill_(0xFF)
    held = []
    for T in sizes:
        _, w, b = routes(rng, T, E, k)
        held.append([torch.zeros((T, H), dtype=torch.bfloat16, device=DEV), sme.empty_fp8_tokens(T, H, DEV), dev(w), b,
                     torch.empty((T, 70), dtype=torch.bfloat16, device=DEV), torch.empty((T, H), dtype=torch.bfloat16, device=DEV)])

    def run(x, tokens, w, b, p, y):
        sme.moe_block_quantize(x, tokens)
        sme.moe_block_linear(tokens, lin, None, p, lws)
        sme.moe_block_expert_ffn(tokens, experts, w, b, ws, y)

    graphs = []
    for h in held:
        run(*h)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(*h)
    for _ in range(3):
        want = []
        for h in held:
            h[0].copy_(torch.from_numpy(rng.standard_normal(tuple(h[0].shape))).to(DEV, torch.bfloat16))
            tokens = sme.moe_block_quantize(h[0])
            want.append((sme.moe_block_linear(tokens, lin), sme.moe_block_expert_ffn(tokens, experts, h[2], h[3])))
            h[4].fill_(0.0)
            h[5].fill_(0.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for h, (p, y) in zip(held, want):
            assert same_bits(h[4], p) and same_bits(h[5], y)


@pytest.mark.parametrize("T", [4, 300])
def test_two_streams(T):
    """Calls at once on streams of their own, behind work queued there, with workspaces of their own."""
    rng = np.random.default_rng(T)
    H, I, E, k = 512, 256, 6, 2  # noqa: E741
    cases = [ffn_case(rng, T, H, I, E, k, 0) for _ in range(2)]
    lin = dev_weight(random_weight(rng, 300, H))
    held = [(dev_tokens(c[0]), dev_experts(*c[1:4]), dev(c[5]), c[6]) for c in cases]
    want = [(sme.moe_block_linear(x, lin), sme.moe_block_expert_ffn(x, e, w, b)) for x, e, w, b in held]
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    xs = [sme.empty_fp8_tokens(T, H, DEV) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, x, (src, e, w, b) in zip(streams, xs, held):
            with torch.cuda.stream(s):
                x.q.copy_(src.q)
                x.scale.copy_(src.scale)
                got.append((sme.moe_block_linear(x, lin), sme.moe_block_expert_ffn(x, e, w, b)))
    torch.cuda.synchronize()
    for i, (p, y) in enumerate(got):
        assert same_bits(p, want[i % 2][0]) and same_bits(y, want[i % 2][1])


@pytest.mark.parametrize("T,grouped,stream", [(4, False, torch.bfloat16), (37, True, torch.float32), (300, False, torch.float32)])
def test_step(T, grouped, stream):
    """Fp8MoeStep: each operator against the oracle on what the one before gave, then two layers' worth captured and
    replayed, the residual carried from one to the next."""
    from gpu_harness import to_dev
    from test_gpu_router import _check_logits
    rng = np.random.default_rng(T)
    H, I, E, k = 256, 144, 24, 4  # noqa: E741
    rule = sme.RouteRule(k, "sigmoid", 4, 2, 2, True, 1.5) if grouped else None
    gate, up, down = random_weight(rng, E, I, H), random_weight(rng, E, I, H), random_weight(rng, E, H, I)
    experts = dev_experts(gate, up, down)
    norm_w, w_router = bits(1 + 0.1 * rng.standard_normal(H)), (rng.standard_normal((E, H)) / 16).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    x = dev_bf16(bits(rng.standard_normal((T, H))))
    res = torch.from_numpy(rng.standard_normal((T, H)) * 3).to(DEV, stream)
    hw, hr, hb = dev_bf16(norm_w), to_dev(w_router), to_dev(bias)
    step = sme.Fp8MoeStep(T, H, I, E, k, DEV, rule, stream, eps=1e-5)
    step.run(x, res, hw, hr, hb, experts)
    torch.cuda.synchronize()
    tokens, r = sme.moe_norm_quantize(x, hw, res, 1e-5)
    assert same_bits(tokens.q, step.tokens.q) and torch.equal(r, step.residual)
    _check_logits(step.logits.cpu().numpy(), step.hidden.view(torch.int16).cpu().numpy().view(np.uint16), w_router)
    logits = step.logits.cpu().numpy()
    idx, w = oracle.route_grouped(logits, bias, k, "sigmoid", 4, 2, 2, True, 1.5) if grouped else oracle.route_topk(logits, bias, k)
    assert np.array_equal(step.topk_idx.cpu().numpy(), idx)
    xq = as_f64(tokens.q)
    deq = oracle.block.weight
    ref, tol = ffn_reference(oracle.block.tokens(xq, tokens.scale.cpu().numpy()), deq(*gate), deq(*up), deq(*down), idx,
                             step.topk_w.cpu().numpy())
    assert_near(as_f64(step.y), ref, tol, "step")

    other = sme.Fp8MoeStep(T, H, I, E, k, DEV, rule, stream, eps=1e-5)

    def layers(a, b):
        a.run(x, res, hw, hr, hb, experts)
        return b.run(a.y, a.residual, hw, hr, hb, experts)

    layers(step, other)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers(step, other)
    for i in range(3):
        x.copy_(torch.roll(x, 1 + i, 1))
        graph.replay()
        torch.cuda.synchronize()
        y, r = other.y.clone(), other.residual.clone()
        a, b = (sme.Fp8MoeStep(T, H, I, E, k, DEV, rule, stream, eps=1e-5) for _ in range(2))
        layers(a, b)
        torch.cuda.synchronize()
        assert same_bits(b.y, y) and torch.equal(b.residual, r)


# ------------------------------------------------------------------ beyond 2^31

def random_codes(*shape):
    """Random finite e4m3 codes of [0.0625, 448), either sign, made on the device."""
    q = torch.empty(shape, dtype=torch.uint8, device=DEV)
    for part in q.view(-1).split(1 << 30):
        part.random_(0x20 << 1, 0x7E << 1)
    return torch.bitwise_or(q >> 1, q << 7, out=q).view(E4M3)


def random_scales(*shape, of):
    return (torch.rand(shape, device=DEV) + 0.5) * of


@pytest.mark.parametrize("T,N,K", [(2, 1 << 18, 16384), (70, 1 << 18, 16384), (300, 1 << 18, 16384), (70000, 65600, 16),
                                   (1 << 17, 200, 32768)])
def test_linear_beyond_32_bits(T, N, K):
    """Weights, outputs, or tokens of more than 2^31 values (their first and last rows and some between are compared)."""
    rng = np.random.default_rng(T)
    torch.manual_seed(T)
    x = sme.Fp8Tokens(random_codes(T, K), random_scales(T, blocks(K), of=1 / 256))
    w = sme.Fp8Weight(random_codes(N, K), random_scales(blocks(N), blocks(K), of=1 / (128 * K ** 0.5)))
    y = sme.moe_block_linear(x, w)
    t, n = (np.unique(np.concatenate([[0, m - 1], rng.integers(0, m, 30), rng.integers(m * 7 // 8, m, 30)])) for m in (T, N))
    dt, dn = dev(t), dev(n)
    bytes_at = lambda q, at: q.view(torch.uint8)[at].view(E4M3)  # noqa: E731
    hx = oracle.block.tokens(as_f64(bytes_at(x.q, dt)), x.scale[dt].cpu().numpy())
    s = np.repeat(w.scale[dn // 128].cpu().numpy().astype(np.float64), 128, axis=1)[:, :K]
    ref, tol = linear_reference(hx, as_f64(bytes_at(w.q, dn)) * s)
    assert_near(as_f64(y[dt][:, dn]), ref, tol, (T, N, K))


@pytest.mark.parametrize("T,H,I,E,k", [(3, 4096, 1040, 1024, 2), (150, 4096, 1040, 1024, 2), (1 << 18, 4096, 144, 4, 4),
                                       (1 << 17, 144, 4224, 4, 4)])
def test_ffn_beyond_32_bits(T, H, I, E, k):  # noqa: E741
    """A matrix of all experts, or the routes' sums or hidden values, of more than 2^31 values."""
    rng = np.random.default_rng(T)
    torch.manual_seed(T)
    x = sme.Fp8Tokens(random_codes(T, H), random_scales(T, blocks(H), of=1 / 256))
    mats = []
    for n, kk in ((I, H), (I, H), (H, I)):
        mats += [random_codes(E, n, kk), random_scales(E, blocks(n), blocks(kk), of=1 / (128 * kk ** 0.5))]
    chosen = np.array([0, E - 1])
    idx = np.argsort(rng.standard_normal((T, E)), axis=1).astype(np.int32)[:, :k] if E == k else chosen[
        np.argsort(rng.standard_normal((T, 2)), axis=1)].astype(np.int32)
    w = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    y = sme.moe_block_expert_ffn(x, sme.Fp8Experts(*mats), dev(w), sme.moe_bucket_routes(dev(idx), E))
    t = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 20), rng.integers(T * 7 // 8, T, 20)]))
    hx = oracle.block.tokens(as_f64(x.q.view(torch.uint8)[dev(t)].view(E4M3)), x.scale[dev(t)].cpu().numpy())
    used = np.unique(idx[t])
    gate, up, down = ([oracle.block.weight(as_f64(mats[m].view(torch.uint8)[int(e)].view(E4M3)), mats[m + 1][int(e)].cpu().numpy())
                       for e in used] for m in (0, 2, 4))
    ref, tol = ffn_reference(hx, *(np.stack(m) for m in (gate, up, down)), np.searchsorted(used, idx[t]), w[t])
    assert_near(as_f64(y[dev(t)]), ref, tol, (T, H, I, E, k))


def test_norm_beyond_32_bits():
    torch.manual_seed(5)
    T, H = 140000, 16384
    x = torch.randn((1000, H), dtype=torch.bfloat16, device=DEV).repeat(T // 1000, 1)
    w = torch.rand(H, dtype=torch.bfloat16, device=DEV)
    tokens, r = sme.moe_norm_quantize(x, w, x)
    t, r1 = sme.moe_norm_quantize(x[:1000], w, x[:1000])
    q = sme.moe_block_quantize(x)
    q1 = sme.moe_block_quantize(x[:1000])
    for i in (0, 65000, T - 1000):                                     # (the 131072nd row is the 2^31st value's)
        for a, b in ((tokens.q, t.q), (tokens.scale, t.scale), (r, r1), (q.q, q1.q), (q.scale, q1.scale)):
            assert same_bits(a[i:i + 1000], b)
