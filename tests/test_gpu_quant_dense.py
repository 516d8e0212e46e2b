"""moe_quant_linear and moe_quant_shared_expert against the fp64 oracle, with
tolerances counted from the arithmetic (layer_testlib)."""

import numpy as np
import pytest
import torch

import oracle
import sparse_moe_expert_amd as sme
from gpu_harness import DEV, to_dev
from layer_testlib import (assert_near, bits, dev_bf16, f64, handle, linear_tolerance, shared_reference, weight)

pytestmark = pytest.mark.gpu

# (T, N, K): one token to hundreds, either side of 1, 4, 8, 16, 32, 64, 128; N of one, odd, and of whole tiles; K of one
# block, of odd numbers of blocks, and long
LINEAR = [
    (1, 1, 32), (1, 7, 64), (1, 2048, 2048), (2, 33, 96), (3, 100, 160), (4, 130, 2560), (5, 17, 32), (7, 300, 672),
    (8, 64, 1056), (9, 129, 288), (15, 65, 4096), (16, 256, 512), (17, 31, 224), (31, 127, 640), (32, 999, 1024),
    (33, 128, 2080), (63, 72, 96), (64, 512, 256), (65, 257, 128), (100, 640, 320), (127, 1, 64), (128, 128, 64),
    (129, 385, 1088), (255, 200, 32), (257, 512, 512), (1, 20, 32768), (40, 20, 16416), (600, 300, 2048),
    (4, 40, 12288), (4, 30, 32768), (600, 6500, 96), (513, 8200, 160), (300, 16390, 64),
    # split reductions: aligned scale rows or not, one to three token tiles, whole and partial steps
    (20, 33, 16384), (17, 1000, 4128), (33, 900, 8224), (60, 700, 8192), (130, 2600, 4160), (24, 130, 32736),
    # rows that take two rounds of smaller tiles; few tokens whose activations do not fit one workgroup
    (20, 16500, 544), (31, 16500, 512), (90, 10300, 544), (90, 10300, 512), (512, 640, 640), (16, 30, 32768),
    (8, 70, 32736),
    # enough tiles of 256 rows by 128 tokens for the chip: partial ones, and either side of a multiple of eight
    (700, 11000, 96), (600, 13200, 1056), (300, 22000, 64), (1025, 7300, 160), (33000, 260, 32),
    (650, 11000, 640), (300, 16384, 448), (1300, 4090, 1152),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear(T, N, K, fmt):
    rng = np.random.default_rng(T * 1000 + N + K)
    w = weight(rng, N, K, fmt)
    x = bits(rng.standard_normal((T, K)))
    bias = bits(rng.standard_normal(N)) if (T + N) % 2 else None
    hw, hx, hb = handle(w, fmt), dev_bf16(x), None if bias is None else dev_bf16(bias)
    out = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((max(sme.moe_quant_linear_workspace_size(T, N, K), 16),), 0xFF, dtype=torch.uint8, device=DEV)
    head = T * N * 2 % 16 == 0
    y = sme.moe_quant_linear(hx, hw, hb, out[:T] if head else None, ws)
    y2 = sme.moe_quant_linear(hx, hw, hb)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))      # bitwise reproducible
    assert torch.all(out[T:] == 7.0)                                   # rows behind the last token
    ref, mag = oracle.quant_linear(x, w, fmt, bias)
    assert_near(f64(y), ref, linear_tolerance(ref, mag, K), (T, N, K, fmt))


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_linear_every_code_and_scale(T):
    """Each e2m1 code under each scale byte, against unit activations: the products are exact."""
    for fmt, group, lo, hi, g in (("nvfp4", 16, 0, 0x7F, np.float32(1.0)), ("mxfp4", 32, 100, 150, None)):
        K = 32
        scales = np.repeat(np.arange(lo, hi, dtype=np.uint8)[:, None], K // group, axis=1)
        N = scales.shape[0]
        codes = np.tile(np.arange(16, dtype=np.uint8) * 0x11, (N, 1))          # both nibbles of byte i: code i
        x = np.zeros((T, K))
        x[np.arange(T), np.arange(T) % K] = 1.0
        y = sme.moe_quant_linear(dev_bf16(bits(x)), handle((codes, scales, g), fmt))
        ref, _ = oracle.quant_linear(bits(x), (codes, scales, g), fmt)
        assert np.array_equal(f64(y), ref), fmt


def test_linear_extreme_scales():
    """MXFP4 scales at the ends of their range, and NVFP4's zero scale."""
    codes = np.full((4, 16), 0x71, np.uint8)                                   # 0.5, 6
    for T in (1, 6, 130):
        scales = np.array([[2], [60], [200], [252]], np.uint8)
        x = np.full((T, 32), 2.0 ** -20)
        y = f64(sme.moe_quant_linear(dev_bf16(bits(x)), handle((codes, scales, None), "mxfp4")))
        assert np.array_equal(y[:, 1:], np.tile([16 * 6.5 * 2.0 ** (e - 147) for e in (60, 200, 252)], (T, 1)))
        # 2^-125 * 2^-20 is below fp32's normal range: the product or zero
        assert np.all((y[:, 0] == 0) | (np.abs(y[:, 0] / (16 * 6.5 * 2.0 ** -145) - 1) < 0.5))
        zero = np.zeros((4, 2), np.uint8)
        y = sme.moe_quant_linear(dev_bf16(bits(x)), handle((codes, zero, np.float32(1)), "nvfp4"))
        assert not f64(y).any()


# (T, H, Is, gated, add)
SHARED = [
    (1, 32, 32, True, True), (1, 2048, 512, False, False), (2, 96, 160, True, False), (4, 2048, 512, True, True),
    (5, 640, 96, False, True), (8, 288, 1056, True, True), (13, 512, 224, True, True), (16, 2560, 640, False, False),
    (32, 64, 2048, True, False), (33, 416, 352, True, True), (64, 256, 256, False, True), (100, 2560, 640, True, True),
    (130, 512, 128, True, True), (257, 160, 416, True, True), (1029, 2080, 2080, True, True),
    (20, 8224, 1056, True, True), (70, 4160, 2112, False, True), (150, 1056, 4192, True, False),
    (24, 512, 8288, True, False), (30, 544, 8416, False, True), (90, 512, 5216, True, True), (90, 544, 5216, False, False),
    (300, 96, 2080, True, True), (9, 5152, 96, True, True), (4100, 2080, 1024, True, True), (1301, 96, 3008, True, False),
    (1300, 640, 3008, True, True), (1281, 896, 2080, False, True),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,H,Is,gated,add", SHARED)
def test_shared(T, H, Is, gated, add, fmt):
    rng = np.random.default_rng(T + H + Is)
    gate, up, down = weight(rng, Is, H, fmt), weight(rng, Is, H, fmt), weight(rng, H, Is, fmt)
    x = bits(rng.standard_normal((T, H)))
    v = bits(rng.standard_normal(H) / np.sqrt(H)) if gated else None
    a = bits(rng.standard_normal((T, H))) if add else None
    dv, da = None if v is None else dev_bf16(v), None if a is None else dev_bf16(a)
    handles = [handle(m, fmt) for m in (gate, up, down)]
    y = sme.moe_quant_shared_expert(dev_bf16(x), *handles, dv, da)
    ref, tol = shared_reference(x, gate, up, down, fmt, v, a)
    assert_near(f64(y), ref, tol, (T, H, Is, fmt))
    # into a given y and workspace, y being `add` itself: the same bits
    out = da.clone() if add else torch.empty_like(y)
    ws = sme.make_quant_shared_workspace(T, H, Is, DEV)
    ws.fill_(0xFF)
    sme.moe_quant_shared_expert(dev_bf16(x), *handles, dv, out if add else None, out, ws)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("T,N,K", [(4, 70, 96), (12, 70, 608), (40, 300, 8224), (130, 2600, 4160), (700, 11000, 96)])
def test_linear_nonfinite_tokens(T, N, K):
    """A token of infinities or NaN is its own row's matter: the others keep their bits, those before it too, whose
    last step of the reduction runs into its row."""
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, K))).to(DEV, torch.bfloat16)
    bad = [1, T // 2, T - 1]
    for fmt in ("nvfp4", "mxfp4"):
        w = handle(weight(rng, N, K, fmt), fmt)
        clean = sme.moe_quant_linear(x, w)
        dirty = x.clone()
        for t, v in zip(bad, (float("inf"), float("nan"), float("-inf"))):
            dirty[t] = v
        y = sme.moe_quant_linear(dirty, w)
        rest = torch.ones(T, dtype=torch.bool, device=DEV)
        rest[bad] = False
        assert torch.equal(y[rest].view(torch.int16), clean[rest].view(torch.int16)), fmt
        assert not torch.isfinite(y[bad].float()).all()


def test_no_tokens():
    rng = np.random.default_rng(0)
    w = handle(weight(rng, 64, 64, "nvfp4"), "nvfp4")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    assert sme.moe_quant_linear(x, w).shape == (0, 64)
    assert sme.moe_quant_shared_expert(x, w, w, w).shape == (0, 64)


def test_refusals():
    rng = np.random.default_rng(0)
    w, mx = handle(weight(rng, 64, 32, "nvfp4"), "nvfp4"), handle(weight(rng, 32, 64, "mxfp4"), "mxfp4")
    down = handle(weight(rng, 32, 64, "nvfp4"), "nvfp4")
    x = torch.zeros((2, 32), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="x"):
        sme.moe_quant_linear(torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV), w)
    with pytest.raises(TypeError, match="x"):
        sme.moe_quant_linear(x.float(), w)
    with pytest.raises(ValueError, match="contiguous"):
        sme.moe_quant_linear(torch.zeros((32, 2), dtype=torch.bfloat16, device=DEV).t(), w)
    with pytest.raises(ValueError, match="y"):
        sme.moe_quant_linear(x, w, None, torch.empty((2, 63), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(sme.MoeError) as e:                       # a misaligned view
        sme.moe_quant_linear(torch.zeros(65, dtype=torch.bfloat16, device=DEV)[1:].view(2, 32), w)
    assert e.value.status == 4
    with pytest.raises(AttributeError, match="QuantWeight"):
        w.codes = w.codes[:1]
    square = handle(weight(rng, 32, 32, "nvfp4"), "nvfp4")
    with pytest.raises(ValueError, match="y must not be x"):
        sme.moe_quant_linear(x, square, None, x)
    with pytest.raises(ValueError, match="y must not be x"):
        sme.moe_quant_shared_expert(x, square, square, square, y=x)
    with pytest.raises(ValueError, match="global scale"):
        sme.QuantWeight(w.codes, w.scales)
    with pytest.raises(ValueError, match="scales"):
        sme.QuantWeight(w.codes, w.scales, format="mxfp4")
    with pytest.raises(ValueError, match="down"):
        sme.moe_quant_shared_expert(x, w, w, w)
    with pytest.raises(ValueError, match="format"):
        sme.moe_quant_shared_expert(x, w, w, mx)
    with pytest.raises(sme.MoeError) as e:
        sme.moe_quant_shared_expert(x, w, w, down, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5


def test_graph_replays():
    """Captured products on one stream, replayed with new activations, eager calls on the same workspace between."""
    rng = np.random.default_rng(9)
    T, H, Is = 6, 256, 128
    gate, up, down = (weight(rng, n, k, "nvfp4") for n, k in ((Is, H), (Is, H), (H, Is)))
    hg, hu, hd = (handle(m, "nvfp4") for m in (gate, up, down))
    v = bits(rng.standard_normal(H) / 16)
    dv = dev_bf16(v)
    x, y, z = (torch.zeros((T, H), dtype=torch.bfloat16, device=DEV) for _ in range(3))
    ws = sme.make_quant_shared_workspace(T, H, Is, DEV)
    p = sme.moe_quant_linear(x, hg)
    sme.moe_quant_shared_expert(x, hg, hu, hd, dv, None, y, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sme.moe_quant_linear(x, hg, None, p)
        sme.moe_quant_shared_expert(x, hg, hu, hd, dv, None, y, ws)
        sme.moe_quant_shared_expert(x, hg, hu, hd, dv, y, y, ws)
    for _ in range(4):
        x.copy_(dev_bf16(bits(rng.standard_normal((T, H)))))
        graph.replay()
        torch.cuda.synchronize()
        sme.moe_quant_shared_expert(x, hg, hu, hd, dv, None, z, ws)
        sme.moe_quant_shared_expert(x, hg, hu, hd, dv, z, z, ws)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), z.view(torch.int16))
        assert torch.equal(p.view(torch.int16), sme.moe_quant_linear(x, hg).view(torch.int16))


def test_split_captured_and_on_two_streams():
    """A split reduction whose workspace the call allocates: captured and replayed, two such graphs in turn, and two
    calls at once on streams of their own."""
    rng = np.random.default_rng(21)
    T, N, K = 40, 300, 8224
    assert sme.moe_quant_linear_workspace_size(T, N, K) > 0
    w = handle(weight(rng, N, K, "nvfp4"), "nvfp4")
    xs = [torch.from_numpy(rng.standard_normal((T, K))).to(DEV, torch.bfloat16) for _ in range(2)]
    want = [sme.moe_quant_linear(x, w) for x in xs]
    torch.cuda.synchronize()
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    graphs, outs, held = [], [], [x.clone() for x in xs]
    for x in held:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(sme.moe_quant_linear(x, w))
    for i in range(4):
        swap = i % 2
        held[0].copy_(xs[swap])
        held[1].copy_(xs[1 - swap])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert same(outs[0], want[swap]) and same(outs[1], want[1 - swap])
        assert same(sme.moe_quant_linear(xs[0], w), want[0])
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(sme.moe_quant_linear(x, w))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert same(y, want[i % 2])


def test_other_stream():
    """On a side stream, behind work queued there."""
    rng = np.random.default_rng(3)
    w = weight(rng, 96, 512, "nvfp4")
    h, x = handle(w, "nvfp4"), bits(rng.standard_normal((3, 512)))
    dx = torch.zeros((3, 512), dtype=torch.bfloat16, device=DEV)
    src = dev_bf16(x)
    side = torch.cuda.Stream(DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        dx.copy_(src)
        y = sme.moe_quant_linear(dx, h)
    side.synchronize()
    ref, mag = oracle.quant_linear(x, w, "nvfp4")
    assert_near(f64(y), ref, linear_tolerance(ref, mag, 512), "side stream")


@pytest.mark.parametrize("path", ["calls", "calls_unfused"])
def test_step_with_rule(path):
    """MoeStep with a rule against the operators called one by one: the same bits, eager and replayed on new inputs."""
    from gpu_harness import device_weights, x_bits
    from moe_inputs import make_workload
    wl = make_workload("tiny")
    T, H, I, E, k = wl.T, wl.H, wl.I, wl.E, wl.k
    rule = sme.RouteRule(k, "softmax", 4, 2, 1, False, 2.0)
    x, logits, bank = x_bits(wl.x), to_dev(wl.logits), device_weights(wl.bank)
    bias = to_dev(np.linspace(-0.1, 0.1, E, dtype=np.float32))
    step = sme.MoeStep(T, H, I, E, k, DEV, path=path, rule=rule)

    def check():
        torch.cuda.synchronize()
        idx, w, b = sme.moe_route_grouped_bucket(logits, bias, rule)
        y = sme.moe_expert_ffn(x, bank, w, b, sme.make_workspace(T, H, I, E, k, DEV))
        torch.cuda.synchronize()
        assert torch.equal(step.topk_idx, idx) and torch.equal(step.topk_w, w)
        assert torch.equal(step.y.view(torch.int16), y.view(torch.int16))

    step.run(x, logits, bias, bank)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(x, logits, bias, bank)
    for i in range(3):
        logits.copy_(torch.roll(logits, 5 + i, 1))
        graph.replay()
        check()


def test_layer():
    """A layer as a user runs it: grouped routing and its buckets, the routed experts, the 4-bit shared expert summed
    onto their output, and a 4-bit projection of the sum, each against the oracle on what the one before gave."""
    from gpu_harness import assert_output, device_weights, x_bits
    from moe_inputs import make_workload
    wl = make_workload("tiny")
    T, H, I, E, k = wl.T, wl.H, wl.I, wl.E, wl.k
    rng = np.random.default_rng(12)
    Is, N = 96, 75
    gate, up, down, proj = (weight(rng, n, m, f) for n, m, f in
                            ((Is, H, "mxfp4"), (Is, H, "mxfp4"), (H, Is, "mxfp4"), (N, H, "nvfp4")))
    v = bits(rng.standard_normal(H) / np.sqrt(H))
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    rule = sme.RouteRule(k, "sigmoid", 4, 2, 2, True, 1.5)
    x = x_bits(wl.x)
    idx, w, b = sme.moe_route_grouped_bucket(to_dev(wl.logits), to_dev(bias), rule)
    routed = sme.moe_expert_ffn(x, device_weights(wl.bank), w, b, sme.make_workspace(T, H, I, E, k, DEV))
    y = sme.moe_quant_shared_expert(x.view(torch.bfloat16), *(handle(m, "mxfp4") for m in (gate, up, down)), dev_bf16(v), routed)
    z = sme.moe_quant_linear(y, handle(proj, "nvfp4"))
    torch.cuda.synchronize()
    ref_idx, ref_w = oracle.route_grouped(wl.logits, bias, k, "sigmoid", 4, 2, 2, True, 1.5)
    assert np.array_equal(idx.cpu().numpy(), ref_idx)
    assert_output(f64(routed), oracle.moe_output(wl.x, wl.bank, ref_idx, ref_w), "routed experts")
    got = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    ref, tol = shared_reference(wl.x, gate, up, down, "mxfp4", v, got(routed))
    assert_near(f64(y), ref, tol, "shared expert on the routed output")
    ref, mag = oracle.quant_linear(got(y), proj, "nvfp4")
    assert_near(f64(z), ref, linear_tolerance(ref, mag, H), "projection")
