"""Host-side refusals of the grouped routing and the 4-bit dense products,
before any launch (no device): the C calls' checks and the binding's."""

import ctypes
import os

import pytest
import torch

import sparse_moe_expert_amd as sme
import sparse_moe_expert_amd.build

P = ctypes.c_void_p
A = P(256)           # a fake, 16-byte aligned, never dereferenced address
OK, NULL, SHAPE, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sme.LIB_PATH):
        sme.build.build_library()
    return sme.load_library()


def _route(lib, fused, logits=A, dtype=0, bias=None, T=0, E=64, k=4, score=1, groups=8, kept=4, top=2, scale=1.0,
           idx=A, w=A, out=A):
    args = (logits, dtype, bias, T, E, k, score, groups, kept, top, 1, scale, idx, w)
    if fused:
        return lib.moe_route_grouped_bucket(*args, A, A, A, A, A, out, None)
    return lib.moe_route_grouped(*args, None)


@pytest.mark.parametrize("fused", [False, True])
def test_route_grouped_host_checks(lib, fused):
    call = lambda **kw: _route(lib, fused, **kw)  # noqa: E731
    assert call() == OK                             # T = 0: nothing launched
    assert call(logits=None, idx=None, w=None) == OK
    for bad in (dict(T=-1), dict(k=0), dict(k=65), dict(E=0), dict(groups=0), dict(groups=7), dict(kept=0),
                dict(kept=9), dict(top=0), dict(top=3), dict(k=9, kept=1), dict(dtype=2), dict(dtype=-1),
                dict(score=2), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(**bad) == SHAPE, bad
    assert call(E=2048) == UNSUPPORTED
    assert call(k=33, kept=8) == UNSUPPORTED
    assert call(E=1024, groups=128, kept=64) == UNSUPPORTED
    assert call(T=1 << 23) == UNSUPPORTED                       # T*k > 2^24
    assert call(E=1023, groups=33, kept=33) == UNSUPPORTED      # 31 experts for the one lane of a group
    assert call(E=1020, groups=17, kept=17) == UNSUPPORTED      # 60 experts for two lanes
    assert call(E=960, groups=15, kept=15) == OK                # 64 experts for four lanes
    assert call(T=2, logits=None) == NULL
    assert call(T=2, idx=None) == NULL
    assert call(T=2, w=None) == NULL
    assert call(T=2, logits=P(264)) == MISALIGNED
    assert call(T=2, bias=P(260)) == MISALIGNED
    if fused:
        assert call(T=2, out=None) == NULL
        assert call(T=2, out=P(260)) == MISALIGNED


def test_quant_linear_host_checks(lib):
    def call(fmt=0, x=A, codes=A, scales=A, g=A, bias=None, T=0, N=7, K=64, y=A, ws=A, ws_bytes=1 << 30):
        return lib.moe_quant_linear(fmt, x, codes, scales, g, bias, T, N, K, ws, ctypes.c_size_t(ws_bytes), y, None)
    assert call() == OK
    assert call(x=None, y=None) == OK               # T = 0: nothing launched
    for bad in (dict(fmt=2), dict(fmt=-1), dict(T=-1), dict(N=0), dict(K=0), dict(K=48), dict(K=-32)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(N=(1 << 20) + 1), dict(K=(1 << 15) + 32), dict(T=(1 << 20) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for name in ("x", "codes", "scales", "g", "y"):
        assert call(T=1, **{name: None}) == NULL, name
    for name in ("x", "codes", "scales", "bias", "y"):
        assert call(T=1, **{name: P(264)}) == MISALIGNED, name
    assert call(T=1, g=P(258)) == MISALIGNED
    size = lib.moe_quant_linear_workspace_size
    assert size(1, 4096, 4096) == size(4, 100, 4096) == size(4096, 4096, 4096) == 0
    assert size(0, 64, 64) == size(8, 0, 64) == size(8, 64, 48) == size((1 << 20) + 1, 64, 64) == 0
    need = size(64, 4100, 8192)                     # parts of fp32 [64, 4224]
    assert need > 0 and need % (64 * 4224 * 4) == 0
    assert call(T=64, N=4100, K=8192, ws_bytes=need - 1) == WORKSPACE
    assert call(T=64, N=4100, K=8192, ws=None) == NULL
    assert call(T=64, N=4100, K=8192, ws=P(264)) == MISALIGNED


def test_quant_shared_host_checks(lib):
    def call(fmt=0, T=0, H=64, Is=32, ws=1 << 20, null_at=None, bad_at=None, g=A, v=None, add=None):
        p = [A] * 9          # x, gate codes, scales, up codes, scales, down codes, scales, workspace, y
        if null_at is not None:
            p[null_at] = None
        if bad_at is not None:
            p[bad_at] = P(264)
        return lib.moe_quant_shared_expert(fmt, p[0], p[1], p[2], g, p[3], p[4], A, p[5], p[6], A, v, add, T, H, Is,
                                           p[7], ctypes.c_size_t(ws), p[8], None)
    assert call() == OK
    for bad in (dict(fmt=2), dict(T=-1), dict(H=0), dict(H=48), dict(Is=40), dict(Is=0)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(H=(1 << 15) + 32), dict(Is=(1 << 15) + 32), dict(T=(1 << 20) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for i in range(9):
        assert call(T=1, null_at=i) == NULL, i
        assert call(T=1, bad_at=i) == MISALIGNED, i
    assert call(T=1, g=None) == NULL
    assert call(T=1, v=P(264)) == MISALIGNED
    assert call(T=1, add=P(264)) == MISALIGNED
    need = lib.moe_quant_shared_expert_workspace_size(5, 64, 96)
    assert need == 1024 + 256                       # 5 * 96 * 2 and 5 * 4, each rounded up to 256; nothing split
    assert call(T=5, Is=96, ws=need - 1) == WORKSPACE
    assert lib.moe_quant_shared_expert_workspace_size(0, 64, 96) == 0


def test_binding_refusals():
    """What the binding refuses before it calls the library, on host tensors."""
    with pytest.raises(ValueError, match="score"):
        sme.RouteRule(4, score="tanh")
    rule = sme.RouteRule(2)
    assert (rule.groups, rule.groups_kept, rule.group_top) == (1, 1, 2)
    with pytest.raises(AttributeError, match="RouteRule"):
        rule.scale = 2.0
    with pytest.raises(TypeError, match="logits"):
        sme.moe_route_grouped(torch.zeros(8), None, rule)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sme.moe_route_grouped(torch.zeros((2, 8), dtype=torch.float16), None, rule)
    with pytest.raises(ValueError, match="device tensor"):
        sme.moe_route_grouped(torch.zeros((2, 8)), None, rule)
    with pytest.raises(ValueError, match="format"):
        sme.QuantWeight(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8), format="int4")
    with pytest.raises(ValueError, match="multiple of 32"):
        sme.QuantWeight(torch.zeros((4, 24), dtype=torch.uint8), torch.zeros((4, 3), dtype=torch.uint8))
    with pytest.raises(ValueError, match="device tensor"):
        sme.QuantWeight(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8))
    with pytest.raises(TypeError, match="codes"):
        sme.QuantWeight(torch.zeros(16, dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8))


def test_step_refusals():
    rule = sme.RouteRule(4)
    for path in ("step", "packed"):
        with pytest.raises(ValueError, match="rule"):
            sme.MoeStep(2, 64, 64, 8, 4, "cpu", path=path, rule=rule)
    with pytest.raises(ValueError, match="rule.k"):
        sme.MoeStep(2, 64, 64, 8, 2, "cpu", path="calls", rule=rule)
