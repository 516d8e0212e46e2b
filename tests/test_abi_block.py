"""Host-side refusals of the block-scaled 8-bit operators, before any launch (no device): the C calls' checks and the
binding's."""

import ctypes
import glob
import hashlib
import os
import re

import pytest
import torch

import sparse_moe_expert_amd as sme
import sparse_moe_expert_amd.build

P = ctypes.c_void_p
A = P(256)           # a fake, 16-byte aligned, never dereferenced address
OK, NULL, SHAPE, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4, 5
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(sme.LIB_PATH):
        sme.build.build_library()
    return sme.load_library()


def test_norm_host_checks(lib):
    def call(x=A, res=None, kind=0, w=A, offset=0.0, eps=1e-6, T=0, H=64, res_out=None, y=None, q=A, scale=A):
        return lib.moe_norm_quantize(x, res, kind, w, offset, eps, T, H, res_out, y, q, scale, None)
    assert call() == OK
    assert call(x=None, w=None, q=None, scale=None) == OK          # T = 0: nothing launched
    for bad in (dict(T=-1), dict(H=0), dict(H=24), dict(H=-16), dict(kind=2), dict(kind=-1), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=NAN), dict(eps=INF), dict(offset=NAN), dict(offset=INF), dict(offset=-INF)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(H=(1 << 15) + 16), dict(T=(1 << 20) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for name in ("x", "w", "q", "scale"):
        assert call(T=1, **{name: None}) == NULL, name
        assert call(T=1, **{name: P(264)}) == MISALIGNED, name
    assert call(T=1, res=A) == NULL                                # a residual without its output, and the other way round
    assert call(T=1, res_out=A) == NULL
    assert call(T=1, res=P(264), res_out=A) == MISALIGNED
    assert call(T=1, res=A, res_out=P(264)) == MISALIGNED
    assert call(T=1, y=P(264)) == MISALIGNED


def test_quantize_host_checks(lib):
    def call(x=A, T=0, K=64, q=A, scale=A):
        return lib.moe_block_quantize(x, T, K, q, scale, None)
    assert call() == call(x=None, q=None, scale=None) == OK
    for bad in (dict(T=-1), dict(K=0), dict(K=24), dict(K=-16)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(K=(1 << 15) + 16), dict(T=(1 << 20) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for name in ("x", "q", "scale"):
        assert call(T=1, **{name: None}) == NULL, name
        assert call(T=1, **{name: P(264)}) == MISALIGNED, name


def test_linear_host_checks(lib):
    def call(x=A, sx=A, w=A, sw=A, bias=None, T=0, N=7, K=64, ws=A, ws_bytes=1 << 30, y=A):
        return lib.moe_block_linear(x, sx, w, sw, bias, T, N, K, ws, ctypes.c_size_t(ws_bytes), y, None)
    assert call() == call(x=None, y=None) == OK
    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(K=24), dict(K=-16)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(N=(1 << 20) + 1), dict(K=(1 << 15) + 16), dict(T=(1 << 20) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for name in ("x", "sx", "w", "sw", "y"):
        assert call(T=1, **{name: None}) == NULL, name
        assert call(T=1, **{name: P(264)}) == MISALIGNED, name
    assert call(T=1, bias=P(264)) == MISALIGNED
    size = lib.moe_block_linear_workspace_size
    assert size(0, 64, 64) == size(8, 0, 64) == size(8, 64, 24) == size((1 << 20) + 1, 64, 64) == 0
    for T in (1, 5, 16, 17, 32, 64, 100, 200, 333, 1000, 5000):
        for N in (1, 100, 640, 2560, 9999, 40000):
            for K in (16, 640, 2048, 5200, 16384, 32768):
                need = size(T, N, K)
                assert 0 <= need <= sme.BLOCK_SUMS_BYTES, (T, N, K)
                if need:
                    assert call(T=T, N=N, K=K, ws_bytes=need - 1) == WORKSPACE
                    assert call(T=T, N=N, K=K, ws=None) == NULL
                    assert call(T=T, N=N, K=K, ws=P(264)) == MISALIGNED


def test_ffn_host_checks(lib):
    def call(T=0, H=64, I=32, E=4, k=2, ws=1 << 30, null_at=None, bad_at=None):  # noqa: E741
        p = [A] * 17          # x, scale, three weights and scales, topk_w, six bucket arrays, workspace, y
        if null_at is not None:
            p[null_at] = None
        if bad_at is not None:
            p[bad_at] = P(264)
        return lib.moe_block_expert_ffn(*p[:15], T, H, I, E, k, p[15], ctypes.c_size_t(ws), p[16], None)
    assert call() == OK
    for bad in (dict(T=-1), dict(H=0), dict(H=24), dict(I=8), dict(I=0), dict(E=0), dict(k=0), dict(k=5)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(H=(1 << 15) + 16), dict(I=(1 << 15) + 16), dict(E=1025), dict(E=64, k=33), dict(T=(1 << 23) + 1),
                dict(T=1 << 20, H=1 << 11)):
        assert call(**bad) == UNSUPPORTED, bad
    for i in range(17):
        assert call(T=1, null_at=i) == NULL, i
        assert call(T=1, bad_at=i) == MISALIGNED, i
    size = lib.moe_block_expert_ffn_workspace_size
    need = size(5, 64, 32, 4, 2)
    assert need > 0 and call(T=5, ws=need - 1) == WORKSPACE
    assert size(0, 64, 32, 4, 2) == size(5, 24, 32, 4, 2) == size(5, 64, 32, 1025, 2) == 0


@pytest.mark.parametrize("H,I,E,k", [(2048, 512, 512, 10), (2560, 640, 512, 10), (64, 48, 3, 1), (4096, 2048, 16, 2), (16, 16, 1, 1)])
def test_workspace_serves_smaller_batches(H, I, E, k):  # noqa: E741
    """A workspace made for a batch is large enough for every smaller one."""
    most = 0
    for T in [*range(1, 300), *range(320, 8400, 61), 16384, 1 << 17]:
        need = sme.moe_block_expert_ffn_workspace_size(T, H, I, E, k)
        assert need >= most, T
        most = need


def test_binding_refusals():
    """What the binding refuses before it calls the library, on host tensors."""
    e4m3 = torch.float8_e4m3fn
    q, s = torch.zeros((4, 32), dtype=e4m3), torch.zeros((1, 1))
    with pytest.raises(ValueError, match="device tensor"):
        sme.Fp8Weight(q, s)
    with pytest.raises(ValueError, match="multiple of 16"):
        sme.Fp8Weight(q[:, :24], s)
    with pytest.raises(TypeError, match="q"):
        sme.Fp8Weight(q[0], s)
    with pytest.raises(TypeError, match="w_gate"):
        sme.Fp8Experts(q, s, q, s, q, s)
    with pytest.raises(ValueError, match="device tensor"):
        sme.moe_block_quantize(torch.zeros((2, 32), dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="bfloat16"):
        sme.moe_block_quantize(torch.zeros((2, 32)))
    with pytest.raises(TypeError, match="x"):
        sme.moe_norm_quantize(torch.zeros(32, dtype=torch.bfloat16), None)
    with pytest.raises(ValueError, match="at most"):
        sme.moe_block_quantize(torch.empty(((1 << 32) + 1, 16), dtype=torch.bfloat16, device="meta"))
    for size, n in ((sme.moe_block_linear_workspace_size, 3), (sme.moe_block_expert_ffn_workspace_size, 5)):
        for i in range(n):
            with pytest.raises(ValueError, match="at most"):
                size(*[(1 << 32) + 64 if j == i else 64 for j in range(n)])


def test_step_refusals():
    with pytest.raises(ValueError, match="rule.k"):
        sme.Fp8MoeStep(2, 64, 64, 8, 2, "cpu", rule=sme.RouteRule(4))
    with pytest.raises(ValueError, match="residual_dtype"):
        sme.Fp8MoeStep(2, 64, 64, 8, 2, "cpu", residual_dtype=torch.float16)


@pytest.mark.parametrize("sizes,status", [
    ((2, 4112, 64, 8, 2), UNSUPPORTED),        # the router ends at 4096, the operators in 8 bits at 2^15
    ((2, 8192, 64, 8, 2), UNSUPPORTED), ((2, 64, (1 << 15) + 16, 8, 2), UNSUPPORTED), ((2, 64, 64, 1025, 2), UNSUPPORTED),
    (((1 << 20) + 1, 64, 64, 8, 2), UNSUPPORTED), ((2, 64, 64, 64, 33), UNSUPPORTED), ((-1, 64, 64, 8, 2), SHAPE),
    ((2, 72, 64, 8, 2), SHAPE), ((2, 64, 40, 8, 2), SHAPE), ((2, 64, 64, 8, 9), SHAPE), ((2, 64, 64, 8, 0), SHAPE)])
def test_step_sizes_refused_when_made(lib, sizes, status):
    with pytest.raises(sme.MoeError) as e:
        sme.Fp8MoeStep(*sizes, "cpu")
    assert e.value.status == status


@pytest.mark.parametrize("sizes", [(0, 64, 64, 8, 2), (1, 16, 16, 1, 1), (3, 4096, 64, 4, 4), (2, 16, 8192, 1, 1)])
def test_step_sizes_taken(lib, sizes):
    step = sme.Fp8MoeStep(*sizes, "cpu")
    assert step.y.shape == sizes[:2]
    with pytest.raises(TypeError, match="zeros"):
        step.run(step.y, None, None, None, None, None)
    with pytest.raises(ValueError, match="at most"):
        sme.Fp8MoeStep(1 << 32, *sizes[1:], "cpu")


def test_profile_names_the_current_sources():
    """The summary of these operators' kernels names the digest of csrc/fp8/*.hip and *.h (contents concatenated in sorted
    path order), which that of csrc/*.hip and *.h does not cover."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fp8 = os.path.join(root, "sparse_moe_expert_amd", "csrc", "fp8")
    h = hashlib.sha256()
    for name in sorted(glob.glob(os.path.join(fp8, "*.hip")) + glob.glob(os.path.join(fp8, "*.h"))):
        with open(name, "rb") as f:
            h.update(f.read())
    with open(os.path.join(root, "profiles", "block_operators_kernel_stats.md")) as f:
        m = re.search(r"csrc/fp8/[^`]*sha256 prefix: `([0-9a-f]{16})`", f.read())
    assert m, "the summary names no digest of csrc/fp8"
    assert m.group(1) == h.hexdigest()[:16], "the summary was taken on other sources"
