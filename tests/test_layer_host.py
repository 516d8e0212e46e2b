"""Host side of the grouped routing and the 4-bit products that needs no device:
workspace sizes over batches, sizes beyond 32 bits, importing the package on a torch
without a GPU; and that the profile of their kernels is of the sources as they stand."""

import glob
import hashlib
import os
import re
import subprocess
import sys

import pytest
import torch

import sparse_moe_expert_amd as sme
import sparse_moe_expert_amd.build


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(sme.LIB_PATH):
        sme.build.build_library()
    return sme.load_library()


# every batch to 300, then ever wider steps, to past the last that is split for any size (128 tiles of 64 tokens)
BATCHES = [*range(1, 300), *(t + d for t in range(320, 8400, 64) for d in (-1, 0, 1)), 16384, 1 << 20]


@pytest.mark.parametrize("H,Is", [(2560, 640), (7168, 2048), (64, 96), (32, 32768), (32768, 32), (4096, 12288), (2048, 512)])
def test_workspace_serves_smaller_batches(H, Is):
    """A workspace made for a batch is large enough for every smaller one; the sums of split reductions never take more
    than what the header says."""
    made = {T: sme.make_quant_shared_workspace(T, H, Is, "meta").numel() for T in BATCHES}
    most = 0
    for T in BATCHES:
        most = max(most, sme.moe_quant_shared_expert_workspace_size(T, H, Is))
        assert made[T] >= most, T
        for N, K in ((H, Is), (Is, H), (9999, H), (257, Is)):
            assert sme.moe_quant_linear_workspace_size(T, N, K) <= sme.QUANT_SUMS_BYTES, (T, N, K)


def test_import_without_gpu_functions():
    """A torch that was built without a GPU lacks the device and stream queries the calls use."""
    code = ("import torch\n"
            "for name in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "import sparse_moe_expert_amd as sme\n"
            "print(sme.RouteRule(4).k)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["4"]


def test_sizes_beyond_32_bits():
    """The library takes sizes of 32 bits; 2^32 + 8 is not 8."""
    for kw in (dict(k=(1 << 32) + 8), dict(k=8, groups=(1 << 32) + 1), dict(k=8, groups=2, groups_kept=1 - (1 << 32)),
               dict(k=8, group_top=(1 << 32) + 2)):
        with pytest.raises(ValueError, match="at most"):
            sme.RouteRule(**kw)
    with pytest.raises(ValueError, match="whole number"):
        sme.RouteRule(4.5)
    assert sme.RouteRule(4.0).k == 4
    for T, E in (((1 << 32) + 1, 1), (1, (1 << 32) + 1)):
        with pytest.raises(ValueError, match="at most"):
            sme.moe_route_grouped(torch.empty((T, E), device="meta"), None, sme.RouteRule(1))
    with pytest.raises(ValueError, match="at most"):
        sme.QuantWeight(torch.empty(((1 << 32) + 1, 16), dtype=torch.uint8, device="meta"),
                        torch.empty(((1 << 32) + 1, 1), dtype=torch.uint8, device="meta"), format="mxfp4")
    for sizes in (((1 << 32) + 64, 4096, 4096), (64, (1 << 32) + 4096, 4096), (64, 4096, (1 << 32) + 4096)):
        for size in (sme.moe_quant_linear_workspace_size, sme.moe_quant_shared_expert_workspace_size):
            with pytest.raises(ValueError, match="at most"):
                size(*sizes)
    assert sme.moe_quant_linear_workspace_size(-1, 64, 64) == 0


def test_profile_names_the_current_sources():
    """The summary of these operators' kernels names the digest of csrc/layer/*.hip and *.h (contents concatenated in
    sorted path order), which that of csrc/*.hip and *.h does not cover."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    layer = os.path.join(root, "sparse_moe_expert_amd", "csrc", "layer")
    h = hashlib.sha256()
    for name in sorted(glob.glob(os.path.join(layer, "*.hip")) + glob.glob(os.path.join(layer, "*.h"))):
        with open(name, "rb") as f:
            h.update(f.read())
    with open(os.path.join(root, "profiles", "layer_operators_kernel_stats.md")) as f:
        m = re.search(r"csrc/layer/[^`]*sha256 prefix: `([0-9a-f]{16})`", f.read())
    assert m, "the summary names no digest of csrc/layer"
    assert m.group(1) == h.hexdigest()[:16], "the summary was taken on other sources"
