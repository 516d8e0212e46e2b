"""Host side of the grouped routing and the 4-bit products that needs no device:
workspace sizes over batches."""

import os

import pytest

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
