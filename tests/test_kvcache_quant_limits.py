"""Limits of the quantised cache's calls that the host decides (CPU)."""
import pytest

import exact_io_aware_94_b200 as fa
from exact_io_aware_94_b200 import build as fa_build

# A fake, 16-byte aligned address: every call is rejected before any CUDA call.
P = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    return fa.load_library()


@pytest.mark.parametrize("d,bits,group", [(64, 4, 4), (64, 8, 8), (64, 4, 9), (128, 8, 1), (128, 4, 16), (128, 8, 17), (256, 4, 8),
                                          (256, 8, 9)])
def test_decode_capacity_limit(d, bits, group):
    """The whole batch at its capacity has to fit the count of units: what is past that has no workspace size and is
    refused, before the workspace is looked at; what fa.h promises to take is taken."""
    B, Hkv, ps = 40, 2000, 16
    H = Hkv * group

    def size(blocks):
        return fa.fa_decode_paged_quant_workspace_size(B, H, Hkv, blocks, ps, d, bits)

    def call(blocks):
        return fa.fa_decode_paged_quant(P, P, P, P, P, P, P, B, H, Hkv, 64, ps, blocks, d, bits, 0.1, 0, None, 0, 0)

    lo, hi = 1, (1 << 31) // ps - 1
    assert size(lo) > 0 and size(hi) == 0
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if size(mid) > 0 else (lo, mid)
    assert call(lo) == fa.FA_ERR_WORKSPACE and call(hi) == fa.FA_ERR_INVALID_ARG
    assert B * Hkv * -(-group // 8) * (lo + 6) >= (1 << 31) - 256  # a block more is past the promise
