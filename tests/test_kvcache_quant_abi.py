"""Refusals of the quantised cache's calls (CPU), and its format's own arithmetic."""
import numpy as np
import pytest
import torch

import exact_io_aware_94_b200 as fa
from exact_io_aware_94_b200 import build as fa_build

from . import kvq_reference as ref

# Fake, 16-byte aligned addresses: every call is rejected before any CUDA call.
P = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    return fa.load_library()


POOL = [
    (dict(kp=0), fa.FA_ERR_INVALID_ARG),
    (dict(vp=P + 8), fa.FA_ERR_INVALID_ARG),
    (dict(bt=0), fa.FA_ERR_INVALID_ARG),
    (dict(kv=0), fa.FA_ERR_INVALID_ARG),
    (dict(kv=P + 2), fa.FA_ERR_INVALID_ARG),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED),
    (dict(bits=3), fa.FA_ERR_UNSUPPORTED),
    (dict(bits=16), fa.FA_ERR_UNSUPPORTED),
    (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=0), fa.FA_ERR_INVALID_ARG),
    (dict(H=4096, Hkv=4096), fa.FA_ERR_INVALID_ARG),
    (dict(pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(blocks=0), fa.FA_ERR_INVALID_ARG),
    (dict(ps=8), fa.FA_ERR_INVALID_ARG),        # less than a tile
    (dict(ps=48), fa.FA_ERR_INVALID_ARG),       # not a power of two
    (dict(ps=1 << 17), fa.FA_ERR_INVALID_ARG),
    (dict(blocks=1 << 26), fa.FA_ERR_INVALID_ARG),  # capacity past int32
]
BASE = dict(kp=P, vp=P, bt=P, kv=P, cu=P, B=2, H=8, Hkv=2, pages=64, ps=32, blocks=32, d=128, bits=4)


@pytest.mark.parametrize("args,code", POOL + [
    (dict(k=0), fa.FA_ERR_INVALID_ARG),
    (dict(v=P + 2), fa.FA_ERR_INVALID_ARG),
    (dict(cu=0), fa.FA_ERR_INVALID_ARG),
    (dict(sk=255), fa.FA_ERR_INVALID_ARG),      # shorter than a row of 2 heads
    (dict(sv=260), fa.FA_ERR_INVALID_ARG),      # rows not 16-byte aligned
    (dict(total=-1), fa.FA_ERR_INVALID_ARG),
    (dict(most=-1), fa.FA_ERR_INVALID_ARG),
    (dict(B=1 << 16, blocks=1, most=1 << 30), fa.FA_ERR_INVALID_ARG),  # more blocks than a grid has
    (dict(total=0), fa.FA_OK),                  # nothing to do: no launch
    (dict(most=0), fa.FA_OK),
])
def test_append_argument_checks(args, code):
    a = dict(BASE, k=P, v=P, sk=256, sv=256, total=10, most=5)
    a.update(args)
    assert fa.fa_kvcache_append_quant(a["k"], a["v"], a["sk"], a["sv"], a["kp"], a["vp"], a["cu"], a["bt"], a["kv"],
                                      a["B"], a["Hkv"], a["total"], a["most"], a["pages"], a["ps"], a["blocks"],
                                      a["d"], a["bits"], 0) == code


@pytest.mark.parametrize("args,code", POOL + [
    (dict(cu=P + 1), fa.FA_ERR_INVALID_ARG),
    (dict(ko=0), fa.FA_ERR_INVALID_ARG),
    (dict(vo=P + 8), fa.FA_ERR_INVALID_ARG),
    (dict(H=7), fa.FA_ERR_INVALID_ARG),         # not a multiple of Hkv
    (dict(dt=2), fa.FA_ERR_UNSUPPORTED),
    (dict(total=-1), fa.FA_ERR_INVALID_ARG),
    (dict(total=0), fa.FA_OK),
    (dict(most=0), fa.FA_OK),
])
def test_read_argument_checks(args, code):
    a = dict(BASE, ko=P, vo=P, total=10, most=5, dt=0)
    a.update(args)
    assert fa.fa_kvcache_read_quant(a["kp"], a["vp"], a["cu"], a["bt"], a["kv"], a["ko"], a["vo"], a["B"], a["H"],
                                    a["Hkv"], a["total"], a["most"], a["pages"], a["ps"], a["blocks"], a["d"],
                                    a["bits"], a["dt"], 0) == code


@pytest.mark.parametrize("args,code", POOL + [
    (dict(q=P + 8), fa.FA_ERR_INVALID_ARG),
    (dict(o=0), fa.FA_ERR_INVALID_ARG),
    (dict(lse=P + 2), fa.FA_ERR_INVALID_ARG),
    (dict(H=7), fa.FA_ERR_INVALID_ARG),
    (dict(dt=2), fa.FA_ERR_UNSUPPORTED),
    (dict(scale=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID_ARG),
    (dict(ws=0), fa.FA_ERR_WORKSPACE),
    (dict(ws=P + 16), fa.FA_ERR_WORKSPACE),
    (dict(nbytes=-1), fa.FA_ERR_WORKSPACE),     # one byte short
])
def test_decode_argument_checks(args, code):
    a = dict(BASE, q=P, o=P, lse=P, scale=0.1, dt=0, ws=P, nbytes=0)
    a.update(args)
    need = fa.fa_decode_paged_quant_workspace_size(2, 8, 2, 32, 32, 128, 4)
    assert need > 0
    assert fa.fa_decode_paged_quant(a["q"], a["kp"], a["vp"], a["bt"], a["kv"], a["o"], a["lse"], a["B"], a["H"],
                                    a["Hkv"], a["pages"], a["ps"], a["blocks"], a["d"], a["bits"], a["scale"], a["dt"],
                                    a["ws"], need + a["nbytes"], 0) == code


def test_sizes():
    assert fa.fa_kvcache_quant_page_bytes(64, 128, 4) == 64 * 80
    assert fa.fa_kvcache_quant_page_bytes(16, 64, 8) == 16 * 72
    assert fa.fa_kvcache_quant_page_bytes(65536, 256, 8) == 65536 * 288
    for bad in ((8, 128, 4), (24, 128, 4), (64, 96, 4), (64, 128, 2)):
        assert fa.fa_kvcache_quant_page_bytes(*bad) == 0
    assert fa.fa_decode_paged_quant_workspace_size(0, 8, 2, 4, 64, 128, 4) == 0
    assert fa.fa_decode_paged_quant_workspace_size(2, 8, 3, 4, 64, 128, 4) == 0


def test_helpers_refuse_cpu_tensors_and_wrong_types():
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(3, 2, 16 * 40, dtype=torch.uint8)
    i32 = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.kvcache_append_quant(k, k, pool, pool, i32[0], i32, i32[0], 4, 4)
    with pytest.raises(ValueError):
        fa.kvcache_read_quant(pool, pool, i32[0], i32, i32[0], 4, 4, 2, 64, 4)
    with pytest.raises(ValueError):
        fa.decode_paged_quant(k, pool, pool, i32, i32[0], 4)
    with pytest.raises(fa.FAError):
        fa.kvcache_quant_pages(4, 2, 24, 128, 4, device="cpu")
    kp, vp = fa.kvcache_quant_pages(4, 2, 32, 128, 4, device="cpu")
    assert kp.shape == vp.shape == (4, 2, 32 * 80) and not kp.any() and not vp.any()


@pytest.mark.parametrize("d,bits", [(64, 4), (64, 8), (128, 4), (128, 8), (256, 4), (256, 8)])
@pytest.mark.parametrize("unit", [ref.K_UNIT, ref.V_UNIT])
def test_reference_places_are_a_permutation(d, bits, unit):
    """Every code of a tile has bits of its own, and they fill the code bytes exactly."""
    first, width, shift = ref.places(d, bits, unit)
    bit = (first[None] + np.arange(16)[:, None] * width) * 8 + shift[None]
    assert sorted(bit.ravel().tolist()) == list(range(0, 16 * d * bits, bits))


@pytest.mark.parametrize("bits", [4, 8])
def test_reference_rounds_to_the_nearest_code(bits):
    """A stored value is within half a step of the input, and a little more where the bf16 step is too short for the
    range: s >= (1 - 2^-8) of the exact step, so the last code may be (2^bits - 1) 2^-8 steps away from the greatest
    value, and rounding (x - lo) / s in fp32 moves a border by less than 2^-20 steps."""
    x = ref.round_bf16(np.random.default_rng(1).normal(0, 3, (500, 128)))
    c, lo, s = ref.quantise(x, bits)
    got = np.repeat(lo.astype(np.float64), 32, -1) + np.repeat(s.astype(np.float64), 32, -1) * c
    bound = max(0.5, (2 ** bits - 1) * 2.0 ** -8 / (1 - 2.0 ** -8)) + 2.0 ** -10
    assert (np.abs(got - x) <= bound * np.repeat(s, 32, -1)).all()


@pytest.mark.parametrize("d,bits", [(64, 4), (128, 8), (256, 4)])
def test_reference_store_and_load_round_trip(d, bits):
    pool = np.full((2, 3, 32 * ref.row_bytes(d, bits)), 0xA5, np.uint8)
    x = ref.round_bf16(np.random.default_rng(2).normal(size=(32, 3, d)))
    for slot in np.random.default_rng(3).permutation(32):
        ref.store(pool, 1, slot, x[slot], bits, ref.V_UNIT)
    assert (pool[0] == 0xA5).all()
    for slot in range(32):
        c, lo, s = ref.load(pool, 1, slot, d, bits, ref.V_UNIT)
        want = ref.quantise(x[slot], bits)
        assert (c == want[0]).all() and (lo == np.repeat(want[1], 32, -1)).all() and (s == np.repeat(want[2], 32, -1)).all()
