"""Decode over the quantised paged cache where outputs are small beside the largest values: tokens of widely different
magnitudes, long sequences, the largest pages."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_94_b200 as fa

from . import kvq_reference as ref
from . import test_kvcache_quant_gpu as kvq
from .parity import to_np

pytestmark = pytest.mark.gpu


def decode64(q, kpool, vpool, table, lens, bits, scale):
    """(o, tolerance of o) in 64 bits for q [B, H, d] (float64).

    Tolerances.  A key's weight u is 2^6 or more for the greatest p of its warp's keys.  It is rounded to fp16, and the output
    is divided by the sum of the rounded weights: p moves by 2^-11 p + min(p, 2^-25 / 2^6 of the greatest p), which weighs
    v - o.  The offset of a group, lo or hi = lo + C s (C the greatest code), is rounded to fp16 over 2^E: by 2^-11 of it or
    2^-25 2^E, whichever is more.  s is held over 2^(E - bits + 1), exactly or to 2^-25 of that, and multiplies c or C - c,
    at most C; u s is rounded to fp16 likewise, by 2^-11 or 2^-31 2^(E - bits + 1) of the greatest p.  2^E is at most twice
    M, the greatest of |lo|, |hi| and 2^(bits - 1) s that the group of dimensions has in the sequence.  Scores are off by
    2^-20 of the sum of their terms' magnitudes, exponentials by 2^-22.  Sums of low nibbles may lose 2^-14 of sum(p s C).
    1 + 2^-8 covers the products of these."""
    B, H, d = q.shape
    G, C, half = H // kpool.shape[1], 2 ** bits - 1, 2.0 ** (bits - 1)
    o, tol = np.zeros((B, H, d)), np.zeros((B, H, d))
    for b in range(B):
        n = int(lens[b])
        kc, klo, ks = ref.rows(kpool, table[b], range(n), d, bits, ref.K_UNIT)
        vc, vlo, vs = ref.rows(vpool, table[b], range(n), d, bits, ref.V_UNIT)
        for h in range(H):
            g = h // G
            x = scale * ((klo + ks * kc)[:, g] @ q[b, h])
            ex = 2.0 ** -20 * scale * ((np.abs(klo) + ks * kc)[:, g] @ np.abs(q[b, h])).max() + 2.0 ** -21
            p = np.exp(x - x.max())
            p /= p.sum()
            lo, s, c = vlo[:, g], vs[:, g], vc[:, g]
            v, hi = lo + s * c, lo + C * s
            o[b, h] = p @ v
            big = np.maximum(np.abs(lo), np.abs(hi))
            M = np.maximum(big, half * s).reshape(n, -1, ref.GROUP).max((0, 2)).repeat(ref.GROUP)
            least = np.minimum(p, 2.0 ** -31 * p.max())[:, None]
            tol[b, h] = (1 + 2.0 ** -8) * (
                ((2.0 ** -11 * p)[:, None] + least).T.reshape(1, n) @ np.abs(v - o[b, h])
                + p @ np.maximum(2.0 ** -11 * big, 2.0 ** -25 * 2 * M)
                + (2.0 ** -11 + 2.0 ** -14) * (p @ (C * s)) + 2.0 ** -25 * 2 * M * C / half
                + np.minimum(p[:, None] * s * C, 2.0 ** -31 * p.max() * 2 * M * C / half).sum(0)
                + 2 * ex * (p @ (np.abs(lo) + s * c)))[0]
    return o, tol


@pytest.mark.parametrize("log2_ratio", [0, 6, 8, 10, 12, 14])
@pytest.mark.parametrize("d,bits,H,Hkv", [(64, 4, 3, 1), (64, 8, 9, 1), (128, 4, 12, 1), (128, 8, 4, 2), (256, 4, 2, 1),
                                          (256, 8, 8, 1)])
def test_decode_beside_large_values_without_weight(cuda_device, d, bits, H, Hkv, log2_ratio):
    """One token of every 16 has values 2^log2_ratio times those of the others and a score some 40 nats below: the output
    is the others' average, and nearly as exact as without that token.  A bound below 2^-6 of every output shows that
    zeros, or the small values' codes lost, would not pass."""
    dev, ps, lens = cuda_device, 16, [64, 33, 700]
    table, pages = kvq.make_table(lens, ps, 1, seed=3)
    gen = torch.Generator().manual_seed(150 + log2_ratio)
    T = sum(lens)
    q = torch.randn(len(lens), H, d, generator=gen).abs().to(torch.bfloat16)
    k = 0.1 * torch.randn(T, Hkv, d, generator=gen)
    sign = torch.where(torch.rand(Hkv, d, generator=gen) < 0.5, -1.0, 1.0)
    v = (1.0 + 0.4 * torch.randn(T, Hkv, d, generator=gen).clamp(-2, 2)) * sign
    at = torch.arange(T)
    loud = at % 16 == at // 16 * 5 % 16
    k[loud] -= 5.0 * math.sqrt(128.0 / d)
    v[loud] *= 2.0 ** log2_ratio
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    kpool, vpool = (np.zeros((pages, Hkv, ps * ref.row_bytes(d, bits)), np.uint8) for _ in range(2))
    cu = np.concatenate(([0], np.cumsum(lens)))
    kvq.append_reference(kpool, vpool, k.float().numpy(), v.float().numpy(), cu, table, lens, bits)
    scale = 1.0 / math.sqrt(d)
    o_ref, tol = decode64(q.double().numpy(), kpool, vpool, table, lens, bits, scale)
    assert (tol <= 2.0 ** -6 * np.abs(o_ref)).all()
    o, _ = fa.decode_paged_quant(q.to(dev), torch.from_numpy(kpool).to(dev), torch.from_numpy(vpool).to(dev),
                                 kvq.i32(table, dev), kvq.i32(lens, dev), bits, scale=scale)
    assert fa.fa_check_status() == fa.FA_OK
    over = np.abs(to_np(o) - o_ref) / tol
    assert over.max() <= 1.0, "o beyond its tolerance by a factor of %.3g" % over.max()


@pytest.mark.parametrize("lens,H,Hkv,ps,d,bits", [
    ([400000], 4, 1, 1024, 64, 4),
    ([400000], 2, 1, 1024, 64, 8),
    ([90000, 3], 2, 2, 65536, 128, 8),
    ([70000, 65536, 65537], 12, 1, 65536, 128, 4),
    ([66000, 131072], 9, 1, 65536, 64, 4),
    ([70000], 3, 1, 65536, 256, 4),
    ([16, 70000], 2, 2, 65536, 256, 8),
])
def test_decode_outputs_of_long_sequences(cuda_device, lens, H, Hkv, ps, d, bits):
    """Each head's error beside its output, in the norm: the roundings of a key (fp16, 2^-12.8 in the mean square, of the
    weight, the offset and the weighted step: terms of at most 4 standard deviations of a value) are independent, and over many
    keys average out as the values do.  They are sqrt(3) 4 2^-12.8 = 2^-10 of an output; 2^-8 leaves a factor of 4.  Values of another page, or
    zeros, would be off by the whole output."""
    dev = cuda_device
    table, pages = kvq.make_table(lens, ps, 2, seed=9)
    kd, vd = (torch.from_numpy(ref.random_pool(pages, Hkv, ps, d, bits, seed=160 + i)).to(dev) for i in (0, 1))
    q = torch.randn(len(lens), H, d, generator=torch.Generator().manual_seed(161)).to(torch.bfloat16).to(dev)
    table, lens = kvq.i32(table, dev), kvq.i32(lens, dev)
    o_ref, _, _, _ = kvq.attention64(q, kd, vd, table, lens, bits, 1.0 / math.sqrt(d), d)
    o, _ = fa.decode_paged_quant(q, kd, vd, table, lens, bits)
    assert fa.fa_check_status() == fa.FA_OK
    off = (o - o_ref).norm(dim=-1) / o_ref.norm(dim=-1)
    assert float(off.max()) <= 2.0 ** -8, "off by %.3g of the output" % float(off.max())


@pytest.mark.parametrize("d,bits,H,Hkv", [(64, 8, 1, 1), (64, 8, 9, 1), (128, 8, 12, 1)])
def test_decode_average_of_many_values_in_the_other_formats(cuda_device, d, bits, H, Hkv):
    kvq.test_decode_average_of_many_values(cuda_device, d, bits, H, Hkv)


def constant_keys(lo, ps, d, bits):
    """Pool of keys that are lo [keys, d / 32] in all dimensions of a group, exactly; page i holds keys ps i and on."""
    n = lo.shape[0]
    pool = np.zeros((-(-n // ps), 1, ps // 16, 16 * ref.row_bytes(d, bits)), np.uint8)
    par = np.zeros((pool.shape[0] * ps, d // 32, 2), np.uint32)
    par[:n, :, 0] = lo.astype(np.float32).view(np.uint32) >> 16
    pool[..., 16 * d * bits // 8:] = par.astype(np.uint16).view(np.uint8).reshape(*pool.shape[:3], -1)
    return pool.reshape(pool.shape[0], 1, -1)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_scores_far_from_zero(cuda_device, d, bits):
    """Equal scores of -2^105 and 2^105.  lse is the score, and a single key's output its value (within 2^-11 of its terms:
    the value, its offset and its range, 8 at most in these pools).  More keys are averaged by each warp, but their parts merged
    by log-sum-exps that end at 2^82, where log2 of a part's number of keys is lost: parts of any size count the same, and the
    outputs lie among the values, as weights that are not negative and sum to 1 have it."""
    dev, ps, lens = cuda_device, 16, [1, 40, 700]
    table, pages = kvq.make_table(lens, ps, 0, seed=1)
    kpool = constant_keys(np.full((pages * ps, d // 32), 2.0 ** 45), ps, d, bits)
    vpool = ref.random_pool(pages, 1, ps, d, bits, seed=170)
    q = torch.full((3, 2, d), 2.0 ** 60, dtype=torch.bfloat16)
    q[:, 0] = -q[:, 0]
    o, lse = fa.decode_paged_quant(q.to(dev), torch.from_numpy(kpool).to(dev), torch.from_numpy(vpool).to(dev),
                                   kvq.i32(table, dev), kvq.i32(lens, dev), bits, scale=1.0 / d)
    assert fa.fa_check_status() == fa.FA_OK
    for b, n in enumerate(lens):
        v = ref.values(vpool, table[b], range(n), d, bits, ref.V_UNIT)[:, 0]
        tol = 3 * 2.0 ** -11 * 8
        assert ((to_np(o)[b] >= v.min(0) - tol) & (to_np(o)[b] <= v.max(0) + tol)).all()
    off = np.abs(to_np(lse) / 2.0 ** 105 - [-1, 1])
    assert off.max() <= 2.0 ** -20


@pytest.mark.parametrize("d,bits,warps", [(64, 4, 12), (64, 8, 16), (128, 4, 12), (128, 8, 12), (256, 4, 8), (256, 8, 8)])
def test_decode_large_scores_that_rise_by_8_bits(cuda_device, d, bits, warps):
    """Scores of 1.5 2^26 in base 2, where fp32 ends at 8, that rise by 8 half-way through each sequence.  They are exact, so the
    output is the average of the values with weights of 2^-8 and 1, but for three roundings of 2^-11 as above.  A sequence that
    is cut between warps is merged by log-sum-exps that end at 8 too, which may move weight from one part to the other: with
    as many sequences as warps those are the fewest, and their outputs still lie among the values."""
    dev, ps, n, rise = cuda_device, 64, 320, 160
    B = torch.cuda.get_device_properties(dev).multi_processor_count * warps
    lo = np.zeros((n, d // 32))
    lo[:, 0] = 1.5 * 2.0 ** 14
    lo[rise:, 1] = 8.0
    kpool = constant_keys(lo, ps, d, bits)
    vpool = ref.random_pool(n // ps, 1, ps, d, bits, seed=171)
    q = torch.zeros(B, 1, d, dtype=torch.bfloat16)
    q[:, :, 0], q[:, :, 32] = 2.0 ** 12, 1.0
    scale = float(np.float32(1.0) / np.float32(1.4426950408889634))
    assert np.float32(scale) * np.float32(1.4426950408889634) == 1.0
    table = torch.arange(n // ps, dtype=torch.int32, device=dev).repeat(B, 1)
    lens = torch.full((B,), n, dtype=torch.int32, device=dev)
    o, _ = fa.decode_paged_quant(q.to(dev), torch.from_numpy(kpool).to(dev), torch.from_numpy(vpool).to(dev), table, lens,
                                 bits, scale=scale)
    assert fa.fa_check_status() == fa.FA_OK
    v = ref.values(vpool, np.arange(n // ps), range(n), d, bits, ref.V_UNIT)[:, 0]
    w = np.where(np.arange(n) < rise, 2.0 ** -8, 1.0)
    tol = 3 * 2.0 ** -11 * 8
    o = to_np(o)[:, 0]
    assert np.isfinite(o).all()
    assert ((o >= v.min(0) - tol) & (o <= v.max(0) + tol)).all()
    exact = np.abs(o - w @ v / w.sum()).max(-1) <= tol
    assert exact.mean() >= 0.5


@pytest.mark.parametrize("log2_spread", [-90, -105, -115])
@pytest.mark.parametrize("d,bits", [(64, 8), (128, 4)])
def test_decode_tiny_values(cuda_device, d, bits, log2_spread):
    """Values near fp32's least: below 2^-100 a group's power of two stays 2^-100, so an offset is off by 2^-125 and a step's
    part by twice that, 2^-123 with the products' roundings (2^-31 2^-100 2 of the greatest weight, of 200 keys)."""
    dev, ps, lens = cuda_device, 16, [200, 37]
    table, pages = kvq.make_table(lens, ps, 1, seed=5)
    kpool = ref.random_pool(pages, 1, ps, d, bits, seed=180)
    vpool = ref.random_pool(pages, 1, ps, d, bits, seed=181, spread=2.0 ** log2_spread)
    q = torch.randn(2, 3, d, generator=torch.Generator().manual_seed(182)).to(torch.bfloat16)
    o_ref, tol = decode64(q.double().numpy(), kpool, vpool, table, lens, bits, 0.1)
    o, _ = fa.decode_paged_quant(q.to(dev), torch.from_numpy(kpool).to(dev), torch.from_numpy(vpool).to(dev),
                                 kvq.i32(table, dev), kvq.i32(lens, dev), bits, scale=0.1)
    assert fa.fa_check_status() == fa.FA_OK
    over = np.abs(to_np(o) - o_ref) / (tol + 2.0 ** -123)
    assert over.max() <= 1.0, "o beyond its tolerance by a factor of %.3g" % over.max()
