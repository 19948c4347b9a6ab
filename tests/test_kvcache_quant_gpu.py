"""The quantised paged cache on the GPU: its writer and its reader bit for bit, decode within derived tolerances."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_94_b200 as fa
import oracle

from . import kvq_reference as ref
from .parity import check_lse, check_o, to_np

pytestmark = pytest.mark.gpu

FORMATS = [(64, 4), (64, 8), (128, 4), (128, 8), (256, 4), (256, 8)]


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def cu_of(rows, dev):
    return i32(np.concatenate(([0], np.cumsum(rows))), dev)


def make_table(lens, ps, spare, seed, extra_blocks=0):
    """Block table with distinct shuffled pages; slots past a sequence's last block point outside the pool."""
    used = [-(-n // ps) for n in lens]
    pool = sum(used) + spare
    perm = np.random.default_rng(seed).permutation(pool).astype(np.int32)
    table = np.full((len(lens), max(1, max(used)) + extra_blocks), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pool


def same_pool(got, want, d, bits):
    """Equal codes, and equal lo and s as numbers (a zero's sign may differ)."""
    rb = ref.row_bytes(d, bits)
    got, want = (x.reshape(-1, 16 * rb) for x in (got, want))
    split = 16 * d * bits // 8
    assert (got[:, :split] == want[:, :split]).all()
    a, b = ((np.ascontiguousarray(x[:, split:]).view(np.uint16).astype(np.uint32) << 16).view(np.float32) for x in (got, want))
    assert np.array_equal(a, b, equal_nan=True)


def append_reference(kpool, vpool, k, v, cu, table, lens, bits):
    d = k.shape[-1]
    ps = kpool.shape[2] // ref.row_bytes(d, bits)
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            pos = lens[b] - n + i
            for pool, x, unit in ((kpool, k, ref.K_UNIT), (vpool, v, ref.V_UNIT)):
                ref.store(pool, table[b, pos // ps], pos % ps, x[cu[b] + i], bits, unit)


@pytest.mark.parametrize("d,bits,Hkv,ps", [(64, 4, 3, 16), (64, 8, 1, 64), (128, 4, 2, 32), (128, 8, 5, 16),
                                           (256, 4, 1, 16), (256, 8, 2, 128)])
def test_append_and_read_bit_for_bit(cuda_device, d, bits, Hkv, ps):
    """Chunks of 0 to 130 rows behind prefixes of any length, rows taken as slices of a fused projection; what the
    call does not own keeps its bytes; then all of it, and its last rows, read back for groups of 3 query heads."""
    dev = cuda_device
    new = [0, 1, 15, 16, 17, 130, 1]
    lens = [5, 1, 40, 16, 100, 130, 33]
    table, pages = make_table(lens, ps, 2, seed=d + bits)
    gen = torch.Generator().manual_seed(d * bits)
    T = sum(new)
    qkv = torch.randn(T, 2 + 2 * Hkv, d, generator=gen).to(torch.bfloat16)
    k, v = qkv[:, 2:2 + Hkv], qkv[:, 2 + Hkv:]
    kpool = ref.random_pool(pages, Hkv, ps, d, bits, seed=1)
    vpool = ref.random_pool(pages, Hkv, ps, d, bits, seed=2)
    kp, vp = (torch.from_numpy(x.copy()).to(dev) for x in (kpool, vpool))
    cu = np.concatenate(([0], np.cumsum(new)))
    append_reference(kpool, vpool, k.float().numpy(), v.float().numpy(), cu, table, lens, bits)
    qd = qkv.to(dev)
    fa.kvcache_append_quant(qd[:, 2:2 + Hkv], qd[:, 2 + Hkv:], kp, vp, i32(cu, dev), i32(table, dev), i32(lens, dev),
                            max(new), bits)
    assert fa.fa_check_status() == fa.FA_OK
    same_pool(kp.cpu().numpy(), kpool, d, bits)
    same_pool(vp.cpu().numpy(), vpool, d, bits)
    for rows in (lens, new):
        want = [np.concatenate([ref.values(pool, table[b], range(lens[b] - rows[b], lens[b]), d, bits, unit)
                                for b in range(len(lens))]) for pool, unit in ((kpool, ref.K_UNIT), (vpool, ref.V_UNIT))]
        for dt in (torch.bfloat16, torch.float32):
            got = fa.kvcache_read_quant(kp, vp, cu_of(rows, dev), i32(table, dev), i32(lens, dev), sum(rows), max(rows),
                                        3 * Hkv, d, bits, out_dtype=dt)
            for g, w in zip(got, want):
                w = ref.round_once(np.repeat(w, 3, 1), dt)
                assert torch.equal(g.cpu(), w)
    assert fa.fa_check_status() == fa.FA_OK


@pytest.mark.parametrize("bits", [4, 8])
def test_append_unusual_values(cuda_device, bits):
    """Groups that are constant, hold zeros of both signs, an infinity or NaN, steps below fp32's least normal, spreads
    past fp32's greatest, and ties between two codes; each beside ordinary groups, which keep their values."""
    dev, d, ps = cuda_device, 128, 16
    x = torch.randn(12, 2, d, generator=torch.Generator().manual_seed(3))
    x[0, 0, :32] = 1.5
    x[1, 1, 32:64] = 0.0
    x[1, 1, 40:44] = -0.0
    x[2, 0, 70] = math.inf
    x[3, 0, 71] = -math.inf
    x[4, 1, 100] = math.nan
    x[5, 0, :32] = torch.linspace(0, 1e-39, 32)
    x[6, 0, :32] = torch.linspace(-3.3e38, 3.3e38, 32)
    x[7, 0, :32] = torch.linspace(-1.6e38, 1.6e38, 32)
    x[8, 0, :32] = torch.arange(32) * 0.5 % (2 ** bits - 0.5)   # halves of a step
    x[8, 0, 31] = 2 ** bits - 1
    x[9, 0, :32] = 1e-30 * torch.arange(32)
    x = x.to(torch.bfloat16)
    table = np.array([[1]], np.int32)
    pool = np.zeros((2, 2, ps * ref.row_bytes(d, bits)), np.uint8)
    kpool, vpool = pool.copy(), pool.copy()
    kp, vp = (torch.from_numpy(pool.copy()).to(dev) for _ in range(2))
    f = x.float().numpy()
    append_reference(kpool, vpool, f, f, [0, 12], table, [12], bits)
    xd = x.to(dev)
    fa.kvcache_append_quant(xd, xd, kp, vp, i32([0, 12], dev), i32(table, dev), i32([12], dev), 12, bits)
    same_pool(kp.cpu().numpy(), kpool, d, bits)
    same_pool(vp.cpu().numpy(), vpool, d, bits)
    k, _ = fa.kvcache_read_quant(kp, vp, i32([0, 12], dev), i32(table, dev), i32([12], dev), 12, 12, 2, d, bits)
    nan = torch.zeros(12, 2, d, dtype=torch.bool)
    for t, h, g in ((2, 0, 2), (3, 0, 2), (4, 1, 3), (6, 0, 0)):
        nan[t, h, 32 * g:32 * g + 32] = True
    assert torch.equal(torch.isnan(k.cpu()), nan)
    assert fa.fa_check_status() == fa.FA_OK


@pytest.mark.parametrize("bits", [4, 8])
def test_append_rounds_as_defined_at_every_exponent(cuda_device, bits):
    """Groups of spreads from 2^-130 to 2^127 (quotient and reciprocal are computed without a division), and every
    8-bit step: bit for bit."""
    dev, d, ps = cuda_device, 128, 64
    gen = torch.Generator().manual_seed(8)
    n = 1024
    x = torch.randn(n, 2, d, generator=gen, dtype=torch.float64)
    x *= 2.0 ** torch.randint(-128, 124, (n, 2, d // 32, 1), generator=gen).expand(-1, -1, -1, 32).reshape(n, 2, d)
    top = (torch.arange(128) / 128.0 + 1.0).repeat(n * 2 * (d // 32) // 128 // 2)  # every significand of hi, lo = 0
    y = x.reshape(-1, 32)
    y[: top.numel()] = y[: top.numel()].abs() / y[: top.numel()].abs().amax(1, keepdim=True)
    y[: top.numel(), 0] = 0.0
    y[: top.numel()] *= (top * (2 ** bits - 1) * 2.0 ** torch.randint(-60, 60, top.shape, generator=gen))[:, None]
    x = y.reshape(n, 2, d).to(torch.bfloat16)
    table = np.random.default_rng(2).permutation(n // ps)[None].astype(np.int32)
    pool = np.zeros((n // ps, 2, ps * ref.row_bytes(d, bits)), np.uint8)
    kpool, vpool = pool.copy(), pool.copy()
    kp, vp = (torch.from_numpy(pool.copy()).to(dev) for _ in range(2))
    f = x.float().numpy()
    append_reference(kpool, vpool, f, f, [0, n], table, [n], bits)
    fa.kvcache_append_quant(x.to(dev), x.to(dev), kp, vp, i32([0, n], dev), i32(table, dev), i32([n], dev), n, bits)
    assert fa.fa_check_status() == fa.FA_OK
    same_pool(kp.cpu().numpy(), kpool, d, bits)
    same_pool(vp.cpu().numpy(), vpool, d, bits)


def test_append_and_read_invalid_sequences(cuda_device):
    """Each invalid sequence or page is flagged and leaves the pools and the outputs as they were; its neighbours are
    served."""
    dev, d, bits, ps, Hkv = cuda_device, 64, 4, 16, 2
    B, blocks = 3, 4
    table = np.arange(B * blocks, dtype=np.int32).reshape(B, blocks)
    k = torch.randn(12, Hkv, d, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    f, kd = k.float().numpy(), k.to(dev)

    def go(cu, lens, most, code, skipped, tab=table):
        pool = np.full((B * blocks, Hkv, ps * ref.row_bytes(d, bits)), 0x21, np.uint8)
        want = pool.copy()
        ok = [b for b in range(B) if b not in skipped]
        for b in ok:
            append_reference(want, pool.copy(), f[cu[b]:cu[b + 1]], f[cu[b]:cu[b + 1]], [0, cu[b + 1] - cu[b]], tab[b:b + 1],
                             [lens[b]], bits)
        kp, vp = (torch.from_numpy(pool.copy()).to(dev) for _ in range(2))
        args = (i32(cu, dev), i32(tab, dev), i32(lens, dev))
        fa.kvcache_append_quant(kd, kd, kp, vp, *args, most, bits)
        assert fa.fa_check_status() == code
        same_pool(kp.cpu().numpy(), want, d, bits)
        ko, vo = (torch.full((14, Hkv, d), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
        rc = fa.fa_kvcache_read_quant(kp, vp, *args, ko, vo, B, Hkv, Hkv, 12, most, B * blocks, ps, blocks, d, bits,
                                      fa.FA_DT_BF16)
        assert rc == fa.FA_OK and fa.fa_check_status() == code
        written = np.zeros(14, bool)
        for b in ok:
            written[cu[b]:cu[b + 1]] = True
        assert (ko.cpu()[~torch.from_numpy(written)] == 7.0).all() and (vo.cpu()[~torch.from_numpy(written)] == 7.0).all()
        for b in ok:
            n = cu[b + 1] - cu[b]
            w = ref.values(want, tab[b], range(lens[b] - n, lens[b]), d, bits, ref.K_UNIT)
            assert torch.equal(ko[cu[b]:cu[b + 1]].cpu(), ref.round_once(w, torch.bfloat16))

    go([0, 4, 8, 12], [4, 30, 64], 4, fa.FA_OK, [])
    go([0, 4, 8, 10], [4, 30, 64], 4, fa.FA_OK, [])              # rows 10, 11 belong to nobody
    go([0, 4, 8, 12], [4, 65, 64], 4, fa.FA_ERR_KV_LEN, [1])     # past the capacity
    go([0, 4, 8, 12], [4, -1, 64], 4, fa.FA_ERR_KV_LEN, [1])
    go([0, 4, 8, 12], [4, 3, 64], 4, fa.FA_ERR_SEQLEN, [1])      # more rows than the length
    go([0, 4, 9, 12], [4, 30, 64], 4, fa.FA_ERR_SEQLEN, [1])     # more rows than max_seqlen_new
    go([0, 4, 2, 5], [4, 30, 64], 4, fa.FA_ERR_SEQLEN, [1])      # decreasing
    go([0, 4, 8, 13], [4, 30, 64], 8, fa.FA_ERR_SEQLEN, [2])     # past the packed rows
    go([-2, 4, 8, 12], [9, 30, 64], 9, fa.FA_ERR_SEQLEN, [0])


@pytest.mark.parametrize("bits", [4, 8])
def test_read_into_outputs_aligned_to_16_bytes_only(cuda_device, bits):
    dev, d, ps, Hkv, n = cuda_device, 64, 16, 3, 21
    pool = ref.random_pool(2, Hkv, ps, d, bits, seed=7)
    kp = torch.from_numpy(pool).to(dev)
    out = torch.full((2, n * Hkv * d + 16), 5.0, dtype=torch.bfloat16, device=dev)
    ko, vo = (o[8:8 + n * Hkv * d] for o in out)
    assert ko.data_ptr() % 32 == 16
    args = (i32([0, n], dev), i32([[1, 0]], dev), i32([n], dev))
    assert fa.fa_kvcache_read_quant(kp, kp, *args, ko, vo, 1, Hkv, Hkv, n, n, 2, ps, 2, d, bits, fa.FA_DT_BF16) == fa.FA_OK
    assert fa.fa_check_status() == fa.FA_OK
    for o, unit in ((ko, ref.K_UNIT), (vo, ref.V_UNIT)):
        w = ref.round_once(ref.values(pool, [1, 0], range(n), d, bits, unit), torch.bfloat16)
        assert torch.equal(o.cpu().reshape(n, Hkv, d), w)
    assert (out[:, :8] == 5.0).all() and (out[:, -8:] == 5.0).all()


@pytest.mark.parametrize("bad", [-1, 12, 1 << 30])
def test_append_bad_page(cuda_device, bad):
    dev, d, bits, ps, Hkv = cuda_device, 64, 4, 16, 2
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    table[1, 1] = bad  # positions 16 to 31 of sequence 1
    k = torch.randn(60, Hkv, d, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    pool = np.full((12, Hkv, ps * ref.row_bytes(d, bits)), 0x21, np.uint8)
    want, f = pool.copy(), k.float().numpy()
    cu, lens = [0, 20, 40, 60], [20, 40, 60]
    for b in range(3):
        for i in range(20):
            pos = lens[b] - 20 + i
            if not (b == 1 and pos // ps == 1):
                ref.store(want, table[b, pos // ps], pos % ps, f[cu[b] + i], bits, ref.K_UNIT)
    kp, vp = (torch.from_numpy(pool.copy()).to(dev) for _ in range(2))
    fa.kvcache_append_quant(k.to(dev), k.to(dev), kp, vp, i32(cu, dev), i32(table, dev), i32(lens, dev), 20, bits)
    assert fa.fa_check_status() == fa.FA_ERR_PAGE
    same_pool(kp.cpu().numpy(), want, d, bits)
    got, _ = fa.kvcache_read_quant(kp, vp, i32(cu, dev), i32(table, dev), i32(lens, dev), 60, 20, Hkv, d, bits)
    assert fa.fa_check_status() == fa.FA_ERR_PAGE
    tab0 = np.where((table < 0) | (table >= 12), 0, table)  # read as page 0
    for b in range(3):
        w = ref.values(want, tab0[b], range(lens[b] - 20, lens[b]), d, bits, ref.K_UNIT)
        assert torch.equal(got[cu[b]:cu[b + 1]].cpu(), ref.round_once(w, torch.bfloat16))


def check_decode(dev, q, kpool, vpool, table, lens, bits, scale, dtypes=(torch.float32, torch.bfloat16), kd=None, vd=None):
    want = ref.decode(q.double().numpy(), kpool, vpool, table, lens, bits, scale)
    o_ref, lse_ref, tol_o, tol_l = want
    kd = torch.from_numpy(kpool).to(dev) if kd is None else kd
    vd = torch.from_numpy(vpool).to(dev) if vd is None else vd
    for dt in dtypes:
        o, lse = fa.decode_paged_quant(q.to(dev), kd, vd, i32(table, dev), i32(lens, dev), bits, scale=scale, out_dtype=dt)
        assert fa.fa_check_status() == fa.FA_OK
        o, lse = to_np(o), to_np(lse)
        assert np.array_equal(np.isnan(o), np.isnan(o_ref)) and np.array_equal(np.isnan(lse), np.isnan(lse_ref))
        tol = tol_o + np.abs(o_ref) * (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -23)
        fine = ~np.isnan(o_ref)
        over = (np.abs(o - o_ref) - tol)[fine]
        assert over.size == 0 or over.max() <= 0, "o beyond its tolerance by %.3g" % over.max()
        inf = np.isneginf(lse_ref)
        assert np.array_equal(np.isneginf(lse), inf)
        fin = ~inf & ~np.isnan(lse_ref)
        assert (np.abs(lse[fin] - lse_ref[fin]) <= tol_l[fin]).all()
    return o_ref, lse_ref


def poison(pool, table, lens, d, bits):
    """A copy of the pool with every byte that no valid position uses set to 0xFF (lo and s read as NaN)."""
    ps = pool.shape[2] // ref.row_bytes(d, bits)
    out = np.full_like(pool, 0xFF)
    for b, n in enumerate(lens):
        for pos in range(n):
            pg = table[b, pos // ps]
            at, _, par = ref.row_places(pos % ps, d, bits, ref.K_UNIT)
            at = np.unique(at)
            par = (par[:, None] + np.arange(4)).ravel()
            at = np.concatenate([at, par])
            out[pg][:, at] = pool[pg][:, at]
    return out


@pytest.mark.parametrize("d,bits,H,Hkv,ps", [
    (128, 4, 8, 2, 64), (128, 8, 8, 2, 16),     # groups of 4
    (64, 4, 3, 1, 16), (64, 8, 6, 2, 128),      # groups of 3
    (256, 4, 16, 2, 32), (256, 8, 8, 1, 16),    # groups of 8
    (128, 4, 12, 1, 32), (256, 8, 11, 1, 32),   # 12 and 11 heads: a second, partly filled set of 8
    (64, 4, 20, 1, 64), (128, 8, 33, 1, 16),    # 20 and 33 heads
    (128, 4, 3, 3, 16), (64, 8, 2, 2, 64),      # a KV head a query head
])
def test_decode_edge_lengths(cuda_device, d, bits, H, Hkv, ps):
    """Lengths around tiles and pages, one key, none; unused slots poisoned, unused table entries outside the pool."""
    lens = [1, 0, 15, 16, 17, 33, ps - 1, ps, ps + 1, 300]
    table, pages = make_table(lens, ps, 2, seed=d + H, extra_blocks=2)
    kpool = ref.random_pool(pages, Hkv, ps, d, bits, seed=10)
    vpool = ref.random_pool(pages, Hkv, ps, d, bits, seed=11)
    q = torch.randn(len(lens), H, d, generator=torch.Generator().manual_seed(12)).to(torch.bfloat16)
    kd, vd = (torch.from_numpy(poison(x, table, lens, d, bits)).to(cuda_device) for x in (kpool, vpool))
    o, lse = check_decode(cuda_device, q, kpool, vpool, table, lens, bits, 1.0 / math.sqrt(d), kd=kd, vd=vd)
    assert (o[1] == 0).all() and np.isneginf(lse[1]).all()


@pytest.mark.parametrize("d,bits", FORMATS)
def test_decode_long_and_many(cuda_device, d, bits):
    """One sequence of 5,000 keys beside many short ones: the sequences are cut over the CTAs at other places, and a
    part of one is merged from several."""
    lens = [5000] + [int(x) for x in np.random.default_rng(d).integers(0, 90, 60)]
    table, pages = make_table(lens, 32, 1, seed=d)
    kpool, vpool = (ref.random_pool(pages, 2, 32, d, bits, seed=s) for s in (20, 21))
    q = torch.randn(len(lens), 4, d, generator=torch.Generator().manual_seed(22)).to(torch.bfloat16)
    check_decode(cuda_device, q, kpool, vpool, table, lens, bits, 1.0 / math.sqrt(d))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("q_scale,v_spread", [(16.0, 1.0), (1.0, 2.0 ** -60), (1.0, 2.0 ** 60), (2.0 ** 40, 1.0), (2.0 ** -80, 1.0)])
def test_decode_magnitudes(cuda_device, bits, q_scale, v_spread):
    """Peaked scores, values far outside fp16's range, queries far outside it (with a scale that undoes it)."""
    d, H, Hkv, ps, lens = 128, 4, 1, 16, [700, 90]
    table, pages = make_table(lens, ps, 1, seed=2)
    kpool = ref.random_pool(pages, Hkv, ps, d, bits, seed=30)
    vpool = ref.random_pool(pages, Hkv, ps, d, bits, seed=31, spread=v_spread)
    q = (torch.randn(2, H, d, generator=torch.Generator().manual_seed(32)) * q_scale).to(torch.bfloat16)
    scale = 1.0 / math.sqrt(d) / (q_scale if not 0.01 < q_scale < 100 else 1.0)
    check_decode(cuda_device, q, kpool, vpool, table, lens, bits, scale)


def test_decode_steps_of_one_sequence_differ_widely(cuda_device):
    """Tokens whose steps are 2^20 apart: the small ones hold the softmax's weight."""
    d, bits, ps, n = 64, 4, 16, 96
    x = torch.randn(n, 1, d, generator=torch.Generator().manual_seed(40))
    y = torch.randn(n, 1, d, generator=torch.Generator().manual_seed(41))
    y[::2] *= 2.0 ** -20
    q = torch.randn(1, 2, d, generator=torch.Generator().manual_seed(42)).to(torch.bfloat16)
    x[::2] += 3.0 * q[0, 0].float()  # those tokens score about 24 nats higher for head 0
    pool = np.zeros((n // ps, 1, ps * ref.row_bytes(d, bits)), np.uint8)
    kpool, vpool = pool.copy(), pool.copy()
    table = np.arange(n // ps, dtype=np.int32)[None]
    f = [t.to(torch.bfloat16).float().numpy() for t in (x, y)]
    append_reference(kpool, vpool, f[0], f[1], [0, n], table, [n], bits)
    check_decode(cuda_device, q, kpool, vpool, table, [n], bits, 0.125, dtypes=(torch.float32,))


@pytest.mark.parametrize("d,bits,H", [(64, 4, 2), (64, 8, 9), (128, 4, 12), (128, 8, 1), (256, 4, 2), (256, 8, 3)])
def test_decode_groups_of_dimensions_differ_widely(cuda_device, d, bits, H):
    """Groups of 32 dimensions whose values are 2^8 to 2^60 apart and grow along the sequence: each is as exact as if alone."""
    ps, lens = 16, [700, 90]
    table, pages = make_table(lens, ps, 1, seed=6)
    kpool, vpool = (ref.random_pool(pages, 1, ps, d, bits, seed=s) for s in (45, 46))
    par = vpool.reshape(pages, -1, 16 * ref.row_bytes(d, bits))[..., 16 * d * bits // 8:]
    f = np.ascontiguousarray(par).view(np.uint16).astype(np.uint32)
    f = (f << 16).view(np.float32).reshape(pages, 1, 16, d // 32, 2)
    f = f * 2.0 ** (-(60 // (d // 32 - 1)) * np.arange(d // 32)[::-1, None].astype(np.float64))
    order = np.concatenate([table[b, :-(-n // ps)] for b, n in enumerate(lens)])
    f[order] *= (2.0 ** (np.arange(len(order)) // 16))[:, None, None, None, None]
    raw = (f.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    par[:] = raw.reshape(pages, -1).view(np.uint8).reshape(par.shape)
    q = torch.randn(2, H, d, generator=torch.Generator().manual_seed(47)).to(torch.bfloat16)
    check_decode(cuda_device, q, kpool, vpool, table, lens, bits, 0.1)


@pytest.mark.parametrize("bits", [4, 8])
def test_decode_nan_rows(cuda_device, bits):
    """A NaN group in a valid key's K makes its head's outputs NaN; one in V the group's 32 columns only."""
    d, H, Hkv, ps, lens = 128, 4, 2, 16, [40, 40, 40]
    table, pages = make_table(lens, ps, 1, seed=3)
    kpool, vpool = (ref.random_pool(pages, Hkv, ps, d, bits, seed=s) for s in (50, 51))
    row = np.random.default_rng(1).normal(size=(Hkv, d)).astype(np.float32)
    row[1, 40] = np.nan
    ref.store(kpool, table[0, 1], 3, row, bits, ref.K_UNIT)
    ref.store(vpool, table[1, 2], 7, row, bits, ref.V_UNIT)
    q = torch.randn(3, H, d, generator=torch.Generator().manual_seed(52)).to(torch.bfloat16)
    o, lse = check_decode(cuda_device, q, kpool, vpool, table, lens, bits, 0.1)
    assert np.isnan(o[0, 2:]).all() and not np.isnan(o[0, :2]).any()
    assert np.isnan(o[1, 2:, 32:64]).all() and np.isnan(o[1]).sum() == 64 and not np.isnan(o[2]).any()
    assert not np.isnan(lse[1:]).any()


def test_decode_bad_lengths_and_pages(cuda_device):
    dev, d, bits, H, Hkv, ps = cuda_device, 128, 4, 4, 2, 16
    table, pages = make_table([64, 64, 64], ps, 1, seed=4)
    kpool, vpool = (ref.random_pool(pages, Hkv, ps, d, bits, seed=s) for s in (60, 61))
    q = torch.randn(3, H, d, generator=torch.Generator().manual_seed(62)).to(torch.bfloat16)
    kd, vd = torch.from_numpy(kpool).to(dev), torch.from_numpy(vpool).to(dev)
    good = ref.decode(q.double().numpy(), kpool, vpool, table, [64, 20, 64], bits, 0.1)

    def call(tab, lens):
        return [to_np(x) for x in fa.decode_paged_quant(q.to(dev), kd, vd, i32(tab, dev), i32(lens, dev), bits, scale=0.1)]

    o, lse = call(table, [-3, 20, 1000])   # clamped to 0 and to the capacity
    assert fa.fa_check_status() == fa.FA_ERR_KV_LEN and fa.fa_check_status() == fa.FA_OK
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all()
    assert (np.abs(o - good[0]) <= good[2] + 1e-6)[1:].all()
    bad = table.copy()
    bad[0, 1], bad[2, 3] = -1, pages
    o, lse = call(bad, [64, 20, 64])       # read as page 0
    assert fa.fa_check_status() == fa.FA_ERR_PAGE and fa.fa_check_status() == fa.FA_OK
    bad[0, 1] = bad[2, 3] = 0
    want = ref.decode(q.double().numpy(), kpool, vpool, bad, [64, 20, 64], bits, 0.1)
    assert (np.abs(o - want[0]) <= want[2] + 1e-6).all()


def test_pool_past_32_bits(cuda_device):
    """Pages whose bytes lie past 2^32: written, read back and attended over."""
    dev, d, bits, Hkv, ps = cuda_device, 128, 8, 2, 64
    block = ps * ref.row_bytes(d, bits)
    pages = (1 << 32) // (Hkv * block) + 10
    kp, vp = fa.kvcache_quant_pages(pages, Hkv, ps, d, bits, device=dev)
    table = i32([[pages - 1, pages - 3]], dev)
    k, v = torch.randn(2, 100, Hkv, d, generator=torch.Generator().manual_seed(70)).to(torch.bfloat16)
    cu, lens = i32([0, 100], dev), i32([100], dev)
    fa.kvcache_append_quant(k.to(dev), v.to(dev), kp, vp, cu, table, lens, 100, bits)
    small_k, small_v = kp[[pages - 1, pages - 3]].cpu().numpy(), vp[[pages - 1, pages - 3]].cpu().numpy()
    assert not kp[:pages - 3].any() and not kp[pages - 2].any()
    c, lo, s = ref.quantise(k.float().numpy(), bits)
    want = np.repeat(lo, 32, -1).astype(np.float64) + np.repeat(s, 32, -1).astype(np.float64) * c
    got, _ = fa.kvcache_read_quant(kp, vp, cu, table, lens, 100, 100, Hkv, d, bits)
    assert torch.equal(got.cpu(), ref.round_once(want, torch.bfloat16))
    q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(71)).to(torch.bfloat16)
    o_ref, lse_ref, tol_o, tol_l = ref.decode(q.double().numpy(), small_k, small_v, np.array([[0, 1]]), [100], bits, 0.1)
    o, lse = fa.decode_paged_quant(q.to(dev), kp, vp, table, lens, bits, scale=0.1)
    assert (np.abs(to_np(o) - o_ref) <= tol_o + 1e-6).all() and (np.abs(to_np(lse) - lse_ref) <= tol_l).all()
    assert fa.fa_check_status() == fa.FA_OK


def test_generation_over_a_quantised_cache(cuda_device):
    """The calls together: a batch of prompts is appended and attended to over the read-back cache by the packed
    forward, a second chunk likewise, then tokens are generated one at a time in a captured graph."""
    dev, d, bits, H, Hkv, ps = cuda_device, 128, 4, 4, 2, 16
    scale, G = 1.0 / math.sqrt(d), 2
    prompts, chunk, steps = [37, 64, 5], [3, 0, 40], 4
    total = [a + c + steps for a, c in zip(prompts, chunk)]
    table, pages = make_table(total, ps, 1, seed=5)
    td = i32(table, dev)
    kp, vp = fa.kvcache_quant_pages(pages, Hkv, ps, d, bits, device=dev)
    gen = torch.Generator().manual_seed(80)
    lens = [0, 0, 0]
    for new in (prompts, chunk):
        lens = [a + n for a, n in zip(lens, new)]
        qkv = torch.randn(sum(new), H + 2 * Hkv, d, generator=gen).to(torch.bfloat16).to(dev)
        cu_q, cu_k, ld = cu_of(new, dev), cu_of(lens, dev), i32(lens, dev)
        fa.kvcache_append_quant(qkv[:, H:H + Hkv], qkv[:, H + Hkv:], kp, vp, cu_q, td, ld, max(new), bits)
        k, v = fa.kvcache_read_quant(kp, vp, cu_k, td, ld, sum(lens), max(lens), H, d, bits)
        q = qkv[:, :H].contiguous()
        o, lse = fa.forward_varlen(q, k, v, cu_q, cu_k, max(new), scale=scale, causal=True)
        assert fa.fa_check_status() == fa.FA_OK
        kn, vn = kp.cpu().numpy(), vp.cpu().numpy()
        kr, vr = (ref.round_once(np.repeat(np.concatenate([
            ref.values(pool, table[b], range(lens[b]), d, bits, unit) for b in range(3)]), G, 1), torch.bfloat16)
            for pool, unit in ((kn, ref.K_UNIT), (vn, ref.V_UNIT)))
        o_ref, lse_ref = oracle.forward_varlen(q.cpu(), kr, vr, cu_q.cpu().numpy(), cu_k.cpu().numpy(), scale, True)
        check_o(o, o_ref, "prefill over the read-back cache")
        check_lse(lse, lse_ref, "prefill over the read-back cache")
    # one step in a graph: the lengths and the new rows are its inputs
    ld = i32(lens, dev)
    qkv = torch.zeros(3, H + 2 * Hkv, d, dtype=torch.bfloat16, device=dev)
    cu1 = cu_of([1, 1, 1], dev)
    ws = fa.workspace(fa.fa_decode_paged_quant_workspace_size(3, H, Hkv, table.shape[1], ps, d, bits), dev)

    def step():
        fa.kvcache_append_quant(qkv[:, H:H + Hkv], qkv[:, H + Hkv:], kp, vp, cu1, td, ld, 1, bits)
        return fa.decode_paged_quant(qkv[:, :H].contiguous(), kp, vp, td, ld, bits, scale=scale, ws=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    for _ in range(steps):
        ws.random_(0, 256)  # nothing is kept in the workspace from one replay to the next
        ld += 1
        qkv.copy_(torch.randn(3, H + 2 * Hkv, d, generator=gen).to(torch.bfloat16))
        graph.replay()
        assert fa.fa_check_status() == fa.FA_OK
        kn, vn = kp.cpu().numpy(), vp.cpu().numpy()
        now = ld.tolist()
        for b in range(3):
            c, lo, s = ref.quantise(qkv[b, H:H + Hkv].float().cpu().numpy(), bits)
            got = ref.load(kn, table[b, (now[b] - 1) // ps], (now[b] - 1) % ps, d, bits, ref.K_UNIT)[0]
            assert (got == c).all()
        o_ref, lse_ref, tol_o, tol_l = ref.decode(qkv[:, :H].double().cpu().numpy(), kn, vn, table, now, bits, scale)
        assert (np.abs(to_np(o) - o_ref) <= tol_o + np.abs(o_ref) * 2.0 ** -23).all()
        assert (np.abs(to_np(lse) - lse_ref) <= tol_l).all()


def test_decode_streams_and_repeats(cuda_device):
    """Calls at once on two streams give what one call gives, bit for bit; a stream passed by handle is used."""
    dev, d, bits, H, Hkv, ps = cuda_device, 128, 4, 8, 2, 64
    lens = [3000, 1, 700, 2222]
    table, pages = make_table(lens, ps, 1, seed=6)
    kd, vd = (torch.from_numpy(ref.random_pool(pages, Hkv, ps, d, bits, seed=s)).to(dev) for s in (90, 91))
    q = torch.randn(4, H, d, generator=torch.Generator().manual_seed(92)).to(torch.bfloat16).to(dev)
    args = (q, kd, vd, i32(table, dev), i32(lens, dev), bits)
    o, lse = fa.decode_paged_quant(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [fa.decode_paged_quant(*args, stream=s if i % 4 < 2 else s.cuda_stream)
           for i in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in got)
    assert fa.fa_check_status() == fa.FA_OK


def test_refused_streams_and_workspaces(cuda_device):
    """A stream of another device, a workspace with gaps, one that is too small or misaligned: nothing is launched."""
    dev, d, bits = cuda_device, 64, 4
    with pytest.raises(ValueError, match="stream"):
        fa._kvq_run(torch.cuda.current_device() + 1, torch.cuda.current_stream(), None)
    kp, vp = fa.kvcache_quant_pages(2, 1, 16, d, bits, device=dev)
    q, table, lens = torch.zeros(1, 1, d, dtype=torch.bfloat16, device=dev), i32([[0, 1]], dev), i32([20], dev)
    n = fa.fa_decode_paged_quant_workspace_size(1, 1, 1, 2, 16, d, bits)
    ws = torch.full((2, n + 256), 9, dtype=torch.uint8, device=dev)
    for bad, error in ((ws[:, :n], ValueError), (ws[0, :n - 256], fa.FAError), (ws[0, 16:16 + n], fa.FAError),
                       (torch.zeros(n, dtype=torch.uint8), ValueError)):
        with pytest.raises(error):
            fa.decode_paged_quant(q, kp, vp, table, lens, bits, ws=bad)
    torch.cuda.synchronize()
    assert (ws == 9).all() and fa.fa_check_status() == fa.FA_OK


def test_decode_graphs_that_share_a_workspace(cuda_device):
    """Two captured graphs of different shapes with one workspace, replayed in turn with eager calls between them: each
    gives what its call alone gave, bit for bit, whatever the workspace held."""
    dev, bits, d, Hkv = cuda_device, 4, 128, 2
    calls = []
    for seed, (lens, H, ps) in enumerate((([2500, 40, 0], 8, 64), ([17, 900], 4, 16))):
        table, pages = make_table(lens, ps, 1, seed=seed)
        kd, vd = (torch.from_numpy(ref.random_pool(pages, Hkv, ps, d, bits, seed=100 + 2 * seed + i)).to(dev) for i in (0, 1))
        q = torch.randn(len(lens), H, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(dev)
        calls.append((q, kd, vd, i32(table, dev), i32(lens, dev), bits))
    ws = fa.workspace(max(fa.fa_decode_paged_quant_workspace_size(c[0].shape[0], c[0].shape[1], Hkv, c[3].shape[1],
                                                                  c[1].shape[2] // ref.row_bytes(d, bits), d, bits)
                          for c in calls), dev)
    alone = [fa.decode_paged_quant(*c) for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.decode_paged_quant(*c, ws=ws))
        graphs.append(g)
    for i in range(6):
        ws.random_(0, 256)
        for x in outs[i % 2]:
            x.fill_(7.0)
        graphs[i % 2].replay()
        fa.decode_paged_quant(*calls[(i + 1) % 2], ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(outs[i % 2], alone[i % 2]))
    assert fa.fa_check_status() == fa.FA_OK


def attention64(q, kp, vp, table, lens, bits, scale, d):
    """(o, lse, greatest |v| and greatest sum of the terms' magnitudes) in 64 bits on the GPU over what the cache reads back as."""
    B, H = q.shape[:2]
    cu = torch.cat([torch.zeros_like(lens[:1]), lens.cumsum(0).to(torch.int32)])
    n = lens.tolist()
    k, v = fa.kvcache_read_quant(kp, vp, cu, table, lens, sum(n), max(n), H, d, bits, out_dtype=torch.float32)
    o = torch.zeros(B, H, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=q.device)
    X = 0.0
    for b in range(B):
        if n[b] == 0:
            continue
        kb, vb = (x[int(cu[b]):int(cu[b + 1])].double() for x in (k, v))
        x = torch.einsum("hd,nhd->hn", q[b].double(), kb) * scale
        # |lo| + s c is at most |value| + 2 |lo|, and |lo| below 4 in these pools
        X = max(X, float((torch.einsum("hd,nhd->hn", q[b].double().abs(), kb.abs() + 8.0) * scale).max()))
        lse[b] = torch.logsumexp(x, 1)
        o[b] = torch.einsum("hn,nhd->hd", torch.softmax(x, 1), vb)
    return o, lse, float(v.abs().max()), X


def test_calls_behind_joins_and_copies(cuda_device):
    """The calls behind what is no kernel of their stream (a fill, a copy, another stream's work), eagerly and captured:
    each sees what was written before it.  A hundred steps back to back give what single steps give."""
    dev, d, bits, H, Hkv, ps, n = cuda_device, 128, 4, 4, 2, 16, 600
    table, pages = make_table([n, 40], ps, 1, seed=9)
    td, lens = i32(table, dev), i32([n, 40], dev)
    cu = i32([0, n, n + 40], dev)
    gen = torch.Generator().manual_seed(130)
    src = torch.randn(3, n + 40, 2, Hkv, d, generator=gen).to(torch.bfloat16).to(dev)
    q = torch.randn(2, H, d, generator=gen).to(torch.bfloat16).to(dev)
    qkv, now = torch.zeros_like(src[0]), torch.zeros_like(lens)
    kp, vp = fa.kvcache_quant_pages(pages, Hkv, ps, d, bits, device=dev)
    ws = fa.workspace(fa.fa_decode_paged_quant_workspace_size(2, H, Hkv, table.shape[1], ps, d, bits), dev)
    side = torch.cuda.Stream(dev)

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            now.copy_(lens)                  # a copy, then the append on another stream
            fa.kvcache_append_quant(qkv[:, 0], qkv[:, 1], kp, vp, cu, td, now, n, bits)
        ws.zero_()                           # a fill, then a join
        main.wait_stream(side)
        a = fa.decode_paged_quant(q, kp, vp, td, now, bits, scale=0.1, ws=ws)
        k, v = fa.kvcache_read_quant(kp, vp, cu, td, now, n + 40, n, Hkv, d, bits)
        kp.zero_(), vp.zero_()               # the next step's pools hold nothing of this one's
        return (*a, k, v)

    want = []
    for x in src:
        qkv.copy_(x)
        torch.cuda.synchronize()
        want.append([t.clone() for t in step()])
        torch.cuda.synchronize()
    kn, vn = (ref.random_pool(pages, Hkv, ps, d, bits, seed=1) for _ in range(2))
    c = src[0].float().cpu().numpy()
    append_reference(kn, vn, c[:, 0], c[:, 1], [0, n, n + 40], table, [n, 40], bits)
    o_ref, lse_ref, tol_o, tol_l = ref.decode(q.double().cpu().numpy(), kn, vn, table, [n, 40], bits, 0.1)
    assert (np.abs(to_np(want[0][0]) - o_ref) <= tol_o + np.abs(o_ref) * 2.0 ** -23).all()
    assert (np.abs(to_np(want[0][1]) - lse_ref) <= tol_l).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for mode in ("eager", "graph"):
        got = []
        for i in range(100):
            qkv.copy_(src[i % 3])
            if mode == "graph":
                graph.replay()
                got.append([t.clone() for t in out])
            else:
                got.append(step())
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            assert all(torch.equal(x, y) for x, y in zip(g, want[i % 3])), (mode, i)
    assert fa.fa_check_status() == fa.FA_OK


def test_default_stream_waits_for_blocking_streams(cuda_device):
    """The legacy default stream waits for a blocking stream's work without an event, and that stream for the default
    stream's: the calls keep to it."""
    import ctypes

    cudart = torch.cuda.cudart()
    handle = ctypes.c_void_p()
    assert int(cudart.cudaStreamCreate(ctypes.addressof(handle))) == 0
    other = torch.cuda.ExternalStream(handle.value, device=cuda_device)
    dev, d, bits, H, Hkv, ps, n = cuda_device, 128, 4, 4, 2, 16, 500
    table, pages = make_table([n], ps, 1, seed=19)
    td, lens, cu = i32(table, dev), i32([n], dev), i32([0, n], dev)
    gen = torch.Generator().manual_seed(140)
    src = torch.randn(3, 2, n, Hkv, d, generator=gen).to(torch.bfloat16).to(dev)
    q = torch.randn(1, H, d, generator=gen).to(torch.bfloat16).to(dev)
    kp, vp = fa.kvcache_quant_pages(pages, Hkv, ps, d, bits, device=dev)
    delay = torch.randn(4096, 4096, device=dev)

    def step(i):
        with torch.cuda.stream(other):
            for _ in range(3):
                torch.mm(delay, delay)
            fa.kvcache_append_quant(src[i, 0], src[i, 1], kp, vp, cu, td, lens, n, bits)
        o, lse = fa.decode_paged_quant(q, kp, vp, td, lens, bits, scale=0.1)
        with torch.cuda.stream(other):
            kp.zero_(), vp.zero_()
        return o, lse

    want = []
    for i in range(3):
        want.append([t.clone() for t in step(i)])
        torch.cuda.synchronize()
    assert all(float((want[0][0] - w[0]).abs().max()) > 0.01 for w in want[1:])
    got = [step(i % 3) for i in range(30)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 3])), i
    assert fa.fa_check_status() == fa.FA_OK
    assert int(cudart.cudaStreamDestroy(handle.value)) == 0


@pytest.mark.parametrize("lens,H,Hkv,ps,d,bits", [
    ([400000], 4, 1, 1024, 64, 4),                    # one long context over all CTAs
    ([90000, 3], 2, 2, 65536, 128, 8),                # the largest pages
    ([i % 7 * (i % 3) for i in range(3000)], 2, 1, 16, 64, 4),  # thousands of tiny sequences, most CTAs with many
    ([70, 0, 1] * 50, 6, 3, 32, 256, 4),
])
def test_decode_sizes(cuda_device, lens, H, Hkv, ps, d, bits):
    """Sizes that a plain loop cannot check: attention in 64 bits over the values that the cache reads back as (fp32,
    2^-24 off).  The tolerances are those of kvq_reference.decode with every |v|, |v - o|, |hi| and s C at twice the
    greatest |v|, and 2^-23 of each score step for the read-back's rounding; a warp's sums have up to 400000 / 16 / 1776
    steps here, 2^-23 * 17 each on the low nibbles."""
    dev = cuda_device
    table, pages = make_table(lens, ps, 1, seed=9)
    kd, vd = (torch.from_numpy(ref.random_pool(pages, Hkv, ps, d, bits, seed=110 + i)).to(dev) for i in (0, 1))
    q = torch.randn(len(lens), H, d, generator=torch.Generator().manual_seed(111)).to(torch.bfloat16).to(dev)
    scale = 1.0 / math.sqrt(d)
    table, lens_t = i32(table, dev), i32(lens, dev)
    o_ref, lse_ref, top, X = attention64(q, kd, vd, table, lens_t, bits, scale, d)
    o, lse = fa.decode_paged_quant(q, kd, vd, table, lens_t, bits)
    assert fa.fa_check_status() == fa.FA_OK
    ex = 2.0 ** -19 * X + 2.0 ** -21
    steps = max(2, max(lens) // 16 // 1776 + 1)
    assert float((o - o_ref).abs().max()) <= 2 * top * (2.0 ** -9 + 2 * ex + steps * 17 * 2.0 ** -23 + max(lens) * 2.0 ** -31 * 31)
    fin = ~torch.isneginf(lse_ref)
    assert torch.equal(torch.isneginf(lse), ~fin)
    assert float((lse - lse_ref)[fin].abs().max()) <= ex + 2.0 ** -22 * float(lse_ref[fin].abs().max())
    zero = lens_t == 0
    assert (o[zero] == 0).all()


@pytest.mark.parametrize("d,bits,H,warps", [(64, 4, 1, 12), (64, 8, 4, 16), (128, 4, 4, 12), (128, 8, 2, 12), (256, 4, 2, 8),
                                            (256, 8, 1, 8), (128, 4, 12, 8), (64, 8, 12, 12)])
def test_decode_sequences_about_as_long_as_a_warps_run(cuda_device, d, bits, H, warps):
    """Equal sequences, 2 % more of them than the GPU's warps: every warp's border cuts one, so a block of `warps` warps
    begins and ends with a part and merges a set more than it has warps."""
    n = torch.cuda.get_device_properties(cuda_device).multi_processor_count * warps * 102 // 100
    test_decode_sizes(cuda_device, [320] * n, H, 1, 64, d, bits)


def test_nothing_is_written_after_a_timeout(cuda_device):
    """Once a wait anywhere in the library has run out (the fault-injection build), the calls write nothing until
    fa_check_status has returned that."""
    import ctypes

    from exact_io_aware_94_b200 import build as fa_build

    lib = ctypes.CDLL(fa_build.build(test_hooks=True))
    vp, i, f, sz, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
    lib.fa_test_inject_fault.argtypes = [i]
    lib.fa_forward.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_kvcache_append_quant.argtypes = [vp, vp, ll, ll, vp, vp, vp, vp, vp] + [i] * 9 + [vp]
    lib.fa_kvcache_read_quant.argtypes = [vp] * 7 + [i] * 11 + [vp]
    lib.fa_decode_paged_quant.argtypes = [vp] * 7 + [i] * 8 + [f, i, vp, sz, vp]
    lib.fa_check_status.argtypes = [vp]
    dev, d, bits, H, Hkv, ps, n = cuda_device, 128, 4, 4, 2, 16, 40
    st = torch.cuda.current_stream().cuda_stream
    x = torch.randn(256, H, d, generator=torch.Generator().manual_seed(120)).to(torch.bfloat16).to(dev)
    out, lse = torch.zeros(1, 1, 256, d, device=dev), torch.zeros(1, 1, 256, device=dev)
    kd, vd = (torch.from_numpy(ref.random_pool(3, Hkv, ps, d, bits, seed=s)).to(dev) for s in (121, 122))
    pools = [kd.clone(), vd.clone()]
    table, lens, cu = i32([[2, 0, 1]], dev), i32([n], dev), i32([0, n], dev)
    o, l, ko, vo = (torch.full(s, 7.0, device=dev) for s in ((1, H, d), (1, H), (n, H, d), (n, H, d)))
    ws = fa.workspace(fa.fa_decode_paged_quant_workspace_size(1, H, Hkv, 3, ps, d, bits), dev)

    def calls():
        k = x[:n, :Hkv].contiguous()
        assert lib.fa_kvcache_append_quant(k.data_ptr(), k.data_ptr(), Hkv * d, Hkv * d, kd.data_ptr(), vd.data_ptr(),
                                           cu.data_ptr(), table.data_ptr(), lens.data_ptr(), 1, Hkv, n, n, 3, ps, 3, d,
                                           bits, st) == fa.FA_OK
        assert lib.fa_kvcache_read_quant(kd.data_ptr(), vd.data_ptr(), cu.data_ptr(), table.data_ptr(), lens.data_ptr(),
                                         ko.data_ptr(), vo.data_ptr(), 1, H, Hkv, n, n, 3, ps, 3, d, bits, fa.FA_DT_F32,
                                         st) == fa.FA_OK
        assert lib.fa_decode_paged_quant(x.data_ptr(), kd.data_ptr(), vd.data_ptr(), table.data_ptr(), lens.data_ptr(),
                                         o.data_ptr(), l.data_ptr(), 1, H, Hkv, 3, ps, 3, d, bits, 0.1, fa.FA_DT_F32,
                                         ws.data_ptr(), ws.numel(), st) == fa.FA_OK
        torch.cuda.synchronize()

    assert lib.fa_check_status(None) == fa.FA_OK
    assert lib.fa_test_inject_fault(1) == fa.FA_OK  # a K tile of the next forward is never loaded
    q = x[:, 0].contiguous()
    assert lib.fa_forward(q.data_ptr(), q.data_ptr(), q.data_ptr(), out.data_ptr(), lse.data_ptr(), 1, 1, 256, 256, d, 0.1,
                          0, fa.FA_DT_F32, st) == fa.FA_OK
    torch.cuda.synchronize()
    calls()
    assert torch.equal(kd, pools[0]) and torch.equal(vd, pools[1])
    assert all((t == 7.0).all() for t in (o, l, ko, vo))
    assert lib.fa_check_status(None) == fa.FA_ERR_TIMEOUT
    calls()
    assert lib.fa_check_status(None) == fa.FA_OK
    assert not torch.equal(kd, pools[0]) and all(torch.isfinite(t).all() and not (t == 7.0).any() for t in (o, l, ko, vo))


@pytest.mark.parametrize("d,bits,H,Hkv", [(128, 4, 4, 1), (128, 8, 2, 1), (64, 4, 9, 1), (256, 4, 4, 1), (256, 8, 4, 1)])
def test_decode_average_of_many_values(cuda_device, d, bits, H, Hkv):
    """An output that is the average of many values of either sign is small beside them, and so must its error be.
    300,000 keys that all but share the probability: the roundings of a key (three of fp16, each 2^-11 at most and so
    2^-12.8 in the mean square, of terms up to the group's range, 4 standard deviations of the values here) are
    independent, so their sum over n keys is to the output, a sum of n values with that deviation, as
    sqrt(3) 4 2^-12.8 = 2^-10 to 1.  A bias of the sums (a truncating accumulator) does not average out: 2^-8 leaves it no room."""
    dev, ps, n = cuda_device, 64, 300000
    pages = -(-n // ps)
    gen = torch.Generator(device=dev).manual_seed(d + bits)
    kp, vp = fa.kvcache_quant_pages(pages, Hkv, ps, d, bits, device=dev)
    table = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)[None]
    k = (0.05 * torch.randn(n, Hkv, d, generator=gen, device=dev)).to(torch.bfloat16)
    v = torch.randn(n, Hkv, d, generator=gen, device=dev).to(torch.bfloat16)
    cu, lens = i32([0, n], dev), i32([n], dev)
    fa.kvcache_append_quant(k, v, kp, vp, cu, table, lens, n, bits)
    q = torch.randn(1, H, d, generator=gen, device=dev).to(torch.bfloat16)
    o, lse = fa.decode_paged_quant(q, kp, vp, table, lens, bits)
    assert fa.fa_check_status() == fa.FA_OK
    o_ref, lse_ref, _, X = attention64(q, kp, vp, table, lens, bits, 1.0 / math.sqrt(d), d)
    assert float((o - o_ref).norm() / o_ref.norm()) <= 2.0 ** -8
    assert float((lse - lse_ref).abs().max()) <= 2.0 ** -20 * X + 2.0 ** -21 + 2.0 ** -22 * float(lse_ref.abs().max())
