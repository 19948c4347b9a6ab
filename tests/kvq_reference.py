"""Plain implementation of the quantised paged cache in numpy, for the tests: quantisation by the format's
definition (fp32 steps), bytes placed dimension by dimension, values and attention in 64 bits."""
import numpy as np
import torch

GROUP, TILE = 32, 16
K_UNIT, V_UNIT = 8, 4


def row_bytes(d, bits):
    return d * bits // 8 + d // GROUP * 4


def round_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def round_once(x, dtype):
    """float64 x rounded once to bf16 or fp32, ties to even (results in the normal range or exact)."""
    x = np.ascontiguousarray(x, dtype=np.float64)
    if dtype == torch.float32:
        return torch.from_numpy(x.astype(np.float32))
    bits = x.view(np.uint64)
    up = bits + np.uint64((1 << 44) - 1) + ((bits >> np.uint64(45)) & np.uint64(1))
    y = np.where(np.isfinite(x), (up & ~np.uint64((1 << 45) - 1)).view(np.float64), x)
    return torch.from_numpy(y.astype(np.float32)).to(torch.bfloat16)


def quantise(x, bits):
    """codes uint8 [..., d], lo and s float32 [..., d / 32] of float32 x [..., d]."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        s = round_bf16((hi - lo) / np.float32(2 ** bits - 1))
        bad = ~np.isfinite(g).all(-1) | ~np.isfinite(s)
        s = np.where(bad | (s < np.float32(2.0 ** -126)), np.float32(0), s)
        inv = np.where(s > 0, np.float32(1) / s, np.float32(0)).astype(np.float32)
        c = np.minimum(np.rint((g - lo[..., None]) * inv[..., None]), 2 ** bits - 1)
    c = np.where((s > 0)[..., None], c, 0).astype(np.uint8)
    return c.reshape(x.shape), np.where(bad, np.float32("nan"), lo), s


def places(d, bits, unit):
    """Of every dimension: byte in the tile for token row 0, bytes from one row to the next, bit shift."""
    width = min(64, d * bits // 8)
    dims = width * 8 // bits
    i = np.arange(d)
    plane, i = i // dims, i % dims
    g, e = i // GROUP, i % GROUP
    bit = (e // unit * (dims // GROUP) + g) * unit * bits + e % unit * bits
    return plane * TILE * width + bit // 8, width, bit % 8


def row_places(slot, d, bits, unit):
    """(bytes of the codes [d], shifts [d], bytes of the first byte of each (lo, s) pair [d / 32]) in a page block."""
    first, width, shift = places(d, bits, unit)
    base = slot // TILE * TILE * row_bytes(d, bits)
    par = base + TILE * d * bits // 8 + slot % TILE * (d // GROUP * 4) + 4 * np.arange(d // GROUP)
    return base + first + slot % TILE * width, shift, par


def store(pool, page, slot, x, bits, unit):
    """Writes the quantised row x [Hkv, d] (float32) to (page, slot) of pool, uint8 [pages, Hkv, bytes]."""
    d = x.shape[-1]
    c, lo, s = quantise(x, bits)
    at, shift, par = row_places(slot, d, bits, unit)
    block = pool[page]
    block[:, at] = 0
    for i in range(d):
        block[:, at[i]] |= (c[:, i] << shift[i]).astype(np.uint8)
    for j, v in ((0, lo), (2, s)):
        raw = (v.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        block[:, par + j] = raw & 255
        block[:, par + j + 1] = raw >> 8


def load(pool, page, slot, d, bits, unit):
    """(codes, lo, s) of the row at (page, slot): float64 [Hkv, d], lo and s repeated over their groups."""
    at, shift, par = row_places(slot, d, bits, unit)
    block = pool[page]
    c = ((block[:, at] >> shift.astype(np.uint8)) & (2 ** bits - 1)).astype(np.float64)
    half = [(block[:, par + j].astype(np.uint32) | (block[:, par + j + 1].astype(np.uint32) << 8)) << 16 for j in (0, 2)]
    lo, s = (np.repeat(np.ascontiguousarray(h).view(np.float32).astype(np.float64), GROUP, -1) for h in half)
    return c, lo, s


def rows(pool, table, positions, d, bits, unit):
    """(codes, lo, s) of a sequence's positions: float64 [n, Hkv, d] each.  pool is a numpy view of a tensor."""
    ps = pool.shape[2] // row_bytes(d, bits)
    got = [load(pool, int(table[p // ps]), int(p % ps), d, bits, unit) for p in positions]
    if not got:
        return tuple(np.zeros((0, pool.shape[1], d)) for _ in range(3))
    return tuple(np.stack(x) for x in zip(*got))


def values(pool, table, positions, d, bits, unit):
    c, lo, s = rows(pool, table, positions, d, bits, unit)
    with np.errstate(invalid="ignore"):
        return lo + s * c


def random_pool(num_pages, Hkv, ps, d, bits, seed, spread=1.0):
    """uint8 pool of random codes; lo ~ N(0, spread), s so that the codes span about 4 spread."""
    rng = np.random.default_rng(seed)
    rb = row_bytes(d, bits)
    pool = rng.integers(0, 256, (num_pages, Hkv, ps // TILE, TILE * rb), dtype=np.uint8)
    n = (num_pages, Hkv, ps // TILE, TILE, d // GROUP)
    lo = round_bf16(rng.normal(-2.0, 0.5, n) * spread)
    s = round_bf16(rng.uniform(0.5, 1.5, n) * 4.0 * spread / (2 ** bits - 1))
    par = np.stack([lo, s], -1).astype(np.float32).view(np.uint32) >> 16
    pool[..., TILE * d * bits // 8:] = par.astype(np.uint16).view(np.uint8).reshape(*n[:3], -1)
    return pool.reshape(num_pages, Hkv, ps * rb)


def decode(q, kpool, vpool, table, lens, bits, scale):
    """(o, lse, tolerance of o, tolerance of lse) in 64 bits for q [B, H, d] (float64).

    Tolerances.  A score is a sum over groups of s (q . c) + lo sum(q): with X the sum of its terms' magnitudes (in
    nats) and at most 14 fp32 roundings on the way (two accumulations a group that may truncate, d / 32 + 2 fused
    sums), it is off by less than 2^-20 X, and the exponential by 2^-22 more.  lse adds its own fp32 rounding.
    A probability's weight u is rounded to fp16 for the output, which is divided by the sum of the rounded weights:
    with u (1 + e), |e| <= 2^-11, the output moves by sum(p e (v - o)) at first order.  Half of the keys enter as
    hi - s (C - c), hi = lo + C s rounded to fp16 and C the greatest code; the product of u and s that weighs c or
    C - c is rounded to fp16 too: 2^-11 of sum(p (|hi| + s C)), which covers either.  fp16 steps end at 2^-24: as the
    greatest u is at least 2^6 and lo, hi and s are scaled by the power of two above the greatest of their group of dimensions, M, each of n keys
    adds at most 2^-25 / 2^6 (|v - o| + 2 M C), and the rounding of s, lo or hi itself 2^-25 * 2 M (C + 1) on average
    over the keys.  A code's low nibbles are summed as the difference of two sums up to 16 times as large: at most
    16 steps a warp at these tests' sizes, which may truncate (2^-23), 2^-14 of sum(p s C) in all.
    The factor 1 + 2^-8 covers the products of these errors."""
    B, H, d = q.shape
    Hkv = kpool.shape[1]
    G = H // Hkv
    o, lse = np.zeros((B, H, d)), np.full((B, H), -np.inf)
    tol_o, tol_l = np.zeros((B, H, d)), np.zeros((B, H))
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        kc, klo, ks = rows(kpool, table[b], range(n), d, bits, K_UNIT)
        vc, vlo, vs = rows(vpool, table[b], range(n), d, bits, V_UNIT)
        for h in range(H):
            g = h // G
            with np.errstate(invalid="ignore"):
                x = scale * ((klo + ks * kc)[:, g] @ q[b, h])
                X = scale * ((np.abs(klo) + ks * kc)[:, g] @ np.abs(q[b, h]))
                m = x.max()
                p = np.exp(x - m)
                lse[b, h] = m + np.log(p.sum())
                p /= p.sum()
                ex = 2.0 ** -20 * X.max() + 2.0 ** -21
                v = (vlo + vs * vc)[:, g]
                o[b, h] = p @ v
                top = 2 ** bits - 1
                vhi, spread = np.abs(vlo + top * vs)[:, g], (top * vs)[:, g]
                far = np.abs(v - o[b, h])
                M = np.fmax(np.fmax(vhi, np.abs(vlo[:, g])), vs[:, g])
                M = np.repeat(np.nanmax(M.reshape(n, -1, GROUP), (0, 2)), GROUP)
                tol_o[b, h] = (1 + 2.0 ** -8) * (
                    2.0 ** -11 * (p @ far + p @ vhi) + (2.0 ** -11 + 2.0 ** -14) * (p @ spread)
                    + 2 * ex * (p @ (np.abs(vlo) + vs * vc)[:, g])
                    + n * 2.0 ** -31 * (far.max(0) + 2 * M * top) + 2.0 ** -24 * M * (top + 1))
                tol_l[b, h] = ex + 2.0 ** -22 * abs(lse[b, h])
    return o, lse, tol_o, tol_l
