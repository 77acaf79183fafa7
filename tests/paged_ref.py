"""A plain float64 (numpy) implementation of the paged KV cache operators, and
the tolerances their float results are held to.  Shares no code with the
library."""

import numpy as np

DIM = 128


def sylvester(n=DIM):
    i = np.arange(n)
    bits = np.bitwise_and.outer(i, i)
    parity = np.zeros_like(bits)
    while bits.any():
        parity ^= bits & 1
        bits >>= 1
    return (1.0 - 2.0 * parity) / np.sqrt(n)


H = sylvester()


def bf16(x):
    """float64 values after rounding to bf16 (nearest even)."""
    b = np.asarray(x, np.float32).view(np.uint32)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & np.uint32(0xFFFF0000)
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def unpack(codes, bits):
    """uint8 [..., 16 * bits] -> float64 codes [..., 128]."""
    if bits == 8:
        return codes.view(np.int8).astype(np.float64)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (DIM,)).astype(np.int64)
    return np.where(c > 7, c - 16, c).astype(np.float64)


def values(codes, scales, bits):
    """Rows in the rotated basis, float64 [..., 128]."""
    group = DIM // scales.shape[-1]
    return unpack(codes, bits) * np.repeat(scales.astype(np.float64), group, -1)


def quantize(x, signs, bits, group):
    """Rotated rows y, scales and integer codes of bf16-valued rows x."""
    s = 1.0 if signs is None else signs.astype(np.float64)
    y = (x * s) @ H
    yg = y.reshape(y.shape[:-1] + (DIM // group, group))
    scale = np.abs(yg).max(-1) / (127.0 if bits == 8 else 7.0)
    t = yg / np.where(scale > 0, scale, 1.0)[..., None]
    return y, scale, t.reshape(y.shape), np.round(t).reshape(y.shape)


def slots(cached, new, free, table, page, capacity):
    """Request after request, page after page."""
    table = table.copy()
    taken, short, refused = 0, False, 0
    out, total, cu = [], [], [0]
    for b in range(len(cached)):
        c, n = max(int(cached[b]), 0), max(int(new[b]), 0)
        old, every = -(-c // page), -(-(c + n) // page)
        need = every - old
        ok = every <= table.shape[1]
        if ok and need:
            short = short or taken + need > len(free)
            ok = not short
        if ok:
            table[b, old:every] = free[taken:taken + need]
            taken += need
        refused += not ok
        for pos in range(c, c + n):
            p = table[b, pos // page] if ok else -1
            out.append(p * page + pos % page if p >= 0 else -1)
        total.append(c + n if ok else 0)
        cu.append(cu[-1] + n)
    out = (out + [-1] * capacity)[:capacity]
    return (table, np.array(out, np.int32), np.array(total, np.int32), np.array(cu, np.int32),
            np.array([taken, refused], np.int32))


def attention(q, k_pool, v_pool, table, lens, cu, page, causal=True, window=0, sinks=0, signs=None, scale=None):
    """q: float64 [rows, heads, 128]; pools: (codes, scales, bits).  Returns the
    output (NaN in rows of no request) and, per row and head, the 2-norm that
    the kernels' internal roundings may put on it.

    Those are, beside the bf16 rounding of the result: the query to one part in
    2^11 per entry or 2^-16 of its largest entry, keys to 2^-11 (group ratios
    and scaled keys are f16), float32 sums; weights and scaled values to 2^-11
    each.  A score error d changes a weight by at most a factor exp(2 d) - 1
    after normalisation, and the rotation keeps 2-norms.
    """
    n_pages, nkv = k_pool[0].shape[:2]
    rows, nqh, _ = q.shape
    g = nqh // nkv
    s = 1.0 if signs is None else signs.astype(np.float64)
    scale = DIM ** -0.5 if scale is None else scale
    qr = (q * s) @ H
    out = np.full(q.shape, np.nan)
    room = np.full(q.shape[:2], np.nan)
    for b in range(len(lens)):
        r0, n, ln = int(cu[b]), int(cu[b + 1] - cu[b]), max(0, int(lens[b]))
        ln = min(ln, table.shape[1] * page)
        pos = np.arange(ln)
        pg = table[b, pos // page] if ln else pos
        there = (pg >= 0) & (pg < n_pages)
        pgc = np.where(there, pg, 0)
        for h in range(nkv):
            k = values(k_pool[0][pgc, h, pos % page], k_pool[1][pgc, h, pos % page], k_pool[2])
            v = values(v_pool[0][pgc, h, pos % page], v_pool[1][pgc, h, pos % page], v_pool[2])
            k = np.where(there[:, None], k, 0.0)
            v = np.where(there[:, None], v, 0.0)
            for i in range(n):
                see = there.copy()
                if causal:
                    p = ln - n + i
                    ok = pos <= p
                    if window:
                        ok &= (pos > p - window) | (pos < sinks)
                    see &= ok
                for hh in range(h * g, h * g + g):
                    x = qr[r0 + i, hh]
                    if not see.any():
                        out[r0 + i, hh] = 0.0
                        room[r0 + i, hh] = 0.0
                        continue
                    sc = scale * (k[see] @ x)
                    w = np.exp(sc - sc.max())
                    w /= w.sum()
                    out[r0 + i, hh] = (w @ v[see]) @ H * s
                    ak = np.abs(k[see])
                    d = scale * (ak @ (np.abs(x) * 2.0 ** -10) + ak.sum(-1) * np.abs(x).max() * 2.0 ** -16)
                    rel = np.expm1(2 * (w @ d) + 2 * d) + 2.0 ** -10 + 2.0 ** -11
                    room[r0 + i, hh] = np.linalg.norm((w * rel) @ np.abs(v[see]))
    return out, room


def check_attention(got, want, room, what=""):
    """Every row within half a bf16 step (2^-8 relative) plus `room`; all rows
    together within half a step plus the two 11-bit roundings."""
    live = ~np.isnan(want[..., 0])
    w, g, r = want[live], got[live], room[live]
    assert np.isfinite(g).all(), what
    err = np.linalg.norm(g - w, axis=-1)
    lim = 2.0 ** -8 * np.linalg.norm(w, axis=-1) + r
    bad = err > lim * (1 + 1e-6) + 1e-30
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} rows off, worst {np.max(err / np.maximum(lim, 1e-300)):.3g} of the limit"
