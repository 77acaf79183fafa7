"""Paged attention in float64 with a close bound of what the kernels' own
roundings do to it, and the check that holds outputs to it.

The bound is a root mean square, made of every rounding's own: an operand
rounded to n bits is off by at most half a step h = 2^-n of its value, evenly
spread, which is h / sqrt(3) of it.  Independent ones add up as squares.

 * Query, kernel for few rows: 32000 steps to its largest rotated entry, half a
   step of 2^-15.9 of that entry; kernel for many rows: f16, 2^-11 of each.
   The error is the same for all keys, so it moves an output row by
   (sum_t w_t k_t x (v_t - out)) times it.
 * Keys, many rows: the scale and the scaled code as f16, 2^-11 each; few rows:
   exact.  The error is a key's own: it moves a row by w_t (v_t - out) times
   the score's.
 * Weights and (many rows) scaled values: f16, 2^-11 each, or 2^-33 of the
   largest weight where that is more (f16 has no more room below).
 * Float32 sums and exponentials: 2^-22 of a score's magnitude, 2^-20 of a row.
Scores that are off by d change a weight by exp(d), not 1 + d: errors are taken
at five times their own size, expm1(5 d) / 5.
"""

import numpy as np

from paged_ref import DIM, H, values

FEW = 32         # query rows per KV head up to which the kernel for few rows serves a request (of several)
SIGMAS = 5.0     # what one row may be off by, in root mean squares
STEP = 2.0 ** -8  # half a step of the bf16 result, at most


def attention(q, k_pool, v_pool, table, lens, cu, page, causal=True, window=0, sinks=0, signs=None, scale=None, short=0, skip=()):
    """q: float64 [rows, heads, 128]; pools: (codes, scales, bits).  Returns
    the output (NaN in rows of no request) and each row's root mean square of
    the roundings beside that of the result.  `short` keys fewer at the end of
    every mask and `skip`ped positions are the mistakes that a check has to
    find."""
    n_pages, nkv = k_pool[0].shape[:2]
    nqh = q.shape[1]
    g = nqh // nkv
    s = 1.0 if signs is None else signs.astype(np.float64)
    scale = DIM ** -0.5 if scale is None else scale
    qr = (q * s) @ H
    out, rms = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    for b in range(len(lens)):
        r0, n = int(cu[b]), int(cu[b + 1] - cu[b])
        ln = min(max(0, int(lens[b])), table.shape[1] * page)
        many = n * g > FEW
        pos = np.arange(ln)
        pg = table[b, pos // page] if ln else pos
        there = (pg >= 0) & (pg < n_pages) & ~np.isin(pos, skip)
        pgc = np.where(there, pg, 0)
        for h in range(nkv):
            k = np.where(there[:, None], values(k_pool[0][pgc, h, pos % page], k_pool[1][pgc, h, pos % page], k_pool[2]), 0.0)
            v = np.where(there[:, None], values(v_pool[0][pgc, h, pos % page], v_pool[1][pgc, h, pos % page], v_pool[2]), 0.0)
            groups = k_pool[1].shape[-1]
            for i in range(n):
                see = there.copy()
                if causal:
                    p = ln - n + i
                    ok = pos <= p - short
                    if window:
                        ok &= (pos > p - window) | (pos < sinks)
                    see &= ok
                kk, vv = k[see], v[see]
                for hh in range(h * g, h * g + g):
                    if not len(kk):
                        out[r0 + i, hh], rms[r0 + i, hh] = 0.0, 0.0
                        continue
                    x = qr[r0 + i, hh]
                    parts = scale * kk * x
                    sc = parts.sum(-1)
                    w = np.exp(sc - sc.max())
                    w /= w.sum()
                    o = w @ vv
                    out[r0 + i, hh] = o @ H * s
                    sq = np.maximum(2.0 ** -11 * many * np.abs(x), 2.0 ** -15.9 * np.abs(x).max()) / 3 ** 0.5
                    dev = vv - o
                    live = w > 1e-9
                    dq = scale * np.sqrt((kk[live] ** 2 @ sq ** 2).max(initial=0.0))
                    e2 = (np.expm1(SIGMAS * dq) / (SIGMAS * dq) if dq > 0 else 1.0) ** 2
                    e2 *= (((scale * (kk * w[:, None]).T @ dev) ** 2).sum(-1) * sq ** 2).sum()
                    dk2 = (2.0 ** -22 * np.abs(sc)) ** 2
                    if many:
                        dk2 = dk2 + 2.0 ** -22 / 3 * ((parts.reshape(-1, groups, DIM // groups).sum(-1) ** 2).sum(-1) + (parts ** 2).sum(-1))
                    dk = np.expm1(SIGMAS * np.minimum(np.sqrt(dk2), 100.0)) / SIGMAS
                    n2 = (vv ** 2).sum(-1)
                    e2 += (w ** 2 * dk ** 2 * (dev ** 2).sum(-1)).sum()
                    e2 += (w ** 2 * n2).sum() * 2.0 ** -22 / 3 * (3 if many else 1)
                    e2 += (2.0 ** -33 * w.max()) ** 2 / 3 * n2.max() * len(w)
                    rms[r0 + i, hh] = np.sqrt(e2) + 2.0 ** -20 * np.linalg.norm(o)
    return out, rms


def check(got, want, rms, what=""):
    """Every row within half a bf16 step plus SIGMAS root mean squares; all rows
    together within the root mean square of the bf16 rounding (a step over
    sqrt(12), a step 2^-7 of the value at most) and twice their own."""
    live = ~np.isnan(want[..., 0])
    w, g, r = want[live], got[live], rms[live]
    assert np.isfinite(g).all(), what
    err, size = np.linalg.norm(g - w, axis=-1), np.linalg.norm(w, axis=-1)
    lim = STEP * size + SIGMAS * r + 1e-36
    assert np.all(err <= lim), f"{what}: {(err > lim).sum()} of {err.size} rows off, worst {np.max(err / lim):.3g} of the limit"
    if err.size >= 8:
        top = size.max()  # (rows of very different size: every one counts relative to its own limit too)
        for a, b, c in ((err / top, size / top, r / top), (err / np.maximum(size, 1e-36), np.where(size > 0, 1.0, 0.0), r / np.maximum(size, 1e-36))):
            total, room = np.sqrt((a ** 2).sum()), 1.1 * 2.0 ** -7 / 12 ** 0.5 * np.sqrt((b ** 2).sum()) + 2 * np.sqrt((c ** 2).sum())
            assert total <= room + 1e-30, f"{what}: all rows together {total / room:.3g} of the limit"
