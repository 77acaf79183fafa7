"""The paged KV cache on the GPU against a plain float64 implementation:
slots, append, gather, attention, and a serving step of all of them."""

import numpy as np
import pytest
import torch

import hadamard_rotation_outlier_b200 as hq
from hadamard_rotation_outlier_b200 import binding as B

import paged_ref as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DIM = 128


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).cuda().to(torch.bfloat16)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def signs_of(rng, on):
    return rng.choice(np.array([-1, 1], np.int8), DIM) if on else None


# -------------------------------------------------------------------- slots

def run_slots(cached, new, free, table, page, capacity):
    t = dev(np.asarray(table, np.int32))
    s, total, cu, counts = hq.hadq_paged_slots(dev(np.asarray(cached, np.int32)), dev(np.asarray(new, np.int32)),
                                               dev(np.asarray(free, np.int32)), t, page, capacity=capacity)
    got = [x.cpu().numpy() for x in (t, s, total, cu, counts)]
    want = R.slots(cached, new, free, np.asarray(table, np.int32), page, capacity)
    for name, a, b in zip(("table", "slots", "total", "cu", "counts"), got, want):
        assert np.array_equal(a, b), name


def tables(rng, cached, new, page, width, spare):
    old = -(-np.maximum(cached, 0) // page)
    need = int((-(-(np.maximum(cached, 0) + np.maximum(new, 0)) // page)).sum()) + 8
    ids = rng.permutation(need + int(old.sum())).astype(np.int32)
    table = np.full((len(cached), width), -7, np.int32)
    at = 0
    for b, n in enumerate(old):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, ids[at:at + spare]


@pytest.mark.parametrize("batch,new_max,ctx_max,page", [(1, 1, 0, 16), (1, 1000, 5, 16), (7, 3, 40, 16), (33, 70, 300, 64),
                                                        (511, 5, 100, 32), (513, 9, 1000, 128), (1500, 40, 600, 256)])
def test_slots(batch, new_max, ctx_max, page):
    rng = np.random.default_rng(batch)
    cached, new = rng.integers(0, ctx_max + 1, batch), rng.integers(0, new_max + 1, batch)
    width = -(-(ctx_max + new_max) // page) + 1
    table, free = tables(rng, cached, new, page, width, spare=10 ** 6)
    run_slots(cached, new, free, table, page, int(new.sum()) + 5)


def test_slots_without_room():
    rng = np.random.default_rng(3)
    cached = np.array([0, 15, 16, 0, 100, 3, -4, 31])
    new = np.array([20, 1, 1, 0, 200, 2, 5, -3])
    table, free = tables(rng, cached, new, 16, 12, spare=100)
    for n_free in (0, 1, 2, 3, 4, 5, 40):
        run_slots(cached, new, free[:n_free], table, 16, 300)
    run_slots(cached, new, free, table, 16, 0)       # no rows asked for
    run_slots(cached, new, free, table, 16, 7)       # fewer rows than tokens
    run_slots(np.zeros(0, int), np.zeros(0, int), free, np.zeros((0, 4), np.int32), 16, 9)  # no requests


def test_slots_page_of_a_grown_request_missing():
    # a half-full page the table does not name: its tokens get no slot
    run_slots(np.array([5]), np.array([20]), np.array([9, 8], np.int32), np.full((1, 4), -1, np.int32), 16, 30)


# --------------------------------------------------------- append and gather

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("group", [128, 64, 32])
@pytest.mark.parametrize("tokens,heads,page,with_signs", [(1, 1, 16, True), (5, 3, 16, False), (67, 8, 64, True), (300, 5, 1024, True)])
def test_append_and_gather(bits, group, tokens, heads, page, with_signs):
    rng = np.random.default_rng(tokens * bits + group)
    signs = signs_of(rng, with_signs)
    x = rng.standard_normal((2, tokens, heads, DIM))
    x[..., 17] *= 40.0
    x[:, 0, 0] = 0.0                # a zero row
    if tokens > 4:
        x[:, 3] *= 1e-37            # a tiny one
        x[:, 4] *= 1e30
    x = R.bf16(x)
    pages = -(-tokens // page) + 2
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    bad = []
    if tokens > 4:
        slots[1], slots[2] = -1, pages * page   # no place
        bad = [1, 2]
    # K and V are slices of a wider projection
    wide = torch.zeros(tokens, 3 * heads + 1, DIM, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:1 + heads] = dev_bf16(x[0])
    wide[:, 1 + heads:1 + 2 * heads] = dev_bf16(x[1])
    k, v = wide[:, 1:1 + heads], wide[:, 1 + heads:1 + 2 * heads]
    pool = [torch.full((pages, heads, page, 16 * bits), 0x5A, dtype=torch.uint8, device="cuda"),
            torch.full((pages, heads, page, DIM // group), -3.0, device="cuda")]
    kc, ks, vc, vs = pool[0].clone(), pool[1].clone(), pool[0].clone(), pool[1].clone()
    sg = None if signs is None else dev(signs)
    hq.hadq_paged_append(k, v, dev(slots), kc, ks, vc, vs, signs=sg, bits=bits, group=group)
    live = [t for t in range(tokens) if t not in bad]
    for src, codes, scales in ((x[0], kc, ks), (x[1], vc, vs)):
        y, scale, t, want = R.quantize(src, signs, bits, group)
        c, s = codes.cpu().numpy(), scales.cpu().numpy()
        p, o = slots[live] // page, slots[live] % page
        # float32 sums of 128 terms, then one product: 2^-24 each, 8 levels deep
        assert np.allclose(s[p, :, o], scale[live], rtol=2.0 ** -20, atol=2.0 ** -149)
        d = R.unpack(c[p, :, o], bits) - want[live]
        # another code only next to a .5 boundary: |t| <= 127 carries 2^-20 of itself
        near = np.abs(np.abs(t[live] - np.floor(t[live])) - 0.5) <= 127 * 2.0 ** -19
        assert np.all((d == 0) | (near & (np.abs(d) == 1)))
        assert np.count_nonzero(d) <= 16
        # everything else in the pool is as it was
        rest = np.ones((pages, page), bool)
        rest[p, o] = False
        pi, oi = np.nonzero(rest)
        assert np.all(c[pi, :, oi] == 0x5A) and np.all(s[pi, :, oi] == -3.0)
        # reading back: within float32 of the codes' values, rows without a slot untouched
        for dtype in (torch.float32, torch.bfloat16):
            out = torch.full((tokens, heads, DIM), 7.0, dtype=dtype, device="cuda")
            got = hq.hadq_paged_gather(codes, scales, dev(slots), signs=sg, bits=bits, group=group, out=out)
            assert got is out
            val = R.values(c[p, :, o], s[p, :, o], bits) @ R.H * (1.0 if signs is None else signs)
            g = host(out)
            top = np.linalg.norm(val, axis=-1, keepdims=True)
            tol = top * 2.0 ** -20 + (2.0 ** -8 * np.abs(val) if dtype == torch.bfloat16 else 0.0) + 2.0 ** -126
            assert np.all(np.abs(g[live] - val) <= tol)
            assert np.all(g[bad] == 7.0)


def test_append_matches_rotate_quantize():
    """The same codes and scales as quantising the rows on their own."""
    g = torch.Generator(device="cuda").manual_seed(5)
    k = torch.randn(130, 4, DIM, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(130, 4, DIM, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(160, generator=g, device="cuda")[:130].to(torch.int32)
    kc = torch.zeros(10, 4, 16, 64, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(10, 4, 16, device="cuda")
    vc, vs = torch.zeros_like(kc), torch.zeros_like(ks)
    hq.hadq_paged_append(k, v, slots, kc, ks, vc, vs, bits=4, group=128)
    p, o = slots.long() // 16, slots.long() % 16
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        codes, scales = hq.hadq_rotate_quantize(x, block=128, bits=4, group=128)
        assert torch.allclose(s[p, :, o], scales[..., 0], rtol=2.0 ** -20, atol=0)
        assert (c[p, :, o] != codes).float().mean() < 1e-3


# ---------------------------------------------------------------- attention

def pool_of(rng, pages, heads, page, bits, group, spread=0.5):
    top = 127 if bits == 8 else 7
    c = np.clip(np.round(rng.standard_normal((pages, heads, page, DIM)) * top / 3), -top, top).astype(np.int64)
    codes = (c & 255).astype(np.uint8) if bits == 8 else ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).astype(np.uint8)
    scales = (np.exp(spread * rng.standard_normal((pages, heads, page, DIM // group))) * 3 / top).astype(np.float32)
    return codes, scales, bits


class Case:
    """Requests of the given (new, length) on shuffled pages."""

    def __init__(self, seed, reqs, nqh, nkv, page=16, bits=4, group=128, with_signs=True, spare_rows=3, spread=0.5, q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.page, self.bits, self.group, self.nqh, self.nkv = rng, page, bits, group, nqh, nkv
        self.new = np.array([r[0] for r in reqs])
        self.lens = np.array([r[1] for r in reqs], np.int32)
        need = -(-self.lens // page)
        pages = int(need.sum()) + 3
        ids = rng.permutation(pages)
        self.table = np.full((len(reqs), max(1, int(need.max(initial=0))) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        rows = int(self.new.sum()) + spare_rows
        self.q = R.bf16(rng.standard_normal((rows, nqh, DIM)) * q_scale)
        self.k, self.v = pool_of(rng, pages, nkv, page, bits, group, spread), pool_of(rng, pages, nkv, page, bits, group, spread)
        self.signs = signs_of(rng, with_signs)

    def run(self, max_new=None, **how):
        rows = self.q.shape[0]
        wide = torch.zeros(rows, self.nqh + 2 * self.nkv, DIM, dtype=torch.bfloat16, device="cuda")
        wide[:, :self.nqh] = dev_bf16(self.q)
        out = torch.full((rows, self.nqh, DIM), 99.0, dtype=torch.bfloat16, device="cuda")
        if max_new is None:
            max_new = int(self.new.max(initial=0))
        args = [wide[:, :self.nqh], dev(self.k[0]), dev(self.k[1]), dev(self.v[0]), dev(self.v[1]), dev(self.table), dev(self.lens), dev(self.cu)]
        sg = None if self.signs is None else dev(self.signs)
        torch.cuda.synchronize()  # (a stream of the caller's may be given)
        hq.hadq_paged_attention(*args, max_new, signs=sg, bits=self.bits, group=self.group, out=out, **how)
        torch.cuda.synchronize()
        got = host(out)
        assert np.all(got[int(self.cu[-1]):] == 99.0)  # rows behind the last request
        return got

    def check(self, max_new=None, **how):
        got = self.run(max_new, **dict(how))
        how.pop("workspace", None)
        scale = how.pop("softmax_scale", None)
        want, room = R.attention(self.q, self.k, self.v, self.table, self.lens, self.cu, self.page, signs=self.signs, scale=scale, **how)
        R.check_attention(got, want, room, str(how))
        return got, want


DECODE = [(1, 1), (1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (0, 40), (1, 300), (1, 129)]


@pytest.mark.parametrize("bits,group", [(4, 128), (4, 64), (4, 32), (8, 128), (8, 64), (8, 32)])
@pytest.mark.parametrize("nqh,nkv", [(4, 4), (8, 2), (5, 1), (16, 2), (7, 1)])
def test_decode(bits, group, nqh, nkv):
    Case(nqh * bits + group, DECODE, nqh, nkv, bits=bits, group=group).check()


CHUNKS = [(3, 3), (1, 700), (40, 40), (17, 300), (0, 0), (130, 257), (64, 64), (2, 2000)]


@pytest.mark.parametrize("bits,group", [(4, 128), (4, 64), (4, 32), (8, 128), (8, 64), (8, 32)])
@pytest.mark.parametrize("nqh,nkv,page", [(4, 1, 16), (3, 3, 128), (10, 2, 32)])
def test_chunks(bits, group, nqh, nkv, page):
    Case(nqh + bits + group, CHUNKS, nqh, nkv, bits=bits, group=group, page=page, with_signs=bits == 4).check()


@pytest.mark.parametrize("new", [1, 2, 3, 5, 8, 9, 16, 31, 33, 64, 65, 129, 200, 256, 300])
@pytest.mark.parametrize("g", [1, 6])
def test_row_counts(new, g):
    """Query rows around every tile size of the kernels."""
    Case(new * g, [(new, new + 77), (new, new)], g, 1, bits=8, page=64).check()


@pytest.mark.parametrize("batch", [1, 2, 40])
def test_same_result_in_any_batch(batch):
    """A request's result lies within the rounding room, alone or in a batch
    whose CTAs it shares; max_new beyond the largest count changes nothing."""
    reqs = [(1, 5 + 37 * b) for b in range(batch)]
    Case(batch, reqs, 8, 2).check(max_new=1)
    Case(batch, reqs, 8, 2).check(max_new=500)


@pytest.mark.parametrize("nqh,nkv", [(200, 1), (256, 1), (300, 1), (72, 2)])
def test_many_heads_per_kv_head(nqh, nkv):
    """One query token of such a group fills a tile, or more than one."""
    Case(nqh, [(1, 70), (3, 200), (2, 2)], nqh, nkv, bits=8, page=32).check()


def test_many_requests():
    """More requests than a CTA has threads, most of them short or empty."""
    rng = np.random.default_rng(4)
    reqs = [(1, int(n)) for n in rng.integers(1, 90, 300)]
    Case(31, reqs, 2, 1).check()
    new = rng.integers(0, 3, 900)
    new[[5, 650, 899]] = [40, 33, 70]
    Case(32, [(int(n), int(n) + int(c)) for n, c in zip(new, rng.integers(0, 60, 900))], 1, 1, bits=8).check()


@pytest.mark.parametrize("new", [1, 50])
def test_pages_beyond_four_gigabytes(new):
    """Byte offsets past 32 bits: the same bits from the far end of a pool of
    4.3 GB codes per tensor as from a small one."""
    c = Case(33, [(new, 300)], 2, 1, bits=4, page=16, spare_rows=0)
    want = c.run()
    far = (1 << 22) + 64
    n = c.k[0].shape[0]
    pools = []
    for codes, scales, _ in (c.k, c.v):
        big = torch.empty((far, 1, 16, 64), dtype=torch.uint8, device="cuda")
        sc = torch.empty((far, 1, 16, 1), device="cuda")
        big[far - n:], sc[far - n:] = dev(codes), dev(scales)
        pools += [big, sc]
    table = np.where(c.table >= 0, c.table + far - n, c.table).astype(np.int32)
    sg = dev(c.signs)
    out = hq.hadq_paged_attention(dev_bf16(c.q), *pools, dev(table), dev(c.lens), dev(c.cu), new, signs=sg, bits=4, group=128)
    assert np.array_equal(host(out), want)
    pos = np.arange(300)
    at = dev((table[0, pos // 16] * 16 + pos % 16).astype(np.int32))
    near = dev((c.table[0, pos // 16] * 16 + pos % 16).astype(np.int32))
    for i, (codes, scales, _) in enumerate((c.k, c.v)):
        assert torch.equal(hq.hadq_paged_gather(pools[2 * i], pools[2 * i + 1], at, signs=sg, bits=4, group=128),
                           hq.hadq_paged_gather(dev(codes), dev(scales), near, signs=sg, bits=4, group=128))
    k = dev_bf16(R.bf16(c.rng.standard_normal((300, 1, DIM))))
    small = [torch.zeros_like(dev(a)) for a in (c.k[0], c.k[1], c.v[0], c.v[1])]
    hq.hadq_paged_append(k, -k, near, *small, signs=sg, bits=4, group=128)
    hq.hadq_paged_append(k, -k, at, *pools, signs=sg, bits=4, group=128)
    used = torch.from_numpy(c.table[0][c.table[0] >= 0]).long().cuda()[:-1]  # (the last page is not full)
    for a, b in zip(small, pools):
        assert torch.equal(a[used], b[used + far - n])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (64, 64), (100, 0), (100, 33), (1000, 4), (128, 500)])
@pytest.mark.parametrize("reqs", [[(1, 1), (1, 400), (3, 260), (1, 1100)], [(150, 500), (64, 64), (1, 900), (33, 1290)]])
def test_window_and_sinks(window, sinks, reqs):
    Case(window + sinks, reqs, 4, 2, bits=8).check(window=window, sinks=sinks)


@pytest.mark.parametrize("window", [2 ** 30 - 1, 2 ** 31 - 1])
def test_window_longer_than_any_request(window):
    """The largest windows limit nothing, queries before the start of their
    request among them (their positions are negative)."""
    c = Case(23, [(6, 4), (40, 10), (1, 70), (50, 300)], 4, 2)
    assert np.array_equal(c.check(window=window)[0], c.run())


@pytest.mark.parametrize("bits", [4, 8])
def test_cross(bits):
    Case(bits, [(1, 33), (7, 1), (50, 200), (3, 0), (129, 64), (20, 1500)], 4, 4, bits=bits).check(causal=False)


def test_rows_that_see_nothing():
    """More queries than cached tokens (the first ones are before the start),
    no cached tokens, and pages outside the pool: zeros, and no read there."""
    c = Case(1, [(6, 4), (2, 0), (1, 40), (3, 90), (40, 10)], 4, 2)
    c.table[2, :] = [-1, 10 ** 6, -(2 ** 31)] + [2 ** 31 - 1] * (c.table.shape[1] - 3)
    c.table[3, 1] = -5
    got, want = c.check()
    assert np.all(got[0] == 0.0) and np.all(got[6:8] == 0.0) and np.all(got[8] == 0.0) and np.any(got[9])
    assert np.all(got[12:12 + 30] == 0.0) and np.all(got[12 + 30:52].any(-1))


@pytest.mark.parametrize("new", [1, 70])
def test_mask_edges_are_exact(new):
    """The keys just outside what a query sees hold huge values and would win
    the softmax: one key too many, or too few, shows at once."""
    for ln, window, sinks in ((new + 200, 0, 0), (new + 200, 96, 0), (new + 200, 65, 3)):
        c = Case(ln, [(new, ln)], 2, 1, bits=8, with_signs=False)
        # every 16th key loud in both K (along its own code pattern) and V
        c.v[1][:] = np.where(c.rng.random(c.v[1].shape) < 0.2, 1000.0, 0.01)
        c.check(window=window, sinks=sinks)


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("group", [128, 32])
def test_nan_where_nobody_looks(new, group):
    """Scales that are not finite behind the last token, in unused pages and
    in masked places reach no output."""
    c = Case(5, [(new, new + 70)], 4, 1, bits=8, group=group)
    last = int(c.lens[0]) - 1
    p, o = c.table[0, last // 16], last % 16
    seen = c.table[0][c.table[0] >= 0]
    for pool in (c.k, c.v):
        pool[1][[i for i in range(pool[1].shape[0]) if i not in seen]] = np.nan
        pool[1][p, :, o + 1:] = np.inf
    c.check()
    for pool in (c.k, c.v):  # the last token's own row: only its own query sees it
        pool[1][p, :, o] = np.nan
    got = c.run()
    want, room = R.attention(c.q, c.k, c.v, c.table, c.lens, c.cu, 16, signs=c.signs)
    want[new - 1] = np.nan
    R.check_attention(got, want, room)


@pytest.mark.parametrize("new", [5, 60])
@pytest.mark.parametrize("bits,group", [(4, 128), (8, 32)])
@pytest.mark.parametrize("lens", [30, 400])
def test_queries_that_are_not_finite(new, bits, group, lens):
    """A query with a NaN or an infinity gets NaN, or zeros where it sees no
    key; the rows beside it are as without it."""
    c = Case(21, [(new, lens), (new, new - 2)], 4, 2, bits=bits, group=group)
    c.q[1, 0, 7] = np.nan
    c.q[2, 3] = np.nan
    c.q[3, 1, 100] = np.inf
    c.q[4, 2, 64] = -np.inf
    c.q[new, 0, 5] = np.nan       # before the start: sees nothing
    c.q[new + 1, 3, 9] = np.inf   # the same
    got = c.run()
    with np.errstate(invalid="ignore"):
        want, room = R.attention(c.q, c.k, c.v, c.table, c.lens, c.cu, 16, signs=c.signs)
    low = max(0, new - lens)      # rows of the first request before its start
    for r, h in ((1, 0), (2, 3), (3, 1), (4, 2)):
        if r >= low:
            assert np.isnan(got[r, h]).all(), (r, h)
            want[r, h] = np.nan
    assert np.all(got[new:new + 2] == 0.0)
    R.check_attention(got, want, room)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("k_scale,v_scale,q_scale", [(1e-6, 1.0, 1.0), (1.0, 1e-12, 1.0), (1.0, 1e12, 1.0), (1.0, 1.0, 1e-20), (1e8, 1.0, 1e-8),
                                                     (1e-10, 1.0, 1e10), (0.0, 0.0, 1.0), (1.0, 1.0, 0.0)])
def test_ranges(new, k_scale, v_scale, q_scale):
    """Scales and queries far from one, and all zero."""
    c = Case(7, [(new, 200)], 4, 2, bits=4, q_scale=q_scale)
    c.k[1][:] = (c.k[1].astype(np.float64) * k_scale).astype(np.float32)
    c.v[1][:] = (c.v[1].astype(np.float64) * v_scale).astype(np.float32)
    c.check()


@pytest.mark.parametrize("new", [1, 40])
def test_peaked_softmax(new):
    """Scores of +-60 and value rows of very different size."""
    c = Case(11, [(new, 500)], 4, 1, bits=8, spread=2.0, q_scale=6.0)
    c.check()


def test_value_scales_of_different_size():
    """Keys with tiny value rows (attention sinks) that take most of the weight."""
    for new in (1, 40):
        c = Case(12, [(new, 300)], 4, 1, bits=8)
        c.v[1][c.table[0, 0], :, :4] *= 2.0 ** -9
        c.k[1][c.table[0, 0], :, :4] *= 4.0
        c.check()


@pytest.mark.parametrize("new,lens", [(1, 70000), (33, 20000)])
def test_long(new, lens):
    """One request over all CTAs, many splits to join."""
    c = Case(13, [(new, lens)], 1, 1, bits=4, page=64)
    c.check()


def test_workspace_is_reused_and_left_ready():
    ws = torch.zeros(hq.hadq_paged_workspace_size(64, 8, 2), dtype=torch.uint8, device="cuda")
    c = Case(14, [(1, 900), (64, 700), (5, 33)], 8, 2)
    first = c.run(workspace=ws)
    for _ in range(3):
        assert np.array_equal(c.run(workspace=ws), first)   # the same bits every time
    assert not ws[:8192].any()
    B.hadq_device_status()  # no wait ran out


def test_output_in_place_of_the_queries():
    c = Case(24, [(1, 2000), (60, 900), (3, 33)], 4, 2, spare_rows=0)
    want = c.run()
    q = dev_bf16(c.q)
    args = [dev(x) for x in (c.k[0], c.k[1], c.v[0], c.v[1], c.table, c.lens, c.cu)]
    assert hq.hadq_paged_attention(q, *args, 60, signs=dev(c.signs), out=q) is q
    assert np.array_equal(host(q), want)


@pytest.mark.parametrize("bits", [4, 8])
def test_rows_aligned_to_16_bytes_only(bits):
    """q and out that start 16 bytes behind a 32-byte boundary."""
    c = Case(25, [(1, 200), (70, 300), (200, 210)], 4, 2, bits=bits, spare_rows=2)
    want = c.run()
    n = c.q.size

    def behind(fill):
        t = torch.full((n + 16,), fill, dtype=torch.bfloat16, device="cuda")
        return t, t[8:8 + n].view(c.q.shape)

    (qb, q), (ob, out) = behind(0.0), behind(99.0)
    q.copy_(dev_bf16(c.q))
    assert q.data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16
    args = [dev(x) for x in (c.k[0], c.k[1], c.v[0], c.v[1], c.table, c.lens, c.cu)]
    hq.hadq_paged_attention(q, *args, 200, signs=dev(c.signs), bits=bits, out=out)
    assert np.array_equal(host(out), want)
    assert np.all(host(ob[:8]) == 99.0) and np.all(host(ob[8 + n:]) == 99.0)


def test_other_stream():
    c = Case(15, [(1, 300), (20, 300)], 4, 2)
    want = c.run()
    s = torch.cuda.Stream()
    assert np.array_equal(c.run(stream=s), want)
    with torch.cuda.stream(s):
        assert np.array_equal(c.run(), want)


# -------------------------------------------------------- a serving step

@pytest.mark.parametrize("bits,group,new", [(4, 128, [1, 1, 1, 1]), (8, 64, [5, 0, 130, 1])])
def test_serving_steps(bits, group, new):
    """slots -> append -> attention over three steps, against attention over
    what gather reads back; then the same step captured once and replayed."""
    rng = np.random.default_rng(bits)
    nkv, g, page, batch, pages = 2, 4, 16, 4, 200
    free = dev(rng.permutation(pages).astype(np.int32))
    table = torch.full((batch, 60), -1, dtype=torch.int32, device="cuda")
    kc = torch.zeros(pages, nkv, page, 16 * bits, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(pages, nkv, page, DIM // group, device="cuda")
    vc, vs = torch.zeros_like(kc), torch.zeros_like(ks)
    sg = dev(signs_of(rng, True))
    how = {"signs": sg, "bits": bits, "group": group}
    lens = np.array([100, 0, 37, 16])
    cap = 160
    ws = torch.zeros(hq.hadq_paged_workspace_size(cap, nkv * g, nkv), dtype=torch.uint8, device="cuda")

    def step(cached, fresh, freelist, k, v, q):
        slots, total, cu, counts = hq.hadq_paged_slots(cached, fresh, freelist, table, page, capacity=k.shape[0])
        hq.hadq_paged_append(k, v, slots, kc, ks, vc, vs, **how)
        out = hq.hadq_paged_attention(q, kc, ks, vc, vs, table, total, cu, cap, workspace=ws, out=torch.zeros_like(q), **how)
        return out, total, cu, counts

    taken = 0
    history = [[np.zeros((0, nkv, DIM)), np.zeros((0, nkv, DIM))] for _ in range(batch)]
    cached = np.zeros(batch, np.int32)
    for fresh in (lens, np.array(new), np.array(new)[::-1].copy()):
        rows = int(fresh.sum()) + 2
        x = [rng.standard_normal((rows, n, DIM)) for n in (nkv, nkv, nkv * g)]
        k, v, q = (dev_bf16(a) for a in x)
        out, total, cu, counts = step(dev(cached.astype(np.int32)), dev(fresh.astype(np.int32)), free[taken:], k, v, q)
        taken += int(counts[0])
        assert int(counts[1]) == 0
        c = cu.cpu().numpy()
        for b in range(batch):
            for i, a in enumerate((k, v)):
                history[b][i] = np.concatenate([history[b][i], host(a)[c[b]:c[b + 1]]])
        cached = cached + fresh
        assert np.array_equal(total.cpu().numpy(), cached)
        # the cache holds each request's own rows, quantised
        want, room = R.attention(host(q), (kc.cpu().numpy(), ks.cpu().numpy(), bits), (vc.cpu().numpy(), vs.cpu().numpy(), bits),
                                 table.cpu().numpy(), total.cpu().numpy(), c, page, signs=sg.cpu().numpy())
        R.check_attention(host(out), want, room)
        t = table.cpu().numpy()
        for b in range(batch):
            pos = np.arange(int(cached[b]))
            at = dev((t[b, pos // page] * page + pos % page).astype(np.int32))
            for i, (codes, scales) in enumerate(((kc, ks), (vc, vs))):
                back = host(hq.hadq_paged_gather(codes, scales, at, out_dtype=torch.float32, **how))
                _, scale, _, _ = R.quantize(history[b][i], sg.cpu().numpy(), bits, group)
                # half a step of every code, as a 2-norm over the row
                step_norm = np.sqrt((scale ** 2).sum(-1) * group) * 0.5
                assert np.all(np.linalg.norm(back - history[b][i], axis=-1) <= step_norm * (1 + 1e-4))

    # captured once, replayed with other lengths and inputs
    fresh_t, cached_t = dev(np.array([1, 1, 1, 1], np.int32)), dev(cached.astype(np.int32))
    k, v, q = (dev_bf16(rng.standard_normal((8, n, DIM))) for n in (nkv, nkv, nkv * g))
    rest = free[taken:].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(cached_t, fresh_t, rest, k, v, q)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, total, cu, counts = step(cached_t, fresh_t, rest, k, v, q)
    fresh_t.copy_(dev(np.array([3, 0, 1, 4], np.int32)))
    for a in (k, v, q):
        a.copy_(dev_bf16(rng.standard_normal(tuple(a.shape))))
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(total.cpu().numpy(), cached + [3, 0, 1, 4])
    want, room = R.attention(host(q), (kc.cpu().numpy(), ks.cpu().numpy(), bits), (vc.cpu().numpy(), vs.cpu().numpy(), bits),
                             table.cpu().numpy(), total.cpu().numpy(), cu.cpu().numpy(), page, signs=sg.cpu().numpy())
    R.check_attention(host(out), want, room)


def test_agrees_with_contiguous_decode():
    """A page table in order is the contiguous cache: the same attention."""
    c = Case(21, [(1, 1024)] * 2, 8, 2, page=1024, spare_rows=0)
    c.table[:, 0] = [0, 1]
    out = host(B.hadq_kv_decode_attention(dev_bf16(c.q), dev(c.k[0][:2]), dev(c.k[1][:2]), dev(c.v[0][:2]), dev(c.v[1][:2]),
                                          signs=dev(c.signs), bits=4, group=128))
    _, room = R.attention(c.q, c.k, c.v, c.table, c.lens, c.cu, 1024, signs=c.signs)
    got = c.run()
    err = np.linalg.norm(got - out, axis=-1)
    assert np.all(err <= 2.0 ** -7 * np.linalg.norm(out, axis=-1) + room)
