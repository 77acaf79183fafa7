"""Paged attention over caches and queries of extreme size: value scales that
span the float32 range, keys that take nearly all weight, signed key scales,
queries that are not finite."""

import numpy as np
import pytest
import torch

import hadamard_rotation_outlier_b200 as hq

import paged_bounds as A
from test_paged_bounds_gpu import held
from test_paged_gpu import Case, dev, dev_bf16

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


NONE = None  # value scales of zero
SPANS = {
    "zeros behind": [30, NONE, NONE, NONE],
    "zeros before": [NONE, 30],
    "zeros far behind": [100, NONE, NONE],
    "tiny behind": [60, -60, -90],
    "tiny before": [-90, 96],
    "up and down": [-60, 40, 0, 90, -90, NONE, 20],
    "one size": [-85],
    "down": [90, 50, 10, -30, -70],
}


def spans(c, blocks):
    """Value scales times 2^e, e by blocks of 128 keys."""
    scales = c.v[1]
    for b, n in enumerate(c.lens):
        for pos in range(0, n, c.page):
            e = blocks[(pos // 128) % len(blocks)]
            scales[c.table[b, pos // c.page]] *= 0.0 if e is NONE else 2.0 ** e


@pytest.mark.parametrize("name", SPANS)
@pytest.mark.parametrize("quiet", [True, False])
@pytest.mark.parametrize("new", [1, 40])
def test_value_scales_that_span(name, quiet, new):
    """Keys hold their part of the weight whatever their values' size: with
    scores of zero (quiet) the output is the plain mean."""
    few = new == 1
    c = Case(len(name) + new, [(new, 1024 - 37 * b % 400) for b in range(56 if few else 10)], 8 if few else 2, 8 if few else 2,
             page=64, bits=8, group=64 if quiet else 128)
    spans(c, SPANS[name])
    if quiet:
        c.k[1][:] = 0.0
    held(c)


def test_value_scales_join():
    """The same over one request that all CTAs share."""
    for new, lens in ((1, 20000), (40, 3000)):
        for name in SPANS:
            c = Case(len(name) + new, [(new, lens)], 2, 1, page=64, bits=4)
            spans(c, SPANS[name])
            held(c)


# ------------------------------------------- nearly all weight on one key

def one_loud_key(c, gap, value):
    """Key 0 of every request has a score `gap` log2 units above the others',
    which are near zero; its value row is `value` times as large."""
    c.signs = None
    c.q[:] = 0.0
    c.k[1][:] *= 2.0 ** -5
    c.q[..., 0] = 8.0                                # rotated: 8 / sqrt(128) in every column
    for b in range(len(c.lens)):
        p = c.table[b, 0]
        c.k[0][p, :, 0] = 0x77 if c.bits == 4 else 127
        c.k[1][p, :, 0] = gap * np.log(2.0) / ((7 if c.bits == 4 else 127) * 8.0)   # 128 columns, times 1 / sqrt(128) twice
        c.v[1][p, :, 0] *= value


@pytest.mark.parametrize("gap,value", [(20, 0.0), (24, 0.0), (24, 2.0 ** -6)])
@pytest.mark.parametrize("new,lens,batch,heads", [(1, 2048, 60, 8), (33, 4096, 4, 4)])
def test_one_key_with_nearly_all_weight(gap, value, new, lens, batch, heads):
    """A sink: what it adds to the output is nothing, or little, and the output
    is made of weights down to 2^-24 of its own.  (Enough requests for one CTA
    to see the sink and thousands of other keys of its request.)"""
    c = Case(gap, [(new, lens)] * batch, heads, heads, page=64, bits=4)
    one_loud_key(c, gap, value)
    held(c)


# ---------------------------------------------------- large value scales

@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("e", [99, 103, 118])
def test_large_value_scales(new, bits, e):
    """Value rows up to the largest that bf16 holds."""
    c = Case(43, [(new, 300), (new, 90)], 4, 2, bits=bits)
    c.v[1][:] *= np.float32(2.0 ** e)
    held(c)


# ------------------------------------------------------- signed key scales

@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("bits,group", [(4, 128), (8, 32)])
def test_negative_key_scales(new, bits, group):
    """A key scale's sign counts in both kernels."""
    c = Case(41, [(new, 300), (new, 90)], 4, 2, bits=bits, group=group)
    c.k[1][:] *= np.where(c.rng.random(c.k[1].shape) < 0.5, -1.0, 1.0).astype(np.float32)
    held(c)


# ------------------------------------------- queries that are not finite

@pytest.mark.parametrize("new", [5, 40])
@pytest.mark.parametrize("bits", [4, 8])
def test_infinite_query_whose_scores_are_all_low(new, bits):
    """An infinity in one column, against keys that give it the score minus
    infinity: still NaN, and no other row changes."""
    c = Case(42, [(new, new + 3), (new, 200)], 4, 2, bits=bits, with_signs=False)
    c.k[0][c.table[0, :4]] = 0x99 if bits == 4 else 0x81   # code -7 or -127 in every column
    c.k[1][:] = 0.01
    want, rms = A.attention(c.q, c.k, c.v, c.table, c.lens, c.cu, c.page)
    c.q[2, 1] = 0.0
    c.q[2, 1, 0] = np.inf         # rotated: infinity in every column
    c.q[3, 2] = 1.0
    c.q[3, 2, 0] = np.inf
    got = c.run()
    for r, h in ((2, 1), (3, 2)):
        assert np.isnan(got[r, h]).all()
        want[r, h] = np.nan
    A.check(got, want, rms)


# ------------------------------------------------ scores that rise with the position

def rising(c, gain):
    """Scores 0 in the first 64 keys of each request, `gain` log2 units after."""
    c.signs = None
    c.q[:] = 0.0
    c.q[..., 0] = 8.0
    c.k[0][:] = 0x77
    c.k[1][:] = gain * np.log(2.0) / (7 * 8.0)
    for b in range(len(c.lens)):
        c.k[1][c.table[b, :64 // c.page]] = 0.0


@pytest.mark.parametrize("gain", [0.0, 1.5, 3.0, 6.9, 9.0, -5.0])
def test_rising_scores(gain):
    c = Case(51, [(64, 700), (40, 900)], 2, 1)
    rising(c, gain)
    held(c)


def test_rising_scores_cost_no_more():
    """Scores that pass the first keys' by a few units leave the fast path once,
    not in every tile after."""
    c = Case(52, [(512, 4096)] * 4, 8, 2)
    out = {}
    for gain in (0.0, 3.0):
        rising(c, gain)
        args = [dev(x) for x in (c.k[0], c.k[1], c.v[0], c.v[1], c.table, c.lens, c.cu)]
        q, ws = dev_bf16(c.q), torch.zeros(hq.hadq_paged_workspace_size(512, 8, 2), dtype=torch.uint8, device="cuda")
        o = torch.empty_like(q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hq.hadq_paged_attention(q, *args, 512, workspace=ws, out=o)
        out[gain] = (g, args, q, ws, o)
    best = {}
    for _ in range(9):  # in turn, so that clocks and neighbours weigh on both
        for gain, (g, *_) in out.items():
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                g.replay()
            b.record()
            b.synchronize()
            best[gain] = min(best.get(gain, 1e9), a.elapsed_time(b))
    assert best[3.0] <= 1.15 * best[0.0], best


# ----------------------------------------------------------- short units

@pytest.mark.parametrize("bits", [4, 8])
def test_many_units_of_one_to_three_tiles(bits):
    """The warps that plan tiles ahead pass from unit to unit without waiting
    for the rows: no wait may be left behind."""
    rng = np.random.default_rng(bits)
    lens = rng.integers(40, 190, 700)
    c = Case(53, [(34 + b % 7, int(n)) for b, n in enumerate(lens)], 1, 1, bits=bits)
    held(c)
    hq.hadq_device_status()  # (raises if a wait ran out)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale", [1e30, np.inf, np.nan])
def test_key_scale_past_the_limit_reaches_no_other_query(new, scale):
    """The last token's key scale, which only its own query sees."""
    c = Case(54, [(new, 300), (new, 90)], 4, 2, bits=8)
    want, rms = A.attention(c.q, c.k, c.v, c.table, c.lens, c.cu, c.page, signs=c.signs)
    for b, n in enumerate(c.lens):
        c.k[1][c.table[b, (n - 1) // c.page], :, (n - 1) % c.page] = scale
        want[c.cu[b + 1] - 1] = np.nan
    A.check(c.run(), want, rms)
