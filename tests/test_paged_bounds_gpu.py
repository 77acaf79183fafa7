"""Paged attention on the GPU within a close bound of float64 (paged_bounds.py)."""

import pytest
import torch

import paged_bounds as A
from test_paged_gpu import CHUNKS, DECODE, Case

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def held(c, max_new=None, **how):
    got = c.run(max_new, **how)
    scale = how.pop("softmax_scale", None)
    want, rms = A.attention(c.q, c.k, c.v, c.table, c.lens, c.cu, c.page, signs=c.signs, scale=scale, **how)
    A.check(got, want, rms, str(how))
    return got, want


FORMS = [(4, 128), (4, 64), (4, 32), (8, 128), (8, 64), (8, 32)]


@pytest.mark.parametrize("bits,group", FORMS)
@pytest.mark.parametrize("nqh,nkv", [(8, 2), (7, 1)])
def test_single_tokens(bits, group, nqh, nkv):
    held(Case(100 + nqh * bits + group, DECODE, nqh, nkv, bits=bits, group=group))


@pytest.mark.parametrize("bits,group", FORMS)
@pytest.mark.parametrize("nqh,nkv,page", [(4, 1, 16), (10, 2, 32)])
def test_several_tokens(bits, group, nqh, nkv, page):
    held(Case(200 + nqh + bits + group, CHUNKS, nqh, nkv, bits=bits, group=group, page=page, with_signs=bits == 4))


@pytest.mark.parametrize("window,sinks", [(1, 1), (64, 64), (100, 0), (100, 33), (128, 500)])
@pytest.mark.parametrize("reqs", [[(1, 1), (1, 400), (3, 260), (1, 1100)], [(150, 500), (64, 64), (1, 900), (33, 1290)]])
def test_window_and_sinks(window, sinks, reqs):
    held(Case(300 + window + sinks, reqs, 4, 2, bits=8), window=window, sinks=sinks)


@pytest.mark.parametrize("bits", [4, 8])
def test_cross(bits):
    held(Case(400 + bits, [(1, 33), (7, 1), (50, 200), (3, 0), (129, 64), (20, 1500)], 4, 4, bits=bits), causal=False)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("batch", [1, 2])
def test_peaked_softmax(new, batch):
    """Scores of hundreds: most rows see one key, some weigh two."""
    held(Case(500 + new, [(new, 500)] * batch, 4, 1, bits=8, spread=2.0, q_scale=6.0))
    held(Case(600 + new, [(new, 500)] * batch, 4, 1, bits=4, q_scale=8.0))


@pytest.mark.parametrize("new,lens", [(1, 70000), (33, 20000)])
def test_long(new, lens):
    """One request over all CTAs, many splits to join."""
    held(Case(700 + new, [(new, lens)], 16 if new == 1 else 1, 1, bits=4, page=64))


@pytest.mark.parametrize("new", [1, 64])
def test_mask_edges(new):
    """The keys on both sides of every border of the masks are loud in V, the
    others quiet, so that one key too many, or too few, shows."""
    for ln, window, sinks in ((new + 200, 0, 0), (new + 200, 96, 0), (new + 200, 65, 3)):
        c = Case(800 + ln, [(new, ln)] * 2, 2, 1, bits=8, with_signs=False)
        c.v[1][:] = 0.01
        for b in range(2):
            for pos in (ln - new - 1, ln - new, ln - 1, ln - new - window, ln - new - window + 1, ln - window - 1, sinks - 1, sinks):
                if 0 <= pos < ln:
                    c.v[1][c.table[b, pos // 16], :, pos % 16] = 3.0
        held(c, window=window, sinks=sinks)
