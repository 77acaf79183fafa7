"""The bound that attention outputs are held to: it lets a correctly rounded
result pass and turns down the mistakes a kernel could make (planted in the
float64 implementation)."""

import numpy as np
import pytest

import paged_bounds as A
import paged_ref as R
from test_paged_gpu import Case

# what is made, how it is called, and the mistakes that change the result at all
SCALE, SHORT, LONG = ("softmax scale", dict(scale=1.02 * R.DIM ** -0.5)), ("mask one key short", dict(short=1)), ("mask one key long", dict(short=-1))
DROP = ("keys dropped", dict(skip=range(16, 32)))
CASES = {
    "decode": (dict(seed=61, reqs=[(1, 300), (1, 129), (1, 64), (1, 640)], nqh=8, nkv=2), {}, [SCALE, SHORT, DROP]),
    "chunk": (dict(seed=62, reqs=[(40, 300), (64, 64)], nqh=4, nkv=2, bits=8, group=64), {}, [SCALE, SHORT, LONG, DROP]),
    "window": (dict(seed=63, reqs=[(1, 500), (70, 400)], nqh=2, nkv=1), dict(window=100, sinks=20), [SCALE, SHORT, LONG, DROP]),
    "cross": (dict(seed=64, reqs=[(20, 90), (9, 200)], nqh=2, nkv=2, bits=8), dict(causal=False), [SCALE, DROP]),
    "peaked": (dict(seed=65, reqs=[(1, 500), (1, 400)], nqh=4, nkv=1, q_scale=8.0), {}, [SCALE]),
    "peaked chunk": (dict(seed=11, reqs=[(40, 500)], nqh=4, nkv=1, bits=8, spread=2.0, q_scale=6.0), {}, [SHORT, LONG]),
    "long": (dict(seed=13, reqs=[(1, 70000)], nqh=8, nkv=1, page=64), {}, [SCALE, ("keys dropped", dict(skip=range(16, 1040)))]),
}


def make(name):
    made, how, mistakes = CASES[name]
    made = dict(made)
    return Case(made.pop("seed"), made.pop("reqs"), made.pop("nqh"), made.pop("nkv"), **made), how, mistakes


def oracle(c, how, **mistake):
    return A.attention(c.q, c.k, c.v, c.table, c.lens, c.cu, c.page, signs=c.signs, **{**how, **mistake})


@pytest.mark.parametrize("name", CASES)
def test_mistakes_are_found(name):
    c, how, mistakes = make(name)
    want, rms = oracle(c, how)
    other, _ = R.attention(c.q, c.k, c.v, c.table, c.lens, c.cu, c.page, signs=c.signs, **how)
    live = ~np.isnan(want)
    assert np.array_equal(live, ~np.isnan(other)) and np.allclose(want[live], other[live], rtol=1e-9, atol=1e-12)
    A.check(R.bf16(want), want, rms)

    def found(wrong, what):
        with pytest.raises(AssertionError):
            A.check(R.bf16(np.nan_to_num(wrong)), want, rms, what)

    found(np.zeros_like(want), "zeros")
    found(want * 0.96, "a factor")
    found(want * 1.01, "a small factor")
    for what, mistake in mistakes:
        found(oracle(c, how, **mistake)[0], what)


def test_the_bound_is_close():
    """Beside the bf16 rounding a row may be off by a few tenths of a percent,
    not by the worst case of every key's error at once."""
    for name in ("decode", "chunk", "window", "cross", "long"):
        c, how, _ = make(name)
        want, rms = oracle(c, how)
        size = np.linalg.norm(want, axis=-1)
        live = size > 0
        own = A.SIGMAS * rms[live] / size[live]
        assert np.median(own) < 2.0 ** -7 and np.max(own) < 2.0 ** -6, name
