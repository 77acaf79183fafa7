"""Refusals of the paged-cache entry points: every bad argument is turned down
on the host, before any launch (no GPU needed: the pointers are never read)."""

import ctypes

import numpy as np
import pytest
import torch

from hadamard_rotation_outlier_b200 import binding as B

import paged_ref as R

INVALID, UNSUPPORTED, MISALIGNED, OK = B.HADQ_ERR_INVALID_ARG, B.HADQ_ERR_UNSUPPORTED, B.HADQ_ERR_MISALIGNED, B.HADQ_OK
P = 0x10000  # an address that is aligned to everything; no call below gets as far as a launch


@pytest.fixture(scope="module")
def lib():
    from hadamard_rotation_outlier_b200.build import build
    build()
    return B.load_library()


SLOTS = dict(cached=P, new=2 * P, batch=2, free=3 * P, n_free=4, page=16, table=4 * P, max_pages=8, total=5 * P, cu=6 * P, slots=7 * P,
             capacity=4, counts=8 * P)
APPEND = dict(k=P, v=P, tokens=2, k_stride=256, v_stride=256, heads=2, dim=128, block=128, signs=None, bits=4, group=128, slots=P, kc=P, ks=P,
              vc=P, vs=P, pages=3, page=16)
GATHER = dict(codes=P, scales=P, pages=3, page=16, heads=2, dim=128, block=-1, signs=None, bits=8, group=-1, slots=P, tokens=2, out=P, dtype=0)
ATTENTION = dict(q=P, rows=4, stride=1024, cu=P, lens=P, batch=2, max_new=1, kc=P, ks=P, vc=P, vs=P, pages=3, page=16, table=P, max_pages=4,
                 nqh=8, nkv=2, dim=128, block=128, signs=None, bits=4, group=128, causal=1, window=0, sinks=0, scale=0.1, out=P, ws=P,
                 ws_bytes=1 << 40)


def call(lib, fn, base, **change):
    n0 = B.hadq_launch_count()
    args = dict(base, **change)
    st = getattr(lib, fn)(*args.values(), None)
    assert B.hadq_launch_count() == n0
    if st != OK:
        assert B.hadq_last_error()
    return st


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), INVALID), (dict(n_free=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(capacity=-1), INVALID),
    (dict(page=0), INVALID), (dict(page=8), INVALID), (dict(page=24), INVALID), (dict(page=2048), INVALID), (dict(batch=16385), UNSUPPORTED),
    (dict(capacity=1 << 31), UNSUPPORTED), (dict(cached=None), INVALID), (dict(new=None), INVALID), (dict(free=None), INVALID),
    (dict(table=None), INVALID), (dict(total=None), INVALID), (dict(cu=None), INVALID), (dict(slots=None), INVALID),
    (dict(counts=None), INVALID), (dict(cached=P + 2), MISALIGNED), (dict(table=P + 1), MISALIGNED), (dict(total=P), INVALID),
    (dict(total=2 * P), INVALID)])
def test_slots_refusals(lib, change, status):
    assert call(lib, "hadq_paged_slots", SLOTS, **change) == status


CACHE = [(dict(page=8), INVALID), (dict(page=48), INVALID), (dict(page=4096), INVALID), (dict(pages=-1), INVALID), (dict(dim=64, block=64, group=64), UNSUPPORTED),
         (dict(dim=127), INVALID), (dict(block=64), UNSUPPORTED), (dict(block=3), INVALID), (dict(bits=5), INVALID), (dict(group=16), UNSUPPORTED),
         (dict(group=48), INVALID), (dict(pages=1 << 27), UNSUPPORTED), (dict(pages=1 << 40), UNSUPPORTED)]


@pytest.mark.parametrize("change,status", CACHE + [
    (dict(heads=0), INVALID), (dict(tokens=-1), INVALID), (dict(k_stride=255), INVALID), (dict(v_stride=128), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(kc=None), INVALID), (dict(vs=None), INVALID), (dict(k=P + 8), MISALIGNED),
    (dict(k_stride=260), MISALIGNED), (dict(kc=P + 8), MISALIGNED), (dict(vs=P + 2), MISALIGNED), (dict(slots=P + 1), MISALIGNED),
    (dict(tokens=1 << 30), UNSUPPORTED),
    (dict(tokens=0, k=None, v=None, slots=None), OK), (dict(pages=0, kc=None, ks=None), OK)])
def test_append_refusals(lib, change, status):
    assert call(lib, "hadq_paged_append", APPEND, **change) == status


@pytest.mark.parametrize("change,status", CACHE + [
    (dict(heads=0), INVALID), (dict(tokens=-1), INVALID), (dict(dtype=2), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(slots=None), INVALID), (dict(out=None), INVALID), (dict(codes=P + 8), MISALIGNED), (dict(out=P + 8), MISALIGNED),
    (dict(scales=P + 1), MISALIGNED), (dict(tokens=1 << 40), UNSUPPORTED), (dict(tokens=0, out=None, codes=None), OK), (dict(pages=0, codes=None), OK)])
def test_gather_refusals(lib, change, status):
    assert call(lib, "hadq_paged_gather", GATHER, **change) == status


@pytest.mark.parametrize("change,status", CACHE + [
    (dict(nkv=0), INVALID), (dict(nqh=0), INVALID), (dict(nqh=9), INVALID), (dict(batch=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(max_new=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(stride=1016), INVALID), (dict(stride=1028), MISALIGNED),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(causal=0, window=5), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=-1.0), INVALID), (dict(rows=1 << 29), UNSUPPORTED),
    (dict(max_pages=1 << 27), UNSUPPORTED),
    (dict(pages=1 << 25, nkv=8), UNSUPPORTED), (dict(q=None), INVALID), (dict(cu=None), INVALID), (dict(lens=None), INVALID),
    (dict(kc=None), INVALID), (dict(vs=None), INVALID), (dict(table=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
    (dict(q=P + 8), MISALIGNED), (dict(kc=P + 8), MISALIGNED), (dict(ks=P + 4), MISALIGNED), (dict(out=P + 8), MISALIGNED),
    (dict(ws=P + 128), MISALIGNED), (dict(lens=P + 2), MISALIGNED), (dict(ws_bytes=100), INVALID), (dict(batch=0, q=None), OK),
    (dict(rows=0, q=None, out=None), OK), (dict(max_new=0, q=None), OK)])
def test_attention_refusals(lib, change, status):
    assert call(lib, "hadq_paged_attention", ATTENTION, **change) == status


@pytest.mark.parametrize("change", [
    dict(total=P + 4), dict(cu=2 * P + 4), dict(cu=5 * P + 4), dict(slots=6 * P + 8), dict(slots=3 * P), dict(counts=7 * P + 12), dict(counts=P),
    dict(table=3 * P - 4), dict(table=5 * P - 60), dict(new=6 * P), dict(free=4 * P + 60)])
def test_slots_outputs_stand_alone(lib, change):
    """CTAs read the inputs while others write: no output may overlap an input
    or another output, nor may it start inside one."""
    assert call(lib, "hadq_paged_slots", SLOTS, **change) == INVALID
    assert "overlap" in B.hadq_last_error()


def test_slots_of_a_table_past_32_bits(lib):
    """Page counts are summed in 32 bits."""
    assert call(lib, "hadq_paged_slots", SLOTS, batch=16384, max_pages=1 << 17) == UNSUPPORTED


@pytest.mark.parametrize("change", [dict(stride=1032), dict(out=P + 16), dict(out=P + 4 * 2048 - 16), dict(out=P + 5 * 2048, stride=2048),
                                    dict(q=P + 4 * 2048 - 16)])
def test_attention_output_over_its_queries(lib, change):
    assert call(lib, "hadq_paged_attention", ATTENTION, **change) == INVALID
    assert "overlap" in B.hadq_last_error()


def test_workspace_size(lib):
    a, b = B.hadq_paged_workspace_size(1, 32, 8), B.hadq_paged_workspace_size(2048, 32, 8)
    assert 0 < a <= b <= 48 << 20
    for bad in ((-1, 8, 8), (1, 0, 1), (1, 3, 2)):
        with pytest.raises(B.HadqError):
            B.hadq_paged_workspace_size(*bad)
    assert lib.hadq_paged_workspace_size(1, 8, 8, None) == INVALID


def test_binding_refuses_cpu_tensors_and_wrong_types():
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    c = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    s = torch.zeros(2, 2, 16)
    with pytest.raises(ValueError, match="CUDA"):
        B.hadq_paged_slots(i, i, i, torch.zeros(2, 2, dtype=torch.int32), 16, capacity=4)
    with pytest.raises(ValueError, match="CUDA"):
        B.hadq_paged_append(q, q, i, c, s, c, s)
    with pytest.raises(ValueError, match="CUDA"):
        B.hadq_paged_gather(c, s, i)
    with pytest.raises(ValueError, match="CUDA"):
        B.hadq_paged_attention(q, c, s, c, s, torch.zeros(2, 2, dtype=torch.int32), i, torch.zeros(3, dtype=torch.int32), 1)
    cpu = -1  # what get_device() says of CPU tensors
    with pytest.raises(TypeError):
        B._rows_view(q.float(), "q", cpu, None)
    with pytest.raises(ValueError, match="contiguously"):
        B._rows_view(q.transpose(0, 1), "q", cpu, None)
    with pytest.raises(ValueError):
        B._rows_view(q, "k", cpu, 3)
    assert B._rows_view(torch.zeros(3, 10, 128, dtype=torch.bfloat16)[:, 2:6], "k", cpu, 4) == 1280
    with pytest.raises(ValueError, match="bytes"):
        B._pool(c, s, "k", cpu, 8, 128)
    with pytest.raises(ValueError, match="scales"):
        B._pool(c, s, "k", cpu, 4, 64)
    with pytest.raises(TypeError):
        B._pool(c.to(torch.int16), s, "k", cpu, 4, 128)
    with pytest.raises(ValueError, match="shape"):
        B._pool(c, s, "v", cpu, 4, 128, (3, 2, 16, 64))


# ------------------------------------------ the reference implementation itself

def test_reference_slots_by_hand():
    table, slots, total, cu, counts = R.slots([3, 0, 16], [2, 17, 1], [9, 5, 7, 4], np.array([[2, -1], [-1, -1], [6, -1]], np.int32), 16, 22)
    assert table.tolist() == [[2, -1], [9, 5], [6, 7]]
    assert slots.tolist() == [35, 36] + [144 + i for i in range(16)] + [80, 112, -1, -1]
    assert total.tolist() == [5, 17, 17] and cu.tolist() == [0, 2, 19, 20] and counts.tolist() == [3, 0]


def test_reference_attention_by_hand():
    """One key: the output is its value row, rotated back; equal keys: the mean."""
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 256, (1, 1, 16, 128)).astype(np.uint8)
    scales = np.ones((1, 1, 16, 1), np.float32)
    q = R.bf16(rng.standard_normal((2, 1, 128)))
    table = np.zeros((1, 1), np.int32)
    zero = (np.zeros_like(codes), scales, 8)
    out, _ = R.attention(q, zero, (codes, scales, 8), table, [2], [0, 2], 16)
    v = codes[0, 0].view(np.int8).astype(np.float64) @ R.H
    assert np.allclose(out[0, 0], v[0]) and np.allclose(out[1, 0], (v[0] + v[1]) / 2)
    out, _ = R.attention(q, zero, (codes, scales, 8), table, [5], [0, 2], 16, window=1, sinks=1)
    assert np.allclose(out[0, 0], (v[0] + v[3]) / 2) and np.allclose(out[1, 0], (v[0] + v[4]) / 2)
    assert np.allclose(R.H @ R.H, np.eye(128))


def test_bf16_rounding_of_the_reference():
    x = np.random.default_rng(1).standard_normal(1000)
    assert np.array_equal(R.bf16(x), torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).double().numpy())
