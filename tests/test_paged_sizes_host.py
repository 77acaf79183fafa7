"""Numbers that do not fit a C int are refused by the binding, not wrapped."""

import pytest
import torch

import hadamard_rotation_outlier_b200 as hq

WRAP = 1 << 32  # what a C int drops


@pytest.fixture
def made():
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    pool = [torch.zeros(2, 2, 16, 64, dtype=torch.uint8), torch.zeros(2, 2, 16)] * 2
    return i, q, pool, torch.zeros(2, 2, dtype=torch.int32)


@pytest.mark.parametrize("name,value", [("group", WRAP + 32), ("group", 32 - WRAP), ("block", WRAP + 128), ("bits", WRAP + 4), ("window", 5 - WRAP),
                                        ("window", 1 << 31), ("sinks", 1 - WRAP), ("max_new", WRAP + 1), ("max_new", 1 - WRAP)])
def test_attention(made, name, value):
    i, q, pool, table = made
    with pytest.raises(ValueError, match="32 bits"):
        hq.hadq_paged_attention(q, *pool, table, i, torch.zeros(3, dtype=torch.int32), **{"max_new": 1, name: value})


@pytest.mark.parametrize("name,value", [("group", WRAP + 32), ("block", WRAP + 128), ("bits", 4 - WRAP)])
def test_append_and_gather(made, name, value):
    i, q, pool, _ = made
    with pytest.raises(ValueError, match="32 bits"):
        hq.hadq_paged_append(q, q, i, *pool, **{name: value})
    with pytest.raises(ValueError, match="32 bits"):
        hq.hadq_paged_gather(*pool[:2], i, **{name: value})


def test_slots_and_workspace(made):
    i, _, _, table = made
    with pytest.raises(ValueError, match="32 bits"):
        hq.hadq_paged_slots(i, i, i, table, WRAP + 16, capacity=4)
    for sizes in ((WRAP + 1, 8, 8), (1, WRAP + 8, 8), (1, 8, 8 - WRAP)):
        with pytest.raises(ValueError, match="32 bits"):
            hq.hadq_paged_workspace_size(*sizes)
