"""Routing tables with choices that were not made (-1), as Router returns them, through the dispatch
and combine namings."""

import numpy as np
import pytest

import collective_datapath_copy_gb300 as cdc
from collective_datapath_copy_gb300 import namings

# tables [R, T, k] of two ranks with two experts each, and the tokens (rank, token) that no expert takes
TABLES = [([[[3, 0], [1, -1]], [[-1, -1], [2, 3]]], {(1, 0)}),
          ([[[-1, -1], [-1, 2]], [[0, -1], [-1, -1]]], {(0, 0), (1, 1)}),
          ([[[-1, -1], [-1, -1]], [[-1, -1], [-1, -1]]], {(0, 0), (0, 1), (1, 0), (1, 1)}),
          ([[[3, 0], [1, -1]], [[1, -1], [2, 3]]], set())]


@pytest.mark.parametrize("zero_copy", [0, 1])
@pytest.mark.parametrize("table,left_out", TABLES)
def test_both_ways_plan_and_tokens_without_an_expert_receive_nothing(table, left_out, zero_copy):
    routing = np.array(table, dtype=np.int32)
    there, back = (f(routing, 2, 8) for f in (namings.moe_dispatch, namings.moe_combine))
    for nm in (there, back):
        cdc.validate(nm, zero_copy=zero_copy)
    tokens = [(s, t) for s in range(2) for t in range(2) if (s, t) not in left_out]
    assert back.rows("out") == [(s, t * 8, 8, s * 2 + t) for s, t in tokens]
    assert back.rows("in") == there.rows("out") and back.in_len == there.out_len
    assert {tuple(i) for i in np.argwhere(~back.meta["dest"].any(2)).tolist()} == left_out
    assert cdc.validate(back, zero_copy=zero_copy).n_names == len(tokens)
