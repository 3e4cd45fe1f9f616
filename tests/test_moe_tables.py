"""Routing tables with choices that were not made (-1), as Router returns them, through the dispatch
and combine namings."""

import numpy as np
import pytest

import collective_datapath_copy_gb300 as cdc
import synth
from collective_datapath_copy_gb300 import namings
from oracle import collectives
from oracle.naming import run_naming

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


def _on(nm, ins):
    """The outputs of a naming by its definition, over zeros."""
    outs = [np.zeros(n, dtype=np.uint16) for n in nm.out_len]
    assert run_naming(nm.R, nm.op, nm.dtype, nm.in_len, nm.rows("in"), nm.out_len, nm.rows("out"),
                      ins, outs) == 0
    return outs


def _tables():
    for table, _ in TABLES:
        yield np.array(table, dtype=np.int32), 2
    for seed, share in ((1, 0.3), (2, 0.8)):
        rng = np.random.default_rng(seed)
        routing = rng.integers(0, 12, (3, 20, 4)).astype(np.int32)
        routing[rng.random(routing.shape) < share] = -1
        yield routing, 4


@pytest.mark.parametrize("routing,per_rank", list(_tables()))
def test_the_namings_agree_with_the_oracle(routing, per_rank):
    R, T, _ = routing.shape
    H = 8
    rng = synth.seeded_rng(5)
    xs = [synth.normal_bf16(rng, (T, H)) for _ in range(R)]
    there = namings.moe_dispatch(routing, per_rank, H)
    assert np.array_equal(there.meta["dest"], collectives.moe_dest_ranks(routing, per_rank))
    want, counts = collectives.moe_dispatch(xs, routing, per_rank)
    assert there.meta["counts"] == counts
    for got, w, c in zip(_on(there, [x.ravel() for x in xs]), want, counts):
        assert np.array_equal(got[:c * H], w.ravel())
    back = namings.moe_combine(routing, per_rank, H)
    ys = [synth.normal_bf16(rng, (max(c, 1), H)) for c in counts]
    want = collectives.moe_combine_sum([y[:c] for y, c in zip(ys, counts)], routing, per_rank, "bf16")
    for got, w in zip(_on(back, [y.ravel() for y in ys]), want):
        assert np.array_equal(got, w.ravel())


def test_the_oracle_sends_a_choice_that_was_not_made_nowhere():
    dest = collectives.moe_dest_ranks(np.array([[[3, 0], [1, -1]], [[-1, -1], [2, 3]]]), 2)
    assert dest.tolist() == [[[True, True], [True, False]], [[False, False], [False, True]]]
