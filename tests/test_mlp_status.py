"""TensorParallelMLP.status (no GPU: weights on the host, sums that are stand-ins)."""

import pytest
import torch

from collective_datapath_copy_gb300 import _lib, dense, mlp

TIMED_OUT = _lib.D["COLL_ETIMEDOUT"]


class Sum:
    def __init__(self, naming, **cfg):
        self.code = _lib.OK

    def status(self):
        return {"code": self.code}


@pytest.fixture(params=[torch.bfloat16, torch.float16])
def layer(monkeypatch, request):
    """float16 sums its gradients in binary32, as it does its outputs; bfloat16 here has two."""
    monkeypatch.setattr(mlp, "Plan", Sum)
    monkeypatch.setattr(dense, "_weight", lambda name, w: w)
    w, d = torch.zeros(64, 32, dtype=request.param), torch.zeros(32, 64, dtype=request.param)
    return mlp.TensorParallelMLP(4, w, w, d, 8, partials="f32")


def test_a_layer_whose_waits_all_ended(layer):
    assert layer.status() == _lib.OK


def test_an_expired_wait_of_any_operator_shows(layer):
    for op in layer.up + layer.down:
        op._status.fill_(TIMED_OUT)
        assert layer.status() == TIMED_OUT and op.status() == TIMED_OUT
        assert sum(o.status() != _lib.OK for o in layer.up + layer.down) == 1
        op._status.zero_()
    assert layer.status() == _lib.OK


def test_an_expired_wait_of_a_sum_shows(layer):
    for plan in (layer._sum, layer._gsum):
        plan.code = TIMED_OUT
        assert layer.status() == TIMED_OUT
        plan.code = _lib.OK
