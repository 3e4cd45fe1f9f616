"""TensorParallelMLP plans and runs its sums on the device of its weights (no GPU: weights on the
host, device -1, while device 0 is current; the sums are stand-ins)."""

import pytest
import torch

from collective_datapath_copy_gb300 import dense, mlp
from test_dense_binding import Machine


@pytest.mark.parametrize("partials", ["f32", "bf16"])
def test_sums_run_where_the_weights_are(monkeypatch, partials):
    m = Machine(monkeypatch, 0)
    where = []

    class Sum:
        def __init__(self, naming, **cfg):
            where.append(("plan", m.current))

        def run(self, ins, outs):
            where.append(("run", m.current))

    monkeypatch.setattr(mlp, "Plan", Sum)
    monkeypatch.setattr(dense, "_weight", lambda name, w: w)
    w, d = torch.zeros(64, 32, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    layer = mlp.TensorParallelMLP(2, w, w, d, 8, partials=partials)
    x = torch.zeros(8, 32, dtype=torch.bfloat16)
    layer.forward(x, residual=x, keep=True)
    layer.backward(x)
    assert len(where) >= 3 and {dev for _, dev in where} == {-1}
    assert {dev for dev, _ in m.launches} == {-1} and len(m.launches) == 8
    assert m.current == 0
