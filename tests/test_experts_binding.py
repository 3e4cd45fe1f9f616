"""GatedExperts' Python face without a GPU: stacks that are given other storage between calls."""

import pytest
import torch

from collective_datapath_copy_gb300 import dense, experts

BF = torch.bfloat16


class Device(torch.Tensor):
    """A CPU tensor that says it is on a GPU unless told otherwise."""

    is_cuda = property(lambda self: getattr(self, "gpu", True))


def stack(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Device)


@pytest.fixture
def op(monkeypatch):
    monkeypatch.setattr(dense, "_current_device", lambda: -1)
    made = experts.GatedExperts(stack(4, 24, 16), stack(4, 24, 16), stack(4, 32, 24), first=3)
    made.calls = []
    made._launch = lambda where, pack, fields: made.calls.append(fields)
    return made


def call(op, k=16):
    op.forward(torch.zeros(5, k, dtype=BF), torch.zeros(5, 2, dtype=torch.int32), torch.zeros(5, 2))
    return op.calls.pop()


def want(op):
    wg, wu, wd = op.w_gate, op.w_up, op.w_down
    (E, F, K), N = wg.shape, wd.shape[1]
    return ((5, N, K, F, E, 3, 2),
            tuple(v for w in (wg, wu, wd) for v in (w.data_ptr(), w.stride(0), w.stride(1))))


def check(op, k=16):
    f = call(op, k)
    assert (f[:7], f[10:19]) == want(op)


def test_sizes_and_strides_are_those_of_the_call(op):
    check(op)
    op.w_up.data = torch.zeros(4, 30, 20, dtype=BF)[:, 2:26, :16]  # other strides
    check(op)
    # fewer experts, more inner features, longer rows and outputs
    for w, shape in ((op.w_gate, (2, 40, 48)), (op.w_up, (2, 40, 48)), (op.w_down, (2, 72, 40))):
        w.data = torch.zeros(*shape, dtype=BF)
    check(op, 48)
    # the same memory seen in another way
    op.w_gate.data = op.w_gate.data.view(2, 48, 40).transpose(0, 1).reshape(48, 2, 40)[:2, :1, :]
    with pytest.raises(ValueError):
        call(op, 40)
    for w in (op.w_gate, op.w_up):
        w.data = w.data.reshape(-1)[:2 * 24].view(2, 1, 24)
    op.w_down.data = op.w_down.data[:, :, :1]
    check(op, 24)
    op.w_down.data = op.w_down.data[:, ::2]  # in place, half of the rows
    check(op, 24)


def test_storage_that_does_not_fit_is_refused_before_the_library(op):
    check(op)
    kept = [w.data for w in (op.w_gate, op.w_up, op.w_down)]

    def refused(match, **to):
        for name, t in to.items():
            getattr(op, name).data = t
        with pytest.raises(ValueError, match=match):
            call(op)
        assert op.calls == []
        for w, t in zip((op.w_gate, op.w_up, op.w_down), kept):
            w.data = t
        check(op)
    refused("must be", w_gate=torch.zeros(4, 12, 16, dtype=BF))
    refused("must be", w_up=torch.zeros(3, 24, 16, dtype=BF))
    refused("must be", w_down=torch.zeros(4, 32, 16, dtype=BF))
    refused("contiguous", w_down=torch.zeros(4, 24, 32, dtype=BF).transpose(1, 2))
    refused("bfloat16 or float16", w_gate=torch.zeros(4, 24, 16))
    refused("w_up must be", w_up=torch.zeros(4, 24, 16, dtype=torch.float16))
    refused("three dimensions", w_up=torch.zeros(0, dtype=BF))
    op.w_up.gpu = False
    refused("CUDA", w_up=torch.zeros(4, 24, 16, dtype=BF))
    del op.w_up.gpu
    check(op)


def test_a_stack_that_moved_to_another_device_is_refused(op, monkeypatch):
    check(op)
    monkeypatch.setattr(Device, "get_device", lambda w: 1)
    for w in (op.w_gate, op.w_up, op.w_down):
        w.data = torch.zeros(w.shape, dtype=BF)
    with pytest.raises(ValueError, match="cuda:1"):
        call(op)
    assert op.calls == []
