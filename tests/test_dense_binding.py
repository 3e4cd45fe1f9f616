"""Host half of the dense operators' Python face: which device a call is launched on. No GPU: the
entry points and torch's device functions are stand-ins that record what they are asked for."""

import contextlib

import pytest
import torch

from collective_datapath_copy_gb300 import dense


class Machine:
    """Two devices, one of them current, and an entry point that notes where it is launched."""

    def __init__(self, monkeypatch, current):
        self.current, self.launches = current, []

        @contextlib.contextmanager
        def device(d):
            before, self.current = self.current, d
            yield
            self.current = before

        def call(packed, stream):
            self.launches.append((self.current, stream))
            return 0

        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(dense, "_current_device", lambda: self.current, raising=False)
        monkeypatch.setattr(dense, "_raw_stream", lambda d: 100 + d)
        monkeypatch.setattr(dense, "_entries", {})
        monkeypatch.setattr(dense, "_entry", lambda name: (call, lambda packed: 0))


def operator(dev):
    """An operator whose weights are on device `dev`, as far as a launch can tell."""
    op = object.__new__(dense.Linear)
    op._start(torch.device("cpu"))
    op._dev = dev
    return op


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("dev", [0, 1])
def test_a_call_is_launched_on_the_device_of_the_weights(monkeypatch, current, dev):
    m = Machine(monkeypatch, current)
    operator(dev)._launch("coll_linear", lambda *fields: fields, (8, 32, 64))
    assert m.launches == [(dev, 100 + dev)]
    assert m.current == current


class Stream:
    def __init__(self, dev):
        self.device_index = dev


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Its handle would be ignored: the call looks up the current stream of the weights' device."""
    m = Machine(monkeypatch, 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    w = torch.zeros(8, 16, dtype=torch.bfloat16)
    lin, ffn = operator(-1), object.__new__(dense.GatedFFN)   # -1: where torch's CPU tensors are
    m.current = -1
    lin.weight, lin.bias, lin.act = w, None, "none"
    ffn.w_gate, ffn.w_up, ffn.act = w, w, "silu"
    ffn._start(torch.device("cpu"))
    x, y = torch.zeros(4, 16, dtype=w.dtype), torch.zeros(4, 8, dtype=w.dtype)
    calls = [lambda s: lin.forward(x, out=y, stream=s), lambda s: lin.backward(y, x, stream=s),
             lambda s: ffn.forward(x, out=y, stream=s),
             lambda s: ffn.backward(y, x, y, y, stream=s)]
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    for call in calls:
        with pytest.raises(ValueError, match="stream"):
            call(Stream(1))
    assert m.launches == []
    for call in calls:
        call(Stream(-1))
    assert len(m.launches) == len(calls)
