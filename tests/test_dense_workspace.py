"""The workspace that a dense operator's call is given, call after call (no GPU: the library's own
sizes, and an entry point that takes what it is given)."""

import struct

import pytest
import torch

from collective_datapath_copy_gb300 import _lib, dense
from collective_datapath_copy_gb300.build import build

BF, F32 = _lib.D["COLL_BF16"], _lib.D["COLL_F32"]
A = 1 << 32
NO = (0, 0, 0)


def linear(m, n, k, off=0, res=NO, out=BF):
    return ("coll_linear", dense._LINEAR.pack,
            (m, n, k, BF, out, 0, A + off, k, 1, 2 * A, k, 1, *res, *NO, 4 * A, n, 1, 0, 0),
            res != NO)


def linear_bwd(m, n, k, dx=True, db=False):
    return ("coll_linear_backward", dense._LINEAR_BWD.pack,
            (m, n, k, BF, BF, 4, A, n, 1, 2 * A, n, 1, 3 * A, k, 1, 4 * A, k, 1,
             *((5 * A, k, 1) if dx else NO), 6 * A, k, 1, 7 * A if db else 0), db)


def gated(m, n, k, off=0):
    return ("coll_gated_ffn", dense._GATED.pack,
            (m, n, k, BF, 4, A + off, k, 1, 2 * A, k, 1, 3 * A, k, 1, *NO, *NO, 4 * A, n, 1), False)


def gated_bwd(m, n, k, dw=True):
    return ("coll_gated_ffn_backward", dense._GATED_BWD.pack,
            (m, n, k, BF, BF, 4, A, n, 1, 2 * A, n, 1, 3 * A, n, 1, 4 * A, k, 1, 5 * A, k, 1,
             6 * A, k, 1, 7 * A, k, 1, *((8 * A, k, 1, 9 * A, k, 1) if dw else NO + NO)), False)


class Calls:
    """An operator whose calls are noted: what each was given, and how often sizes were asked."""

    def __init__(self, monkeypatch):
        build()
        self.given, self.asked = [], 0
        self.op = object.__new__(dense.Linear)
        self.op._start(torch.device("cpu"))
        monkeypatch.setattr(dense, "_current_device", lambda: self.op._dev, raising=False)
        monkeypatch.setattr(dense, "_raw_stream", lambda d: 0)
        monkeypatch.setattr(dense, "_entries", {})
        monkeypatch.setattr(dense, "_entry", self.entry)

    def entry(self, name):
        size = getattr(_lib.lib(), name + "_workspace")

        def call(packed, stream):
            ws, got, _ = struct.unpack("3q", packed[-24:])
            if got < size(packed):
                return _lib.D["COLL_EWORKSPACE"]
            self.given.append(got)
            return 0

        def ask(packed):
            self.asked += 1
            return size(packed)
        return call, ask

    def __call__(self, where, pack, fields, given):
        """The workspace the call was given, and what it needs."""
        self.op._launch(where, pack, fields, given)
        need = getattr(_lib.lib(), where + "_workspace")(pack(*fields, 0, 0, 0))
        return self.given[-1], need


SEQUENCES = [
    # a prompt that lays out its operand or shares k, then a token that needs nothing
    [linear(2048, 4096, 4097), linear(1, 4096, 4096), linear(1, 4096, 4096)],
    [gated(300, 512, 4096, off=2), gated(1, 512, 4096), gated(300, 512, 4096)],
    [linear(20, 40, 9000), linear(20, 40, 9000, out=F32), linear(20, 40, 512)],
    # one size, other operands: a base off 16 bytes, a residual that is one number for all
    [linear(300, 512, 4096, off=2), linear(300, 512, 4096), linear(300, 512, 4096, off=4)],
    [linear(130, 72, 4096, res=(3 * A, 0, 0)), linear(130, 72, 4096)],
    [linear_bwd(4096, 512, 256, db=True), linear_bwd(2, 512, 256), linear_bwd(2, 512, 256, db=True)],
    [linear_bwd(300, 512, 9000, db=True), linear_bwd(300, 512, 9000),
     linear_bwd(300, 512, 9000, dx=False)],
    [gated_bwd(4096, 14336, 64), gated_bwd(2, 14336, 64), gated_bwd(2, 14336, 64, dw=False)],
]


@pytest.mark.parametrize("calls", SEQUENCES)
def test_a_call_is_given_what_it_needs(monkeypatch, calls):
    c = Calls(monkeypatch)
    for call in calls + calls[::-1]:
        given, need = c(*call)
        assert given == need, call


def test_a_loop_over_one_size_asks_once(monkeypatch):
    c = Calls(monkeypatch)
    for _ in range(5):
        c(*gated_bwd(512, 1024, 256))
        c(*linear(8, 256, 256))
    assert c.asked == 1


def test_two_entry_points_do_not_disturb_each_other(monkeypatch):
    c = Calls(monkeypatch)
    for _ in range(3):
        for call in (linear(2048, 4096, 4097), linear_bwd(777, 1530, 1016, db=True)):
            given, need = c(*call)
            assert given == need
    assert c.asked == 2
