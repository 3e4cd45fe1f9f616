"""The mixture-of-experts operators' host half, without a GPU: refusals of the C entry points, what a
call launches over a fake CUDA runtime, workspaces, and which device a Python call runs on."""

import contextlib

import numpy as np
import pytest
import torch

import fake_cuda
from collective_datapath_copy_gb300 import _lib, dense, experts, namings

D = _lib.D
BF, HF, F32 = D["COLL_BF16"], D["COLL_F16"], D["COLL_F32"]
A = 1 << 40
NO = (0, 0, 0)


_linked = None


@pytest.fixture
def rt(tmp_path, monkeypatch):
    global _linked
    monkeypatch.setattr(fake_cuda, "OBJECTS", ["route.cu.o", "experts.cu.o", "experts_direct.cu.o"])
    monkeypatch.setattr(fake_cuda, "_built", _linked)
    h = fake_cuda.load(str(tmp_path))
    _linked = fake_cuda._built
    h.fake_reset(-1)
    return h


def call(m, n, k, f, e, top, dtype=BF, out=None, first=0, act=4, off=0, w_off=0, **over):
    """The fields of a coll_gated_experts call, every array at its own address."""
    v = dict(head=(m, n, k, f, e, first, top, dtype, dtype if out is None else out, act),
             gate=(A + w_off, f * k, k), up=(2 * A, f * k, k), down=(3 * A, n * f, f),
             x=(4 * A + off, k, 1), ids=(5 * A, top, 1), weights=(6 * A, top, 1), res=NO,
             y=(7 * A, n, 1), status=0)
    v.update(over)
    return v


def pack(v, ws=8 * A, size=1 << 34):
    flat = [*v["head"]]
    for name in ("gate", "up", "down", "x", "ids", "weights", "res", "y"):
        flat += v[name]
    return experts._EXPERTS.pack(*flat, ws, size, v["status"])


def run(h, v, refused=-1):
    need = h.coll_gated_experts_workspace(pack(v))
    assert need >= 0, need
    h.fake_reset(refused)
    return h.coll_gated_experts(pack(v, size=need), None)


def names(h):
    return [n for n, _ in fake_cuda.launches(h)]


BAD = [({"head": (-1, 64, 64, 64, 4, 0, 2, BF, BF, 4)}, "COLL_EINVAL"),
       ({"head": (5, 1 << 40, 64, 64, 4, 0, 2, BF, BF, 4)}, "COLL_EINVAL"),
       ({"head": (5, 64, 64, 64, 0, 0, 2, BF, BF, 4)}, "COLL_EINVAL"),
       ({"head": (5, 64, 64, 64, 1025, 0, 2, BF, BF, 4)}, "COLL_EINVAL"),
       ({"head": (5, 64, 64, 64, 4, -1, 2, BF, BF, 4)}, "COLL_EINVAL"),
       ({"head": (5, 64, 64, 64, 4, 0, 0, BF, BF, 4)}, "COLL_EINVAL"),
       ({"head": (5, 64, 64, 64, 4, 0, 33, BF, BF, 4)}, "COLL_EINVAL"),
       ({"head": (5, 64, 64, 64, 4, 0, 2, F32, F32, 4)}, "COLL_EINVAL"),
       ({"head": (5, 64, 64, 64, 4, 0, 2, BF, HF, 4)}, "COLL_EINVAL"),
       ({"head": (5, 64, 64, 64, 4, 0, 2, BF, BF, 0)}, "COLL_EINVAL"),
       ({"gate": (0, 64 * 64, 64)}, "COLL_EINVAL"), ({"down": (0, 64 * 64, 64)}, "COLL_EINVAL"),
       ({"up": (2 * A, -64 * 64, 64)}, "COLL_EINVAL"), ({"up": (2 * A, 1 << 50, 64)}, "COLL_EINVAL"),
       ({"x": NO}, "COLL_EINVAL"), ({"ids": NO}, "COLL_EINVAL"), ({"weights": NO}, "COLL_EINVAL"),
       ({"y": NO}, "COLL_EINVAL"), ({"y": (7 * A, 63, 1)}, "COLL_EINVAL"),
       ({"y": (7 * A, 64, 2)}, "COLL_EINVAL"), ({"up": (2 * A + 1, 64 * 64, 64)}, "COLL_EALIGN"),
       ({"x": (4 * A + 1, 64, 1)}, "COLL_EALIGN"), ({"ids": (5 * A + 2, 2, 1)}, "COLL_EALIGN"),
       ({"weights": (6 * A + 2, 2, 1)}, "COLL_EALIGN"), ({"status": 2}, "COLL_EALIGN"),
       ({"y": (4 * A, 64, 1)}, "COLL_EOVERLAP"), ({"y": (5 * A, 64, 1)}, "COLL_EOVERLAP"),
       ({"y": (6 * A, 64, 1)}, "COLL_EOVERLAP"), ({"y": (3 * A + 64, 64, 1)}, "COLL_EOVERLAP"),
       ({"res": (7 * A + 2, 64, 1)}, "COLL_EOVERLAP")]


@pytest.mark.parametrize("over,code", BAD)
def test_refusals(rt, over, code):
    v = call(5, 64, 64, 64, 4, 2, **over)
    assert rt.coll_gated_experts_workspace(pack(v)) == D[code]
    assert rt.coll_gated_experts(pack(v), None) == D[code]
    assert names(rt) == []


def test_null_and_workspace(rt):
    assert rt.coll_gated_experts(None, None) == D["COLL_EINVAL"]
    assert rt.coll_gated_experts_workspace(None) == D["COLL_EINVAL"]
    for v in (call(5, 64, 64, 64, 4, 2), call(50, 64, 64, 64, 4, 2)):
        need = rt.coll_gated_experts_workspace(pack(v, 0, 0))
        assert need > 0
        rt.fake_reset(-1)
        for ws, size in ((0, need), (8 * A, need - 1), (8 * A + 8, need), (8 * A, 0)):
            assert rt.coll_gated_experts(pack(v, ws, size), None) == D["COLL_EWORKSPACE"]
        assert names(rt) == []
        for ws in (8 * A, 8 * A + 16, 8 * A + 112):
            assert rt.coll_gated_experts(pack(v, ws, need), None) == _lib.OK
    for v in (call(0, 64, 64, 64, 4, 2), call(5, 0, 64, 64, 4, 2)):
        rt.fake_reset(-1)
        assert rt.coll_gated_experts_workspace(pack(v)) == 0
        assert rt.coll_gated_experts(pack(v, 0, 0), None) == _lib.OK and names(rt) == []


def test_residual_in_place_is_allowed(rt):
    assert run(rt, call(5, 64, 64, 64, 4, 2, res=(7 * A, 64, 1))) == _lib.OK


DIRECT = ["direct_inner", "direct_outer"]
CUT = ["product_kernelILb1E", "join_kernelILb1E", "product_kernelILb0E", "join_kernelILb0E"]


def test_what_a_call_launches(rt):
    for v, want in ((call(1, 2048, 2048, 176, 64, 6), DIRECT),
                    (call(5, 1001, 1001, 517, 20, 4), DIRECT),
                    (call(5, 64, 64, 64, 3, 2, off=2), DIRECT),
                    (call(1, 7168, 7168, 2048, 32, 8), DIRECT), (call(16, 4096, 4096, 1792, 8, 2), DIRECT),
                    (call(17, 4096, 4096, 14336, 8, 2), CUT),        # 34 choices
                    (call(5, 64, 64, 14336, 3, 2, x=(4 * A, 200, 3)), ["plan_kernel", CUT[0]] + CUT[2:]),
                    (call(9, 64, 64, 64, 3, 2), None),
                    (call(128, 4096, 4096, 14336, 8, 2), CUT),
                    (call(128, 4096, 4096, 14336, 8, 3), ["plan_kernel"] + CUT),  # 384 choices
                    # x off 16 bytes is laid out; inner tiles whole
                    (call(40, 1024, 1024, 14336, 8, 2, off=2), ["plan_kernel", CUT[0]] + CUT[2:]),
                    (call(300, 4096, 4096, 14336, 8, 2), CUT * 3),
                    (call(5, 64, 0, 64, 3, 2, x=(4 * A, 1, 1)), ["product_kernelILb0E"]),
                    (call(5, 64, 64, 0, 3, 2), ["product_kernelILb0E"])):
        assert run(rt, v) == _lib.OK
        got = names(rt)
        if want is not None:
            assert len(got) == len(want) and all(w in g for w, g in zip(want, got)), got
    # weights on 16 bytes go by tensor copies (the second template argument), others by loader warps
    for v, inner, outer in ((call(40, 64, 64, 14336, 8, 2), 1, 1),
                            (call(40, 64, 68, 14336, 8, 2), 0, 1),
                            (call(40, 64, 64, 14340, 8, 2), 1, 0),
                            (call(40, 64, 64, 14336, 8, 2, w_off=8), 0, 1),
                            (call(40, 64, 64, 14336, 8, 2, down=(3 * A, 0, 14336)), 1, 0)):
        assert run(rt, v) == _lib.OK
        got = [n for n in names(rt) if "product" in n]
        assert f"ILb1ELb{inner}E" in got[0] and f"ILb0ELb{outer}E" in got[1], got


@pytest.mark.parametrize("v", [call(50, 64, 64, 64, 4, 2), call(128, 64, 72, 328, 4, 8),
                               call(40, 64, 68, 64, 4, 2)], ids=["own", "planned", "loaders"])
def test_a_refused_tensor_map_or_set_up_stops_the_call_before_its_first_launch(rt, v):
    # the limits on shared memory are set at the first launch on a device, and kept
    rt.fake_fail_attributes(1)
    assert run(rt, v) == D["COLL_ECUDA"]
    assert names(rt) == []
    assert run(rt, v) == _lib.OK
    maps, all_of_it = rt.fake_maps(), names(rt)
    assert maps >= 3 and all_of_it
    for i in range(maps):
        assert run(rt, v, i) == D["COLL_EINVAL"]
        assert names(rt) == [], i
    assert run(rt, v) == _lib.OK and names(rt) == all_of_it


def test_every_shape_is_taken(rt):
    """Shapes, shared memory and grids stay within the device's limits (the fake runtime checks)."""
    for m in (1, 2, 8, 9, 16, 17, 32, 33, 64, 65, 127, 128, 129, 1000):
        for e, top in ((1, 1), (3, 2), (8, 8), (64, 6), (1024, 32)):
            for n, k, f in ((1, 1, 1), (8, 8, 8), (4096, 4096, 14336), (7168, 7168, 2048),
                            (333, 77, 129), (64, 16384, 8), (16384, 64, 16384)):
                v = call(m, n, k, f, e, min(top, 32))
                assert run(rt, v) == _lib.OK, (m, e, top, n, k, f)


def route(t, e, top, dtype=F32, score=0, norm=1, scale=1.0, logits=None, ids=None, w=None):
    return experts._ROUTE.pack(t, e, top, dtype, score, norm, scale, *(logits or (A, e, 1)),
                               *(ids or (2 * A, top, 1)), *(w or (3 * A, top, 1)))


def route_bwd(t, e, top, dtype=F32, score=0, norm=1, scale=1.0, dw=None, logits=None, ids=None,
              out=None):
    return experts._ROUTE_BWD.pack(t, e, top, dtype, score, norm, scale, *(dw or (4 * A, top, 1)),
                                   *(logits or (A, e, 1)), *(ids or (2 * A, top, 1)),
                                   *(out or (5 * A, e, 1)))


def test_route_refusals(rt):
    for fn, make in ((rt.coll_route, route), (rt.coll_route_backward, route_bwd)):
        assert fn(None, None) == D["COLL_EINVAL"]
        for bad in ((-1, 8, 2), (5, 8, 0), (5, 8, 9), (5, 1025, 2), (5, 64, 33), (1 << 40, 8, 2)):
            assert fn(make(*bad), None) == D["COLL_EINVAL"], bad
        for over in (dict(dtype=D["COLL_BYTES"]), dict(score=2), dict(norm=2),
                     dict(scale=float("inf")), dict(scale=float("nan")), dict(logits=(0, 8, 1)),
                     dict(ids=(0, 2, 1)), dict(logits=(A, 1 << 45, 1))):
            assert fn(make(5, 8, 2, **over), None) == D["COLL_EINVAL"], over
        assert fn(make(5, 8, 2, logits=(A + 2, 8, 1)), None) == D["COLL_EALIGN"]
        assert fn(make(5, 8, 2, ids=(2 * A + 1, 2, 1)), None) == D["COLL_EALIGN"]
        assert names(rt) == []
        assert fn(make(0, 8, 2), None) == _lib.OK and names(rt) == []
        assert fn(make(5, 8, 2), None) == _lib.OK and len(names(rt)) == 1
        rt.fake_reset(-1)
    assert rt.coll_route(route(5, 8, 2, ids=(A, 2, 1)), None) == D["COLL_EOVERLAP"]
    assert rt.coll_route(route(5, 8, 2, w=(2 * A, 2, 1)), None) == D["COLL_EOVERLAP"]
    assert rt.coll_route(route(5, 8, 2, ids=(2 * A, 1, 1)), None) == D["COLL_EINVAL"]
    assert rt.coll_route(route(5, 8, 2, w=(3 * A, 4, 2)), None) == D["COLL_EINVAL"]
    assert rt.coll_route_backward(route_bwd(5, 8, 2, out=(A, 8, 1)), None) == D["COLL_EOVERLAP"]
    assert rt.coll_route_backward(route_bwd(5, 8, 2, out=(5 * A, 7, 1)), None) == D["COLL_EINVAL"]
    assert rt.coll_route_backward(route_bwd(5, 8, 2, dw=(0, 2, 1)), None) == D["COLL_EINVAL"]
    assert names(rt) == []


class Machine:
    """Two devices, one of them current, and entry points that note where they are called."""

    def __init__(self, monkeypatch, current):
        self.current, self.calls = current, []

        @contextlib.contextmanager
        def device(d):
            before, self.current = self.current, d
            yield
            self.current = before

        class Library:
            def __getattr__(lib, name):
                return lambda packed, stream: self.calls.append((name, self.current, stream)) or 0

        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(dense, "_current_device", lambda: self.current)
        monkeypatch.setattr(dense, "_raw_stream", lambda d: 100 + d)
        monkeypatch.setattr(experts, "lib", Library)
        monkeypatch.setattr(experts, "_entries", {})


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("dev", [0, 1])
def test_the_router_runs_on_the_device_of_its_logits(monkeypatch, current, dev):
    m = Machine(monkeypatch, current)
    experts.Router(2)._launch("coll_route", b"", dev)
    assert m.calls == [("coll_route", dev, 100 + dev)] and m.current == current


class Stream:
    def __init__(self, dev):
        self.device_index = dev


def test_a_stream_of_another_device_is_refused(monkeypatch):
    m = Machine(monkeypatch, -1)  # where torch's CPU tensors are
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(experts.Router, "_logits", staticmethod(lambda t: -1))
    r, logits = experts.Router(2), torch.zeros(3, 8)
    ids, w = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    calls = [lambda s: r.forward(logits, stream=s), lambda s: r.backward(w, logits, ids, stream=s)]
    for c in calls:
        with pytest.raises(ValueError, match="stream"):
            c(Stream(1))
    assert m.calls == []
    for c in calls:
        c(Stream(-1))
    assert [n for n, _, _ in m.calls] == ["coll_route", "coll_route_backward"]


@pytest.mark.parametrize("code", [0, D["COLL_ECUDA"]])
@pytest.mark.parametrize("current", [0, 1])
def test_a_workspace_is_of_the_calls_device_and_stream_and_freed(monkeypatch, current, code):
    m, op = Machine(monkeypatch, current), object.__new__(experts.GatedExperts)
    op._start(torch.device("cpu"))
    op._dev = 1
    seen = []
    monkeypatch.setattr(experts, "_alloc", lambda n, s: seen.append((n, m.current, s)) or 5 * A)
    monkeypatch.setattr(experts, "_free", lambda p: seen.append(("free", p)))
    fields = (8, 256, 256, 128, 4, 0, 2, BF, BF, D["COLL_ACT_SILU"], A, 128 * 256, 256, 2 * A,
              128 * 256, 256, 3 * A, 256 * 128, 128, 4 * A, 256, 1, 5 * A, 2, 1, 6 * A, 2, 1, *NO,
              7 * A, 256, 1)

    def call(packed, stream):
        given = packed[-24:]
        if given[:16] == bytes(16):
            return D["COLL_EWORKSPACE"]
        seen.append((given, m.current, stream))
        return code

    monkeypatch.setattr(dense, "_entries", {"coll_gated_experts": (call, lambda packed: 4096)})
    for _ in range(2):
        seen.clear()
        with contextlib.nullcontext() if code == 0 else pytest.raises(_lib.CollError):
            op._launch("coll_gated_experts", experts._EXPERTS.pack, fields)
        given = np.array([5 * A, 4096, op._word], np.int64).tobytes()
        assert seen == [(4096, 1, 101), (given, 1, 101), ("free", 5 * A)]


def test_arguments_before_any_device_is_asked():
    w = torch.zeros(4, 8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        experts.GatedExperts(w, w, w.transpose(1, 2).contiguous())
    with pytest.raises(ValueError, match="three dimensions"):
        experts.GatedExperts(w[0], w, w)
    with pytest.raises(ValueError, match="CUDA"):
        experts.Router(2).forward(torch.zeros(3, 8))
    with pytest.raises(ValueError, match="top_k"):
        experts.Router(0)
    with pytest.raises(ValueError, match="score"):
        experts.Router(2, "max")


def test_choices_that_were_not_made_go_to_no_rank():
    """The router's table as moe_dispatch takes it: -1 ends the choices of a token with few experts."""
    routing = np.array([[[3, 0], [1, -1]], [[-1, -1], [2, 3]]], dtype=np.int32)
    nm = namings.moe_dispatch(routing, 2, 4)
    assert nm.meta["counts"] == [2, 2]
    assert nm.rows("out") == [(0, 0, 4, 0), (0, 4, 4, 1), (1, 0, 4, 0), (1, 4, 4, 3)]


def test_the_structures_are_as_long_as_the_header_says():
    assert experts._ROUTE.size == 16 * 8
    assert experts._ROUTE_BWD.size == 19 * 8
    assert experts._EXPERTS.size == 37 * 8
