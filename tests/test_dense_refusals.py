"""A refused call has enqueued nothing, and what a call launches, over a fake CUDA runtime (no
GPU)."""

import pytest

import fake_cuda
from collective_datapath_copy_gb300 import _lib, dense

BF, F32 = _lib.D["COLL_BF16"], _lib.D["COLL_F32"]
A = 1 << 32
NO = (0, 0, 0)


@pytest.fixture
def rt(tmp_path):
    h = fake_cuda.load(str(tmp_path))
    h.fake_reset(-1)
    return h


def linear(m, n, k, off=0):
    return ("coll_linear", dense._LINEAR,
            (m, n, k, BF, BF, 2, A + off, k, 1, 2 * A, k, 1, *NO, *NO, 4 * A, n, 1, 0, 0))


def linear_bwd(m, n, k, off=0, act=4):
    return ("coll_linear_backward", dense._LINEAR_BWD,
            (m, n, k, BF, F32, act, A, n, 1, 2 * A, n, 1, 3 * A + off, k, 1, 4 * A, k, 1,
             5 * A, k, 1, 6 * A, k, 1, 7 * A))


def gated(m, n, k, off=0):
    return ("coll_gated_ffn", dense._GATED,
            (m, n, k, BF, 4, A + off, k, 1, 2 * A, k, 1, 3 * A, k, 1, *NO, *NO, 4 * A, n, 1))


def gated_bwd(m, n, k, off=0):
    return ("coll_gated_ffn_backward", dense._GATED_BWD,
            (m, n, k, BF, BF, 4, A, n, 1, 2 * A, n, 1, 3 * A, n, 1, 4 * A + off, k, 1, 5 * A, k, 1,
             6 * A, k, 1, 7 * A, k, 1, 8 * A, k, 1, 9 * A, k, 1))


def run(h, call, refused=-1):
    name, args, vals = call
    need = getattr(h, name + "_workspace")(args.pack(*vals, 0, 0, 0))
    assert need >= 0
    h.fake_reset(refused)
    return getattr(h, name)(args.pack(*vals, 16 * A, need, 0), None)


CALLS = [linear(512, 512, 512), linear(512, 512, 512, off=2), linear(20, 40, 9001),
         linear(48, 9728, 512), linear(48, 9728, 513), gated(300, 512, 256), gated(300, 512, 251),
         gated(48, 9728, 251), linear_bwd(300, 512, 256), linear_bwd(300, 511, 255, off=2),
         linear_bwd(300, 512, 256, act=0), gated_bwd(513, 512, 1000), gated_bwd(513, 271, 1001),
         gated_bwd(4000, 40, 24)]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: f"{c[0]}-{c[2][:3]}")
def test_a_refused_tensor_map_stops_the_call_before_its_first_launch(rt, call):
    assert run(rt, call) == _lib.OK
    maps, all_of_it = rt.fake_maps(), fake_cuda.launches(rt)
    assert maps >= 2 and all_of_it
    for i in range(maps):
        assert run(rt, call, i) == _lib.D["COLL_EINVAL"]
        assert fake_cuda.launches(rt) == [], i
    assert run(rt, call) == _lib.OK and fake_cuda.launches(rt) == all_of_it


@pytest.mark.parametrize("call", CALLS, ids=lambda c: f"{c[0]}-{c[2][:3]}")
def test_a_failed_set_up_stops_it_too(rt, call):
    rt.fake_fail_attributes(1)
    assert run(rt, call) == _lib.D["COLL_ECUDA"]
    assert fake_cuda.launches(rt) == []


def names(h):
    return [n for n, _ in fake_cuda.launches(h)]


def test_what_a_call_launches(rt):
    for call, want in ((linear(1, 512, 512), ["gemv_kernel"]),
                       (linear(512, 512, 512), ["tc_kernel"]),
                       (linear(512, 512, 512, off=2), ["pack_kernel", "tc_kernel"]),
                       (linear(20, 40, 9001), ["pack_kernel", "tc_kernel", "share_join_kernel"]),
                       (linear(512, 512, 0), ["empty_sum_kernel"]), (linear(0, 512, 512), []),
                       (gated(48, 9728, 251), ["pack_kernel", "skinny_kernel"]),
                       (linear_bwd(300, 512, 256), ["act_bwd_kernel", "tc_kernel"]),
                       (linear_bwd(300, 512, 0), ["act_bwd_kernel", "join_kernel"]),
                       (linear_bwd(0, 512, 256), ["empty_sum_kernel", "act_bwd_kernel"]),
                       (gated_bwd(300, 0, 256), ["empty_sum_kernel"])):
        assert run(rt, call) == _lib.OK
        got = names(rt)
        assert len(got) == len(want) and all(w in g for w, g in zip(want, got)), (call[0], got)
