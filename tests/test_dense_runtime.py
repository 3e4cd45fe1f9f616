"""What the dense operators ask of the CUDA runtime, over a fake one (no GPU)."""

import pytest

import fake_cuda
from collective_datapath_copy_gb300 import _lib, dense

BF = _lib.D["COLL_BF16"]
A = 1 << 32   # addresses far apart
NO = (0, 0, 0)


@pytest.fixture
def rt(tmp_path):
    h = fake_cuda.load(str(tmp_path))
    h.fake_reset(-1)
    return h


def linear(h, m, n, k):
    """A forward product of aligned rows."""
    vals = (m, n, k, BF, BF, 0, A, k, 1, 2 * A, k, 1, *NO, *NO, 3 * A, n, 1, 0, 0)
    need = h.coll_linear_workspace(dense._LINEAR.pack(*vals, 0, 0, 0))
    return h.coll_linear(dense._LINEAR.pack(*vals, 4 * A, need, 0), None)


def gated(h, m, n, k):
    vals = (m, n, k, BF, 4, A, k, 1, 2 * A, k, 1, 3 * A, k, 1, *NO, *NO, 4 * A, n, 1)
    need = h.coll_gated_ffn_workspace(dense._GATED.pack(*vals, 0, 0, 0))
    return h.coll_gated_ffn(dense._GATED.pack(*vals, 5 * A, need, 0), None)


# the pair kernel and the small-batch kernel, whose rings need the larger shared memory
@pytest.mark.parametrize("call", [linear, gated])
@pytest.mark.parametrize("m,n,k,kernel", [(512, 512, 512, "tc_kernel"),
                                          (48, 9728, 512, "skinny_kernel")])
def test_large_kernels_launch_on_every_device(rt, call, m, n, k, kernel):
    for dev in (0, 1, 0, 3):
        rt.fake_device(dev)
        assert call(rt, m, n, k) == _lib.OK, dev
    got = fake_cuda.launches(rt)
    assert [d for _, d in got] == [0, 1, 0, 3] and all(kernel in name for name, _ in got)
    assert rt.fake_attribute_calls() == 3      # once a device


@pytest.mark.parametrize("m,n,k", [(512, 512, 512), (48, 9728, 512)])
def test_a_failed_set_up_is_tried_again(rt, m, n, k):
    rt.fake_fail_attributes(1)
    assert linear(rt, m, n, k) == _lib.D["COLL_ECUDA"] and fake_cuda.launches(rt) == []
    assert linear(rt, m, n, k) == _lib.OK
