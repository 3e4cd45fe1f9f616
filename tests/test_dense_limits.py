"""Sizes whose scratch no device holds, of inputs that take no memory (broadcast, stride 0), by the
argument check (no GPU: the addresses are made up)."""

import pytest

from collective_datapath_copy_gb300 import _lib, dense
from collective_datapath_copy_gb300.build import build
from test_dense_host import A, EALIGN, EINVAL, F32, gated, gated_bwd, linear, linear_bwd

NO = (0, 0, 0)
MOST = 0x7FFFFFFF - 4096


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def zero(i):
    return (i * A, 0, 0)


@pytest.mark.parametrize("m,n", [(MOST, MOST), (MOST, MOST // 2), (MOST // 2, MOST),
                                 (1 << 20, 1 << 21)])
def test_gradients_that_are_rounded_on_the_way(m, n):
    """dz, dg and du would take 2^42 bytes and more: 2^64 for the two of the largest."""
    kw = dict(m=m, n=n, k=1)
    wide = dict(x=zero(100), dx=(1000 * A, 1, 1))
    assert gated_bwd(dh=zero(1), gate=zero(2), up=zero(3), wg=zero(101), wu=zero(102),
                     dg=(2000 * A, 1, 1), du=(3000 * A, 1, 1), **wide, **kw) == EINVAL
    assert linear_bwd(act=1, dy=zero(1), pre=zero(2), w=zero(101), dw=(2000 * A, 1, 1), **wide,
                      **kw) == EINVAL


@pytest.mark.parametrize("m,k", [(MOST, MOST), (1 << 21, 1 << 21)])
def test_operands_that_are_laid_out(m, k):
    assert linear(m=m, n=8, k=k, x=zero(1), w=zero(2), y=(1000 * A, 8, 1)) == EINVAL
    assert linear(m=m, n=8, k=k, out=F32, x=zero(1), w=zero(2), y=(1000 * A, 8, 1)) == EINVAL
    assert gated(m=m, n=8, k=k, x=zero(1), wg=zero(2), wu=zero(3), h=(1000 * A, 8, 1)) == EINVAL


def test_large_scratch_that_a_device_might_hold():
    need = gated_bwd(m=1 << 17, n=1 << 17, k=8, dh=zero(1), gate=zero(2), up=zero(3),
                     dx=(1000 * A, 8, 1), dg=(2000 * A, 8, 1), du=(3000 * A, 8, 1))
    assert need >= 2 * (1 << 35)
    assert linear_bwd(m=1 << 17, n=1 << 17, k=8, act=1, dy=zero(1), pre=zero(2),
                      dx=(1000 * A, 8, 1), dw=(2000 * A, 8, 1)) >= 1 << 35


def test_a_status_word_is_four_bytes_on_four():
    """It is only written when a wait expires, where an odd address would fault."""
    vals = (8, 32, 64, 0, 0, 0, A, 64, 1, 2 * A, 64, 1, *NO, *NO, 3 * A, 32, 1, 0, 0)
    for off in (0, 4, 2, 1):
        got = _lib.lib().coll_linear_workspace(dense._LINEAR.pack(*vals, 0, 0, 4 * A + off))
        assert got == (EALIGN if off % 4 else 0)
