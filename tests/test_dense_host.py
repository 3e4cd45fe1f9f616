"""Host half of the dense operators: argument codes and workspace sizes, without a GPU.

The *_workspace entry points run every check of the call and touch no memory, so the addresses
below are made up."""

import pytest

from collective_datapath_copy_gb300 import _lib
from collective_datapath_copy_gb300.build import build

BF, F32, F16, BYTES = (_lib.D[k] for k in ("COLL_BF16", "COLL_F32", "COLL_F16", "COLL_BYTES"))
A = 1 << 32   # addresses far apart
NO = (0, 0, 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def pack(name, vals):
    from collective_datapath_copy_gb300 import dense
    return getattr(dense, name).pack(*vals, 0, 0, 0)


def linear(m=8, n=32, k=64, dtype=BF, out=None, act=0, x=None, w=None, res=NO, pre=NO, y=None,
           bias=0, bstride=1):
    vals = (m, n, k, dtype, dtype if out is None else out, act, *(x or (A, k, 1)),
            *(w or (2 * A, k, 1)), *res, *pre, *(y or (3 * A, n, 1)), bias, bstride)
    return _lib.lib().coll_linear_workspace(pack("_LINEAR", vals))


def linear_bwd(m=8, n=32, k=64, dtype=BF, gd=None, act=0, dy=None, pre=NO, x=None, w=None,
               dx=None, dw=None, db=0):
    vals = (m, n, k, dtype, dtype if gd is None else gd, act, *(dy or (A, n, 1)), *pre,
            *(x or (2 * A, k, 1)), *(w or (3 * A, k, 1)), *(dx or (4 * A, k, 1)),
            *(dw or (5 * A, k, 1)), db)
    return _lib.lib().coll_linear_backward_workspace(pack("_LINEAR_BWD", vals))


def gated(m=8, n=32, k=64, dtype=BF, act=4, x=None, wg=None, wu=None, gate=NO, up=NO, h=None):
    vals = (m, n, k, dtype, act, *(x or (A, k, 1)), *(wg or (2 * A, k, 1)),
            *(wu or (3 * A, k, 1)), *gate, *up, *(h or (4 * A, n, 1)))
    return _lib.lib().coll_gated_ffn_workspace(pack("_GATED", vals))


def gated_bwd(m=8, n=32, k=64, dtype=BF, gd=None, act=4, dh=None, gate=None, up=None, x=None,
              wg=None, wu=None, dx=None, dg=None, du=None):
    vals = (m, n, k, dtype, dtype if gd is None else gd, act, *(dh or (A, n, 1)),
            *(gate or (2 * A, n, 1)), *(up or (3 * A, n, 1)), *(x or (4 * A, k, 1)),
            *(wg or (5 * A, k, 1)), *(wu or (6 * A, k, 1)), *(dx or (7 * A, k, 1)),
            *(dg or (8 * A, k, 1)), *(du or (9 * A, k, 1)))
    return _lib.lib().coll_gated_ffn_backward_workspace(pack("_GATED_BWD", vals))


EINVAL, EALIGN, EOVERLAP = (_lib.D["COLL_" + c] for c in ("EINVAL", "EALIGN", "EOVERLAP"))


def test_plain_calls_pass():
    assert linear() >= 0 and gated() >= 0 and linear_bwd() >= 0
    assert gated_bwd() >= 2 * 8 * 32 * 2          # dg and du
    assert linear(out=F32) >= 0 and linear(dtype=F16) >= 0
    assert linear_bwd(act=2, pre=(6 * A, 32, 1)) >= 8 * 32 * 2   # dz


def test_null_arguments():
    for f in ("coll_linear", "coll_linear_backward", "coll_gated_ffn", "coll_gated_ffn_backward"):
        assert getattr(_lib.lib(), f)(None, None) == EINVAL
        assert getattr(_lib.lib(), f + "_workspace")(None) == EINVAL


@pytest.mark.parametrize("f", [linear, linear_bwd, gated, gated_bwd])
def test_sizes_and_types(f):
    for kw in (dict(m=-1), dict(n=-1), dict(k=-1), dict(m=1 << 31), dict(dtype=F32),
               dict(dtype=BYTES), dict(dtype=9), dict(act=9), dict(act=-1)):
        assert f(**kw) == EINVAL, kw
    for kw in (dict(m=0), dict(n=0), dict(k=0)):
        assert f(**kw) >= 0, kw


def test_activations_by_operator():
    assert linear(act=5) == EINVAL and linear_bwd(act=5, pre=(6 * A, 32, 1)) == EINVAL
    assert gated(act=0) == EINVAL and gated_bwd(act=0) == EINVAL
    assert gated(act=5) >= 0 and linear(act=4) >= 0


def test_output_types():
    assert linear(out=F16) == EINVAL and linear(out=BYTES) == EINVAL
    assert linear_bwd(gd=F32) >= 0 and linear_bwd(gd=F16) == EINVAL
    assert gated_bwd(gd=F32) >= 0 and gated_bwd(gd=7) == EINVAL


def test_missing_matrices():
    z = (0, 64, 1)
    assert linear(x=z) == EINVAL and linear(w=z) == EINVAL and linear(y=z) == EINVAL
    assert linear_bwd(dy=z) == EINVAL and linear_bwd(act=1) == EINVAL
    assert linear_bwd(x=z) == EINVAL and linear_bwd(x=z, dw=z) >= 0
    assert linear_bwd(w=z) == EINVAL and linear_bwd(w=z, dx=z) >= 0
    assert gated(wu=z) == EINVAL and gated(gate=(5 * A, 32, 1)) == EINVAL
    assert gated_bwd(gate=z) == EINVAL and gated_bwd(dg=z) == EINVAL
    assert gated_bwd(dg=z, du=z) >= 0
    assert linear(k=0, x=z, w=z) >= 0


def test_bases_and_strides():
    assert linear(x=(A + 1, 64, 1)) == EALIGN and linear(out=F32, y=(3 * A + 2, 32, 1)) == EALIGN
    assert linear(y=(3 * A, 31, 1)) == EINVAL          # rows overlap
    assert linear(y=(3 * A, 64, 2)) == EINVAL          # columns apart
    assert linear(m=1, y=(3 * A, 0, 1)) >= 0           # one row: its stride is not used
    assert linear(n=1, y=(3 * A, 5, 7)) >= 0
    assert linear(x=(A, 1 << 41, 1)) == EINVAL
    assert linear(x=(A, 0, 0)) >= 0                    # a broadcast input


def test_overlaps():
    y = (3 * A, 32, 1)
    assert linear(x=y, y=y) == EOVERLAP and linear(w=y) == EOVERLAP
    assert linear(res=y) >= 0                                     # in place
    assert linear(res=(3 * A, 0, 1)) == EOVERLAP                  # not the same view
    assert linear(res=(3 * A + 2, 32, 1)) == EOVERLAP
    assert linear(pre=y) == EOVERLAP and linear(bias=3 * A + 64) == EOVERLAP
    assert linear(pre=y, res=(4 * A, 32, 1)) == EOVERLAP
    # column slices of one buffer
    assert linear(x=(A, 128, 1), y=(A + 128, 128, 1)) >= 0
    assert linear(x=(A, 128, 1), y=(A + 126, 128, 1)) == EOVERLAP
    assert linear(x=(A + 64, 128, 1), y=(A, 128, 1)) >= 0
    assert linear(x=(A + 62, 128, 1), y=(A, 128, 1)) == EOVERLAP
    assert linear(x=(A, -64, 1), y=(A - 1024, 32, 1)) == EOVERLAP  # rows that go down
    assert gated(gate=(5 * A, 32, 1), up=(5 * A, 32, 1)) == EOVERLAP
    assert linear_bwd(dx=(5 * A, 64, 1)) == EOVERLAP and linear_bwd(db=5 * A) == EOVERLAP
    assert gated_bwd(du=(8 * A, 64, 1)) == EOVERLAP and gated_bwd(dx=(A, 64, 1)) == EOVERLAP


def test_a_missing_workspace_is_refused():
    from collective_datapath_copy_gb300 import dense
    vals = (8, 32, 64, BF, BF, 4, A, 32, 1, 2 * A, 32, 1, 3 * A, 32, 1, 4 * A, 64, 1, 5 * A, 64,
            1, 6 * A, 64, 1, 7 * A, 64, 1, 8 * A, 64, 1, 9 * A, 64, 1)
    need = _lib.lib().coll_gated_ffn_backward_workspace(dense._GATED_BWD.pack(*vals, 0, 0, 0))
    assert need > 0
    for ws, size in ((0, need), (10 * A, need - 1), (10 * A + 8, need)):
        assert _lib.lib().coll_gated_ffn_backward(
            dense._GATED_BWD.pack(*vals, ws, size, 0), None) == _lib.D["COLL_EWORKSPACE"]
