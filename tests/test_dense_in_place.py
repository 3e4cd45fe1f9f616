"""What a dense call may write over, by its argument check (no GPU: the addresses are made up)."""

import pytest

from collective_datapath_copy_gb300.build import build
from test_dense_host import A, EOVERLAP, linear


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


Y = (3 * A, 64, 1)


def test_the_residual_may_be_the_output():
    assert linear(m=64, n=64, k=64, res=Y, y=Y) >= 0
    assert linear(m=64, n=64, k=64, x=Y, res=Y, y=(4 * A, 64, 1)) >= 0   # read twice


@pytest.mark.parametrize("also", [dict(x=Y), dict(w=Y), dict(bias=3 * A), dict(x=Y, w=Y)])
@pytest.mark.parametrize("m", [1, 64])
def test_no_other_input_may_be_the_output_beside_it(m, also):
    """y written over x, w or the bias while other rows still read them: y = x would be lost."""
    assert linear(m=m, n=64, k=64, res=Y, y=Y, **also) == EOVERLAP


def test_nor_one_of_another_width():
    assert linear(n=32, k=64, x=(3 * A, 64, 1), res=Y, y=Y) == EOVERLAP
