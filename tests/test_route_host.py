"""Router's refusals that need no GPU, beside those in test_experts_host."""

import pytest

import test_experts_host as host
from collective_datapath_copy_gb300 import _lib, experts
from test_experts_host import rt  # noqa: F401 (a fixture)

D = _lib.D
MOST = (2.0 - 2.0 ** -23) * 2.0 ** 127  # binary32's largest


@pytest.mark.parametrize("scale", [MOST * (1 + 2.0 ** -24), 1e39, -1e39, 1e308])
def test_a_scale_that_binary32_does_not_hold_is_refused(rt, scale):  # noqa: F811
    """It would be infinite, and every weight with it."""
    for fn, make in ((rt.coll_route, host.route), (rt.coll_route_backward, host.route_bwd)):
        assert fn(make(5, 8, 2, scale=scale), None) == D["COLL_EINVAL"]
    assert host.names(rt) == []
    with pytest.raises(ValueError, match="scale"):
        experts.Router(2, scale=scale)


@pytest.mark.parametrize("scale", [MOST, -MOST, 0.0, 2.0 ** -149, 1e-60])
def test_scales_that_it_holds_are_taken(rt, scale):  # noqa: F811
    for fn, make in ((rt.coll_route, host.route), (rt.coll_route_backward, host.route_bwd)):
        assert fn(make(5, 8, 2, scale=scale), None) == _lib.OK
    assert experts.Router(2, scale=scale).scale == scale
