"""GatedExperts on the tensor cores where offsets pass 32 bits and sums are long: weights by tensor copies
and through loader warps, whose ring goes round many times."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300 import _lib  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import dense_ref as ref  # noqa: E402
import experts_ref as er  # noqa: E402

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def normal(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def routing(g, m, e, top):
    v, ids = torch.topk(torch.randn(m, e, generator=g, device="cuda"), top, dim=1)
    return ids.int(), torch.softmax(v, 1)


def test_rows_past_30_bits():
    """Rows of 2^30 elements and more, off 16 bytes, two tokens of 17 choices of the one expert: a k
    block's place in its row passes 31 bits."""
    k, n, m, top = 2 ** 30 + 2 ** 27 + 1, 24, 2, 17
    w = torch.zeros(1, 1, k, dtype=BF, device="cuda")
    x = torch.zeros(m, k, dtype=BF, device="cuda")
    # a few values, at the start, around 2^30 and at the end, and no others
    at = torch.tensor([0, 63, 64, 2 ** 29 + 7, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 65, 2 ** 30 + 2 ** 26 + 3,
                       k - 66, k - 2, k - 1], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    w[0, 0, at] = normal(g, len(at))
    x[:, at] = normal(g, m, len(at))
    wd = normal(g, 1, n, 1)
    op = cdc.GatedExperts(w, w, wd)
    ids = torch.zeros(m, top, dtype=torch.int32, device="cuda")
    s = torch.rand(m, top, generator=g, device="cuda")
    y = op.forward(x, ids, s)
    assert op.status() == _lib.OK
    want = er.experts(x[:, at], ids, s, w[:, :, at], w[:, :, at], wd, "silu", 0, None, BF)
    ref.assert_close(y, want, "y")
