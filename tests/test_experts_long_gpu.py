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


@pytest.mark.parametrize("n,k", [(512, 8192), (8192, 512)])
@pytest.mark.parametrize("odd", [0, 1])
def test_stacks_past_32_bits(n, k, odd):
    """2^31 elements and more in gate and up, then in down; odd: rows that only loader warps bring."""
    E, f, m, k = 20, 14336 + odd, 20, k + odd
    wg = torch.zeros(E, f, k, dtype=BF, device="cuda")
    wu, wd = torch.zeros_like(wg), torch.zeros(E, n, f, dtype=BF, device="cuda")
    assert max(wg.numel(), wd.numel()) > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(n + odd)
    for e in (0, E - 1):
        for w in (wg, wu):
            w[e] = normal(g, f, k, scale=k ** -0.5)
        wd[e] = normal(g, n, f, scale=f ** -0.5)
    op = cdc.GatedExperts(wg, wu, wd)
    ids = torch.tensor([[0, E - 1], [E - 1, 5], [7, 3], [E - 1, 0]], dtype=torch.int32, device="cuda")
    ids = ids.repeat(m // 4, 1)
    x, s = normal(g, m, k), torch.rand(m, 2, generator=g, device="cuda")
    y = op.forward(x, ids, s)
    assert op.status() == _lib.OK
    at = torch.where(ids == 0, 0, torch.where(ids == E - 1, 1, -1)).int()  # the others' are zero
    rows = torch.tensor([0, E - 1], device="cuda")
    want = er.experts(x, at, s, wg[rows], wu[rows], wd[rows], "silu", 0, None, BF)
    ref.assert_close(y, want, "y")
    ref.assert_rms(y, want, BF, "y", 2.0)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m", [20, 32, 64, 128])  # 32, 64 and 128 columns
@pytest.mark.parametrize("n,k,f", [(2064, 8192, 4096), (2064, 4099, 2051), (259, 8200, 2049),
                                   (520, 4097, 8200)])
def test_long_sums(m, n, k, f, dtype):
    g = torch.Generator(device="cuda").manual_seed(m + k)
    E = 2
    wg, wu = (normal(g, E, f, k, dtype=dtype, scale=k ** -0.5) for _ in range(2))
    wd = normal(g, E, n, f, dtype=dtype, scale=f ** -0.5)
    op = cdc.GatedExperts(wg, wu, wd)
    ids, s = routing(g, m, E, 2)
    x, r = normal(g, m, k, dtype=dtype), normal(g, m, n, dtype=dtype)
    y = op.forward(x, ids, s, residual=r)
    assert op.status() == _lib.OK
    want = er.experts(x, ids, s, wg, wu, wd, "silu", 0, r, dtype)
    ref.assert_close(y, want, "y")
    ref.assert_rms(y, want, dtype, "y", 2.0)
