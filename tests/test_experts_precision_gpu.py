"""GatedExperts keeps its inner values to twice their type's bits: in binary32 the result shows it, in
the operands' type it is off by little more than its own rounding."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300 import _lib  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import experts_ref as er  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
# A pair of numbers is off by 2^-16 (bf16) or 2^-22 (f16) of the value; the activation is good to 2^-19 of
# its argument and the sums to 2^-22 of their terms: twice the larger for bf16, four times for f16.
BOUND = {BF: 2.0 ** -15, HF: 2.0 ** -17}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    yield
    torch.cuda.synchronize()


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# tokens, outputs, inputs, inner features, experts, chosen: few choices of an expert and more than four,
# then 16 to 128 columns; rows on 16, 4 and 2 bytes; sums long enough that their tiles are cut
SIZES = [(1, 256, 256, 176, 8, 2), (1, 2048, 2048, 176, 64, 6), (8, 264, 264, 200, 2, 1),
         (16, 512, 512, 256, 2, 2), (5, 258, 258, 178, 3, 2), (16, 129, 257, 177, 2, 2),
         (16, 512, 256, 512, 8, 4), (32, 1024, 512, 1024, 8, 2), (64, 520, 264, 2056, 8, 2),
         (128, 512, 256, 1024, 2, 2), (128, 129, 257, 1025, 2, 2), (100, 1000, 136, 520, 64, 4),
         (300, 256, 128, 136, 16, 4), (40, 64, 64, 8192, 4, 2)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("size", SIZES)
def test_inner_values_keep_twice_their_types_bits(size, dtype, act):
    m, n, k, f, E, top = size
    g = torch.Generator(device="cuda").manual_seed(m + n)
    wg, wu = (normal(g, E, f, k, dtype=dtype, scale=k ** -0.5) for _ in range(2))
    wd = normal(g, E, n, f, dtype=dtype, scale=f ** -0.5)
    v, ids = torch.topk(normal(g, m, E), top, dim=1)
    ids, w = ids.int(), torch.softmax(v, 1)
    x = normal(g, m, k, dtype=dtype)
    op = cdc.GatedExperts(wg, wu, wd, act=act)
    want, _ = er.experts(x, ids, w, wg, wu, wd, act, 0, None, F32)
    size = float(want.square().mean().sqrt())

    def off(y):
        return float((y.double() - want).square().mean().sqrt()) / size
    assert off(op.forward(x, ids, w, out_dtype=F32)) <= BOUND[dtype]
    # rounded to nearest, nothing comes closer than want itself rounded
    assert off(op.forward(x, ids, w)) <= off(want.to(dtype)) + BOUND[dtype]
    assert op.status() == _lib.OK


@pytest.mark.parametrize("m", [1, 6, 40])
def test_inner_values_past_their_types_range_are_infinite(m):
    """One past 65504 in float16: that value's outputs are infinite and no NaN, the others' untouched."""
    g = torch.Generator(device="cuda").manual_seed(m)
    E, k, f, n = 2, 64, 24, 40
    wg, wu = (normal(g, E, f, k, dtype=HF, scale=k ** -0.5) for _ in range(2))
    wd = normal(g, E, n, f, dtype=HF, scale=f ** -0.5)
    ids = torch.zeros(m, 2, dtype=torch.int32, device="cuda")
    ids[:, 1] = -1
    w, x = torch.ones(m, 2, device="cuda"), normal(g, m, k, dtype=HF)
    op = cdc.GatedExperts(wg, wu, wd, act="relu")
    clean = op.forward(x, ids, w).clone()
    x[m // 2] = 2000 * (wg[0, 3].float() + wu[0, 3].float()).to(HF)
    h = torch.relu(x[m // 2].double() @ wg[0].double().t()) * (x[m // 2].double() @ wu[0].double().t())
    far = h.abs() > 65520  # where the nearest number of the type is infinite
    assert bool(far[3]) and not bool(((h.abs() > 65000) & ~far).any())
    signs = torch.sign(wd[0].double() * torch.where(far, h, torch.zeros_like(h)))
    y = op.forward(x, ids, w)
    rows = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(y[rows], clean[rows])
    plus, minus = (signs > 0).any(1), (signs < 0).any(1)
    assert torch.equal(y[m // 2] == float("inf"), plus & ~minus)
    assert torch.equal(y[m // 2] == -float("inf"), minus & ~plus)
