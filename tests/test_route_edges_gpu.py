"""Router at the edges of what it documents: gradients of choices that were not made, scores below
binary32's normal range."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import experts_ref as er  # noqa: E402

F32 = torch.float32
INF = float("inf")
KINDS = [("softmax", True, 1.0), ("softmax", False, 1.0), ("sigmoid", True, 2.5),
         ("sigmoid", False, 0.7)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("e,top", [(9, 6), (60, 4), (256, 8), (700, 20)])
@pytest.mark.parametrize("value", [float("nan"), INF, -INF])
def test_the_gradient_of_a_choice_that_was_not_made_is_unread(kind, e, top, value):
    """An id outside the experts has no part in the gradient, whatever stands in its place."""
    g = torch.Generator(device="cuda").manual_seed(e)
    logits = torch.randn(40, e, generator=g, device="cuda")
    logits[:, 3:] = torch.where(torch.rand(40, 1, generator=g, device="cuda") < 0.5,
                                logits[:, 3:], torch.full_like(logits[:, 3:], -INF))
    logits[7] = -INF
    r = cdc.Router(top, *kind)
    ids, w = r.forward(logits)
    assert bool((ids < 0).any())
    ids[5, 1] = e  # of another table
    dw = torch.randn(40, top, generator=g, device="cuda")
    out = (ids < 0) | (ids >= e)
    want = r.backward(torch.where(out, torch.zeros_like(dw), dw), logits, ids)
    got = r.backward(torch.where(out, torch.full_like(dw, value), dw), logits, ids)
    assert bool(want.isfinite().all())
    assert torch.equal(got, want)


def test_sigmoid_scores_below_the_normal_range():
    """Down to the last subnormal: a score is good to 2^-20 of itself or two steps of 2^-149."""
    logits = -torch.arange(80.0, 104.0, 0.25, device="cuda").repeat(4, 1)
    logits[1:] += torch.tensor([[0.1], [0.17], [-0.05]], device="cuda")
    r = cdc.Router(32, "sigmoid", False)
    ids, w = r.forward(logits)
    assert torch.equal(ids.long(), er.choose(logits, 32))
    for part in (logits[:, :32], logits[:, 32:64], logits[:, 64:]):
        ids, w = r.forward(part)
        s = torch.special.expit(torch.gather(part, 1, ids.long()).double())
        # a product by 1 and the rounding of a subnormal are below a step, expf good to two of them
        assert bool(((w.double() - s).abs() <= 2.0 ** -20 * s + 2 * 2.0 ** -149).all())
        # the slope s (1 - s) at -l and at l is the smaller of s and 1 - s
        for l in (part, -part):
            dl = torch.gather(r.backward(torch.ones_like(w), l, ids), 1, ids.long()).double()
            assert bool(((dl - s).abs() <= 2.0 ** -19 * s + 4 * 2.0 ** -149).all())


@pytest.mark.parametrize("normalize", [True, False])
def test_softmax_scores_below_the_normal_range(normalize):
    """The same for probabilities, next to one of nearly 1."""
    logits = torch.zeros(60, 32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    logits[:, 1:] = -84 - 20 * torch.rand(60, 31, generator=g, device="cuda")
    ids, w = cdc.Router(32, normalize=normalize).forward(logits)
    assert torch.equal(ids.long(), er.choose(logits, 32))
    p = torch.gather(torch.softmax(logits.double(), 1), 1, ids.long())
    assert bool(((w.double() - p).abs() <= 2.0 ** -20 * p + 2 * 2.0 ** -149).all())
