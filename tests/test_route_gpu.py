"""The router's choice and its gradient on the GPU, against 64-bit references (experts_ref has the
bounds)."""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import dense_ref as ref  # noqa: E402
import experts_ref as er  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    yield
    torch.cuda.synchronize()


def draw(seed, t, e, dtype, scale=1.5, layout="rows"):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)
    if layout == "rows":
        return make(t, e)
    if layout == "slice":
        return make(t, e + 5)[:, 3:3 + e]
    if layout == "cols":
        return make(e, t).t()
    if layout == "every2":
        return make(2 * t, 3 * e)[::2, ::3]
    if layout == "row0":
        return make(1, e).expand(t, e)
    raise KeyError(layout)


def check_forward(logits, top, score, normalize, scale):
    r = cdc.Router(top, score, normalize, scale)
    t = logits.shape[0]
    # outputs inside larger buffers, whose rest has to stay
    ids = torch.full((t + 2, top + 3), -7, dtype=torch.int32, device="cuda")
    w = torch.full((t + 2, top + 3), -7.0, device="cuda")
    r.forward(logits, ids=ids[1:1 + t, 1:1 + top], weights=w[1:1 + t, 1:1 + top])
    got, gw = ids[1:1 + t, 1:1 + top].clone(), w[1:1 + t, 1:1 + top].clone()
    ids[1:1 + t, 1:1 + top] = -7
    w[1:1 + t, 1:1 + top] = -7
    assert bool((ids == -7).all()) and bool((w == -7).all())
    want, ww = er.route(logits, top, score, normalize, scale)
    assert torch.equal(got.long(), want.long())
    ref.assert_close(gw, ww, "weights")
    return got, gw


def check_backward(logits, ids, score, normalize, scale, seed=0):
    t, top = ids.shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    dw = torch.randn(t, top, generator=g, device="cuda")
    r = cdc.Router(top, score, normalize, scale)
    buf = torch.full((t + 2, logits.shape[1] + 5), -7.0, dtype=logits.dtype, device="cuda")
    out = buf[1:1 + t, 3:3 + logits.shape[1]]
    r.backward(dw, logits, ids, dlogits=out)
    got = out.clone()
    ref.assert_close(got, er.route_bwd(dw, logits, ids, score, normalize, scale), "dlogits")
    out.fill_(-7)
    assert bool((buf == -7).all())


SIZES = [(1, 1, 1), (1, 8, 2), (1, 256, 8), (3, 5, 5), (7, 31, 4), (8, 32, 32), (9, 33, 3),
         (64, 60, 6), (65, 64, 8), (100, 65, 1), (33, 127, 9), (257, 128, 4), (1000, 160, 6),
         (1001, 256, 8), (5, 257, 10), (64, 384, 32), (31, 512, 8), (17, 513, 2), (40, 1000, 22),
         (129, 1024, 8)]
KINDS = [("softmax", True, 1.0), ("softmax", False, 1.0), ("sigmoid", True, 2.5),
         ("sigmoid", False, 0.7)]


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)))
@pytest.mark.parametrize("kind", KINDS)
def test_sizes(i, size, kind):
    t, e, top = size
    for dtype in (F32, (BF, HF)[i % 2]):
        logits = draw(i, t, e, dtype)
        ids, _ = check_forward(logits, top, *kind)
        check_backward(logits, ids, *kind, seed=i)


@pytest.mark.parametrize("layout", ["slice", "cols", "every2", "row0"])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("e", [60, 256])
def test_layouts(layout, dtype, e):
    logits = draw(3, 77, e, dtype, layout=layout)
    for kind in KINDS:
        ids, _ = check_forward(logits, 6, *kind)
        check_backward(logits, ids, *kind)


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("kind", KINDS)
def test_ties_go_to_the_lowest_index(dtype, kind):
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randint(-2, 3, (300, 200), generator=g, device="cuda").to(dtype)
    logits = torch.where((logits == 0) & (torch.rand(300, 200, generator=g, device="cuda") < 0.5),
                         -logits, logits)  # both zeros
    ids, _ = check_forward(logits, 12, *kind)
    check_backward(logits, ids, *kind)
    same = torch.zeros(4, 77, dtype=dtype, device="cuda")
    ids, w = check_forward(same, 8, *kind)
    assert torch.equal(ids, torch.arange(8, device="cuda", dtype=torch.int32).expand(4, 8))


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("kind", KINDS)
def test_masked(dtype, kind):
    logits = draw(5, 64, 100, dtype)
    low = torch.finfo(dtype).min
    for row in range(64):  # 0 .. 12 experts left, the others -inf or the type's lowest value
        logits[row, (row % 13):] = -INF if row % 2 else low
    logits[0] = -INF
    ids, w = check_forward(logits, 8, *kind)
    assert bool((ids[0] == -1).all()) and bool((w[0] == 0).all())
    check_backward(logits, ids, *kind)


@pytest.mark.parametrize("kind", KINDS)
def test_far_logits(kind):
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn(200, 64, generator=g, device="cuda") * 40
    logits[:50] -= 500     # every sigmoid far below binary32's range
    logits[50:100] += 500
    logits[100:110] = torch.finfo(F32).min
    logits[110:120, 5] = torch.finfo(F32).max
    ids, _ = check_forward(logits, 6, *kind)
    check_backward(logits, ids, *kind)


@pytest.mark.parametrize("kind", KINDS)
def test_nan_and_infinity(kind):
    logits = draw(6, 6, 40, F32)
    logits[1, 7] = float("nan")
    logits[2, 9] = -float("nan")
    logits[2, 30] = INF
    logits[3, 4] = INF
    r = cdc.Router(4, *kind)
    ids, w = r.forward(logits)
    assert torch.equal(ids.long(), er.choose(logits, 4))
    assert [int(ids[i, 0]) for i in (1, 2, 3)] == [7, 9, 4] and int(ids[2, 1]) == 30
    clean = torch.tensor([0, 4, 5], device="cuda")
    want = er.weights(logits[clean], ids[clean].long(), kind[0], kind[1])[0] * kind[2]
    assert torch.allclose(w[clean].double(), want, rtol=1e-5)
    assert bool(w[1, 0].isnan()) and bool(w[2, 0].isnan())
    if kind[0] == "softmax" or kind[1]:
        assert bool(w[1].isnan().all()) and bool(w[2].isnan().all())
    dl = r.backward(torch.ones_like(w), logits, ids)
    assert bool(dl[clean].isfinite().all())


@pytest.mark.parametrize("e", [100, 256, 500, 1000])
@pytest.mark.parametrize("kind", KINDS)
def test_odd_rows_among_many_experts(kind, e):
    """NaN, infinities, equal leaders and zeros of both signs between ordinary rows."""
    logits = draw(8, 3000, e, F32)
    places = torch.randperm(e, generator=torch.Generator().manual_seed(e))[:12].cuda()
    ties = torch.arange(0, 3000, 7, device="cuda")
    logits[ties[:, None], places] = torch.tensor([9.0, 8.0, 9.0, 7.0, 9.0, 8.0] * 2, device="cuda")
    zeros = ties[:-1] + 1
    logits[zeros] = -logits[zeros].abs() - 1
    logits[zeros[:, None], places] = torch.tensor([0.0, -0.0] * 6, device="cuda")
    high = ties[:-1] + 2
    logits[high] = -INF
    logits[high[:, None], places[:5]] = torch.arange(5.0, device="cuda")
    check_forward(logits, 8, *kind)
    nan = ties[:-1] + 3
    logits[nan, places[0]] = -float("nan")
    logits[nan[::2], places[1]] = INF
    logits[nan[1::2], places[2]] = float("nan")
    logits[ties[:-1] + 4, places[3]] = INF
    r = cdc.Router(8, *kind)
    ids, w = r.forward(logits)
    assert torch.equal(ids.long(), er.choose(logits, 8))
    assert bool(w[nan, 0].isnan().all())


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("e", [40, 128, 256, 1000])
def test_subnormal_logits(dtype, e):
    tiny = torch.finfo(dtype).smallest_normal
    g = torch.Generator(device="cuda").manual_seed(e)
    logits = (torch.randn(200, e, generator=g, device="cuda") * (tiny / 4)).to(dtype)
    logits[100:] = -logits[100:].abs()
    assert bool((logits != 0).any()) and float(logits.abs().max()) < 2 * tiny
    for kind in KINDS:
        ids, _ = check_forward(logits, 8, *kind)
        check_backward(logits, ids, *kind)


@pytest.mark.parametrize("normalize", [True, False])
def test_sigmoids_around_where_their_logarithms_are_taken(normalize):
    rows = [[-58.0, -59.5, -60.0, -60.5], [-59.9, -59.99, -59.0, -59.5], [0.0, -59.9, 3.0, -60.1],
            [-61.0, -88.0, -104.0, -120.0], [20.0, -100.0, -1.0, -59.0], [90.0, 100.0, -59.0, 0.5]]
    logits = torch.tensor(rows, device="cuda").repeat(1, 20) - torch.arange(80, device="cuda") * 1e-3
    ids, _ = check_forward(logits, 6, "sigmoid", normalize, 1.0)
    check_backward(logits, ids, "sigmoid", normalize, 1.0)
    ids, _ = check_forward(logits, 32, "sigmoid", normalize, 1.0)
    check_backward(logits, ids, "sigmoid", normalize, 1.0)


def test_backward_takes_any_ids():
    """Out of order, outside the experts, the same one twice."""
    logits = draw(7, 50, 33, F32)
    g = torch.Generator(device="cuda").manual_seed(7)
    ids = torch.randint(-3, 36, (50, 10), generator=g, device="cuda", dtype=torch.int32)
    ids[3] = 5
    ids[4] = -1
    for kind in KINDS:
        check_backward(logits, ids, *kind)
    wide = torch.full((50, 20), -9, dtype=torch.int32, device="cuda")
    wide[:, ::2] = ids
    check_backward(logits, wide[:, ::2], *KINDS[0])


@pytest.mark.parametrize("kind", KINDS)
def test_gradient_against_differences(kind):
    score, normalize, scale = kind
    g = torch.Generator(device="cuda").manual_seed(8)
    logits = torch.randn(5, 12, generator=g, device="cuda")
    dw = torch.randn(5, 4, generator=g, device="cuda")
    r = cdc.Router(4, score, normalize, scale)
    ids, _ = r.forward(logits)
    got = r.backward(dw, logits, ids).double()

    def loss(l):  # the weights of the same choice, in 64 bits
        return (er.weights(l, ids.long(), score, normalize)[0] * scale * dw.double()).sum(1)

    step = 2.0 ** -16
    for e in range(12):
        d = torch.zeros(5, 12, dtype=torch.float64, device="cuda")
        d[:, e] = step
        l = logits.double()
        slope = (loss(l + d) - loss(l - d)) / (2 * step)
        # the third derivative is below 8 of the gradient's size, the products' rounding 2^-19
        assert float((got[:, e] - slope).abs().max()) <= (8 * step ** 2 + 2.0 ** -19) * float(
            dw.abs().sum(1).max()) * scale


def test_leading_dimensions_and_empty():
    logits = draw(9, 24, 16, BF)
    r = cdc.Router(3)
    ids, w = r.forward(logits)
    i3, w3 = r.forward(logits.view(2, 3, 4, 16))
    assert i3.shape == (2, 3, 4, 3) and torch.equal(i3.view(24, 3), ids)
    assert torch.equal(w3.view(24, 3), w)
    dw = torch.ones(2, 3, 4, 3, device="cuda")
    d3 = r.backward(dw, logits.view(2, 3, 4, 16), i3)
    assert torch.equal(d3.view(24, 16), r.backward(dw.view(24, 3), logits, ids))
    i1, _ = r.forward(logits[0])
    assert i1.shape == (3,) and torch.equal(i1, ids[0])
    ids0, w0 = r.forward(logits[:0])
    assert ids0.shape == (0, 3) and r.backward(w0, logits[:0], ids0).shape == (0, 16)


def test_rows_past_32_bits():
    t, e = 4_300_000, 1024  # 2^32 elements and more
    logits = torch.zeros(t, e, dtype=BF, device="cuda")
    logits[-1, 77] = 3
    logits[-2, 1023] = 2
    r = cdc.Router(2)
    ids, w = r.forward(logits)
    assert ids[-1].tolist() == [77, 0] and ids[-2].tolist() == [1023, 0]
    assert ids[0].tolist() == [0, 1]
    dl = r.backward(torch.ones_like(w) * torch.tensor([1.0, 0.0], device="cuda"), logits, ids)
    want = float(w[-1, 0] * w[-1, 1])
    assert abs(float(dl[-1, 77]) - want) <= want * 2 ** -7
    assert float(dl[-1].abs().sum()) <= 2.02 * want


def test_graph_and_streams():
    logits = draw(10, 300, 64, F32)
    r = cdc.Router(4, "sigmoid", True, 2.5)
    ids, w = r.forward(logits)
    dw = torch.randn_like(w)
    dl = r.backward(dw, logits, ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    i2, w2 = r.forward(logits, stream=side)
    d2 = r.backward(dw, logits, i2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(ids, i2) and torch.equal(w, w2) and torch.equal(dl, d2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        i3, w3 = r.forward(logits)
        d3 = r.backward(dw, logits, i3)
    logits.copy_(draw(11, 300, 64, F32))
    graph.replay()
    graph.replay()
    ids, w = r.forward(logits)
    assert torch.equal(ids, i3) and torch.equal(w, w3)
    assert torch.equal(r.backward(dw, logits, ids), d3)


def test_refusals():
    logits = draw(12, 4, 16, F32)
    for args in ((0,), (33,), (2, "tanh"), (2, "softmax", True, INF)):
        with pytest.raises(ValueError):
            cdc.Router(*args)
    r = cdc.Router(4)
    ids, w = r.forward(logits)
    bad = [lambda: r.forward(logits.double()), lambda: r.forward(logits.cpu()),
           lambda: r.forward(logits, ids=ids.long()), lambda: r.forward(logits, ids=ids[:2]),
           lambda: r.forward(logits, weights=w.half()), lambda: r.forward(torch.tensor(1.0).cuda()),
           lambda: r.backward(w[:, :3], logits, ids), lambda: r.backward(w, logits, ids.long()),
           lambda: r.backward(w, logits, ids, dlogits=logits.half())]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(cdc.CollError):
        r.forward(logits[:, :3])                          # fewer experts than are chosen
    with pytest.raises(cdc.CollError):
        r.forward(draw(12, 1, 1025, F32))
    with pytest.raises(cdc.CollError):
        r.backward(w, logits, ids, dlogits=logits)        # over its input
