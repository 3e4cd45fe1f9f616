"""GatedExperts on the GPU against 64-bit references (experts_ref has the bounds). Every output is
a view of a larger buffer filled with a canary, which has to survive."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300 import _lib  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import dense_ref as ref  # noqa: E402
import experts_ref as er  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")
CANARY = -77.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def stacks(g, E, n, k, f, dtype):
    return (normal(g, E, f, k, dtype=dtype, scale=k ** -0.5),
            normal(g, E, f, k, dtype=dtype, scale=k ** -0.5),
            normal(g, E, n, f, dtype=dtype, scale=f ** -0.5))


def routing(g, m, e, top):
    v, ids = torch.topk(normal(g, m, e), top, dim=1)
    return ids.int(), torch.softmax(v, 1)


class Out:
    def __init__(self, rows, cols, dtype, slack=0, shift=0):
        self.buf = torch.full((rows + 2, cols + slack + 8), CANARY, dtype=dtype, device="cuda")
        self.shift = shift
        self.v = self.buf[1:1 + rows, shift:shift + cols]
        self.v.fill_(float("nan"))

    def untouched(self):
        b = self.buf.clone()
        b[1:1 + self.v.shape[0], self.shift:self.shift + self.v.shape[1]] = CANARY
        return bool((b == CANARY).all())


def check(op, x, ids, w, residual=None, out_dtype=None, slack=0, shift=0, rms=True):
    wg, wu, wd = op.w_gate, op.w_up, op.w_down
    ot = out_dtype or wg.dtype
    y = Out(x.shape[0], wd.shape[1], ot, slack, shift)
    op.forward(x, ids, w, residual=residual, out=y.v)
    want = er.experts(x, ids, w, wg, wu, wd, op.act, op.first, residual, ot)
    ref.assert_close(y.v, want, "y")
    if rms:  # the inner rounding, and that of the output
        ref.assert_rms(y.v, want, wg.dtype, "y", 2.0)
    assert y.untouched()
    assert op.status() == _lib.OK
    return y.v


# tokens, outputs, inputs, inner features, experts, chosen
SIZES = [(1, 1, 1, 1, 1, 1), (1, 64, 64, 64, 1, 1), (1, 512, 512, 176, 8, 2),
         (1, 2048, 2048, 176, 64, 6), (2, 100, 264, 40, 4, 2), (3, 130, 72, 136, 5, 5),
         (4, 4096, 1024, 96, 8, 2), (5, 128, 128, 128, 16, 4), (8, 264, 1032, 72, 3, 1),
         (13, 256, 520, 200, 20, 3), (16, 384, 256, 640, 8, 8), (17, 128, 64, 128, 2, 1),
         (31, 72, 136, 88, 32, 4), (33, 1000, 328, 264, 7, 2), (37, 1001, 1001, 517, 20, 4),
         (64, 512, 512, 256, 8, 2), (65, 77, 33, 51, 6, 3), (100, 136, 192, 1288, 4, 2),
         (127, 520, 64, 64, 64, 8), (128, 256, 512, 384, 8, 2), (128, 64, 64, 72, 128, 8),
         (129, 128, 136, 72, 8, 2), (300, 256, 128, 136, 16, 4), (6, 3, 7, 5, 2, 2),
         (1, 128, 8192, 64, 4, 1), (2, 64, 64, 8192, 4, 2), (7, 257, 255, 511, 9, 3)]


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)))
@pytest.mark.parametrize("dtype", [BF, HF])
def test_sizes(i, size, dtype):
    m, n, k, f, E, top = size
    g = gen(i)
    op = cdc.GatedExperts(*stacks(g, E, n, k, f, dtype), act=ACTS[i % 5])
    ids, w = routing(g, m, E, top)
    x = normal(g, m, k, dtype=dtype)
    ot = F32 if i % 4 == 3 else dtype
    r = normal(g, m, n, dtype=ot) if i % 3 else None
    slack, shift = ((-n % 8, 0), (3, 1), (5, 0))[i % 3]
    check(op, x, ids, w, r, ot, slack, shift)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("size", [(1, 136, 128, 72), (40, 264, 200, 136), (150, 72, 136, 64)])
@pytest.mark.parametrize("layout", ["slice8", "slice3", "cols", "every2", "row0"])
def test_layouts(dtype, size, layout):
    m, n, k, f = size
    g = gen(m)
    if layout == "slice8":
        x = normal(g, m, k + 16, dtype=dtype)[:, 8:8 + k]
    elif layout == "slice3":
        x = normal(g, m, k + 5, dtype=dtype)[:, 3:3 + k]
    elif layout == "cols":
        x = normal(g, k, m, dtype=dtype).t()
    elif layout == "every2":
        x = normal(g, 2 * m, 3 * k, dtype=dtype)[::2, ::3]
    else:
        x = normal(g, 1, k, dtype=dtype).expand(m, k)
    # gate and up in one buffer; down a slice; ids and weights of a wider table, by column
    both = normal(g, 6, 2 * f, k, dtype=dtype, scale=k ** -0.5)
    down = normal(g, 6, n + 3, f + 8, dtype=dtype, scale=f ** -0.5)[:, 1:1 + n, :f]
    op = cdc.GatedExperts(both[:, :f], both[:, f:], down)
    ids, w = routing(g, m, 6, 3)
    ids = ids.t().contiguous().t()
    w = w.repeat_interleave(2, 1)[:, ::2]
    r = normal(g, n, m, dtype=dtype).t()
    check(op, x, ids, w, r)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("off", [(0, 1), (1, 0), (4, 8), (8, 2)])
def test_weights_off_alignment(dtype, off):
    """Rows and bases of the stacks on 2, 4, 8 and 16 bytes."""
    base, pad = off
    g = gen(base + pad)
    m, n, k, f, E = 20, 136, 264, 72, 5

    def stack(rows, cols):
        w = normal(g, E, rows, cols + pad, dtype=dtype, scale=cols ** -0.5)
        flat = torch.cat([torch.zeros(base, dtype=dtype, device="cuda"), w.reshape(-1)])
        return flat[base:].view(E, rows, cols + pad)[:, :, :cols]
    op = cdc.GatedExperts(stack(f, k), stack(f, k), stack(n, f))
    for m in (1, 20):
        ids, w = routing(g, m, E, 2)
        check(op, normal(g, m, k, dtype=dtype), ids, w)


def test_order_of_experts_and_rows_in_memory():
    """[F, E, K] seen as [E, F, K], and one expert for all."""
    g = gen(3)
    wg, wu = (normal(g, 72, 6, 128, dtype=BF, scale=0.1).transpose(0, 1) for _ in range(2))
    wd = normal(g, 1, 136, 72, dtype=BF, scale=0.1).expand(6, 136, 72)
    op = cdc.GatedExperts(wg, wu, wd)
    ids, w = routing(g, 30, 6, 2)
    check(op, normal(g, 30, 128, dtype=BF), ids, w)


@pytest.mark.parametrize("m", [1, 19, 140])
def test_other_ranks_experts(m):
    g = gen(m)
    E, e, top = 32, 8, 4
    wg, wu, wd = stacks(g, E, 136, 128, 72, BF)
    x, (ids, w) = normal(g, m, 128, dtype=BF), routing(g, m, E, top)
    whole = torch.zeros(m, 136, dtype=torch.float64, device="cuda")
    for r in range(E // e):
        s = slice(r * e, (r + 1) * e)
        op = cdc.GatedExperts(wg[s], wu[s], wd[s], first=r * e)
        whole += check(op, x, ids, w, out_dtype=F32, rms=False).double()
    want, bound = er.experts(x, ids, w, wg, wu, wd, "silu", 0, None, F32)
    ref.assert_close(whole, (want, bound * 2), "ranks")


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m", [1, 37, 200])
def test_tokens_without_an_expert(m, residual):
    g = gen(4)
    op = cdc.GatedExperts(*stacks(g, 4, 200, 64, 72, BF), first=10)
    x = normal(g, m, 64, dtype=BF)
    r = normal(g, m, 200, dtype=BF) if residual else None
    w = torch.rand(m, 3, generator=g, device="cuda")
    w[:, 0] = float("nan")  # of an expert that is not here: unread
    for ids in (-1, 9, 14, -2 ** 31, 2 ** 31 - 1):
        i = torch.full((m, 3), ids, dtype=torch.int32, device="cuda")
        y = check(op, x, i, w, r)
        assert torch.equal(y, r if residual else torch.zeros_like(y))
    i = torch.full((m, 3), -1, dtype=torch.int32, device="cuda")
    i[m // 2, 1] = 12  # one choice in all
    check(op, x, i, w, r, rms=False)


@pytest.mark.parametrize("m,top", [(1, 4), (40, 4), (128, 2), (128, 32), (260, 3)])
def test_all_choose_the_same(m, top):
    """Every token one expert, and the same expert more than once."""
    g = gen(m)
    op = cdc.GatedExperts(*stacks(g, 5, 136, 128, 72, BF))
    x = normal(g, m, 128, dtype=BF)
    w = normal(g, m, top)
    check(op, x, torch.full((m, top), 3, dtype=torch.int32, device="cuda"), w)
    ids = torch.full((m, top), 3, dtype=torch.int32, device="cuda")
    ids[:, 0] = 1
    check(op, x, ids, w)


@pytest.mark.parametrize("k,f", [(128, 72), (131, 75)])
@pytest.mark.parametrize("m", [40, 100, 128])
def test_a_hot_expert_among_many(m, k, f):
    """More tokens on one expert than a chunk has columns, where the others have one or none."""
    g = gen(m + k)
    op = cdc.GatedExperts(*stacks(g, 64, 136, k, f, BF))
    ids, w = routing(g, m, 64, 3)
    ids[:, 1] = 7
    ids[::3, 2] = 63
    check(op, normal(g, m, k, dtype=BF), ids, w)


@pytest.mark.parametrize("m,E,top,k,f", [(128, 40, 32, 64, 72), (128, 1024, 32, 64, 8),
                                         (97, 1000, 7, 72, 40), (33, 300, 20, 67, 9),
                                         (8, 1024, 4, 64, 16), (3, 1024, 32, 64, 16)])
def test_many_experts_and_choices(m, E, top, k, f):
    g = gen(E + top)
    op = cdc.GatedExperts(*stacks(g, E, 72, k, f, BF))
    ids, w = routing(g, m, E, top)
    check(op, normal(g, m, k, dtype=BF), ids, w)


def test_nan_stays_where_it_is():
    g = gen(6)
    wg, wu, wd = stacks(g, 8, 136, 128, 72, BF)
    x, (ids, w) = normal(g, 40, 128, dtype=BF), routing(g, 40, 7, 2)
    for t in (wg, wu, wd):
        t[7] = float("nan")      # no token's expert
    op = cdc.GatedExperts(wg, wu, wd)
    clean = check(op, x, ids, w).clone()
    x[11] = float("nan")
    x[12] = float("inf")
    w[13, 0] = float("nan")
    y = op.forward(x, ids, w)
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[11:14] = False
    assert torch.equal(y[rows], clean[rows])
    assert bool(y[11].isnan().all()) and bool(y[13].isnan().all())
    ids[20, 0], ids[20, 1] = 7, -1
    y = op.forward(x, ids, w)
    rows[20] = False
    assert bool(y[20].isnan().all()) and torch.equal(y[rows], clean[rows])


def test_nothing_to_sum_over():
    g = gen(7)
    r = normal(g, 5, 40, dtype=BF)
    ids, w = routing(g, 5, 3, 2)
    for k, f in ((0, 16), (16, 0), (0, 0)):
        op = cdc.GatedExperts(*stacks(g, 3, 40, max(k, 1), max(f, 1), BF))
        op = cdc.GatedExperts(op.w_gate[:, :f, :k], op.w_up[:, :f, :k], op.w_down[:, :, :f])
        y = op.forward(normal(g, 5, k, dtype=BF), ids, w, residual=r)
        assert torch.equal(y, r)
    op = cdc.GatedExperts(*stacks(g, 3, 40, 16, 16, BF))
    x = normal(g, 5, 16, dtype=BF)
    assert op.forward(x[:0], ids[:0], w[:0]).shape == (0, 40)
    op0 = cdc.GatedExperts(op.w_gate, op.w_up, op.w_down[:, :0])
    assert op0.forward(x, ids, w).shape == (5, 0)


def test_residual_in_place_and_leading_dimensions():
    g = gen(8)
    op = cdc.GatedExperts(*stacks(g, 6, 128, 128, 72, BF))
    x, (ids, w) = normal(g, 140, 128, dtype=BF), routing(g, 140, 6, 2)
    y = x.clone()
    r = normal(g, 140, 128, dtype=BF)
    want = op.forward(x, ids, w, residual=r)
    out = r.clone()
    assert op.forward(x, ids, w, residual=out, out=out) is out
    assert torch.equal(out, want) and torch.equal(x, y)
    y4 = op.forward(x.view(7, 20, 128), ids.view(7, 20, 2), w.view(7, 20, 2),
                    residual=r.view(7, 20, 128))
    assert y4.shape == (7, 20, 128) and torch.equal(y4.view(140, 128), want)
    one = op.forward(x[0], ids[0], w[0])
    assert one.shape == (128,)
    assert torch.equal(op.forward(x[:1], ids[:1], w[:1])[0], one)
    assert torch.equal(op.forward(x, ids, w, residual=r[0]),
                       op.forward(x, ids, w, residual=r[:1].expand(140, 128).contiguous()))


@pytest.mark.parametrize("m", [1, 24, 140])
def test_same_bits_every_time(m):
    g = gen(9)
    for shape in ((8, 512, 1024, 712, BF), (4, 333, 129, 77, HF)):
        op = cdc.GatedExperts(*stacks(g, *shape))
        x, (ids, w) = normal(g, m, shape[2], dtype=shape[4]), routing(g, m, shape[0], 2)
        first = op.forward(x, ids, w)
        for _ in range(20):
            assert torch.equal(op.forward(x, ids, w), first)


def test_graphs_and_streams():
    """Two graphs of one object, replayed in turn with calls between; calls on two streams."""
    g = gen(10)
    op = cdc.GatedExperts(*stacks(g, 8, 512, 512, 264, BF))
    xs = [normal(g, m, 512, dtype=BF) for m in (1, 40)]
    rs = [routing(g, m, 8, 2) for m in (1, 40)]
    for x, (ids, w) in zip(xs, rs):
        op.forward(x, ids, w)
    graphs, outs = [], []
    for x, (ids, w) in zip(xs, rs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(op.forward(x, ids, w))
        graphs.append(graph)
    for i in range(2):
        xs[i].copy_(normal(g, *xs[i].shape, dtype=BF))
        ids, w = routing(g, xs[i].shape[0], 8, 2)
        rs[i][0].copy_(ids)
        rs[i][1].copy_(w)
    want = [op.forward(x, ids, w) for x, (ids, w) in zip(xs, rs)]
    for _ in range(5):
        for i in (0, 1, 1, 0):
            graphs[i].replay()
            assert torch.equal(op.forward(xs[1 - i], *rs[1 - i]), want[1 - i])
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[op.forward(xs[i], *rs[i], stream=streams[i]) for i in (0, 1)] for _ in range(10)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


def test_updates_in_place_are_seen():
    g = gen(11)
    op = cdc.GatedExperts(*stacks(g, 4, 128, 128, 64, BF))
    x, (ids, w) = normal(g, 3, 128, dtype=BF), routing(g, 3, 4, 2)
    y = op.forward(x, ids, w)
    op.w_down.mul_(2)
    assert torch.equal(op.forward(x, ids, w), 2 * y)


def test_stacks_past_32_bits():
    E, n, k, f = 20, 512, 8192, 14336  # 2^31 elements and more in gate and up
    wg = torch.zeros(E, f, k, dtype=BF, device="cuda")
    wu, wd = torch.zeros_like(wg), torch.zeros(E, n, f, dtype=BF, device="cuda")
    g = gen(12)
    for e in (0, E - 1):
        for w in (wg, wu):
            w[e] = normal(g, f, k, dtype=BF, scale=k ** -0.5)
        wd[e] = normal(g, n, f, dtype=BF, scale=f ** -0.5)
    op = cdc.GatedExperts(wg, wu, wd)
    ids = torch.tensor([[0, E - 1], [E - 1, 5], [7, 3]], dtype=torch.int32, device="cuda")
    x, w = normal(g, 3, k, dtype=BF), torch.rand(3, 2, generator=g, device="cuda")
    y = op.forward(x, ids, w)
    rows = torch.tensor([0, E - 1], device="cuda")
    at = torch.tensor([[0, 1], [1, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    want = er.experts(x, at, w, wg[rows], wu[rows], wd[rows], "silu", 0, None, BF)
    ref.assert_close(y, want, "y")
    ref.assert_rms(y, want, BF, "y", 2.0)


def test_refusals():
    g = gen(13)
    wg, wu, wd = stacks(g, 4, 128, 64, 72, BF)
    for args in ((wg[0], wu, wd), (wg, wu[:3], wd), (wg, wu, wd[:, :, :70]), (wg, wu, wd.half()),
                 (wg.float(), wu.float(), wd.float()), (wg.cpu(), wu.cpu(), wd.cpu()),
                 (wg.transpose(1, 2), wu.transpose(1, 2), wd)):
        with pytest.raises(ValueError):
            cdc.GatedExperts(*args)
    with pytest.raises(ValueError):
        cdc.GatedExperts(wg, wu, wd, act="none")
    with pytest.raises(ValueError):
        cdc.GatedExperts(wg, wu, wd, first=-1)
    op = cdc.GatedExperts(wg, wu, wd)
    x, (ids, w) = normal(g, 5, 64, dtype=BF), routing(g, 5, 4, 2)
    out = torch.empty(5, 128, dtype=BF, device="cuda")
    for call in (lambda: op.forward(x.half(), ids, w), lambda: op.forward(x[:, :60], ids, w),
                 lambda: op.forward(x, ids.long(), w), lambda: op.forward(x, ids, w.bfloat16()),
                 lambda: op.forward(x, ids[:4], w), lambda: op.forward(x, ids, w[:, :1]),
                 lambda: op.forward(x, ids, w, out=out[:4]),
                 lambda: op.forward(x, ids, w, out=out, out_dtype=F32),
                 lambda: op.forward(x, ids, w, out_dtype=HF),
                 lambda: op.forward(x, ids, w, residual=out.float()),
                 lambda: op.forward(x.cpu(), ids, w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: op.forward(x, ids, w, out=torch.empty(128, 5, dtype=BF, device="cuda").t()),
                 lambda: op.forward(wd[0, :5, :64], ids, w, out=wd[0].t()[:5, :128]),
                 lambda: op.forward(x, ids[:, :0], w[:, :0])):
        with pytest.raises(cdc.CollError):
            call()
