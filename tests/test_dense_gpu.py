"""Linear and GatedFFN on the GPU against 64-bit references (tests/dense_ref.py has the bounds).

Every output buffer is a view of a larger one filled with a canary, which has to survive."""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300 import _lib  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import dense_ref as ref  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
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


def rnd(g, rows, cols, dtype, scale=1.0, layout="rows"):
    """A matrix in one of the layouts an input may come in."""
    def make(r, c):
        return (torch.randn(r, c, generator=g, device="cuda") * scale).to(dtype)
    if layout == "rows":
        return make(rows, cols)
    if layout == "cols":
        return make(cols, rows).t()
    if layout == "slice8":      # aligned rows inside a wider buffer
        return make(rows, (cols + 7) // 8 * 8 + 16)[:, 8:8 + cols]
    if layout == "slice3":      # nothing lines up
        return make(rows, cols + 5)[:, 3:3 + cols]
    if layout == "cols3":
        return make(cols, rows + 5)[:, 3:3 + rows].t()
    if layout == "every2":      # no unit stride at all
        return make(rows * 2, cols * 3)[::2, ::3]
    if layout == "row0":        # one row for all (stride 0)
        return make(1, cols).expand(rows, cols)
    raise KeyError(layout)


class Out:
    """An output view inside a canary-filled buffer."""

    def __init__(self, rows, cols, dtype, slack=0, shift=0):
        self.buf = torch.full((rows + 2, cols + slack + 8), CANARY, dtype=dtype, device="cuda")
        self.v = self.buf[1:1 + rows, shift:shift + cols]
        self.v.fill_(float("nan"))

    def untouched(self):
        b = self.buf.clone()
        b[1:1 + self.v.shape[0], self.v.storage_offset() % self.buf.shape[1]:
          self.v.storage_offset() % self.buf.shape[1] + self.v.shape[1]] = CANARY
        return bool((b == CANARY).all())


def aligned(cols):
    return -cols % 8


SIZES = [(1, 1, 1), (1, 64, 64), (1, 4096, 512), (2, 100, 264), (3, 130, 72), (5, 33, 1),
         (7, 8, 4104), (8, 257, 256), (9, 1000, 1000), (16, 512, 2048), (17, 96, 96),
         (31, 640, 333), (33, 127, 129), (64, 256, 512), (65, 520, 64), (100, 1, 100),
         (127, 128, 31), (128, 128, 128), (129, 257, 65), (200, 1025, 40), (256, 256, 256),
         (257, 100, 1024), (300, 521, 2056), (1000, 72, 7), (512, 768, 64), (1, 2, 16384),
         (640, 2304, 320)]
LAYOUTS = [("rows", "rows"), ("slice8", "cols"), ("slice3", "rows"), ("rows", "slice3"),
           ("cols", "cols3"), ("every2", "slice8"), ("row0", "every2")]
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
GACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)))
def test_linear_sizes(i, size):
    m, n, k = size
    dtype = (BF, HF)[i % 2]
    g = gen(i)
    x, w = rnd(g, m, k, dtype), rnd(g, n, k, dtype, k ** -0.5)
    b = rnd(g, 1, n, dtype)[0] if i % 3 else None
    r = rnd(g, m, n, dtype) if i % 4 < 2 else None
    act = ACTS[i % 5]
    slack, shift = ((aligned(n), 0), (3, 1), (5, 0))[i % 3]
    y, p = Out(m, n, dtype, slack, shift), Out(m, n, dtype, slack, shift)
    lin = cdc.Linear(w, b, act)
    lin.forward(x, residual=r, out=y.v, save=True, pre=p.v)
    want, pre = ref.linear(x, w, b, r, act, dtype, dtype)
    ref.assert_close(y.v, want, "y")
    ref.assert_close(p.v, pre, "pre")
    ref.assert_rms(p.v, pre, dtype, "pre")
    assert y.untouched() and p.untouched()
    assert lin.status() == _lib.OK


@pytest.mark.parametrize("size", [(1, 200, 328), (6, 520, 1000), (24, 72, 2048), (40, 300, 136),
                                  (150, 264, 200), (300, 384, 520)])
@pytest.mark.parametrize("layouts", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_linear_layouts(size, layouts, dtype):
    m, n, k = size
    g = gen(m + n)
    x, w = rnd(g, m, k, dtype, 1.0, layouts[0]), rnd(g, n, k, dtype, k ** -0.5, layouts[1])
    b = rnd(g, 1, 2 * n, dtype)[0, ::2]
    r = rnd(g, m, n, dtype, 1.0, layouts[0])
    y = Out(m, n, dtype, 1, 1)
    cdc.Linear(w, b, "silu").forward(x, residual=r, out=y.v)
    ref.assert_close(y.v, ref.linear(x, w, b, r, "silu", dtype, dtype)[0])
    assert y.untouched()


@pytest.mark.parametrize("m", [1, 4, 16, 40, 130, 400])
@pytest.mark.parametrize("act", ACTS)
def test_linear_f32_output(m, act):
    g = gen(m)
    n, k = 264, 520
    x, w, b = rnd(g, m, k, BF), rnd(g, n, k, BF, k ** -0.5), rnd(g, 1, n, BF)[0]
    r = torch.randn(m, n, generator=g, device="cuda")
    y = cdc.Linear(w, b, act).forward(x, residual=r, out_dtype=F32)
    assert y.dtype is F32
    ref.assert_close(y, ref.linear(x, w, b, r, act, F32, BF)[0])


@pytest.mark.parametrize("m", [1, 20, 200, 600])
def test_linear_in_place_residual_and_leading_dimensions(m):
    g = gen(3)
    x, w = rnd(g, 3 * m, 96, BF).view(3, m, 96), rnd(g, 80, 96, BF, 0.1)
    r = rnd(g, 3 * m, 80, BF).view(3, m, 80)
    want = ref.linear(x.reshape(-1, 96), w, None, r.reshape(-1, 80), "none", BF, BF)[0]
    y = r.clone()
    out = cdc.Linear(w).forward(x, residual=y, out=y)
    assert out is y
    ref.assert_close(y.view(-1, 80), want)
    fresh = cdc.Linear(w).forward(x, residual=r)
    assert fresh.shape == (3, m, 80) and torch.equal(fresh, y)
    one = cdc.Linear(w).forward(x[0, 0], residual=r[0, 0])   # a vector
    assert one.shape == (80,)
    ref.assert_close(one[None], (want[0][:1], want[1][:1]))
    wide = cdc.Linear(w).forward(x, residual=r[:1, :1])       # a broadcast residual
    ref.assert_close(wide.view(-1, 80), ref.linear(
        x.reshape(-1, 96), w, None, r[:1, :1].expand(3, m, 80).reshape(-1, 80), "none", BF, BF)[0])


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)))
def test_linear_backward_sizes(i, size):
    m, n, k = size
    dtype = (HF, BF)[i % 2]
    act = ACTS[(i + 2) % 5]
    g = gen(100 + i)
    x, w, dy = rnd(g, m, k, dtype), rnd(g, n, k, dtype, k ** -0.5), rnd(g, m, n, dtype)
    z = rnd(g, m, n, dtype)
    gt = F32 if i % 4 == 1 else dtype
    slack, shift = ((3, 1), (aligned(k), 0), (2, 0))[i % 3]
    dx, dw = Out(m, k, dtype, slack, shift), Out(n, k, gt, slack, shift)
    db = Out(1, n, gt, 1, 1)
    lin = cdc.Linear(w, None, act)
    lin.backward(dy, x, pre=z, dx=dx.v, dw=dw.v, db=db.v[0])
    rdx, rdw, rdb = ref.linear_bwd(dy, z, x, w, act, dtype, gt)
    ref.assert_close(dx.v, rdx, "dx")
    ref.assert_close(dw.v, rdw, "dw")
    ref.assert_close(db.v[0], rdb, "db")
    ref.assert_rms(dx.v, rdx, dtype, "dx", 2.0)
    ref.assert_rms(dw.v, rdw, dtype, "dw", 2.0)
    assert dx.untouched() and dw.untouched() and db.untouched()
    assert lin.status() == _lib.OK


@pytest.mark.parametrize("layouts", LAYOUTS)
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_backward_layouts(layouts, act):
    m, n, k = 150, 136, 210
    g = gen(7)
    x, w = rnd(g, m, k, BF, 1.0, layouts[0]), rnd(g, n, k, BF, k ** -0.5, layouts[1])
    dy, z = rnd(g, m, n, BF, 1.0, layouts[1]), rnd(g, m, n, BF, 1.0, layouts[0])
    got = cdc.Linear(w, None, act).backward(dy, x, pre=z, need_db=True)
    for a, b in zip(got, ref.linear_bwd(dy, z, x, w, act, BF, BF)):
        ref.assert_close(a, b)


def test_linear_backward_of_a_broadcast_gradient():
    """dy with stride 0 everywhere, as the gradient of a sum has it."""
    g = gen(8)
    x, w = rnd(g, 130, 64, BF), rnd(g, 72, 64, BF, 0.1)
    dy = torch.ones(1, 1, dtype=BF, device="cuda").expand(130, 72)
    got = cdc.Linear(w).backward(dy, x, need_db=True)
    for a, b in zip(got, ref.linear_bwd(dy, None, x, w, "none", BF, BF)):
        ref.assert_close(a, b)


def test_linear_backward_parts():
    """Any subset of the gradients, with the values of all three."""
    g = gen(9)
    x, w, dy, z = (rnd(g, *s, BF) for s in ((70, 40), (48, 40), (70, 48), (70, 48)))
    lin = cdc.Linear(w, None, "silu")
    full = lin.backward(dy, x, pre=z, need_db=True)
    for which in range(8):
        want = [bool(which >> b & 1) for b in range(3)]
        got = lin.backward(dy, x, pre=z, need_dx=want[0], need_dw=want[1], need_db=want[2])
        for have, a, b in zip(want, got, full):
            assert (a is not None) == have and (a is None or torch.equal(a, b))


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)))
def test_gated_sizes(i, size):
    m, n, k = size
    dtype = (BF, HF)[i % 2]
    act = GACTS[i % 5]
    g = gen(200 + i)
    x = rnd(g, m, k, dtype)
    wg, wu = rnd(g, n, k, dtype, k ** -0.5), rnd(g, n, k, dtype, k ** -0.5)
    slack, shift = ((aligned(n), 0), (3, 1), (5, 0))[i % 3]
    h, gate, up = (Out(m, n, dtype, slack, shift) for _ in range(3))
    ffn = cdc.GatedFFN(wg, wu, act)
    ffn.forward(x, out=h.v, gate=gate.v, up=up.v)
    rh, rg, ru = ref.gated(x, wg, wu, act, dtype)
    ref.assert_close(h.v, rh, "h")
    ref.assert_close(gate.v, rg, "gate")
    ref.assert_close(up.v, ru, "up")
    ref.assert_rms(gate.v, rg, dtype, "gate")
    ref.assert_rms(up.v, ru, dtype, "up")
    assert h.untouched() and gate.untouched() and up.untouched()
    assert torch.equal(ffn.forward(x), h.v)          # without keeping anything
    assert ffn.status() == _lib.OK


@pytest.mark.parametrize("size", [(1, 200, 328), (6, 520, 1000), (24, 72, 2048), (40, 300, 136),
                                  (150, 264, 200), (300, 384, 520)])
@pytest.mark.parametrize("layouts", LAYOUTS)
def test_gated_layouts(size, layouts):
    m, n, k = size
    g = gen(m + n)
    x = rnd(g, m, k, HF, 1.0, layouts[0])
    wg, wu = rnd(g, n, k, HF, k ** -0.5, layouts[1]), rnd(g, n, k, HF, k ** -0.5, layouts[0])
    h = Out(m, n, HF, 1, 1)
    cdc.GatedFFN(wg, wu, "gelu").forward(x, out=h.v)
    ref.assert_close(h.v, ref.gated(x, wg, wu, "gelu", HF)[0])
    assert h.untouched()


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)))
def test_gated_backward_sizes(i, size):
    m, n, k = size
    dtype = (HF, BF)[i % 2]
    act = GACTS[(i + 1) % 5]
    g = gen(300 + i)
    x = rnd(g, m, k, dtype)
    wg, wu = rnd(g, n, k, dtype, k ** -0.5), rnd(g, n, k, dtype, k ** -0.5)
    dh, gate, up = (rnd(g, m, n, dtype) for _ in range(3))
    gt = F32 if i % 4 == 1 else dtype
    slack, shift = ((3, 1), (aligned(k), 0), (2, 0))[i % 3]
    dx, dg, du = (Out(r, k, t, slack, shift) for r, t in ((m, dtype), (n, gt), (n, gt)))
    ffn = cdc.GatedFFN(wg, wu, act)
    ffn.backward(dh, x, gate, up, dx=dx.v, dw_gate=dg.v, dw_up=du.v)
    want = ref.gated_bwd(dh, gate, up, x, wg, wu, act, dtype, gt)
    for o, b, t, what in zip((dx, dg, du), want, (dtype, gt, gt), ("dx", "dw_gate", "dw_up")):
        ref.assert_close(o.v, b, what)
        ref.assert_rms(o.v, b, dtype, what, 2.0)
        assert o.untouched()
    assert ffn.status() == _lib.OK


@pytest.mark.parametrize("layouts", LAYOUTS)
def test_gated_backward_layouts(layouts):
    m, n, k = 150, 136, 210
    g = gen(17)
    x = rnd(g, m, k, BF, 1.0, layouts[0])
    wg, wu = rnd(g, n, k, BF, k ** -0.5, layouts[1]), rnd(g, n, k, BF, k ** -0.5, layouts[0])
    dh, gate, up = (rnd(g, m, n, BF, 1.0, s) for s in (layouts[1], layouts[0], "rows"))
    got = cdc.GatedFFN(wg, wu, "silu").backward(dh, x, gate, up)
    for a, b in zip(got, ref.gated_bwd(dh, gate, up, x, wg, wu, "silu", BF, BF)):
        ref.assert_close(a, b)
    dx, none, _ = cdc.GatedFFN(wg, wu, "silu").backward(dh, x, gate, up, need_dw=False)
    assert none is None and torch.equal(dx, got[0])


# few output tiles and a long sum: k is shared between the tiles of several clusters
LONG = [(20, 40, 9000), (130, 72, 4100), (200, 130, 16384), (257, 520, 5000), (150, 33, 20001),
        (600, 300, 3000)]


@pytest.mark.parametrize("i,size", list(enumerate(LONG)))
def test_long_sums(i, size):
    m, n, k = size
    dtype = (BF, HF)[i % 2]
    g = gen(500 + i)
    x, w, w2 = rnd(g, m, k, dtype), rnd(g, n, k, dtype, k ** -0.5), rnd(g, n, k, dtype, k ** -0.5)
    b, r = rnd(g, 1, n, dtype)[0], rnd(g, m, n, dtype)
    y, p = Out(m, n, dtype, 3, 1), Out(m, n, dtype, aligned(n), 0)
    cdc.Linear(w, b, ACTS[i % 5]).forward(x, residual=r, out=y.v, pre=p.v)
    want, pre = ref.linear(x, w, b, r, ACTS[i % 5], dtype, dtype)
    ref.assert_close(y.v, want, "y")
    ref.assert_close(p.v, pre, "pre")
    ref.assert_rms(p.v, pre, dtype, "pre")
    f = cdc.Linear(w, b, ACTS[i % 5]).forward(x, residual=r.float(), out_dtype=F32)
    ref.assert_close(f, ref.linear(x, w, b, r, ACTS[i % 5], F32, dtype)[0], "f32")
    h, gate, up = (Out(m, n, dtype, 1, 1) for _ in range(3))
    cdc.GatedFFN(w, w2, GACTS[i % 5]).forward(x, out=h.v, gate=gate.v, up=up.v)
    for o, q, what in zip((h, gate, up), ref.gated(x, w, w2, GACTS[i % 5], dtype),
                          ("h", "gate", "up")):
        ref.assert_close(o.v, q, what)
        assert o.untouched()
    assert y.untouched() and p.untouched()


@pytest.mark.parametrize("i,size", list(enumerate(LONG)))
def test_long_sums_backward(i, size):
    """dx sums over n, dW over m: each axis in turn is the long one."""
    a, b, c = size
    dtype = (HF, BF)[i % 2]
    g = gen(600 + i)
    for m, n, k in ((a, c, b), (c, a, b)):
        x, w, w2 = rnd(g, m, k, dtype), rnd(g, n, k, dtype, .05), rnd(g, n, k, dtype, .05)
        dy, z, u = (rnd(g, m, n, dtype) for _ in range(3))
        act = ACTS[i % 5]
        dx, dw, db = Out(m, k, dtype, 3, 1), Out(n, k, dtype, 3, 1), Out(1, n, dtype, 1, 1)
        cdc.Linear(w, None, act).backward(dy, x, pre=z, dx=dx.v, dw=dw.v, db=db.v[0])
        for o, q, what in zip((dx.v, dw.v, db.v[0]),
                              ref.linear_bwd(dy, z, x, w, act, dtype, dtype), ("dx", "dw", "db")):
            ref.assert_close(o, q, what)
        assert dx.untouched() and dw.untouched() and db.untouched()
        alone = cdc.Linear(w, None, act)
        ref.assert_close(alone.backward(dy, x, pre=z, need_dw=False, need_db=True)[0],
                         ref.linear_bwd(dy, z, x, w, act, dtype, dtype)[0])
        got = cdc.GatedFFN(w, w2, GACTS[i % 5]).backward(dy, x, z, u, grad_dtype=F32)
        for o, q, what in zip(got, ref.gated_bwd(dy, z, u, x, w, w2, GACTS[i % 5], dtype, F32),
                              ("dx", "dw_gate", "dw_up")):
            ref.assert_close(o, q, what)


# a small batch against many outputs: the weights' rows are the wide side
@pytest.mark.parametrize("m,n,k", [(17, 9728, 72), (33, 9800, 200), (48, 10003, 136),
                                   (64, 12296, 328), (50, 9984, 1000)])
@pytest.mark.parametrize("layouts", [("rows", "rows"), ("slice3", "cols"), ("cols", "slice8")])
def test_wide_outputs_for_a_small_batch(m, n, k, layouts):
    for dtype, act, i in ((BF, "gelu", 0), (HF, "silu", 1)):
        g = gen(m + i)
        x = rnd(g, m, k, dtype, 1.0, layouts[0])
        w, w2 = (rnd(g, n, k, dtype, k ** -0.5, layouts[1]) for _ in range(2))
        b, r = rnd(g, 1, n, dtype)[0], rnd(g, m, n, dtype)
        y, p = Out(m, n, dtype, 3, 1), Out(m, n, dtype, aligned(n), 0)
        lin = cdc.Linear(w, b, act)
        lin.forward(x, residual=r, out=y.v, pre=p.v)
        want, pre = ref.linear(x, w, b, r, act, dtype, dtype)
        ref.assert_close(y.v, want, "y")
        ref.assert_close(p.v, pre, "pre")
        ref.assert_rms(p.v, pre, dtype, "pre")
        f = lin.forward(x, residual=r.float(), out_dtype=F32)
        ref.assert_close(f, ref.linear(x, w, b, r, act, F32, dtype)[0], "f32")
        h, gate, up = (Out(m, n, dtype, 1, 1) for _ in range(3))
        ffn = cdc.GatedFFN(w, w2, act)
        ffn.forward(x, out=h.v, gate=gate.v, up=up.v)
        for o, q, what in zip((h, gate, up), ref.gated(x, w, w2, act, dtype), ("h", "gate", "up")):
            ref.assert_close(o.v, q, what)
            assert o.untouched()
        assert y.untouched() and p.untouched()
        assert lin.status() == _lib.OK and ffn.status() == _lib.OK


@pytest.mark.parametrize("m,n,k", [(1, 96, 128), (3, 100, 1024), (9, 264, 300), (16, 33, 77)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_few_tokens_over_transposed_weights(m, n, k, dtype):
    g = gen(m)
    for layout in ("cols", "cols3"):
        x = rnd(g, m, k, dtype, 1.0, "rows" if layout == "cols" else "slice3")
        w, w2 = (rnd(g, n, k, dtype, k ** -0.5, layout) for _ in range(2))
        r = rnd(g, m, n, dtype)
        y, h = Out(m, n, dtype, 1, 1), Out(m, n, dtype, 1, 1)
        cdc.Linear(w, None, "relu").forward(x, residual=r, out=y.v)
        ref.assert_close(y.v, ref.linear(x, w, None, r, "relu", dtype, dtype)[0])
        cdc.GatedFFN(w, w2, "sigmoid").forward(x, out=h.v)
        ref.assert_close(h.v, ref.gated(x, w, w2, "sigmoid", dtype)[0])
        assert y.untouched() and h.untouched()


def test_offsets_beyond_32_bits():
    """More than 2^32 bytes and 2^31 elements in the output and in the gradient's scratch."""
    m, n, k = 66000, 33000, 40
    g = gen(2)
    x, w = rnd(g, m, k, BF), rnd(g, n, k, BF, k ** -0.5)
    lin = cdc.Linear(w, None, "relu")
    y, z = lin.forward(x, save=True)
    rows = torch.tensor([0, 1, 32537, 32538, 65000, m - 1], device="cuda")
    want, pre = ref.linear(x[rows], w, None, None, "relu", BF, BF)
    ref.assert_close(y[rows], want)
    ref.assert_close(z[rows], pre)
    del y
    dy = rnd(g, 1, n, BF).expand(m, n)
    dx, dw, _ = lin.backward(dy, x, pre=z)
    rdx = ref.linear_bwd(dy[rows], z[rows], x[rows], w, "relu", BF, BF)[0]
    ref.assert_close(dx[rows], rdx)
    cols = torch.tensor([0, 7, n - 1], device="cuda")
    rdw = ref.linear_bwd(dy[:, cols], z[:, cols], x, w[cols], "relu", BF, BF)[1]
    ref.assert_close(dw[cols], rdw)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,n,k", [(0, 40, 64), (5, 0, 64), (5, 40, 0), (0, 0, 0), (200, 300, 0)])
def test_empty_axes(m, n, k):
    """No tokens, no outputs, nothing to sum over: zeros, the bias and the residual remain."""
    g = gen(1)
    x, w, b, r = rnd(g, m, k, BF), rnd(g, n, k, BF), rnd(g, 1, n, BF)[0], rnd(g, m, n, BF)
    lin = cdc.Linear(w, b, "silu")
    y, z = lin.forward(x, residual=r, save=True)
    ref.assert_close(y, ref.linear(x, w, b, r, "silu", BF, BF)[0])
    for a, q in zip(lin.backward(r, x, pre=z), ref.linear_bwd(r, z, x, w, "silu", BF, BF)):
        ref.assert_close(a, q)
    ffn = cdc.GatedFFN(w, w.clone())
    h, gate, up = ffn.forward(x, save=True)
    ref.assert_close(h, ref.gated(x, w, w, "silu", BF)[0])
    for a, q in zip(ffn.backward(r, x, gate, up),
                    ref.gated_bwd(r, gate, up, x, w, w, "silu", BF, BF)):
        ref.assert_close(a, q)
    torch.cuda.synchronize()


@pytest.mark.parametrize("m", [1, 12, 40, 300])
def test_gradients_against_differences(m):
    """Central differences of the 64-bit loss along random directions; the step's own error is
    below the bound's share from rounding dz and the result. relu has no derivative at zero: its
    step is halved until no argument changes sign within it."""
    g = gen(m)
    n, k, h = 48, 40, 1e-4
    x, w, w2 = rnd(g, m, k, HF), rnd(g, n, k, HF, 0.15), rnd(g, n, k, HF, 0.15)
    b, c = rnd(g, 1, n, HF)[0], rnd(g, m, n, HF)

    def check(got, loss, args, scale, kink=None):
        for i, grad in enumerate(got):
            d = torch.randn(args[i].shape, generator=g, device="cuda", dtype=torch.float64)
            step = h
            while True:
                up, dn = ([a.double() + t * d if j == i else a.double()
                           for j, a in enumerate(args)] for t in (step, -step))
                if kink is None or torch.equal(kink(*up) > 0, kink(*dn) > 0):
                    break
                step /= 2
            num = float((loss(*up) - loss(*dn)) / (2 * step))
            have = float((grad.double() * d).sum())
            # independent roundings: u of each element of dz and of the result, along d
            tol = 4 * 2.0 ** -11 * float(grad.double().norm() + scale) + 1e-5 * abs(num)
            assert abs(num - have) <= tol, (i, num, have, tol)

    for act in ACTS:
        lin = cdc.Linear(w, b, act)
        # pre in 16 bits moves the slope; hand over z's rounding and differentiate there
        z = (x.double() @ w.double().t() + b.double()).to(HF)
        off = z.double() - (x.double() @ w.double().t() + b.double())
        got = lin.backward(c, x, pre=z)
        check(got, lambda xx, ww, bb: (ref.act(xx @ ww.t() + bb + off, act)[0] * c.double()).sum(),
              (x, w, b), float(c.double().norm()),
              (lambda xx, ww, bb: xx @ ww.t() + bb + off) if act == "relu" else None)
    for act in GACTS:
        ffn = cdc.GatedFFN(w, w2, act)
        zg, zu = x.double() @ w.double().t(), x.double() @ w2.double().t()
        gate, up = zg.to(HF), zu.to(HF)
        og, ou = gate.double() - zg, up.double() - zu
        got = ffn.backward(c, x, gate, up)
        check(got, lambda xx, a, bb: (ref.act(xx @ a.t() + og, act)[0] * (xx @ bb.t() + ou)
                                      * c.double()).sum(), (x, w, w2), float(c.double().norm()),
              (lambda xx, a, bb: xx @ a.t() + og) if act == "relu" else None)


@pytest.mark.parametrize("m,n,k", [(1, 96, 1024), (40, 264, 1000), (300, 300, 600)])
def test_infinities_and_nan_stay_in_their_rows(m, n, k):
    g = gen(4)
    x, w = rnd(g, m, k, BF), rnd(g, n, k, BF, k ** -0.5)
    wu = rnd(g, n, k, BF, k ** -0.5)
    w[n - 1, k - 1] = float("inf")
    wu[3, 0] = float("nan")
    if m > 1:
        x[m - 1, k // 2] = float("nan")
    x[0, k - 1] = 2.0
    y = cdc.Linear(w).forward(x)
    rows = slice(0, m - 1 if m > 1 else 1)
    assert torch.isfinite(y[rows, :n - 1]).all()
    assert (y[0, n - 1] == float("inf"))
    if m > 1:
        assert torch.isnan(y[m - 1]).all()
    h = cdc.GatedFFN(w, wu).forward(x)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[3] = keep[n - 1] = False
    assert torch.isfinite(h[rows][:, keep]).all()
    assert torch.isnan(h[:, 3]).all()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "sigmoid"])
def test_activations_far_out(act):
    """Large arguments of both signs, through an identity product."""
    v = torch.tensor([0.0, -0.0, 1e-3, -1e-3, 5, -5, 12, -12, 60, -60, 90, -90, 300, -300, 6e4,
                      -6e4], device="cuda").to(HF)
    eye = torch.eye(16, device="cuda", dtype=HF)
    x = torch.diag(v)
    if act != "sigmoid":
        y = cdc.Linear(eye, None, act).forward(x).diagonal()
        want = ref.act(v.double(), act)[0]
        assert torch.allclose(y.double(), want, rtol=2.0 ** -10, atol=2.0 ** -20)
    h = cdc.GatedFFN(eye, torch.eye(16, device="cuda", dtype=HF), act).forward(
        torch.diag(v.clamp(-200, 200))).diagonal()
    c = v.clamp(-200, 200).double()
    assert torch.allclose(h.double(), ref.act(c, act)[0] * c, rtol=2.0 ** -10, atol=2.0 ** -17)


@pytest.mark.parametrize("m,n,k", [(1, 512, 1024), (20, 512, 1024), (100, 264, 2048),
                                   (700, 520, 328)])
def test_same_call_same_bits(m, n, k):
    g = gen(5)
    x, w, r = rnd(g, m, k, BF), rnd(g, n, k, BF, k ** -0.5), rnd(g, m, n, BF)
    lin, ffn = cdc.Linear(w, None, "gelu"), cdc.GatedFFN(w, w.flip(0).contiguous())
    first = None
    for _ in range(5):
        y, z = lin.forward(x, residual=r, save=True)
        h, gate, up = ffn.forward(x, save=True)
        now = (y, z, h, *lin.backward(r, x, pre=z, need_db=True), *ffn.backward(r, x, gate, up))
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("m", [1, 16, 64, 400])
def test_other_streams_and_graphs(m):
    """A call on a stream given, and calls captured into a graph that sees new inputs."""
    g = gen(6)
    n, k = 264, 392
    x, w, r = rnd(g, m, k, BF), rnd(g, n, k, BF, k ** -0.5), rnd(g, m, n, BF)
    lin, ffn = cdc.Linear(w, None, "silu"), cdc.GatedFFN(w, w.flip(0).contiguous())
    y, z = lin.forward(x, residual=r, save=True)
    h, gate, up = ffn.forward(x, save=True)
    grads = lin.backward(r, x, pre=z) + ffn.backward(r, x, gate, up)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2, z2 = lin.forward(x, residual=r, save=True, stream=s)
    h2, gate2, up2 = ffn.forward(x, save=True, stream=s)
    grads2 = lin.backward(r, x, pre=z2, stream=s) + ffn.backward(r, x, gate2, up2, stream=s)
    s.synchronize()
    for a, b in zip((y, z, h, gate, up, *grads), (y2, z2, h2, gate2, up2, *grads2)):
        assert (a is None and b is None) or torch.equal(a, b)
    xin, gr = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y3, z3 = lin.forward(xin, residual=r, save=True)
        h3, gate3, up3 = ffn.forward(xin, save=True)
        grads3 = lin.backward(r, xin, pre=z3) + ffn.backward(r, xin, gate3, up3)
    for _ in range(2):
        xin.copy_(x)
        gr.replay()
    torch.cuda.synchronize()
    for a, b in zip((y, z, h, gate, up, *grads), (y3, z3, h3, gate3, up3, *grads3)):
        assert (a is None and b is None) or torch.equal(a, b)


def test_weights_updated_in_place_are_seen():
    g = gen(11)
    x, w = rnd(g, 40, 64, BF), rnd(g, 72, 64, BF)
    lin = cdc.Linear(w)
    lin.forward(x)
    w.mul_(2)
    ref.assert_close(lin.forward(x), ref.linear(x, w, None, None, "none", BF, BF)[0])


def test_refusals():
    g = gen(12)
    w, x = rnd(g, 32, 64, BF), rnd(g, 8, 64, BF)
    lin, ffn = cdc.Linear(w, None, "silu"), cdc.GatedFFN(w, w.clone())
    bad = [
        lambda: cdc.Linear(w.float()), lambda: cdc.Linear(w[0]), lambda: cdc.Linear(w.cpu()),
        lambda: cdc.Linear(w, act="sigmoid"), lambda: cdc.Linear(w, bias=w[0]),
        lambda: cdc.Linear(w, bias=w[:, 0].float()), lambda: cdc.GatedFFN(w, w[:16]),
        lambda: cdc.GatedFFN(w, w.half()), lambda: cdc.GatedFFN(w, w, act="none"),
        lambda: lin.forward(x.half()), lambda: lin.forward(x[:, :32]), lambda: lin.forward(x.cpu()),
        lambda: lin.forward(x, out=torch.empty(8, 31, dtype=BF, device="cuda")),
        lambda: lin.forward(x, out=torch.empty(8, 32, dtype=HF, device="cuda")),
        lambda: lin.forward(x, out_dtype=HF), lambda: lin.forward(x, residual=x.half()),
        lambda: lin.backward(rnd(g, 8, 32, BF), x),                     # pre is missing
        lambda: lin.backward(rnd(g, 7, 32, BF), x, pre=rnd(g, 8, 32, BF)),
        lambda: ffn.backward(rnd(g, 8, 32, BF), x, rnd(g, 8, 32, BF), rnd(g, 7, 32, BF)),
    ]
    for f in bad:
        with pytest.raises((ValueError, RuntimeError)):
            f()
    buf = torch.zeros(8, 128, dtype=BF, device="cuda")
    for f in (lambda: cdc.Linear(w[:, :32]).forward(buf[:, :32], out=buf[:, 16:48]),
              lambda: cdc.GatedFFN(w, w).forward(buf[:, :64], out=buf[:, 96:], gate=buf[:, 64:96],
                                                 up=buf[:, 64:96]),
              lambda: lin.forward(x, residual=buf[:, 1:33], out=buf[:, :32])):
        with pytest.raises(cdc.CollError) as e:
            f()
        assert e.value.code == _lib.D["COLL_EOVERLAP"]
    # column slices of one buffer that do not meet are fine
    buf[:, :64] = x
    cdc.Linear(w).forward(buf[:, :64], out=buf[:, 64:96])
    ref.assert_close(buf[:, 64:96], ref.linear(x, w, None, None, "none", BF, BF)[0])
    with pytest.raises(cdc.CollError) as e:   # rows of an output that overlap
        lin.forward(x, out=torch.zeros(64, dtype=BF, device="cuda").as_strided((8, 32), (4, 1)))
    assert e.value.code == _lib.D["COLL_EINVAL"]


FEW = [(1, 76, 12289), (4, 40, 9000), (16, 76, 13679), (32, 76, 13679), (32, 64, 12288),
       (64, 76, 4099), (64, 40, 4096), (24, 33, 4001), (12, 50, 1027), (48, 90, 611)]


@pytest.mark.parametrize("m,n,k", FEW)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_few_tokens_over_long_sums(m, n, k, dtype):
    g = gen(k + m)
    x, w = rnd(g, m, k, dtype), rnd(g, n, k, dtype, k ** -0.5)
    wu, b = rnd(g, n, k, dtype, k ** -0.5), rnd(g, 1, n, dtype)[0]
    y = Out(m, n, dtype, 1, 1)
    cdc.Linear(w, b, "gelu").forward(x, out=y.v)
    ref.assert_close(y.v, ref.linear(x, w, b, None, "gelu", dtype, dtype)[0])
    assert y.untouched()
    h = Out(m, n, dtype)
    cdc.GatedFFN(w, wu, "silu").forward(x, out=h.v)
    ref.assert_close(h.v, ref.gated(x, w, wu, "silu", dtype)[0])
    assert h.untouched()


@pytest.mark.parametrize("shift", range(8))
@pytest.mark.parametrize("m", [1, 12, 30, 60])
def test_few_tokens_at_any_offset(m, shift):
    """Rows that start on every even byte, with infinities around them that must not be read in."""
    g = gen(shift)
    n, k = 35, 301
    def inside(rows):
        buf = torch.full((rows, k + 16), float("inf"), dtype=BF, device="cuda")
        v = buf[:, shift:shift + k]
        v.copy_(rnd(g, rows, k, BF, k ** -0.5))
        return v
    x, w = inside(m), inside(n)
    y = cdc.Linear(w).forward(x)
    ref.assert_close(y, ref.linear(x, w, None, None, "none", BF, BF)[0])
