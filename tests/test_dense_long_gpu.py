"""Long sums in the root mean square. A bound on each element grows with K and the error does not: a
lost block of k passes it (tests/test_dense_bounds.py), and these see it. Limits: an output rounded
once, u of its type; one whose dz was rounded on the way, twice that; binary32 outputs sqrt(K) 2^-22
(K adds of independent errors of 2^-23 of the sum, twice), and u of the operands' type where dz was
rounded."""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import dense_ref as ref  # noqa: E402
from test_dense_gpu import ACTS, FEW, GACTS, LONG, gen, rnd  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    yield
    torch.cuda.synchronize()


def f32_rms(got, want, k, what):
    ref.assert_rms(got, want, F32, what, 4 * math.sqrt(k))


@pytest.mark.parametrize("m,n,k", LONG + FEW)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward(m, n, k, dtype):
    i = m + n
    g = gen(k + m)
    x, w, w2 = rnd(g, m, k, dtype), rnd(g, n, k, dtype, k ** -0.5), rnd(g, n, k, dtype, k ** -0.5)
    b, r = rnd(g, 1, n, dtype)[0], rnd(g, m, n, dtype)
    act, gact = ACTS[i % 5], GACTS[i % 5]
    lin = cdc.Linear(w, b, act)
    y, p = lin.forward(x, residual=r, save=True)
    want, pre = ref.linear(x, w, b, r, act, dtype, dtype)
    ref.assert_rms(y, want, dtype, "y")
    ref.assert_rms(p, pre, dtype, "pre")
    f32_rms(lin.forward(x, residual=r.float(), out_dtype=F32), want, k, "f32")
    for o, q, what in zip(cdc.GatedFFN(w, w2, gact).forward(x, save=True),
                          ref.gated(x, w, w2, gact, dtype), ("h", "gate", "up")):
        ref.assert_rms(o, q, dtype, what)


@pytest.mark.parametrize("i,size", list(enumerate(LONG)))
@pytest.mark.parametrize("dtype", [BF, HF])
def test_backward(i, size, dtype):
    a, b, c = size
    g = gen(700 + i)
    for m, n, k in ((a, c, b), (c, a, b)):
        x, w, w2 = rnd(g, m, k, dtype), rnd(g, n, k, dtype, .05), rnd(g, n, k, dtype, .05)
        dy, z, u = (rnd(g, m, n, dtype) for _ in range(3))
        for act in (ACTS[i % 5], "none"):
            lin = cdc.Linear(w, None, act)
            want = ref.linear_bwd(dy, z, x, w, act, dtype, dtype)
            for o, q, what, t in zip(lin.backward(dy, x, pre=z, need_db=True), want,
                                     ("dx", "dw", "db"), (2, 2, 1)):
                ref.assert_rms(o, q, dtype, what, t)
            _, dw, db = lin.backward(dy, x, pre=z, need_db=True, grad_dtype=F32)
            if act == "none":
                f32_rms(dw, want[1], m, "dw in binary32")
            else:
                ref.assert_rms(dw, want[1], dtype, "dw in binary32")
            f32_rms(db, want[2], m, "db in binary32")
        ffn = cdc.GatedFFN(w, w2, GACTS[i % 5])
        want = ref.gated_bwd(dy, z, u, x, w, w2, GACTS[i % 5], dtype, F32)
        for o, q, what in zip(ffn.backward(dy, x, z, u), want, ("dx", "dw_gate", "dw_up")):
            ref.assert_rms(o, q, dtype, what, 2)
        for o, q, what in zip(ffn.backward(dy, x, z, u, grad_dtype=F32)[1:], want[1:],
                              ("dw_gate", "dw_up")):
            ref.assert_rms(o, q, dtype, what + " in binary32")
