"""Slopes and values of the activations at the ends of the types' ranges."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import dense_ref as ref  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
FAR = [s * v for v in (300.0, 1e3, 6e4, 1e10, 1e19, 1e20, 1e30, 3.3e38) for s in (1, -1)]
LEAST = 2.0 ** -126   # results below the normal range are zero


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("n", [16, 15])
def test_slopes_of_linear(act, n):
    """One token and dy = 1: db is the slope itself, in binary32. It is 0 or 1 this far out."""
    z = torch.tensor(FAR[:n], device="cuda").to(BF)[None]
    w, x = torch.ones(n, 8, dtype=BF, device="cuda"), torch.zeros(1, 8, dtype=BF, device="cuda")
    lin = cdc.Linear(w, None, act)
    db = lin.backward(torch.ones_like(z), x, pre=z, need_dx=False, need_dw=False, need_db=True,
                      grad_dtype=F32)[2]
    assert ((db.double() - ref.act(z[0].double(), act)[1]).abs() <= LEAST).all()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "sigmoid"])
@pytest.mark.parametrize("n", [16, 15])
def test_slopes_and_values_of_the_gated_block(act, n):
    """x = 1 and one token: dw_gate is dh u act'(g), dw_up is dh act(g)."""
    g = torch.tensor(FAR[:n], device="cuda").to(BF)[None]
    w, x = torch.ones(n, 8, dtype=BF, device="cuda"), torch.ones(1, 8, dtype=BF, device="cuda")
    ffn = cdc.GatedFFN(w, w.clone(), act)
    _, dg, du = ffn.backward(torch.ones_like(g), x, g, torch.ones_like(g), need_dx=False,
                             grad_dtype=F32)
    value, slope = ref.act(g[0].double(), act)
    assert ((dg[:, 0].double() - slope).abs() <= LEAST).all()
    assert ((du[:, 0].double() - value).abs() <= LEAST).all()


# relative error of gelu for negative arguments: the polynomial's own in each range (its ratio to
# the distribution function in 64 bits, at the far end: 3.04e-6, 5.13e-5, 4.671e-4, 1.582e-3, 3.582e-3,
# 1.025e-2), and 2^-19 for its evaluation
@pytest.mark.parametrize("lo,hi,own", [(-2, -0.01, 3.2e-6), (-3, -2, 5.2e-5), (-4, -3, 4.7e-4),
                                       (-5, -4, 1.59e-3), (-6, -5, 3.6e-3), (-8, -6, 1.03e-2)])
def test_gelu_of_negative_arguments(lo, hi, own):
    x = torch.linspace(lo, hi, 500, device="cuda").to(torch.float16).clamp(lo, hi)[:, None]
    y = cdc.Linear(torch.ones_like(x[:1]), None, "gelu").forward(x, out_dtype=F32)
    want = ref.act(x.double(), "gelu")[0]
    assert float(((y.double() - want) / want).abs().max()) <= own + 2.0 ** -19
