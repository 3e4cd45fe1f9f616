"""The tensor-parallel MLP: dense operators around the all-reduce, against a 64-bit reference."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import dense_ref as ref  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    yield
    torch.cuda.synchronize()


def normal(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


CASES = [(1, 4, 256, 512, "bf16"), (8, 8, 512, 1024, "f32"), (40, 2, 128, 320, "bf16"),
         (200, 4, 512, 768, "bf16"), (300, 3, 264, 600, "f32")]


@pytest.mark.parametrize("tokens,R,K,F,partials", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_forward_and_backward(tokens, R, K, F, partials, dtype):
    if dtype is torch.float16:
        partials = "f32"
    g = torch.Generator(device="cuda").manual_seed(tokens)
    wg, wu = (normal(g, F, K, dtype=dtype, scale=K ** -0.5) for _ in range(2))
    wd = normal(g, K, F, dtype=dtype, scale=F ** -0.5)
    x, res, dy = (normal(g, tokens, K, dtype=dtype) for _ in range(3))
    mlp = cdc.TensorParallelMLP(R, wg, wu, wd, tokens, partials=partials)
    ys = mlp.forward(x, residual=res, keep=True)
    dxs, grads = mlp.backward(dy)
    assert all(torch.equal(ys[0], y) for y in ys) and all(torch.equal(dxs[0], d) for d in dxs)
    f, u = F // R, ref.U[dtype]
    ptype = torch.bfloat16 if partials == "bf16" else torch.float32
    y, ey = res.double(), torch.zeros(tokens, K, dtype=torch.float64, device="cuda")
    dx, ex = torch.zeros_like(y), torch.zeros_like(y)
    for r in range(R):
        s = slice(r * f, (r + 1) * f)
        (h, eh), (gate, _), (up, _) = ref.gated(x, wg[s], wu[s], "silu", dtype)
        p, ep = ref.mm(h, wd[:, s].double())
        ep = ep + eh @ wd[:, s].double().abs().t()
        y = y + p
        # rank 0's partial is rounded with the residual in it
        ey = ey + ep + ref.rounded(p + (res.double() if r == 0 else 0), ptype)
        # backward from what the forward kept
        hk, gk, uk = mlp._kept[1][r]
        (dh, edh), (dwd, edwd), _ = ref.linear_bwd(dy, None, hk, wd[:, s], "none", dtype, dtype)
        ref.assert_close(grads[r][2], (dwd, edwd), "dw_down")
        dhk = mlp.down[r].backward(dy, hk, need_dw=False)[0]
        ref.assert_close(dhk, (dh, edh), "dh")
        want = ref.gated_bwd(dhk, gk, uk, x, wg[s], wu[s], "silu", dtype, dtype)
        ref.assert_close(grads[r][0], want[1], "dw_gate")
        ref.assert_close(grads[r][1], want[2], "dw_up")
        dx, ex = dx + want[0][0], ex + want[0][1]
    sums = R * 2.0 ** -23
    ref.assert_close(ys[0], (y, ey + sums * (y.abs() + ey) + ref.rounded(y, ptype)), "y")
    gt = torch.bfloat16 if dtype is torch.bfloat16 else torch.float32
    ref.assert_close(dxs[0], (dx, ex + sums * (dx.abs() + ex) + ref.rounded(dx, gt) * 1.01
                              + u * ex), "dx")


def test_shards_follow_the_weights():
    g = torch.Generator(device="cuda").manual_seed(5)
    BF = torch.bfloat16
    wg, wu, wd = (normal(g, *s, dtype=BF, scale=0.1) for s in ((64, 32), (64, 32), (32, 64)))
    x = normal(g, 8, 32, dtype=BF)
    mlp = cdc.TensorParallelMLP(2, wg, wu, wd, 8)
    y = mlp.forward(x)[0].clone()
    wd.mul_(2)
    assert torch.equal(mlp.forward(x)[0], y * 2)


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(6)
    BF = torch.bfloat16
    wg, wd = normal(g, 64, 32, dtype=BF), normal(g, 32, 64, dtype=BF)
    for args in ((3, wg, wg, wd, 8), (2, wg, wg, wg, 8), (0, wg, wg, wd, 8)):
        with pytest.raises(ValueError):
            cdc.TensorParallelMLP(*args)
    with pytest.raises(ValueError):
        cdc.TensorParallelMLP(2, wg.half(), wg.half(), wd.half(), 8)
    with pytest.raises(ValueError):
        cdc.TensorParallelMLP(2, wg, wg, wd, 8, partials="f64")
    with pytest.raises(RuntimeError):
        cdc.TensorParallelMLP(2, wg, wg, wd, 8).backward(wg)
