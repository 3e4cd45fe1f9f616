"""The expert-parallel mixture of experts: Linear, Router, GatedExperts and the all-reduce together,
against a 64-bit reference."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300 import _lib  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import dense_ref as ref  # noqa: E402
import experts_ref as er  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    yield
    torch.cuda.synchronize()


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


CASES = [(1, 4, 16, 256, 72, 4, "softmax", True, "bf16", BF),
         (8, 8, 64, 512, 96, 8, "sigmoid", True, "bf16", BF),
         (33, 2, 8, 264, 136, 2, "softmax", False, "f32", BF),
         (40, 3, 12, 128, 77, 3, "sigmoid", False, "f32", HF),
         (150, 4, 32, 512, 128, 6, "softmax", True, "bf16", BF)]


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    tokens, R, E, K, F, top, score, norm, partials, dtype = case
    g = torch.Generator(device="cuda").manual_seed(tokens)
    wr = normal(g, E, K, dtype=dtype, scale=K ** -0.5)
    wg, wu = (normal(g, E, F, K, dtype=dtype, scale=K ** -0.5) for _ in range(2))
    wd = normal(g, E, K, F, dtype=dtype, scale=F ** -0.5)
    x, res = (normal(g, tokens, K, dtype=dtype) for _ in range(2))
    moe = cdc.ExpertParallelMoE(R, wr, wg, wu, wd, top, tokens, score=score, normalize=norm,
                                scale=1.5, partials=partials)
    ys, ids, w = moe.forward(x, residual=res, routing=True)
    assert all(torch.equal(ys[0], y) for y in ys)
    # the choice: by the logits that Linear gives, which are held to their own bound
    logits = moe.gate.forward(x, out_dtype=F32)
    ref.assert_close(logits, ref.linear(x, wr, None, None, "none", F32, dtype)[0], "logits")
    want_ids, want_w = er.route(logits, top, score, norm, 1.5)
    assert torch.equal(ids.long(), want_ids)
    ref.assert_close(w, want_w, "weights")
    ptype = F32 if partials == "f32" else BF
    e = E // R
    y = torch.zeros(tokens, K, dtype=torch.float64, device="cuda")
    ey = torch.zeros_like(y)
    for r in range(R):
        s = slice(r * e, (r + 1) * e)
        p, ep = er.experts(x, ids, w, wg[s], wu[s], wd[s], "silu", r * e,
                           res.to(ptype) if r == 0 else None, ptype)
        y, ey = y + p, ey + ep
    ey = ey + R * 2.0 ** -23 * (y.abs() + ey) + ref.rounded(y.abs() + ey, ptype)
    ref.assert_close(ys[0], (y, ey), "y")
    assert moe.status() == _lib.OK
    again = moe.forward(x, residual=res)
    assert torch.equal(again[0], ys[0])


def test_one_rank_is_the_whole():
    g = torch.Generator(device="cuda").manual_seed(3)
    wr, x = normal(g, 8, 128, dtype=BF), normal(g, 20, 128, dtype=BF)
    wg, wu, wd = (normal(g, 8, *s, dtype=BF, scale=0.1) for s in ((72, 128), (72, 128), (128, 72)))
    one = cdc.ExpertParallelMoE(1, wr, wg, wu, wd, 3, 20)
    y, ids, w = one.forward(x, routing=True)
    assert torch.equal(y[0], cdc.GatedExperts(wg, wu, wd).forward(x, ids, w))
    wd.mul_(2)  # the shards are views
    assert torch.equal(one.forward(x)[0], cdc.GatedExperts(wg, wu, wd).forward(x, ids, w))


def test_a_training_steps_routing_gradient():
    """Choice, dispatch order, experts one by one with their gradients, and the router's gradient
    from theirs, against autograd of the whole in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(4)
    T, E, K, F, top = 48, 6, 64, 96, 2
    wr = normal(g, E, K, dtype=BF, scale=K ** -0.5)
    wg, wu = (normal(g, E, F, K, dtype=BF, scale=K ** -0.5) for _ in range(2))
    wd = normal(g, E, K, F, dtype=BF, scale=F ** -0.5)
    x, dy = normal(g, T, K, dtype=BF), normal(g, T, K, dtype=BF)
    router, gate = cdc.Router(top), cdc.Linear(wr)
    logits = gate.forward(x, out_dtype=F32)
    ids, w = router.forward(logits)
    dw = torch.zeros_like(w)
    for e in range(E):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if len(tok):
            out = cdc.Linear(wd[e]).forward(cdc.GatedFFN(wg[e], wu[e]).forward(x[tok]),
                                            out_dtype=F32)
            dw[tok, slot] = (out * dy[tok].float()).sum(1)
    dlogits = router.backward(dw, logits, ids)
    _, dwr, _ = gate.backward(dlogits.bfloat16(), x, need_dx=False, grad_dtype=F32)
    r64 = wr.double().requires_grad_()
    l64 = x.double() @ r64.t()
    w64 = torch.softmax(torch.gather(l64, 1, ids.long()), 1)
    loss = torch.zeros((), dtype=torch.float64, device="cuda")
    for e in range(E):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        xe = x[tok].double()
        h = torch.nn.functional.silu(xe @ wg[e].double().t()) * (xe @ wu[e].double().t())
        loss = loss + (w64[tok, slot][:, None] * (h @ wd[e].double().t()) * dy[tok].double()).sum()
    loss.backward()
    err = (dwr.double() - r64.grad).norm() / r64.grad.norm()
    # the inner values and dlogits are rounded to bf16 on the way, 2^-8 at most each; as much again
    # for the binary32 logits and sums
    assert float(err) <= 3 * 2.0 ** -8


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(6)
    wr, wg, wd = (normal(g, *s, dtype=BF) for s in ((8, 32), (8, 64, 32), (8, 32, 64)))
    for args in ((3, wr, wg, wg, wd, 2, 8), (2, wr[:4], wg, wg, wd, 2, 8),
                 (2, wr, wg, wg, wg, 2, 8), (2, wr, wg, wg, wd, 9, 8), (0, wr, wg, wg, wd, 2, 8)):
        with pytest.raises(ValueError):
            cdc.ExpertParallelMoE(*args)
    with pytest.raises(ValueError):
        cdc.ExpertParallelMoE(2, wr.half(), wg.half(), wg.half(), wd.half(), 2, 8)
    with pytest.raises(ValueError):
        cdc.ExpertParallelMoE(2, wr, wg, wg, wd, 2, 8, partials="f64")
