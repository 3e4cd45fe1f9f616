"""A prompt's way through a mixture of experts: Router's ids as the table of a dispatch plan, the rows
through their experts on the ranks they went to, and a combine plan, against a 64-bit reference."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import collective_datapath_copy_gb300 as cdc  # noqa: E402
from collective_datapath_copy_gb300.build import build  # noqa: E402
import dense_ref as ref  # noqa: E402
import experts_ref as er  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    yield
    torch.cuda.synchronize()


def by_experts(rows, ids, w, wg, wu, wd, first):
    return cdc.GatedExperts(wg, wu, wd, first=first).forward(rows, ids, w)


def by_products(rows, ids, w, wg, wu, wd, first):
    y = torch.zeros(len(rows), wd.shape[1], device="cuda")
    for e in range(len(wg)):
        tok, slot = torch.nonzero(ids == first + e, as_tuple=True)
        if len(tok):
            h = cdc.GatedFFN(wg[e], wu[e]).forward(rows[tok])
            out = cdc.Linear(wd[e]).forward(h, out_dtype=F32)
            y.index_add_(0, tok, out * w[tok, slot][:, None])
    return y.to(BF)


@pytest.mark.parametrize("zero_copy", [0, 1])
@pytest.mark.parametrize("through", [by_experts, by_products])
@pytest.mark.parametrize("R,T,E,K,F,top", [(2, 24, 8, 128, 72, 2), (4, 50, 16, 256, 96, 3)])
def test_router_dispatch_experts_combine(R, T, E, K, F, top, through, zero_copy):
    g = torch.Generator(device="cuda").manual_seed(T)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)
    wg, wu = (normal(E, F, K, scale=K ** -0.5) for _ in range(2))
    wd = normal(E, K, F, scale=F ** -0.5)
    x = normal(R, T, K)
    logits = torch.randn(R, T, E, generator=g, device="cuda")
    logits[0, 3] = logits[1, :2] = -float("inf")  # no expert for these
    logits[1, 5, 1:] = -float("inf")              # one
    ids, w = cdc.Router(top).forward(logits)
    e = E // R
    table = ids.cpu().numpy()
    there, back = cdc.moe_dispatch(table, e, K), cdc.moe_combine(table, e, K)
    dest = torch.from_numpy(there.meta["dest"]).cuda()
    counts = there.meta["counts"]
    assert int((~dest.any(2)).sum()) == 3

    def buffers(lens):
        return [torch.full((n,), -7, dtype=torch.int16, device="cuda") for n in lens]
    got, out = buffers(there.out_len), buffers(back.out_len)
    plan = cdc.Plan(there, zero_copy=zero_copy)
    plan.run([t.view(torch.int16).reshape(-1) for t in x], got)
    parts = []
    for d in range(R):
        here = dest[:, :, d]  # in the order of the rows
        rows = got[d].view(BF).view(-1, K)[:counts[d]]
        assert torch.equal(rows, x[here])
        y = torch.zeros(back.in_len[d], dtype=BF, device="cuda")
        y[:counts[d] * K] = through(rows, ids[here], w[here], wg[d * e:][:e], wu[d * e:][:e],
                                    wd[d * e:][:e], d * e).reshape(-1)
        parts.append(y.view(torch.int16))
    combine = cdc.Plan(back, zero_copy=zero_copy)
    combine.run(parts, out)
    assert plan.status()["code"] == 0 and combine.status()["code"] == 0
    y = torch.stack([t.view(BF).view(T, K) for t in out])
    # the ranks' partials are rounded, and then their sum in binary32
    want = torch.zeros(R * T, K, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    for d in range(R):
        s = slice(d * e, (d + 1) * e)
        p, ep = er.experts(x.view(-1, K), ids.view(-1, top), w.view(-1, top), wg[s], wu[s], wd[s],
                           "silu", d * e, None, BF)
        want, bound = want + p, bound + ep
    bound = bound + R * 2.0 ** -23 * (want.abs() + bound)
    bound = bound + ref.rounded(want.abs() + bound, BF)
    routed = dest.any(2).view(-1)
    ref.assert_close(y.view(-1, K)[routed], (want[routed], bound[routed]), "y")
    assert bool((y.view(torch.int16).view(-1, K)[~routed] == -7).all())  # as they were
