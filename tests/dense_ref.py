"""64-bit references of the dense operators and the error bounds their tests use.

u(T) is the unit roundoff of an output type: 2^-8 (bf16), 2^-11 (f16), 2^-24 (f32). A product of
length K accumulated in binary32, in any order and with truncating adders, is off by at most
K * 2^-22 * (|a| |b|): each of its K adds loses less than 2^-23 of the running magnitude, doubled
for the alignment inside a matrix instruction. An activation's value has a slope of at most 1.13
and its evaluation is good to 2^-19 of the argument's magnitude. A rounding to T adds u(T) of the
value, and in f16 2^-25 below the normal range.
"""

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def act(z, name):
    """(value, slope) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return (0.5 * z * (1 + t),
                0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z))
    s = torch.sigmoid(z)
    return (s, s * (1 - s)) if name == "sigmoid" else (z * s, s + z * s * (1 - s))


def mm(a, b):
    """Product and its accumulation bound."""
    k = a.shape[-1]
    return a @ b.t(), (k + 1) * 2.0 ** -22 * (a.abs() @ b.abs().t())


def rounded(v, dtype):
    return U[dtype] * v.abs() + TINY[dtype]


def linear(x, w, b, r, name, out_dtype, pre_dtype):
    """[(value, bound)] of y and pre."""
    x, w = x.double(), w.double()
    z, ez = mm(x, w)
    if b is not None:
        z = z + b.double()
        ez = ez + 2.0 ** -23 * z.abs()
    y, _ = act(z, name)
    ey = 1.13 * ez + 2.0 ** -19 * z.abs() * (name != "none")
    if r is not None:
        y = y + r.double()
        ey = ey + 2.0 ** -23 * y.abs()
    return (y, (ey + rounded(y, out_dtype)) * 1.01), (z, (ez + rounded(z, pre_dtype)) * 1.01)


def _slope_bound(z):
    return 2.0 ** -18 * (1 + z.abs())


def linear_bwd(dy, z, x, w, name, dtype, grad_dtype):
    """[(value, bound)] of dx, dw and db; dz is rounded to dtype before the products."""
    dy, x, w = dy.double(), x.double(), w.double()
    if name == "none":
        dz, ed = dy, torch.zeros_like(dy)
        er = ed
    else:
        d = act(z.double(), name)[1]
        dz = dy * d
        ed = dy.abs() * _slope_bound(z.double())
        er = ed + rounded(dz, dtype)
    dx, e1 = mm(dz, w.t())
    dw, e2 = mm(dz.t(), x.t())
    db = dz.sum(0)
    e1 = e1 + er @ w.abs()
    e2 = e2 + er.t() @ x.abs()
    e3 = ed.sum(0) + (dz.shape[0] + 1) * 2.0 ** -23 * dz.abs().sum(0)
    return [(v, (e + rounded(v, t)) * 1.02) for v, e, t in
            ((dx, e1, dtype), (dw, e2, grad_dtype), (db, e3, grad_dtype))]


def gated(x, wg, wu, name, dtype):
    """[(value, bound)] of h, gate and up."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, eg = mm(x, wg)
    u, eu = mm(x, wu)
    a, _ = act(g, name)
    h = a * u
    ea = 1.13 * eg + 2.0 ** -19 * (1 + g.abs())
    eh = ea * u.abs() + a.abs() * eu + ea * eu
    return [(v, (e + rounded(v, dtype)) * 1.01) for v, e in ((h, eh), (g, eg), (u, eu))]


def gated_bwd(dh, g, u, x, wg, wu, name, dtype, grad_dtype):
    """[(value, bound)] of dx, dw_gate and dw_up."""
    dh, g, u, x, wg, wu = (t.double() for t in (dh, g, u, x, wg, wu))
    a, d = act(g, name)
    dg, du = dh * u * d, dh * a
    eg = (dh * u).abs() * _slope_bound(g) + rounded(dg, dtype)
    eu = dh.abs() * _slope_bound(g) + rounded(du, dtype)
    p, ep = mm(dg, wg.t())
    q, eq = mm(du, wu.t())
    dx = p + q
    ex = ep + eq + eg @ wg.abs() + eu @ wu.abs() + 2.0 ** -22 * (p.abs() + q.abs())
    dwg, e1 = mm(dg.t(), x.t())
    dwu, e2 = mm(du.t(), x.t())
    return [(v, (e + rounded(v, t)) * 1.02) for v, e, t in
            ((dx, ex, dtype), (dwg, e1 + eg.t() @ x.abs(), grad_dtype),
             (dwu, e2 + eu.t() @ x.abs(), grad_dtype))]


def assert_close(got, ref, what=""):
    """Every element within its bound. The bound grows with K and the error does not: over a long
    sum a lost block of k passes it, and assert_rms has to look at the whole."""
    want, bound = ref
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if want.numel() == 0:
        return
    err = (got - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(err[bad].max()) if bad.any() else 0,
                           tuple(torch.nonzero(bad)[0].tolist()))


def assert_rms(got, ref, dtype, what="", times=1.0):
    """The root mean square of the error within `times` the rounding of `dtype` (2 for an output
    whose dz was rounded on the way)."""
    want = ref[0]
    err = (got.double() - want).square().mean().sqrt()
    size = want.square().mean().sqrt()
    assert float(err) <= times * U[dtype] * float(size) + TINY[dtype] + 1e-300, \
        (what, float(err), float(size))
