"""64-bit references of the mixture-of-experts operators and the error bounds their tests use.

u = 2^-24 is half a step of binary32. The exponential, log1p and a division are good to two steps, 2^-22
relative; a sum of n binary32 terms in any order to (n + 4) u of the terms' magnitudes.

Weights over the chosen: exp(a_j - a_0) / sum. The difference is rounded (u |a_j - a_0|); for the
sigmoid a = min(l, 0) - log1p(exp(-|l|)) is itself off by at most 2^-21 + u |a|. So a term is off by
2^-20 + 2^-23 D relative, D the largest |a| in play, and a quotient by twice that and the sum's share.
"""

import math

import torch

import dense_ref as ref

U32 = 2.0 ** -24
TINY32 = 2.0 ** -124  # below it binary32 exponentials lose their relative precision


def choose(logits, top):
    """ids by definition: largest first, ties to the lowest index, NaN the largest, -inf never."""
    l = logits.double()
    key = torch.where(l.isnan(), torch.full_like(l, math.inf), l)
    # NaN above +inf: a second, stable sort on that alone
    order = torch.sort(key, dim=1, descending=True, stable=True)[1]
    nan = torch.gather(l, 1, order).isnan()
    order = torch.gather(order, 1, torch.sort(nan.int(), dim=1, descending=True, stable=True)[1])
    ids = order[:, :top]
    return torch.where(torch.gather(l, 1, ids) == -math.inf, torch.full_like(ids, -1), ids)


def _from_most(logits):
    """64 bits next to a type's lowest value are coarse, so the logits relative to the largest."""
    l = logits.double()
    most = l.amax(1, keepdim=True)
    return torch.where(most.isfinite(), l - most, l)


def _chosen(logits, ids, score):
    l = logits.double()
    if score == "softmax":
        l = _from_most(logits)
    there = (ids >= 0) & (ids < l.shape[1])
    lc = torch.gather(l, 1, ids.clamp(0, l.shape[1] - 1).long())
    if score == "sigmoid":
        a = -torch.logaddexp(torch.zeros_like(lc), -lc)
        lse = torch.zeros(l.shape[0], 1, dtype=l.dtype, device=l.device)
    else:
        a = lc
        lse = torch.logsumexp(l, 1, keepdim=True)
    return there, lc, a, lse


def weights(logits, ids, score, normalize):
    """(w, relative bound) without the scale, of shape [t, top]."""
    there, lc, a, lse = _chosen(logits, ids, score)
    low = torch.full_like(a, -math.inf)
    if normalize:
        a = torch.where(there, a, low)
        most = a.amax(1, keepdim=True)
        a = torch.where(most.isfinite(), a - most, a)
        lse = torch.logsumexp(a, 1, keepdim=True)
    w = torch.where(there, torch.exp(a - lse), torch.zeros_like(a))
    top, e = ids.shape[1], logits.shape[1]
    if not normalize and score == "sigmoid":
        return w, torch.full_like(w, 2.0 ** -20)
    if normalize:
        far = torch.where(there, lc, torch.zeros_like(lc)).abs().amax(1, keepdim=True) * 2
    else:
        l = logits.double()
        far = torch.where(l.isfinite(), l, torch.zeros_like(l)).abs().amax(1, keepdim=True) * 2
    # terms too far below the largest to matter: their share of the sum is nothing
    far = far.clamp(max=120.0)
    n = top if normalize else e
    return w, 2 * (2.0 ** -20 + 2.0 ** -23 * far) + (n + 8) * U32 + torch.zeros_like(w)


def route(logits, top, score, normalize, scale):
    """ids, and (weights, bound)."""
    ids = choose(logits, top)
    w, rel = weights(logits, ids, score, normalize)
    return ids, (w * scale, (w * (rel + 4 * U32) + TINY32) * abs(scale) * 1.01)


def route_bwd(dw, logits, ids, score, normalize, scale):
    """(dlogits, bound)."""
    there, lc, a, lse = _chosen(logits, ids, score)
    w, rel = weights(logits, ids, score, normalize)
    g = torch.where(there, dw.double() * scale, torch.zeros_like(w))
    gw, top = g * w, ids.shape[1]
    rest = (top + 8) * U32
    out = torch.zeros(logits.shape, dtype=torch.float64, device=logits.device)
    err = torch.zeros_like(out)
    at = ids.clamp(0, logits.shape[1] - 1).long()

    def scatter(d, ed):
        out.scatter_add_(1, at, torch.where(there, d, torch.zeros_like(d)))
        err.scatter_add_(1, at, torch.where(there, ed + top * U32 * d.abs(), torch.zeros_like(d)))

    s = gw.sum(1, keepdim=True)
    es = (gw.abs() * (rel + rest)).sum(1, keepdim=True)
    if normalize or score == "sigmoid":
        if normalize:
            d = w * (g - s)
            ed = w * (es + 4 * U32 * (g.abs() + s.abs())) + d.abs() * (rel + 8 * U32)
        else:
            d, ed = gw, gw.abs() * (rel + 8 * U32)
        if score == "sigmoid":
            n = torch.special.expit(-lc)
            d, ed = d * n, ed * n + d.abs() * n * 2.0 ** -20
        scatter(d, ed)
    else:
        p = torch.exp(_from_most(logits) - lse)
        p = torch.where(lse == -math.inf, torch.zeros_like(p), p)
        r = rel[:, :1]
        scatter(gw, gw.abs() * (rel + 8 * U32))
        out -= p * s
        err += p * (s.abs() * (r + 8 * U32) + es) + 4 * U32 * (p * s).abs()
    err = err + TINY32 * (1 + g.abs().amax(1, keepdim=True))
    return out, (err + ref.rounded(out, logits.dtype) + U32 * out.abs()) * 1.02


def experts(x, ids, weights, wg, wu, wd, act, first, residual, out_dtype):
    """(y, bound): the inner values are rounded to the operands' type once (dense_ref.gated's bound),
    the sums over features, choices and the residual are in binary32."""
    dt = wg.dtype
    m, n = x.shape[0], wd.shape[1]
    y = torch.zeros(m, n, dtype=torch.float64, device=x.device)
    size, err = torch.zeros_like(y), torch.zeros_like(y)
    for e in range(wg.shape[0]):
        tok, slot = torch.nonzero(ids == first + e, as_tuple=True)
        if len(tok) == 0:
            continue
        (h, eh), _, _ = ref.gated(x[tok], wg[e], wu[e], act, dt)
        p, ep = ref.mm(h, wd[e].double())
        ep = ep + eh @ wd[e].double().abs().t()
        w = weights[tok, slot].double()[:, None]
        y.index_add_(0, tok, w * p)
        size.index_add_(0, tok, (w * p).abs())
        err.index_add_(0, tok, w.abs() * ep)
    if residual is not None:
        y = y + residual.double()
        size = size + residual.double().abs()
    err = err + (ids.shape[1] + 8) * 2.0 ** -22 * (size + err)
    return y, (err + ref.rounded(y, out_dtype)) * 1.02
