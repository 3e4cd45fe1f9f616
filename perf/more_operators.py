"""Cases of the mixture-of-experts operators: the router's choice of experts from logits (Router),
its gradient, and a few tokens through their chosen gated experts (GatedExperts).

A case is a plain dict:
  op        route | route_bwd | experts
  t         tokens
  e, top    experts to choose from; chosen for each token
  dtype     bf16 | f16 | f32 (f32: logits only)
  score     softmax | sigmoid       (router)
  norm      weights of a token add up to `scale`  (router)
  scale     factor of the weights   (router)
  masked    some logits are -inf: experts that a token may not use  (router)
  first, n  experts: the rank holds experts [first, first + n) of e
  k, f      experts: features of a token, of an expert's inner layer
  act       experts: the gate's activation
  residual  experts: added to the sum
  pad       extra elements between the rows of logits or x (a slice of a wider buffer)

`own` chooses between the plain form (elementary torch operations in 32 bits, rounded once) and
the framework's operators.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")


def _route(name, op, t, e, top, dtype="f32", score="softmax", norm=True, scale=1.0, masked=False,
           pad=0):
    c = dict(op=op, t=t, e=e, top=top, dtype=dtype, score=score, norm=norm, scale=scale,
             masked=masked, pad=pad)
    if name:
        c["name"] = name
    return c


def _experts(name, t, e, top, k, f, dtype="bf16", act="silu", first=0, n=None, residual=False,
             pad=0):
    c = dict(op="experts", t=t, e=e, top=top, k=k, f=f, dtype=dtype, act=act, first=first,
             n=e if n is None else n, residual=residual, pad=pad)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token's choice in a decode step: latency
        _route("route decode 1", "route", 1, 256, 8),
        # the prompts of 8 ranks x 4096 tokens
        _route("route prompt 32768", "route", 32768, 256, 8),
        # a ragged batch of 16-bit logits, rows of odd length inside a wider buffer, experts that
        # some tokens may not use
        _route("route odd 5003", "route", 5003, 60, 4, "bf16", "sigmoid", True, 2.5, True, 3),
        # a training step's gradient of probabilities over all experts
        _route("route backward 32768", "route_bwd", 32768, 256, 8, "f32", "softmax", False),
        # a short ragged step's, weights that add up to a scale
        _route("route backward 777", "route_bwd", 777, 60, 6, "bf16", "sigmoid", True, 2.5, True),
        # one token through an eighth of small experts' inner features: latency
        _experts("experts decode 1", 1, 64, 6, 2048, 176),
        # a few tokens through an eighth of 14336-wide experts
        _experts("experts decode 4", 4, 8, 2, 4096, 1792, "f16", residual=True),
        # a serving batch on one of 8 ranks that hold 32 experts each: a rank's partial
        _experts("experts serve 32", 32, 256, 8, 7168, 2048, first=64, n=32),
        # the largest batch over whole wide experts
        _experts("experts serve 128", 128, 8, 2, 4096, 14336, residual=True),
        # odd sizes: rows that no 16-byte load lines up with
        _experts("experts odd 37", 37, 20, 4, 1001, 517, "f16", "gelu", pad=5),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def size(lo, hi):
        v, how = spread(lo, hi), rng.random()
        if how < 0.45:  # most widths are multiples of a power of two, some are anything
            return max(lo, v // 64 * 64)
        return max(lo, v // 8 * 8) if how < 0.75 else v

    op = rng.choice(["route", "route_bwd", "experts", "experts", "experts"])
    if op != "experts":
        e = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512, rng.randint(5, 512)])
        t = min(spread(1, 32768), 32768 * 256 // e)
        return _route(None, op, t, e, rng.randint(1, min(e, 12)),
                      rng.choice(["f32", "f32", "bf16", "f16"]),
                      rng.choice(["softmax", "softmax", "sigmoid"]), rng.random() < 0.6,
                      rng.choice([1.0, 1.0, 2.5, 0.7]), rng.random() < 0.2,
                      rng.choice([0, 0, 0, 8, 3]))
    n = rng.choice([4, 8, 8, 16, 20, 32, 64, 128])
    e = n * rng.choice([1, 1, 2, 8])
    k, f = size(128, 8192), size(64, 16384)
    while 6 * n * k * f > 2.8e9:  # bytes of the largest listed case's weights
        if f > k:
            f = f // 2 + 1
        else:
            k = k // 2 + 1
    return _experts(None, spread(1, 128), e, rng.randint(1, min(e, 8)), k, f,
                    rng.choice(["bf16", "bf16", "f16"]), rng.choice(ACTS),
                    n * rng.randrange(e // n), n, rng.random() < 0.4,
                    rng.choice([0, 0, 0, 8, 3]))


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, e, top, dt = case["t"], case["e"], case["top"], DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] != "experts":
        # some experts are liked more than others
        logits = 1.5 * normal(t, e + case["pad"]) + normal(e + case["pad"])
        if case["masked"]:  # an expert in sixteen; now and then fewer are left than are chosen
            share = torch.rand(t, 1, generator=gen, device="cuda").pow(4)
            out = torch.rand(t, e + case["pad"], generator=gen, device="cuda") < share * 1.02
            logits = torch.where(out, torch.full_like(logits, -math.inf), logits)
        s = {"logits": logits.to(dt)[:, :e]}
        if case["op"] == "route_bwd":
            s["g"] = normal(t, top)
            s["ids"] = _choose(s["logits"], top)[0]
        return s
    n, k, f = case["n"], case["k"], case["f"]
    x = normal(t, k + case["pad"])
    # activations with a few loud channels, as a residual stream has them
    loud = torch.rand(k + case["pad"], generator=gen, device="cuda") < 0.01
    s = {"x": (x * (1 + 5 * loud.float())).to(dt)[:, :k]}
    for name, rows, cols in (("wg", f, k), ("wu", f, k), ("wd", k, f)):
        w = torch.empty(n, rows, cols, dtype=dt, device="cuda")
        for i in range(n):
            w[i] = normal(rows, cols).mul_(cols ** -0.5)
        s[name] = w
    ids, picked = _choose(normal(t, e), top)
    s["ids"] = ids
    s["weights"] = torch.softmax(picked, 1)
    if case["residual"]:
        s["r"] = normal(t, k).to(dt)
    return s


def _choose(logits, top):
    """The `top` largest of each row, largest first, ties to the lowest index; -1 for -inf."""
    v, i = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    v, i = v[:, :top], i[:, :top]
    return torch.where(v == -math.inf, torch.full_like(i, -1), i).int(), v


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import collective_datapath_copy_gb300 as cdc

        t, top = case["t"], case["top"]
        if case["op"] == "experts":
            s["op"] = cdc.GatedExperts(s["wg"], s["wu"], s["wd"], act=case["act"],
                                       first=case["first"])
            s["y"] = torch.empty(t, case["k"], dtype=DT[case["dtype"]], device="cuda")
        else:
            s["op"] = cdc.Router(top, score=case["score"], normalize=case["norm"],
                                 scale=case["scale"])
            if case["op"] == "route":
                s["oi"] = torch.empty(t, top, dtype=torch.int32, device="cuda")
                s["ow"] = torch.empty(t, top, dtype=torch.float32, device="cuda")
            else:
                s["dl"] = torch.empty(t, case["e"], dtype=DT[case["dtype"]], device="cuda")
    return s


def _run_own(s):
    op = s["case"]["op"]
    if op == "route":
        return s["op"].forward(s["logits"], ids=s["oi"], weights=s["ow"])
    if op == "route_bwd":
        return s["op"].backward(s["g"], s["logits"], s["ids"], dlogits=s["dl"])
    return s["op"].forward(s["x"], s["ids"], s["weights"], residual=s.get("r"), out=s["y"])


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 2 ** -0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    s = 1 / (1 + torch.exp(-z))
    return s if act == "sigmoid" else z * s


def _scores(logits, score):
    """In 32 bits, over all experts; a row without any is 0."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    top = logits.amax(1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total)


def _plain_route(s):
    c = s["case"]
    logits = s["logits"].float()
    ids, _ = _choose(logits, c["top"])
    there = ids >= 0
    w = torch.gather(_scores(logits, c["score"]), 1, ids.clamp(min=0).long())
    w = torch.where(there, w, torch.zeros_like(w))
    if c["norm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
    return ids, w * c["scale"]


def _plain_route_bwd(s):
    c = s["case"]
    logits, at = s["logits"].float(), s["ids"].clamp(min=0).long()
    there = s["ids"] >= 0
    p = _scores(logits, c["score"])
    w = torch.gather(p, 1, at)
    w = torch.where(there, w, torch.zeros_like(w))
    g = torch.where(there, s["g"] * c["scale"], torch.zeros_like(w))
    if c["norm"]:  # to the gradient of the score itself
        total = w.sum(1, keepdim=True)
        total = torch.where(total == 0, torch.ones_like(total), total)
        w = w / total
        g = (g - (g * w).sum(1, keepdim=True)) / total
    ds = torch.zeros_like(logits).scatter_add(1, at, torch.where(there, g, torch.zeros_like(g)))
    if c["score"] == "sigmoid":
        dl = ds * p / (1 + torch.exp(logits))  # 1 - p without its cancellation
    else:
        dl = p * (ds - (ds * p).sum(1, keepdim=True))
    return dl.to(s["logits"].dtype)


def _plain_experts(s):
    c = s["case"]
    x = s["x"].float()
    y = torch.zeros_like(x)
    for i in range(c["n"]):
        here = s["ids"] == c["first"] + i
        w = torch.where(here, s["weights"], torch.zeros_like(s["weights"])).sum(1, keepdim=True)
        h = _act(x @ s["wg"][i].float().t(), c["act"]) * (x @ s["wu"][i].float().t())
        part = w * (h @ s["wd"][i].float().t())
        y = y + torch.where(here.any(1, keepdim=True), part, torch.zeros_like(part))
    if "r" in s:
        y = y + s["r"].float()
    return y.to(s["x"].dtype)


def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "route_bwd": _plain_route_bwd,
            "experts": _plain_experts}[state["case"]["op"]](state)


def exact(case, seed):
    """The same outputs from the definitions in 64 bits: probabilities through log-sums, the
    gradient as a product with the scores' Jacobian, each expert over its own tokens."""
    s = _inputs(case, seed)
    if case["op"] == "experts":
        def act(z):
            name = case["act"]
            if name == "relu":
                return z.clamp(min=0)
            if name == "gelu":
                return z * torch.special.ndtr(z)
            if name == "gelu_tanh":  # (1 + tanh(a)) / 2 is the logistic function of 2a
                return z * torch.special.expit(
                    2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            sg = torch.special.expit(z)
            return sg if name == "sigmoid" else z * sg

        y = s["r"].double() if "r" in s else torch.zeros(case["t"], case["k"], device="cuda",
                                                         dtype=torch.float64)
        for i in range(case["n"]):
            tok, slot = torch.nonzero(s["ids"] == case["first"] + i, as_tuple=True)
            if len(tok) == 0:
                continue
            x = s["x"][tok].double()
            h = act(torch.einsum("tk,fk->tf", x, s["wg"][i].double()))
            h = h * torch.einsum("tk,fk->tf", x, s["wu"][i].double())
            part = torch.einsum("tf,kf->tk", h, s["wd"][i].double())
            y.index_add_(0, tok, part * s["weights"][tok, slot].double()[:, None])
        return y
    logits = s["logits"].double()
    if case["score"] == "softmax":
        lse = torch.logsumexp(logits, 1, keepdim=True)
        log_p = torch.where(lse == -math.inf, torch.full_like(logits, -math.inf), logits - lse)
    else:
        log_p = -torch.logaddexp(torch.zeros_like(logits), -logits)
    # one chosen expert after the other: the first largest of those left
    left, chosen, rows = logits.clone(), [], torch.arange(case["t"], device="cuda")
    for _ in range(case["top"]):
        best = left.amax(1, keepdim=True)
        index = torch.arange(case["e"], device="cuda").expand_as(left)
        i = torch.where(left == best, index, torch.full_like(index, case["e"])).amin(1)
        chosen.append(torch.where(best[:, 0] == -math.inf, torch.full_like(i, -1), i))
        left[rows, i] = -math.inf
    ids = torch.stack(chosen, 1)
    there = ids >= 0
    lw = torch.gather(log_p, 1, ids.clamp(min=0))
    lw = torch.where(there, lw, torch.full_like(lw, -math.inf))
    if case["norm"]:
        total = torch.logsumexp(lw, 1, keepdim=True)
        lw = torch.where(there, lw - total, lw)
    w = torch.exp(lw)
    if case["op"] == "route":
        return ids.int(), w * case["scale"]
    gw = torch.where(there, s["g"].double() * w, torch.zeros_like(w)) * case["scale"]
    if case["norm"]:  # gradient of the chosen log-scores
        gw = gw - w * gw.sum(1, keepdim=True)
    d = torch.zeros_like(logits).scatter_add(1, ids.clamp(min=0), torch.where(
        there, gw, torch.zeros_like(gw)))
    if case["score"] == "sigmoid":
        return d * torch.special.expit(-logits)
    return d if case["norm"] else d - torch.exp(log_p) * gw.sum(1, keepdim=True)


def work(case):
    t, e, top = case["t"], case["e"], case["top"]
    if case["op"] != "experts":
        size = SIZE[case["dtype"]]
        if case["op"] == "route":
            return {"bytes": t * e * size + 8 * t * top, "flops": 3 * t * e}
        # normalised weights depend on the chosen logits alone
        read = top if case["norm"] or case["score"] == "sigmoid" else e
        return {"bytes": t * (e + read) * size + 8 * t * top, "flops": 4 * t * e}
    n, k, f = case["n"], case["k"], case["f"]
    # experts are chosen alike: how many of this rank's some token asks for, and how often
    used = n * (1 - (1 - top / e) ** t)
    rows = t * top * n / e
    return {"bytes": int(6 * used * k * f) + 2 * t * k * (3 if case["residual"] else 2)
            + 8 * t * top, "flops": int(6 * rows * k * f)}
