"""Cases of the dense operators beside the collectives: Linear (a matrix product with bias,
activation and residual in its epilogue) and GatedFFN (gate and up projections, activation and
product), forward and backward.

A case is a plain dict:
  op       linear | linear_bwd | gated | gated_bwd
  m, n, k  tokens, output features (of gate and of up for the gated operators), input features
  dtype    bf16 | f16
  act      the activation
  bias, residual, save   Linear: with a bias, with a residual; both: keep what backward needs
  wt       the weights are stored transposed ([k][n]) and passed as a view
  pad      extra elements between the rows of x (a slice of a wider buffer)

`own` chooses between the plain form (elementary torch operations in 32 bits, rounded once) and
the framework's operators.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
LINEAR_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
GATED_ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")


def _case(name, op, m, n, k, dtype="bf16", act="none", bias=False, residual=False, save=False,
          wt=False, pad=0):
    c = dict(op=op, m=m, n=n, k=k, dtype=dtype, act=act, bias=bias, residual=residual, save=save,
             wt=wt, pad=pad)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token through a row-parallel shard (an eighth of a 14336-wide block) into the 8 KiB
        # payload of the decode all-reduce: latency
        _case("linear decode 1", "linear", 1, 4096, 1792, residual=True),
        # a small serving batch through a full projection with a bias
        _case("linear decode 24", "linear", 24, 6144, 4096, "f16", bias=True),
        # a prompt through a projection with everything in the epilogue
        _case("linear prompt 2048", "linear", 2048, 4096, 4096, act="gelu", bias=True,
              residual=True),
        # odd sizes: rows that no 16-byte load lines up with, x a slice of a wider buffer
        _case("linear odd 1237", "linear", 1237, 2050, 1001, "f16", act="gelu_tanh", bias=True,
              pad=5),
        # a training step's backward: dx, dW, db
        _case("linear backward 4096", "linear_bwd", 4096, 4096, 4096, act="gelu", bias=True),
        # a short ragged batch's backward, weights stored transposed
        _case("linear backward 777", "linear_bwd", 777, 1530, 1016, "f16", act="silu", bias=True,
              wt=True),
        # one token through a column-parallel shard of a gated block
        _case("gated decode 1", "gated", 1, 1792, 4096, act="silu"),
        # a serving batch through a whole gated block
        _case("gated decode 48", "gated", 48, 14336, 4096, act="silu"),
        # odd sizes, a prompt chunk
        _case("gated odd 300", "gated", 300, 5461, 2056, "f16", act="gelu"),
        # a training step's forward, keeping gate and up for the backward
        _case("gated train 8192", "gated", 8192, 14336, 4096, act="silu", save=True),
        # its backward over half as many tokens: dx, dWg, dWu
        _case("gated backward 4096", "gated_bwd", 4096, 14336, 4096, act="silu"),
        # a short backward with odd sizes
        _case("gated backward 513", "gated_bwd", 513, 2731, 1000, "f16", act="gelu_tanh"),
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        how = rng.random()
        if how < 0.4:  # most widths are multiples of a power of two, some are anything
            v = max(lo, v // 64 * 64)
        elif how < 0.7:
            v = max(lo, v // 8 * 8)
        return v

    op = rng.choice(["linear", "linear", "linear_bwd", "gated", "gated", "gated_bwd"])
    most = 1.9e12  # flops of the largest listed case
    per = {"linear": 2, "linear_bwd": 4, "gated": 4, "gated_bwd": 8}[op]
    m = int(round(math.exp(rng.uniform(0, math.log(8192)))))
    n, k = size(64, 16384), size(64, 16384)
    while per * m * n * k > most:
        if m > 256 and rng.random() < 0.5:
            m = m // 2 + 1
        elif n > k:
            n = n // 2 + 1
        else:
            k = k // 2 + 1
    if op.endswith("bwd"):
        m = max(m, 2)
    lin = op.startswith("linear")
    return _case(None, op, m, n, k, rng.choice(["bf16", "f16"]),
                 rng.choice(LINEAR_ACTS if lin else GATED_ACTS), bias=lin and rng.random() < 0.6,
                 residual=op == "linear" and rng.random() < 0.5,
                 save=not op.endswith("bwd") and rng.random() < 0.3, wt=rng.random() < 0.2,
                 pad=rng.choice([0, 0, 0, 8, 3]))


def _inputs(case, seed):
    m, n, k, dt = case["m"], case["n"], case["k"], DT[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    # activations with a few loud channels, as a residual stream has them
    x = normal(m, k + case["pad"])
    loud = torch.rand(k + case["pad"], generator=gen, device="cuda") < 0.01
    x = (x * (1 + 5 * loud.float())).to(dt)[:, :k]

    def weight():
        w = (normal(k, n) if case["wt"] else normal(n, k)).mul_(k ** -0.5).to(dt)
        return w.t() if case["wt"] else w

    s = {"x": x, "w": weight()}
    if case["op"].startswith("gated"):
        s["w2"] = weight()
    if case["bias"]:
        s["b"] = normal(n).to(dt)
    if case["residual"]:
        s["r"] = normal(m, n).to(dt)
    if case["op"].endswith("bwd"):
        s["dy"] = normal(m, n).to(dt)
        # what the forward kept: the product before the activation, or gate and up
        if case["op"] == "linear_bwd":
            if case["act"] != "none":
                s["z"] = (x.float() @ s["w"].float().t() + (s["b"].float() if "b" in s else 0)).to(dt)
        else:
            s["g"] = (x.float() @ s["w"].float().t()).to(dt)
            s["u"] = (x.float() @ s["w2"].float().t()).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import collective_datapath_copy_gb300 as cdc

        m, n, k, op = case["m"], case["n"], case["k"], case["op"]

        def buf(*shape):
            return torch.empty(*shape, dtype=s["x"].dtype, device="cuda")

        if op.startswith("linear"):
            s["op"] = cdc.Linear(s["w"], bias=s.get("b"), act=case["act"])
            if op == "linear":
                s["y"] = buf(m, n)
                s["pre"] = buf(m, n) if case["save"] else None
            else:
                s["dx"], s["dw"] = buf(m, k), buf(n, k)
                s["db"] = buf(n) if case["bias"] else None
        else:
            s["op"] = cdc.GatedFFN(s["w"], s["w2"], act=case["act"])
            if op == "gated":
                s["y"] = buf(m, n)
                s["gate"], s["up"] = (buf(m, n), buf(m, n)) if case["save"] else (None, None)
            else:
                s["dx"], s["dw"], s["dw2"] = buf(m, k), buf(n, k), buf(n, k)
    return s


def _run_own(s):
    c = s["case"]
    if c["op"] == "linear":
        return s["op"].forward(s["x"], residual=s.get("r"), out=s["y"], save=c["save"],
                               pre=s["pre"])
    if c["op"] == "linear_bwd":
        dx, dw, db = s["op"].backward(s["dy"], s["x"], pre=s.get("z"), dx=s["dx"], dw=s["dw"],
                                      db=s["db"])
        return (dx, dw) if db is None else (dx, dw, db)
    if c["op"] == "gated":
        return s["op"].forward(s["x"], out=s["y"], save=c["save"], gate=s["gate"], up=s["up"])
    return s["op"].backward(s["dy"], s["x"], s["g"], s["u"], dx=s["dx"], dw_gate=s["dw"],
                            dw_up=s["dw2"])


_RT2 = 2 ** -0.5
_GT0, _GT1 = (2 / math.pi) ** 0.5, 0.044715


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * _RT2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_GT0 * (z + _GT1 * z * z * z)))
    s = 1 / (1 + torch.exp(-z))
    return s if act == "sigmoid" else z * s


def _dact(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * _RT2))
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    if act == "gelu_tanh":
        t = torch.tanh(_GT0 * (z + _GT1 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _GT0 * (1 + 3 * _GT1 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 - s) if act == "sigmoid" else s * (1 + z * (1 - s))


def _run_plain(s):
    c, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    if c["op"] == "linear":
        z = x @ w.t()
        if "b" in s:
            z = z + s["b"].float()
        y = _act(z, c["act"])
        if "r" in s:
            y = y + s["r"].float()
        return (y.to(dt), z.to(dt)) if c["save"] else y.to(dt)
    if c["op"] == "linear_bwd":
        dz = s["dy"].float()
        if "z" in s:
            dz = dz * _dact(s["z"].float(), c["act"])
        out = ((dz @ w).to(dt), (dz.t() @ x).to(dt))
        return out + (dz.sum(0).to(dt),) if c["bias"] else out
    w2 = s["w2"].float()
    if c["op"] == "gated":
        g, u = x @ w.t(), x @ w2.t()
        h = (_act(g, c["act"]) * u).to(dt)
        return (h, g.to(dt), u.to(dt)) if c["save"] else h
    g, u, dh = s["g"].float(), s["u"].float(), s["dy"].float()
    dg, du = dh * u * _dact(g, c["act"]), dh * _act(g, c["act"])
    return (dg @ w + du @ w2).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def exact(case, seed):
    """The same outputs from the definitions in 64 bits: products as einsum over named axes,
    activations through the normal distribution function and the logistic function."""
    s = {a: (t.double() if torch.is_tensor(t) else t) for a, t in _inputs(case, seed).items()}

    def phi(z):
        return torch.special.ndtr(z)

    def value_and_slope(z):
        act = case["act"]
        if act == "none":
            return z, torch.ones_like(z)
        if act == "relu":
            return z.clamp(min=0), (z > 0).double()
        if act == "gelu":
            return z * phi(z), phi(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
        if act == "gelu_tanh":
            # (1 + tanh(a)) / 2 is the logistic function of 2a
            a2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
            sg = torch.special.expit(a2)
            slope = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z.square())
            return z * sg, sg + z * sg * torch.special.expit(-a2) * slope
        sg, sn = torch.special.expit(z), torch.special.expit(-z)
        if act == "sigmoid":
            return sg, sg * sn
        return z * sg, sg + z * sg * sn

    def ein(spec, *t):
        return torch.einsum(spec, *t)

    if case["op"] == "linear":
        z = ein("mk,nk->mn", s["x"], s["w"]) + s.get("b", 0.0)
        y = value_and_slope(z)[0] + s.get("r", 0.0)
        return (y, z) if case["save"] else y
    if case["op"] == "linear_bwd":
        dz = s["dy"] * (value_and_slope(s["z"])[1] if "z" in s else 1.0)
        out = (ein("mn,nk->mk", dz, s["w"]), ein("mn,mk->nk", dz, s["x"]))
        return out + (ein("mn->n", dz),) if case["bias"] else out
    if case["op"] == "gated":
        g, u = ein("mk,nk->mn", s["x"], s["w"]), ein("mk,nk->mn", s["x"], s["w2"])
        h = value_and_slope(g)[0] * u
        return (h, g, u) if case["save"] else h
    a, da = value_and_slope(s["g"])
    dg, du = s["dy"] * s["u"] * da, s["dy"] * a
    return (ein("mn,nk->mk", dg, s["w"]) + ein("mn,nk->mk", du, s["w2"]),
            ein("mn,mk->nk", dg, s["x"]), ein("mn,mk->nk", du, s["x"]))


def work(case):
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    mn, mk, nk = m * n, m * k, n * k
    e = 2  # bytes of an element, either type
    if op == "linear":
        b = mk + nk + mn + n * case["bias"] + mn * case["residual"] + mn * case["save"]
        return {"bytes": e * b, "flops": 2 * m * n * k}
    if op == "linear_bwd":  # dy, the kept product, x, W in; dx, dW, db out
        b = mn + mn * (case["act"] != "none") + 2 * mk + 2 * nk + n * case["bias"]
        return {"bytes": e * b, "flops": 4 * m * n * k}
    if op == "gated":
        return {"bytes": e * (mk + 2 * nk + mn + 2 * mn * case["save"]), "flops": 4 * m * n * k}
    return {"bytes": e * (3 * mn + 2 * mk + 4 * nk), "flops": 8 * m * n * k}
