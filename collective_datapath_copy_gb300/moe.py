"""An expert-parallel mixture of experts over R emulated ranks, for a decode step's few tokens.

Every rank has all tokens; rank r holds experts [r E/R, (r + 1) E/R):

    logits = x w_router^T                        Linear, a binary32 output
    ids, weights = choice(logits)                Router (the same on every rank: computed once here)
    p_r = sum over rank r's chosen experts       GatedExperts (+ residual on rank 0), a partial
    y   = sum over r of p_r                      Plan (all-reduce, fixed rank order)

The shards are views of the whole stacks, so nothing is copied. Prompts go another way: their rows
through moe_dispatch to the ranks, each expert's through GatedFFN and Linear, back through
moe_combine, with plans made from that prompt's table (the Router's ids, copied to the host). Run as
a module for a timing: python -m collective_datapath_copy_gb300.moe [tokens]
"""

from __future__ import annotations

import torch

from .dense import Linear
from .experts import GatedExperts, Router
from .mlp import STAGED_BYTES
from .namings import allreduce
from .plan import Plan


class ExpertParallelMoE:
    """w_router [E, K], w_gate and w_up [E, F, K], w_down [E, K, F], bfloat16 (or float16 with
    partials="f32"); R divides E; `tokens` rows a call. score, normalize and scale: Router's. The
    ranks hold views of the stacks as they are given: updates in place are seen, other storage is not.
    partials: "bf16" sums rounded partials, "f32" sums them in binary32 and returns y in float32."""

    def __init__(self, R, w_router, w_gate, w_up, w_down, top_k, tokens, act="silu",
                 score="softmax", normalize=True, scale=1.0, partials="bf16"):
        E, F, K = w_gate.shape
        if w_router.shape != (E, K) or w_down.shape != (E, K, F):
            raise ValueError(f"w_router must be {(E, K)} and w_down {(E, K, F)}, not "
                             f"{tuple(w_router.shape)} and {tuple(w_down.shape)}")
        if R < 1 or E % R:
            raise ValueError(f"{R} ranks do not divide {E} experts")
        if top_k > E:
            raise ValueError(f"top_k is {top_k} of {E} experts")
        if partials not in ("bf16", "f32"):
            raise ValueError(f'partials must be "bf16" or "f32", not {partials!r}')
        if partials == "bf16" and w_gate.dtype is not torch.bfloat16:
            raise ValueError('partials="bf16" needs bfloat16 weights')
        e, dev = E // R, w_gate.device
        self.R, self.tokens, self.K = R, tokens, K
        self.gate = Linear(w_router)
        self.router = Router(top_k, score, normalize, scale)
        self.experts = [GatedExperts(w_gate[r * e:(r + 1) * e], w_up[r * e:(r + 1) * e],
                                     w_down[r * e:(r + 1) * e], act, first=r * e)
                        for r in range(R)]
        self._words = torch.zeros(R + 1, dtype=torch.int32, device=dev)
        for i, op in enumerate([self.gate] + self.experts):
            op._report_to(self._words[i:i + 1])
        self._ptype = torch.float32 if partials == "f32" else torch.bfloat16
        self._p = [torch.empty(tokens, K, dtype=self._ptype, device=dev) for _ in range(R)]
        self._y = [torch.empty(tokens, K, dtype=self._ptype, device=dev) for _ in range(R)]
        n = tokens * K
        with self._here():
            if n * self._p[0].element_size() <= STAGED_BYTES:
                self._sum = Plan(allreduce(R, n, partials), protocol="spec")
            else:
                self._sum = Plan(allreduce(R, n, partials), zero_copy=1, datapath="twoshot")

    def _here(self):
        """The weights' device as the current one: a plan belongs to the device it was made on."""
        return torch.cuda.device(self.gate._dev)

    def status(self) -> int:
        """COLL_OK, or the code of an operator whose bounded device wait expired in any call so far
        or of a sum whose last run failed. Synchronises with the object's calls."""
        code = int(self._words.min())  # codes are negative
        with self._here():
            return code or self._sum.status()["code"]

    def forward(self, x, residual=None, routing=False):
        """x [tokens, K] -> y, one tensor per rank, all equal (the object's buffers, overwritten by
        the next call). residual is added once, by rank 0. routing: returns (y, ids, weights)."""
        ids, weights = self.router.forward(self.gate.forward(x, out_dtype=torch.float32))
        if residual is not None:
            residual = residual.to(self._ptype)
        for r in range(self.R):
            self.experts[r].forward(x, ids, weights, residual=residual if r == 0 else None,
                                    out=self._p[r])
        carrier = [[t.view(torch.int16) if t.dtype is torch.bfloat16 else t for t in ts]
                   for ts in (self._p, self._y)]
        with self._here():
            self._sum.run(*carrier)
        return (self._y, ids, weights) if routing else self._y


def main(tokens=8, R=8, E=64, K=4096, F=1792, top_k=8, steps=10):
    gen = torch.Generator(device="cuda").manual_seed(0)

    def weight(*shape):
        w = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
        return w.normal_(0, shape[-1] ** -0.5, generator=gen)

    moe = ExpertParallelMoE(R, weight(E, K), weight(E, F, K), weight(E, F, K), weight(E, K, F),
                            top_k, tokens)
    x = torch.randn(tokens, K, generator=gen, device="cuda").bfloat16()
    for _ in range(3):
        moe.forward(x, residual=x)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(steps):
        moe.forward(x, residual=x)
    b.record()
    torch.cuda.synchronize()
    print(f"{a.elapsed_time(b) / steps * 1e3:.1f} us for {tokens} tokens, {top_k} of {E} experts "
          f"of {K} x {F} on {R} emulated ranks")


if __name__ == "__main__":
    import sys
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
