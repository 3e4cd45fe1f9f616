"""A tensor-parallel gated MLP over R emulated ranks: the dense operators around the collective.

Rank r holds rows [r f, (r + 1) f) of w_gate and w_up and the same columns of w_down:

    h_r = act(x w_gate_r^T) * (x w_up_r^T)          GatedFFN   (column-parallel)
    p_r = h_r w_down_r^T  (+ residual on rank 0)     Linear     (row-parallel, a partial)
    y   = sum over r of p_r                          Plan       (all-reduce, fixed rank order)

and backward, with dy the same on every rank:

    dh_r, dw_down_r = Linear.backward(dy);  dx_r, dw_gate_r, dw_up_r = GatedFFN.backward(dh_r)
    dx = sum over r of dx_r                          Plan

The shards are views of the whole weights (w_down's rows keep their stride), so nothing is copied
and an optimiser that updates the whole weights in place updates the shards. Run as a module for a
timing of both directions: python -m collective_datapath_copy_gb300.mlp [tokens]
"""

from __future__ import annotations

import torch

from .dense import GatedFFN, Linear
from .namings import allreduce
from .plan import Plan

# outputs up to this many bytes go through the staged engine (one persistent launch, speculative
# protocol), larger ones through the zero-copy datapath in two steps
STAGED_BYTES = 64 * 1024


class TensorParallelMLP:
    """w_gate, w_up [F, K] and w_down [K, F], bfloat16 (or float16 with partials="f32"); R divides
    F; `tokens` rows a call. partials: "bf16" sums rounded partials (2-byte elements cross the
    collective), "f32" sums them in binary32 and returns y in float32."""

    def __init__(self, R, w_gate, w_up, w_down, tokens, act="silu", partials="bf16"):
        F, K = w_gate.shape
        if w_down.shape != (K, F):
            raise ValueError(f"w_down must be {(K, F)}, not {tuple(w_down.shape)}")
        if R < 1 or F % R:
            raise ValueError(f"{R} ranks do not divide {F} features")
        if partials not in ("bf16", "f32"):
            raise ValueError(f'partials must be "bf16" or "f32", not {partials!r}')
        if partials == "bf16" and w_gate.dtype is not torch.bfloat16:
            raise ValueError('partials="bf16" needs bfloat16 weights')
        f = F // R
        self.R, self.tokens, self.K, self.f = R, tokens, K, f
        self.up = [GatedFFN(w_gate[r * f:(r + 1) * f], w_up[r * f:(r + 1) * f], act)
                   for r in range(R)]
        self.down = [Linear(w_down[:, r * f:(r + 1) * f]) for r in range(R)]
        dev, dt = w_gate.device, w_gate.dtype
        # the operators' status words, side by side
        self._words = torch.zeros(2 * R, dtype=torch.int32, device=dev)
        for i, op in enumerate(self.up + self.down):
            op._report_to(self._words[i:i + 1])
        self._ptype = torch.float32 if partials == "f32" else torch.bfloat16
        self._p = [torch.empty(tokens, K, dtype=self._ptype, device=dev) for _ in range(R)]
        self._y = [torch.empty(tokens, K, dtype=self._ptype, device=dev) for _ in range(R)]
        self._sum = self._plan(partials)
        # gradients of x cross in the operands' type, or f32 where that is float16
        self._gtype = torch.bfloat16 if dt is torch.bfloat16 else torch.float32
        self._g = self._dx = None
        self._gsum = self._sum if self._gtype is self._ptype else self._plan(
            "bf16" if self._gtype is torch.bfloat16 else "f32")
        self._kept = None

    def _here(self):
        """The weights' device as the current one: a plan belongs to the device it was made on,
        and runs only while that is current."""
        return torch.cuda.device(self.up[0]._dev)

    def _plan(self, dtype):
        n = self.tokens * self.K
        with self._here():
            if n * (2 if dtype == "bf16" else 4) <= STAGED_BYTES:
                return Plan(allreduce(self.R, n, dtype), protocol="spec")
            return Plan(allreduce(self.R, n, dtype), zero_copy=1, datapath="twoshot")

    def status(self) -> int:
        """COLL_OK, or the code of an operator whose bounded device wait expired in any call so far
        or of a sum whose last run failed: results are then incomplete. Calls enqueue their sums
        behind their products without looking, so a caller asks before it relies on them.
        Synchronises with the object's calls."""
        code = int(self._words.min())  # codes are negative
        with self._here():
            for plan in (self._sum, self._gsum):
                code = code or plan.status()["code"]
        return code

    @staticmethod
    def _carrier(ts):
        # the collective moves 16-bit patterns
        return [t.view(torch.int16) if t.dtype is torch.bfloat16 else t for t in ts]

    def forward(self, x, residual=None, keep=False):
        """x [tokens, K] -> y, one tensor per rank, all equal (the object's buffers, overwritten by
        the next call). residual is added once, by rank 0's
        epilogue; its gradient is dy. keep: what backward needs."""
        kept = []
        for r in range(self.R):
            if keep:
                h, gate, up = self.up[r].forward(x, save=True)
                kept.append((h, gate, up))
            else:
                h = self.up[r].forward(x)
            res = residual if r == 0 else None
            if res is not None and self._ptype is torch.float32:
                res = res.float()
            self.down[r].forward(h, residual=res, out=self._p[r])
        self._kept = (x, kept) if keep else None
        with self._here():
            self._sum.run(self._carrier(self._p), self._carrier(self._y))
        return self._y

    def backward(self, dy):
        """dx, one tensor per rank (the object's buffers), and (dw_gate_r, dw_up_r, dw_down_r) of
        every rank's shards, for the last forward(keep=True)."""
        if self._kept is None:
            raise RuntimeError("backward needs forward(keep=True) before it")
        x, kept = self._kept
        if self._g is None:
            self._g, self._dx = ([torch.empty(self.tokens, self.K, dtype=self._gtype,
                                              device=x.device) for _ in range(self.R)]
                                 for _ in range(2))
        grads = []
        for r in range(self.R):
            h, gate, up = kept[r]
            dh, dw_down, _ = self.down[r].backward(dy, h)
            direct = self._gtype is x.dtype
            dx, dw_gate, dw_up = self.up[r].backward(dh, x, gate, up,
                                                     dx=self._g[r] if direct else None)
            if not direct:
                self._g[r].copy_(dx)
            grads.append((dw_gate, dw_up, dw_down))
        with self._here():
            self._gsum.run(self._carrier(self._g), self._carrier(self._dx))
        return self._dx, grads


def main(tokens=512, R=8, K=4096, F=14336, steps=10):
    gen = torch.Generator(device="cuda").manual_seed(0)

    def weight(n, k):
        return (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).bfloat16()

    mlp = TensorParallelMLP(R, weight(F, K), weight(F, K), weight(K, F), tokens)
    x = torch.randn(tokens, K, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(tokens, K, generator=gen, device="cuda").bfloat16()
    for what, call in (("forward", lambda: mlp.forward(x, residual=x)),
                       ("forward and backward",
                        lambda: (mlp.forward(x, residual=x, keep=True), mlp.backward(dy)))):
        for _ in range(3):
            call()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(steps):
            call()
        b.record()
        torch.cuda.synchronize()
        print(f"{what}: {a.elapsed_time(b) / steps * 1e3:.1f} us for {tokens} tokens, "
              f"{R} emulated ranks, {K} x {F}")


if __name__ == "__main__":
    import sys
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 512)
