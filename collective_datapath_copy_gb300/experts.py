"""Python face of the mixture-of-experts operators: Router and GatedExperts.

A router's choice of experts from its logits, with its gradient, and a few tokens through their
chosen gated experts, as a decode step runs them. Calls marshal the C entry points
(include/coll.h), enqueue on a stream and return; outputs and workspaces come from PyTorch's
allocator on that stream unless given.

    logits = cdc.Linear(w_router).forward(x, out_dtype=torch.float32)
    ids, weights = cdc.Router(8).forward(logits)          # int32 and binary32, [tokens, 8]
    experts = cdc.GatedExperts(w_gate, w_up, w_down)      # [E, F, K], [E, F, K], [E, N, F]
    y = experts.forward(x, ids, weights, residual=x)

A rank that holds experts [first, first + E) passes over the others' ids; the ranks' outputs add up
(ExpertParallelMoE). `ids`, on the host, is also the routing table that moe_dispatch and
moe_combine take. The operators record nothing for autograd: Router.backward is explicit, and
GatedExperts is for serving.
"""

from __future__ import annotations

import math
import struct

import torch

from . import _lib, dense
from ._lib import check, lib
from .dense import ACT, GATED_ACTS, _NONE, _TYPE, _Dense, _mask, _new, _on, _read, _row_count

_ROUTE = struct.Struct("6qd9q")
_ROUTE_BWD = struct.Struct("6qd12q")
_EXPERTS = struct.Struct("37q")
# What lies behind torch.cuda.caching_allocator_alloc and _delete: blocks of the caching allocator, as
# torch.empty has them (of a graph's pool under capture, reused in the stream's order). A call for one token
# takes 10.6 us with them, 12.4 with those two, which make a device current each time, 15.2 with a tensor.
_alloc = torch._C._cuda_cudaCachingAllocator_raw_alloc
_free = torch._C._cuda_cudaCachingAllocator_raw_delete
_entries = {}
_MOST = (2.0 - 2.0 ** -23) * 2.0 ** 127  # binary32's largest

dense._MASK["coll_gated_experts"] = _mask("." * 10 + "a.." * 8)


def _out(t, m, cols, dtype, dev, what):
    """An output's address and strides as a matrix; never a copy."""
    if t.shape == (m, cols) and t.dtype is dtype and t.get_device() == dev:
        return (t.data_ptr(),) + t.stride()
    if t.dtype is not dtype:
        raise ValueError(f"{what} is {t.dtype}, expected {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, expected cuda:{dev}")
    if t.dim() == 0 or t.shape[-1] != cols or t.numel() != m * cols:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {m} rows of {cols}")
    t = t.view(m, cols)
    return (t.data_ptr(),) + t.stride()


def _stack(name, w, like=None):
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError(f"{name} must have three dimensions")
    if w.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name} must be bfloat16 or float16, not {w.dtype}")
    if not w.is_cuda:
        raise ValueError(f"{name} is not a CUDA tensor")
    if like is not None and (w.dtype != like.dtype or w.device != like.device):
        raise ValueError(f"{name} must be {like.dtype} on {like.device}")
    if w.stride(2) != 1 and w.shape[2] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return w


class Router:
    """Each token's choice of `top_k` experts, by its largest logits, and their weights.

    score: "softmax" (over all experts) or "sigmoid"; normalize: a token's weights add up to `scale`,
    else each is `scale` times its score."""

    def __init__(self, top_k, score="softmax", normalize=True, scale=1.0):
        if not 1 <= top_k <= 32:
            raise ValueError(f"top_k must be 1 to 32, not {top_k}")
        if score not in _lib.SCORE:
            raise ValueError(f"score must be one of {tuple(_lib.SCORE)}, not {score!r}")
        if not abs(scale) <= _MOST:
            raise ValueError(f"scale must be a finite binary32 number, not {scale}")
        self.top_k, self._score = int(top_k), score
        self._how = (_lib.SCORE[score], int(bool(normalize)), float(scale))

    score = property(lambda self: self._score)
    normalize = property(lambda self: bool(self._how[1]))
    scale = property(lambda self: self._how[2])

    @staticmethod
    def _logits(logits):
        if logits.dtype not in _TYPE:
            raise ValueError(f"logits must be one of {tuple(_TYPE)}, not {logits.dtype}")
        dev = logits.get_device()
        if dev < 0:
            raise ValueError("logits is not a CUDA tensor")
        if logits.dim() == 0:
            raise ValueError("logits must have a dimension of experts")
        return dev

    def _head(self, logits, keep):
        """Sizes and how to choose, the first fields of a call, and the logits as a matrix."""
        shape = logits.shape
        e = shape[-1]
        if len(shape) == 2:
            t, rows = shape[0], logits
        else:
            t = math.prod(shape[:-1])
            rows = logits.reshape(t, e)
            keep.append(rows)
        return ((t, e, self.top_k, _TYPE[logits.dtype]) + self._how,
                (rows.data_ptr(),) + rows.stride())

    @staticmethod
    def _launch(where, packed, dev):
        if dense._current_device() != dev:
            with torch.cuda.device(dev):
                return Router._launch(where, packed, dev)
        fn = _entries.get(where)
        if fn is None:
            fn = _entries[where] = getattr(lib(), where)
        code = fn(packed, dense._raw_stream(dev))
        if code:
            check(code, where)

    def forward(self, logits, ids=None, weights=None, stream=None):
        """logits [..., E] (binary32, bfloat16 or float16) -> ids [..., top_k] (int32) and weights
        [..., top_k] (binary32), the largest logit first, equal ones by ascending index. A logit of
        -inf is not chosen: where too few are left, ids ends in -1 with weight 0."""
        dev = self._logits(logits)
        if stream is not None:
            with _on(stream, dev, (logits, ids, weights), "logits are"):
                return self.forward(logits, ids, weights)
        keep, top = [], self.top_k
        head, lm = self._head(logits, keep)
        t = head[0]
        if ids is None:
            ids = torch.empty(*logits.shape[:-1], top, dtype=torch.int32, device=logits.device)
        if weights is None:
            weights = torch.empty(*logits.shape[:-1], top, dtype=torch.float32,
                                  device=logits.device)
        self._launch("coll_route", _ROUTE.pack(*(
            head + lm + _out(ids, t, top, torch.int32, dev, "ids")
            + _out(weights, t, top, torch.float32, dev, "weights"))), dev)
        return ids, weights

    __call__ = forward

    def backward(self, dweights, logits, ids, dlogits=None, stream=None):
        """dlogits [..., E], of the logits' type, for the gradient dweights [..., top_k] (binary32)
        of forward's weights and the ids it returned. The choice itself has no gradient."""
        dev = self._logits(logits)
        if stream is not None:
            with _on(stream, dev, (dweights, logits, ids, dlogits), "logits are"):
                return self.backward(dweights, logits, ids, dlogits)
        keep, top = [], self.top_k
        head, lm = self._head(logits, keep)
        t, e = head[:2]
        gm = _read(dweights, t, top, torch.float32, dev, "dweights", keep)
        im = _read(ids, t, top, torch.int32, dev, "ids", keep)
        if dlogits is None:
            dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        self._launch("coll_route_backward", _ROUTE_BWD.pack(
            *(head + gm + lm + im + _out(dlogits, t, e, logits.dtype, dev, "dlogits"))), dev)
        return dlogits


class GatedExperts(_Dense):
    """y = residual + sum over a token's choices of weight * (act(x w_gate^T) * (x w_up^T)) w_down^T:
    a few tokens through the experts they chose.  w_gate, w_up [E, F, K], w_down [E, N, F],
    bfloat16 or float16, each one's last dimension contiguous. Updates in place and storage that takes
    the place of a stack's are seen by the next call.

    act: "silu", "gelu", "gelu_tanh", "relu" or "sigmoid". first: the id of w_gate[0]; a token's ids
    outside [first, first + E) are passed over. act(...) * (...) is kept to twice the bits of the weights'
    type, in float16 infinite past 65504; everything else is binary32 until y is rounded."""

    def __init__(self, w_gate, w_up, w_down, act="silu", first=0):
        self._w = (_stack("w_gate", w_gate), w_up, w_down)
        self._start(w_gate.device)
        self._take(None)
        if act not in GATED_ACTS:
            raise ValueError(f"act must be one of {GATED_ACTS}, not {act!r}")
        if not 0 <= first < 2 ** 31 - 4096:
            raise ValueError(f"first must be the id of an expert, not {first}")
        self.act, self.first = act, int(first)

    w_gate = property(lambda self: self._w[0])
    w_up = property(lambda self: self._w[1])
    w_down = property(lambda self: self._w[2])

    def _take(self, now):
        """The call's view of the stacks, checked: at first, and when `now`, what a call finds of their
        addresses, shapes, strides and types, is not what the last one found."""
        wg, wu, wd = self._w
        _stack("w_gate", wg)
        _stack("w_up", wu, wg)
        _stack("w_down", wd, wg)
        E, F, K = wg.shape
        if wu.shape != wg.shape or wd.shape[0] != E or wd.shape[2] != F:
            raise ValueError(f"w_up must be {(E, F, K)} and w_down {(E, 'N', F)}, not "
                             f"{tuple(wu.shape)} and {tuple(wd.shape)}")
        if wg.get_device() != self._dev:
            raise ValueError(f"the weights are on cuda:{wg.get_device()}, the object was made on "
                             f"cuda:{self._dev}")
        self._sizes = (wd.shape[1], K, F, E, wg.dtype)
        self._stacks = tuple(v for w in self._w for v in (w.data_ptr(),) + w.stride()[:2])
        self._now = now

    def _lend(self, fn, pack, fields, need, stream):
        # no tensor around it: making one costs as much as the launches
        ws = _alloc(need, stream)
        try:
            return fn(pack(*fields, ws, need, self._word), stream)
        finally:
            _free(ws)

    def forward(self, x, ids, weights, residual=None, out=None, out_dtype=None, stream=None):
        """x [..., K], ids [..., top] (int32) and weights [..., top] (binary32) -> y [..., N].
        out_dtype: the operands' type or torch.float32 (a partial for a binary32 sum; its residual
        is float32 too). residual may be `out` itself. The chosen experts' weights are read once for
        every 128 tokens."""
        wg, wu, wd = self._w
        dev, keep = self._dev, []
        if stream is not None:
            with _on(stream, dev, (x, ids, weights, residual, out, wg, wu, wd, self._status)):
                return self.forward(x, ids, weights, residual, out, out_dtype)
        now = (wg.data_ptr(), wg.shape, wg.stride(), wg.dtype, wu.data_ptr(), wu.shape, wu.stride(),
               wu.dtype, wd.data_ptr(), wd.shape, wd.stride(), wd.dtype)
        if now != self._now:
            self._take(now)
        n, K, F, E, dt = self._sizes
        xm = _read(x, None, K, dt, dev, "x", keep)
        m = _row_count(x)
        if ids.dim() == 0:
            raise ValueError("ids must have a dimension of choices")
        top = ids.shape[-1]
        im = _read(ids, m, top, torch.int32, dev, "ids", keep)
        sm = _read(weights, m, top, torch.float32, dev, "weights", keep)
        ot = out.dtype if out is not None else out_dtype or dt
        if (ot is not dt and ot is not torch.float32) or out_dtype not in (None, ot):
            raise ValueError(f"the output must be {dt} or torch.float32, not "
                             f"{ot if out_dtype in (None, ot) else out_dtype}")
        if out is None:
            out = _new(m, n, ot, wg, x)
        ym = _out(out, m, n, ot, dev, "out")
        rm = _NONE
        if residual is not None:
            if residual.shape != out.shape:
                residual = residual.expand(out.shape)
            rm = _read(residual, m, n, ot, dev, "residual", keep)
        self._launch("coll_gated_experts", _EXPERTS.pack,
                     (m, n, K, F, E, self.first, top, _TYPE[dt], _TYPE[ot], ACT[self.act],
                      *self._stacks, *xm, *im, *sm, *rm, *ym))
        return out

    __call__ = forward
