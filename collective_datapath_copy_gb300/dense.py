"""Python face of the dense operators: Linear and GatedFFN, forward and backward.

The products on either side of a tensor-parallel layer's collective. An object holds a layer's
weights (the tensors themselves: updates in place are seen by the next call) and marshals calls
of the C entry points (include/coll.h); every step runs in the library's kernels. Calls enqueue
on a stream and return. Outputs and workspaces come from PyTorch's allocator on that stream
unless given.

    up = cdc.GatedFFN(w_gate, w_up, act="silu")      # h = silu(x w_gate^T) * (x w_up^T)
    down = cdc.Linear(w_down, act="none")            # y = h w_down^T + residual
    h = up.forward(x)
    y = down.forward(h, residual=x)

Inputs may have any strides and leading dimensions; outputs that a caller passes have unit column
stride. The operators record nothing for autograd: the backward calls are explicit.
"""

from __future__ import annotations

import contextlib
import struct

import torch

from . import _lib
from ._lib import check, lib

ACT = {"none": _lib.D["COLL_ACT_NONE"], "relu": _lib.D["COLL_ACT_RELU"],
       "gelu": _lib.D["COLL_ACT_GELU"], "gelu_tanh": _lib.D["COLL_ACT_GELU_TANH"],
       "silu": _lib.D["COLL_ACT_SILU"], "sigmoid": _lib.D["COLL_ACT_SIGMOID"]}
LINEAR_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
GATED_ACTS = ("relu", "gelu", "gelu_tanh", "silu", "sigmoid")
_TYPE = {torch.bfloat16: _lib.D["COLL_BF16"], torch.float16: _lib.D["COLL_F16"],
         torch.float32: _lib.D["COLL_F32"]}
_EWORKSPACE = _lib.D["COLL_EWORKSPACE"]

# every field of the argument structures is eight bytes wide
_LINEAR = struct.Struct("26q")
_LINEAR_BWD = struct.Struct("28q")
_GATED = struct.Struct("26q")
_GATED_BWD = struct.Struct("36q")
_NONE = (0, 0, 0)
_entries = {}


def _entry(name):
    e = _entries.get(name)
    if e is None:
        h = lib()
        e = _entries[name] = (getattr(h, name), getattr(h, name + "_workspace"))
    return e


_raw_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream, 2 us cheaper


def _weight(name, w):
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    if w.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name} must be bfloat16 or float16, not {w.dtype}")
    if not w.is_cuda:
        raise ValueError(f"{name} is not a CUDA tensor")
    return w


def _rows(t, cols, dtype, device, what):
    """An input as a matrix of `cols` columns (leading dimensions flattened)."""
    if t.dtype is not dtype:
        raise ValueError(f"{what} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the weights are on {device}")
    s = t.shape
    if len(s) == 0 or s[-1] != cols:
        raise ValueError(f"{what} has shape {tuple(s)}, expected {cols} columns")
    if len(s) == 2:
        return t
    m = 1
    for d in s[:-1]:
        m *= d
    return t.reshape(m, cols)


def _dest(t, m, cols, dtypes, device, what):
    """An output the caller passed, as a matrix; never a copy."""
    if t.dtype not in dtypes:
        raise ValueError(f"{what} is {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the weights are on {device}")
    if t.dim() == 0 or t.shape[-1] != cols or t.numel() != m * cols:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {m} rows of {cols}")
    return t if t.dim() == 2 else t.view(m, cols)


def _mat(t):
    if t is None:
        return _NONE
    a, b = t.stride()
    return t.data_ptr(), a, b


@contextlib.contextmanager
def _on(stream, tensors):
    """Run a call on another stream than the current one: allocations belong to that stream, and
    the caller's tensors are not handed out again before it has passed the call."""
    with torch.cuda.stream(stream):
        yield
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


class _Dense:
    def _start(self, device):
        self._status = torch.zeros(1, dtype=torch.int32, device=device)
        self._need = {}

    def status(self) -> int:
        """COLL_OK, or COLL_ETIMEDOUT if a bounded device wait of an earlier call expired (its
        outputs are then incomplete). Synchronises with the object's calls on the current
        stream."""
        return int(self._status.item())

    def _launch(self, where, pack, fields):
        """Call an entry point on the current stream, with a workspace if it asks for one. The
        size it last asked for is offered first, so that a loop over one size makes one call."""
        fn, size = _entry(where)
        device, status = self._status.device, self._status.data_ptr()
        stream = _raw_stream(device.index)  # the current stream's handle
        need = self._need.get(where, 0)
        while True:
            if need:
                ws = torch.empty(need, dtype=torch.uint8, device=device)
                code = fn(pack(*fields, ws.data_ptr(), need, status), stream)
            else:
                code = fn(pack(*fields, 0, 0, status), stream)
            if code != _EWORKSPACE:
                break
            need = int(size(pack(*fields, 0, 0, status)))
            if need < 0:
                check(need, where)
            self._need[where] = need
        if code:
            check(code, where)


class Linear(_Dense):
    """y = act(x weight^T + bias) + residual.  weight [N, K], bias [N], bfloat16 or float16.

    act: "none", "relu", "gelu", "gelu_tanh" or "silu"."""

    def __init__(self, weight, bias=None, act="none"):
        self.weight = _weight("weight", weight)
        if act not in LINEAR_ACTS:
            raise ValueError(f"act must be one of {LINEAR_ACTS}, not {act!r}")
        if bias is not None and (bias.dtype != weight.dtype or bias.device != weight.device
                                 or bias.shape != (weight.shape[0],)):
            raise ValueError(f"bias must be {weight.dtype} with shape ({weight.shape[0]},) on "
                             f"{weight.device}")
        self.bias = bias
        self.act = act
        self._start(weight.device)

    def forward(self, x, residual=None, out=None, out_dtype=None, save=False, pre=None,
                stream=None):
        """x [..., K] -> y [..., N]. With `save`, returns (y, pre): pre is the product before the
        activation, which backward needs unless act is "none". out_dtype: the operands' type or
        torch.float32 (a partial for a binary32 sum; its residual is float32 too). residual may be
        `out` itself."""
        if stream is not None:
            with _on(stream, (x, residual, out, pre, self.weight, self.bias)):
                return self.forward(x, residual, out, out_dtype, save, pre)
        w, b = self.weight, self.bias
        n, k = w.shape
        dt, dev = w.dtype, w.device
        x2 = _rows(x, k, dt, dev, "x")
        m = x2.shape[0]
        if out is not None:
            ot = out.dtype
            if out_dtype is not None and out_dtype is not ot:
                raise ValueError(f"out is {ot}, out_dtype is {out_dtype}")
            y2 = _dest(out, m, n, (dt, torch.float32), dev, "out")
        else:
            ot = out_dtype or dt
            if ot not in (dt, torch.float32):
                raise ValueError(f"out_dtype must be {dt} or torch.float32, not {ot}")
            y2 = torch.empty(m, n, dtype=ot, device=dev)
            out = y2 if x.dim() == 2 else y2.view(*x.shape[:-1], n)
        if pre is not None:
            p2 = _dest(pre, m, n, (dt,), dev, "pre")
        elif save:
            p2 = torch.empty(m, n, dtype=dt, device=dev)
            pre = p2 if x.dim() == 2 else p2.view(*x.shape[:-1], n)
        else:
            p2 = None
        r2 = None
        if residual is not None:
            if residual.shape != out.shape:
                residual = residual.expand(out.shape)
            r2 = _rows(residual, n, ot, dev, "residual")
        self._launch("coll_linear", _LINEAR.pack,
                     (m, n, k, _TYPE[dt], _TYPE[ot], ACT[self.act], *_mat(x2), *_mat(w),
                      *_mat(r2), *_mat(p2), *_mat(y2), 0 if b is None else b.data_ptr(),
                      0 if b is None else b.stride(0)))
        return (out, pre) if save or p2 is not None else out

    __call__ = forward

    def backward(self, dy, x, pre=None, need_dx=True, need_dw=True, need_db=None, dx=None,
                 dw=None, db=None, grad_dtype=None, stream=None):
        """(dx, dw, db) for the gradient dy [..., N] of y; None in the place of one that is not
        needed (db follows the bias unless need_db says otherwise). The residual's gradient is dy
        itself. grad_dtype: the type of dw and db, the operands' or torch.float32."""
        if stream is not None:
            with _on(stream, (dy, x, pre, dx, dw, db, self.weight)):
                return self.backward(dy, x, pre, need_dx, need_dw, need_db, dx, dw, db,
                                     grad_dtype)
        w = self.weight
        n, k = w.shape
        dt, dev = w.dtype, w.device
        x2 = _rows(x, k, dt, dev, "x")
        m = x2.shape[0]
        dy2 = _rows(dy, n, dt, dev, "dy")
        if dy2.shape[0] != m:
            raise ValueError(f"dy has {dy2.shape[0]} rows, x has {m}")
        p2 = None
        if self.act != "none":
            if pre is None:
                raise ValueError(f"backward of act={self.act!r} needs pre")
            p2 = _rows(pre, n, dt, dev, "pre")
            if p2.shape[0] != m:
                raise ValueError(f"pre has {p2.shape[0]} rows, x has {m}")
        if need_db is None:
            need_db = self.bias is not None or db is not None
        gt = grad_dtype or (dw.dtype if dw is not None else db.dtype if db is not None else dt)
        if gt not in (dt, torch.float32):
            raise ValueError(f"grad_dtype must be {dt} or torch.float32, not {gt}")
        dx2 = dw2 = db2 = None
        if need_dx:
            if dx is None:
                dx2 = torch.empty(m, k, dtype=dt, device=dev)
                dx = dx2 if x.dim() == 2 else dx2.view(x.shape)
            else:
                dx2 = _dest(dx, m, k, (dt,), dev, "dx")
        if need_dw:
            dw = torch.empty(n, k, dtype=gt, device=dev) if dw is None else dw
            dw2 = _dest(dw, n, k, (gt,), dev, "dw")
        if need_db:
            db = torch.empty(n, dtype=gt, device=dev) if db is None else db
            db2 = _dest(db, 1, n, (gt,), dev, "db")
            if db.dim() != 1 or (n > 1 and db.stride(0) != 1):
                raise ValueError("db must be a contiguous vector")
        self._launch("coll_linear_backward", _LINEAR_BWD.pack,
                     (m, n, k, _TYPE[dt], _TYPE[gt], ACT[self.act], *_mat(dy2), *_mat(p2),
                      *_mat(x2), *_mat(w), *_mat(dx2), *_mat(dw2),
                      0 if db2 is None else db2.data_ptr()))
        return (dx if need_dx else None, dw if need_dw else None, db if need_db else None)


class GatedFFN(_Dense):
    """h = act(x w_gate^T) * (x w_up^T): both projections of a gated feed-forward block, its
    activation and its product in one launch.  w_gate, w_up [F, K], bfloat16 or float16.

    act: "silu", "gelu", "gelu_tanh", "relu" or "sigmoid"."""

    def __init__(self, w_gate, w_up, act="silu"):
        self.w_gate, self.w_up = _weight("w_gate", w_gate), _weight("w_up", w_up)
        if (w_up.shape != w_gate.shape or w_up.dtype != w_gate.dtype
                or w_up.device != w_gate.device):
            raise ValueError("w_gate and w_up must have one shape, type and device")
        if act not in GATED_ACTS:
            raise ValueError(f"act must be one of {GATED_ACTS}, not {act!r}")
        self.act = act
        self._start(w_gate.device)

    def forward(self, x, out=None, save=False, gate=None, up=None, stream=None):
        """x [..., K] -> h [..., F]. With `save`, returns (h, gate, up): the two products, which
        backward needs."""
        if stream is not None:
            with _on(stream, (x, out, gate, up, self.w_gate, self.w_up)):
                return self.forward(x, out, save, gate, up)
        w = self.w_gate
        n, k = w.shape
        dt, dev = w.dtype, w.device
        x2 = _rows(x, k, dt, dev, "x")
        m = x2.shape[0]
        lead = x.shape[:-1]

        def dest(t, what):
            if t is None:
                t2 = torch.empty(m, n, dtype=dt, device=dev)
                return (t2 if len(lead) == 1 else t2.view(*lead, n)), t2
            return t, _dest(t, m, n, (dt,), dev, what)

        out, h2 = dest(out, "out")
        g2 = u2 = None
        if save or gate is not None or up is not None:
            gate, g2 = dest(gate, "gate")
            up, u2 = dest(up, "up")
        self._launch("coll_gated_ffn", _GATED.pack,
                     (m, n, k, _TYPE[dt], ACT[self.act], *_mat(x2), *_mat(w), *_mat(self.w_up),
                      *_mat(g2), *_mat(u2), *_mat(h2)))
        return out if g2 is None else (out, gate, up)

    __call__ = forward

    def backward(self, dh, x, gate, up, need_dx=True, need_dw=True, dx=None, dw_gate=None,
                 dw_up=None, grad_dtype=None, stream=None):
        """(dx, dw_gate, dw_up) for the gradient dh [..., F] of h; None in the place of one that
        is not needed. gate and up: what forward kept. grad_dtype: the type of dw_gate and dw_up,
        the operands' or torch.float32."""
        if stream is not None:
            with _on(stream, (dh, x, gate, up, dx, dw_gate, dw_up, self.w_gate, self.w_up)):
                return self.backward(dh, x, gate, up, need_dx, need_dw, dx, dw_gate, dw_up,
                                     grad_dtype)
        w = self.w_gate
        n, k = w.shape
        dt, dev = w.dtype, w.device
        x2 = _rows(x, k, dt, dev, "x")
        m = x2.shape[0]
        ins = []
        for t, what in ((dh, "dh"), (gate, "gate"), (up, "up")):
            t2 = _rows(t, n, dt, dev, what)
            if t2.shape[0] != m:
                raise ValueError(f"{what} has {t2.shape[0]} rows, x has {m}")
            ins.append(t2)
        gt = grad_dtype or (dw_gate.dtype if dw_gate is not None else
                            dw_up.dtype if dw_up is not None else dt)
        if gt not in (dt, torch.float32):
            raise ValueError(f"grad_dtype must be {dt} or torch.float32, not {gt}")
        dx2 = dg2 = du2 = None
        if need_dx:
            if dx is None:
                dx2 = torch.empty(m, k, dtype=dt, device=dev)
                dx = dx2 if x.dim() == 2 else dx2.view(x.shape)
            else:
                dx2 = _dest(dx, m, k, (dt,), dev, "dx")
        if need_dw:
            dw_gate = torch.empty(n, k, dtype=gt, device=dev) if dw_gate is None else dw_gate
            dw_up = torch.empty(n, k, dtype=gt, device=dev) if dw_up is None else dw_up
            dg2 = _dest(dw_gate, n, k, (gt,), dev, "dw_gate")
            du2 = _dest(dw_up, n, k, (gt,), dev, "dw_up")
        self._launch("coll_gated_ffn_backward", _GATED_BWD.pack,
                     (m, n, k, _TYPE[dt], _TYPE[gt], ACT[self.act], *_mat(ins[0]),
                      *_mat(ins[1]), *_mat(ins[2]), *_mat(x2), *_mat(w), *_mat(self.w_up),
                      *_mat(dx2), *_mat(dg2), *_mat(du2)))
        return (dx if need_dx else None, dw_gate if need_dw else None,
                dw_up if need_dw else None)
