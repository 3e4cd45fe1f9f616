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
stride. The operators record nothing for autograd: the backward calls are explicit, and an input
that requires a gradient gets none from them. Gradients of the products (dz, dg, du) pass to the
next ones in the operands' type: in float16 one past 65504 is infinite, so scale the loss.
"""

from __future__ import annotations

import contextlib
import math
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


def _mask(kinds):
    """Over a packed structure as one number: whole fields (.), of an address (a) its place within
    16 bytes, nothing of the workspace and status at the end. Two calls alike in this, and in which
    optional arrays are there, need the same workspace."""
    return sum((15 if kind == "a" else 2 ** 64 - 1) << 64 * i for i, kind in enumerate(kinds))


_MASK = {"coll_linear": _mask("......" + "a.." * 5 + "a."),
         "coll_linear_backward": _mask("......" + "a.." * 6 + "a"),
         "coll_gated_ffn": _mask("....." + "a.." * 6),
         "coll_gated_ffn_backward": _mask("......" + "a.." * 9)}


def _entry(name):
    h = lib()
    e = _entries[name] = (getattr(h, name), getattr(h, name + "_workspace"))
    return e


_raw_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream, 2 us cheaper
_current_device = torch._C._cuda_getDevice


def _weight(name, w):
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    if w.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name} must be bfloat16 or float16, not {w.dtype}")
    if not w.is_cuda:
        raise ValueError(f"{name} is not a CUDA tensor")
    return w


def _read(t, m, cols, dtype, dev, what, keep):
    """An input's address and strides as a matrix of `cols` columns (leading dimensions flattened)
    and m rows (any where m is None). What has to be copied for that lives in `keep`."""
    if (t.dtype is dtype and t.get_device() == dev and t.dim() == 2 and t.size(1) == cols
            and (m is None or t.size(0) == m)):
        return (t.data_ptr(), *t.stride())
    if t.dtype is not dtype:
        raise ValueError(f"{what} is {t.dtype}, expected {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, the weights are on cuda:{dev}")
    if t.dim() == 0 or t.shape[-1] != cols:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {cols} columns")
    rows = math.prod(t.shape[:-1])
    if m is not None and rows != m:
        raise ValueError(f"{what} has {rows} rows, x has {m}")
    t = t.reshape(rows, cols)
    keep.append(t)
    return (t.data_ptr(), *t.stride())


def _write(t, m, cols, dtype, dev, what):
    """An output's address and strides as a matrix; never a copy."""
    if (t.dtype is dtype and t.get_device() == dev and t.dim() == 2 and t.size(1) == cols
            and t.size(0) == m):
        return (t.data_ptr(), *t.stride())
    if t.dtype is not dtype:
        raise ValueError(f"{what} is {t.dtype}, expected {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, the weights are on cuda:{dev}")
    if t.dim() == 0 or t.shape[-1] != cols or t.numel() != m * cols:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {m} rows of {cols}")
    t = t.view(m, cols)
    return (t.data_ptr(), *t.stride())


def _row_count(x):
    return x.size(0) if x.dim() == 2 else math.prod(x.shape[:-1])


def _new(m, cols, dtype, weight, like):
    """An output on the current stream, with the leading dimensions of `like`."""
    t = torch.empty(m, cols, dtype=dtype, device=weight.device)
    return t if like.dim() == 2 else t.view(*like.shape[:-1], cols)


@contextlib.contextmanager
def _on(stream, dev, tensors):
    """Run a call on another stream than the current one: allocations belong to that stream, and
    the caller's tensors are not handed out again before it has passed the call."""
    if stream.device_index != dev:
        raise ValueError(f"stream is of cuda:{stream.device_index}, the weights are on cuda:{dev}")
    with torch.cuda.stream(stream):
        yield
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


class _Dense:
    def _start(self, device):
        self._report_to(torch.zeros(1, dtype=torch.int32, device=device))
        self._need = {}

    def _report_to(self, word):
        """`word` is what an expired wait is written to from now on."""
        self._status = word
        self._word = word.data_ptr()
        self._dev = word.get_device()

    def status(self) -> int:
        """COLL_OK, or COLL_ETIMEDOUT if a bounded device wait of an earlier call expired (its
        outputs are then incomplete). Synchronises with the object's calls on the current
        stream."""
        return int(self._status.item())

    def _launch(self, where, pack, fields, given=False):
        """Call an entry point on the current stream, with the workspace it needs. The size of the
        last call is kept with what decided it, so that a loop over one size asks once and a
        smaller call is not given a larger one's workspace; a call after one that needed none is
        first made without. `given`: whether the one optional array is there whose strides do not
        tell. The library launches on the current device, which the weights' is made for the call.
        """
        if _current_device() != self._dev:
            with torch.cuda.device(self._dev):
                return self._launch(where, pack, fields, given)
        fn, size = _entries.get(where) or _entry(where)
        stream = _raw_stream(self._dev)  # the current stream's handle
        need, kept = 0, self._need.get(where)
        if kept is not None and kept[0]:
            need = kept[0] if kept[1] == fields else self._fit(where, pack, size, fields, given)
        if not need:
            code = fn(pack(*fields, 0, 0, self._word), stream)
            if code == _EWORKSPACE:
                need = self._fit(where, pack, size, fields, given)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=self._status.device)
            code = fn(pack(*fields, ws.data_ptr(), need, self._word), stream)
        if code:
            check(code, where)

    def _fit(self, where, pack, size, fields, given):
        """The workspace of a call, asked for unless the last one was alike."""
        args = pack(*fields, 0, 0, self._word)
        key = (int.from_bytes(args, "little") & _MASK[where], given)
        kept = self._need.get(where)  # (workspace, of which call, what decided it)
        need = kept[0] if kept is not None and kept[2] == key else int(size(args))
        if need < 0:
            check(need, where)
        self._need[where] = (need, fields, key)
        return need


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
            with _on(stream, self._dev, (x, residual, out, pre, self.weight, self.bias,
                                         self._status)):
                return self.forward(x, residual, out, out_dtype, save, pre)
        w, b, dev, keep = self.weight, self.bias, self._dev, []
        n, k = w.shape
        dt = w.dtype
        xm = _read(x, None, k, dt, dev, "x", keep)
        m = _row_count(x)
        if out is None:
            ot = out_dtype or dt
            if ot is not dt and ot is not torch.float32:
                raise ValueError(f"out_dtype must be {dt} or torch.float32, not {ot}")
            out = _new(m, n, ot, w, x)
        else:
            ot = out.dtype
            if out_dtype is not None and out_dtype is not ot:
                raise ValueError(f"out is {ot}, out_dtype is {out_dtype}")
            if ot is not dt and ot is not torch.float32:
                raise ValueError(f"out is {ot}, expected {dt} or torch.float32")
        ym = _write(out, m, n, ot, dev, "out")
        if pre is None and save:
            pre = _new(m, n, dt, w, x)
        pm = _NONE if pre is None else _write(pre, m, n, dt, dev, "pre")
        rm = _NONE
        if residual is not None:
            if residual.shape != out.shape:
                residual = residual.expand(out.shape)
            rm = _read(residual, m, n, ot, dev, "residual", keep)
        self._launch("coll_linear", _LINEAR.pack,
                     (m, n, k, _TYPE[dt], _TYPE[ot], ACT[self.act], *xm, w.data_ptr(),
                      *w.stride(), *rm, *pm, *ym, 0 if b is None else b.data_ptr(),
                      0 if b is None else b.stride(0)), residual is not None)
        return out if pre is None else (out, pre)

    __call__ = forward

    def backward(self, dy, x, pre=None, need_dx=True, need_dw=True, need_db=None, dx=None,
                 dw=None, db=None, grad_dtype=None, stream=None):
        """(dx, dw, db) for the gradient dy [..., N] of y; None in the place of one that is not
        needed (db follows the bias unless need_db says otherwise). The residual's gradient is dy
        itself. grad_dtype: the type of dw and db, the operands' or torch.float32."""
        if stream is not None:
            with _on(stream, self._dev, (dy, x, pre, dx, dw, db, self.weight, self._status)):
                return self.backward(dy, x, pre, need_dx, need_dw, need_db, dx, dw, db,
                                     grad_dtype)
        w, dev, keep = self.weight, self._dev, []
        n, k = w.shape
        dt = w.dtype
        xm = _read(x, None, k, dt, dev, "x", keep)
        m = _row_count(x)
        dym = _read(dy, m, n, dt, dev, "dy", keep)
        pm = _NONE
        if self.act != "none":
            if pre is None:
                raise ValueError(f"backward of act={self.act!r} needs pre")
            pm = _read(pre, m, n, dt, dev, "pre", keep)
        if need_db is None:
            need_db = self.bias is not None or db is not None
        gt = grad_dtype or (dw.dtype if dw is not None else db.dtype if db is not None else dt)
        if gt is not dt and gt is not torch.float32:
            raise ValueError(f"grad_dtype must be {dt} or torch.float32, not {gt}")
        dxm = dwm = _NONE
        dbp = 0
        if need_dx:
            dx = _new(m, k, dt, w, x) if dx is None else dx
            dxm = _write(dx, m, k, dt, dev, "dx")
        if need_dw:
            dw = torch.empty(n, k, dtype=gt, device=w.device) if dw is None else dw
            dwm = _write(dw, n, k, gt, dev, "dw")
        if need_db:
            db = torch.empty(n, dtype=gt, device=w.device) if db is None else db
            if (db.dtype is not gt or db.get_device() != dev or db.dim() != 1 or db.size(0) != n
                    or (n > 1 and db.stride(0) != 1)):
                raise ValueError(f"db must be a contiguous vector of {n} {gt} on cuda:{dev}")
            dbp = db.data_ptr()
        self._launch("coll_linear_backward", _LINEAR_BWD.pack,
                     (m, n, k, _TYPE[dt], _TYPE[gt], ACT[self.act], *dym, *pm, *xm, w.data_ptr(),
                      *w.stride(), *dxm, *dwm, dbp), need_db)
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
            with _on(stream, self._dev, (x, out, gate, up, self.w_gate, self.w_up, self._status)):
                return self.forward(x, out, save, gate, up)
        w, wu, dev, keep = self.w_gate, self.w_up, self._dev, []
        n, k = w.shape
        dt = w.dtype
        xm = _read(x, None, k, dt, dev, "x", keep)
        m = _row_count(x)
        out = _new(m, n, dt, w, x) if out is None else out
        hm = _write(out, m, n, dt, dev, "out")
        gm = um = _NONE
        kept = save or gate is not None or up is not None
        if kept:
            gate = _new(m, n, dt, w, x) if gate is None else gate
            up = _new(m, n, dt, w, x) if up is None else up
            gm, um = _write(gate, m, n, dt, dev, "gate"), _write(up, m, n, dt, dev, "up")
        self._launch("coll_gated_ffn", _GATED.pack,
                     (m, n, k, _TYPE[dt], ACT[self.act], *xm, w.data_ptr(), *w.stride(),
                      wu.data_ptr(), *wu.stride(), *gm, *um, *hm))
        return (out, gate, up) if kept else out

    __call__ = forward

    def backward(self, dh, x, gate, up, need_dx=True, need_dw=True, dx=None, dw_gate=None,
                 dw_up=None, grad_dtype=None, stream=None):
        """(dx, dw_gate, dw_up) for the gradient dh [..., F] of h; None in the place of one that
        is not needed. gate and up: what forward kept. grad_dtype: the type of dw_gate and dw_up,
        the operands' or torch.float32."""
        if stream is not None:
            with _on(stream, self._dev, (dh, x, gate, up, dx, dw_gate, dw_up, self.w_gate,
                                         self.w_up, self._status)):
                return self.backward(dh, x, gate, up, need_dx, need_dw, dx, dw_gate, dw_up,
                                     grad_dtype)
        w, wu, dev, keep = self.w_gate, self.w_up, self._dev, []
        n, k = w.shape
        dt = w.dtype
        xm = _read(x, None, k, dt, dev, "x", keep)
        m = _row_count(x)
        dhm = _read(dh, m, n, dt, dev, "dh", keep)
        gm = _read(gate, m, n, dt, dev, "gate", keep)
        um = _read(up, m, n, dt, dev, "up", keep)
        gt = grad_dtype or (dw_gate.dtype if dw_gate is not None else
                            dw_up.dtype if dw_up is not None else dt)
        if gt is not dt and gt is not torch.float32:
            raise ValueError(f"grad_dtype must be {dt} or torch.float32, not {gt}")
        dxm = dgm = dum = _NONE
        if need_dx:
            dx = _new(m, k, dt, w, x) if dx is None else dx
            dxm = _write(dx, m, k, dt, dev, "dx")
        if need_dw:
            dw_gate = torch.empty(n, k, dtype=gt, device=w.device) if dw_gate is None else dw_gate
            dw_up = torch.empty(n, k, dtype=gt, device=w.device) if dw_up is None else dw_up
            dgm = _write(dw_gate, n, k, gt, dev, "dw_gate")
            dum = _write(dw_up, n, k, gt, dev, "dw_up")
        self._launch("coll_gated_ffn_backward", _GATED_BWD.pack,
                     (m, n, k, _TYPE[dt], _TYPE[gt], ACT[self.act], *dhm, *gm, *um, *xm,
                      w.data_ptr(), *w.stride(), wu.data_ptr(), *wu.stride(), *dxm, *dgm, *dum))
        return (dx if need_dx else None, dw_gate if need_dw else None,
                dw_up if need_dw else None)
