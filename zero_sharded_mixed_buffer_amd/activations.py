"""Tensor-level calls of the activation operators (include/zs_act.h) and their autograd form.

What a training program keeps between forward and backward, at 1.03 bytes per element, and the
gradients that backward then writes into the optimizer's gradient buffer:

    Act8                         an 8-bit checkpoint of a rows x cols matrix
    act_pack, act_unpack         write a checkpoint, read it back
    rmsnorm, rmsnorm_backward    the norm with the residual's addition; it writes checkpoints of
                                 its output and of its input in the same pass
    act_wgrad                    a linear layer's weight gradient from its input's checkpoint
    norm, linear                 the same under autograd

The functions work on the current stream of their tensors' device, write into the tensors they
are given, allocate nothing but a workspace that was not passed in, and never wait for the GPU.
What a call writes, a checkpoint's arrays among it, counts as changed in place for autograd.
A wrong type, shape, stride or device is a ValueError before anything is enqueued.
"""

from __future__ import annotations

import ctypes
import threading
import weakref
from collections import namedtuple

import torch
from torch.autograd.function import once_differentiable

from . import _abi as A

GROUP = 32
CODES = {"e4m3": A.ZS_E4M3, "int8": A.ZS_INT8}
HALF = (torch.bfloat16, torch.float16)
_DTYPES = {torch.bfloat16: A.ZS_BF16, torch.float16: A.ZS_FP16, torch.float32: A.ZS_FP32}


class Act8:
    """An 8-bit checkpoint: `codes`, uint8 [rows, cols rounded up to a multiple of 32], and
    `scales`, uint8 [rows, groups of 32], both contiguous on one GPU; `code` is "e4m3" or
    "int8".  The arrays are the caller's, or Act8.empty's."""

    __slots__ = ("codes", "scales", "rows", "cols", "code", "device", "arrays", "address", "source")

    # `arrays` is the struct that the C calls read; every call writes the tensors' present
    # addresses into it, so that storage which was freed and allocated again is found.
    # `source` is what the checkpoint was last taken of, if that is known: a tensor's storage (weakly
    # held), the tensor's version and the codes' version then

    def __init__(self, codes, scales, cols, code="e4m3"):
        if code not in CODES:
            raise ValueError(f"code is 'e4m3' or 'int8', not {code!r}")
        cols = int(cols)
        if cols < 1:
            raise ValueError("cols must be positive")
        groups = -(-cols // GROUP)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise ValueError("codes and scales must be uint8")
        shape = codes.shape
        rows = shape[0] if shape else -1
        if shape != (rows, groups * GROUP) or scales.shape != (rows, groups):
            raise ValueError(f"a checkpoint of {cols} columns holds codes [rows, {groups * GROUP}] and scales "
                             f"[rows, {groups}], got {tuple(codes.shape)} and {tuple(scales.shape)}")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous")
        device = codes.device
        if device != scales.device:
            raise ValueError(f"codes are on {codes.device}, scales on {scales.device}")
        self.codes, self.scales, self.rows, self.cols, self.code = codes, scales, rows, cols, code
        self.device = device
        self.arrays = A.ActArrays(0, 0, CODES[code], 0)
        self.address = ctypes.addressof(self.arrays)
        self.source = None

    def _wrote(self):
        """The arrays that a write gives a new version.  Those that are parts of a larger tensor share
        its version with all other parts, other checkpoints' among them: the fills of such codes are
        counted beside their storage instead."""
        codes, scales = self.codes, self.scales
        if not (codes._is_view() or scales._is_view()):
            return [codes, scales]
        own = [t for t in (codes, scales) if _has_own_version(t)]
        if not own or own[0] is not codes:
            _fills(codes)[0] += 1
        return own

    def _taken_of(self, t):
        if t is None or not _has_own_version(t):
            self.source = None
            return
        try:
            self.source = weakref.ref(t.untyped_storage()), t._version, self.codes._version
        except RuntimeError:  # tensors made in inference mode carry no version
            self.source = None

    def _outlived(self, t):
        """Whether t is known to have been changed since the checkpoint was taken of it.  Versions
        only grow; a smaller one is counted apart (t.data's) and says nothing, and neither does that
        of a part of a larger tensor.  Codes written by other means since then may be anyone's."""
        if self.source is None or t.is_inference():
            return False
        storage, of_t, of_codes = self.source
        return storage() is t.untyped_storage() and t._version > of_t and self.codes._version == of_codes

    @classmethod
    def empty(cls, rows, cols, code="e4m3", device="cuda"):
        """A checkpoint with newly allocated, unwritten arrays."""
        groups = -(-int(cols) // GROUP)
        return cls(torch.empty(int(rows), groups * GROUP, dtype=torch.uint8, device=device),
                   torch.empty(int(rows), groups, dtype=torch.uint8, device=device), cols, code)

    @classmethod
    def of(cls, x, code="e4m3"):
        """The checkpoint of a matrix (bf16, fp16 or fp32)."""
        act = cls.empty(x.shape[0], x.shape[1], code, x.device)
        act_pack(x, act)
        return act

    def unpack(self, dtype=torch.bfloat16):
        """The matrix it stands for, in a new tensor."""
        out = torch.empty(self.rows, self.cols, dtype=dtype, device=self.device)
        act_unpack(self, out)
        return out

    @property
    def nbytes(self):
        return self.codes.numel() + self.scales.numel()


def _need_gpu(device):
    if device.type != "cuda":
        raise ValueError(f"the tensors must live on a GPU, not on {device}")


def _enqueue(name, device, *args):
    """Call a C entry point on the current stream of `device`, made the current device for it.
    (The tensor checks above each call stand in for those of the ctypes wrappers; the raw stream
    and device lookups are the ones that cost a fraction of a microsecond.)"""
    fn = getattr(A.lib(), name)
    index = device.index
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        A._check(status, name)


def _wrote(tensors):
    """Mark what a call has written as changed, as torch's own writes are: autograd then refuses a
    backward pass that would read a saved tensor's later contents."""
    try:
        torch._C._increment_version(tensors)
    except RuntimeError:  # tensors made in inference mode carry no version outside of it
        torch._C._increment_version([t for t in tensors if not t.is_inference()])


def _has_own_version(t):
    """Whether t is no part of a larger tensor, whose version it would share with other parts."""
    return not t._is_view() or t.numel() * t.element_size() == t.untyped_storage().nbytes()


def _fills(codes):
    """How often checkpoint codes that are part of a larger tensor have been filled, as a list of one
    number that all checkpoints in this place share."""
    places = codes.untyped_storage().__dict__.setdefault("_act8_fills", {})
    return places.setdefault(codes.storage_offset(), [0])


def _at(t):
    return t.data_ptr() if t is not None else None


def _matrix(t, what, dtype, rows, cols, device):
    """Check a matrix argument; returns its row stride."""
    if t.dtype != dtype:
        raise ValueError(f"{what} is {t.dtype}, not {dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {(rows, cols)}")
    if t.device != device:
        raise ValueError(f"{what} lives on {t.device}, not on {device}")
    row, col = t.stride()
    if cols > 1 and col != 1:
        raise ValueError(f"{what}: the columns must be consecutive (its stride is {t.stride()})")
    return row


def _vector(t, what, dtypes, n, device):
    if t.dtype not in dtypes:
        raise ValueError(f"{what} is {t.dtype}, not one of {dtypes}")
    if t.shape != (n,) or (n > 1 and not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous vector of {n} elements")
    if t.device != device:
        raise ValueError(f"{what} lives on {t.device}, not on {device}")
    return t


def _checkpoint(act, what, rows, cols, device):
    if (act.rows, act.cols) != (rows, cols):
        raise ValueError(f"{what} is a checkpoint of {act.rows} x {act.cols}, not of {rows} x {cols}")
    if act.device != device:
        raise ValueError(f"{what} lives on {act.device}, not on {device}")
    arrays = act.arrays
    arrays.codes, arrays.scales = act.codes.data_ptr(), act.scales.data_ptr()
    return act.address


def _input(t, what, dtypes):
    """Check the argument that sets a call's sizes; returns its rows, columns, device and row
    stride."""
    shape = t.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"{what} must be a matrix with at least one column, got shape {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{what} is {t.dtype}, not one of {tuple(dtypes)}")
    device = t.device
    if not t.is_cuda:
        _need_gpu(device)
    rows, cols = shape
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise ValueError(f"{what}: the columns must be consecutive (its stride is {t.stride()})")
    return rows, cols, device, row


def _workspace(workspace, need, device):
    """The caller's workspace (any contiguous tensor), or a new one: allocated on the current
    stream, so the caching allocator hands it out again only after this call's kernels."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device), need
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"workspace holds {have} bytes, {need} are needed")
    return workspace, have


def act_pack(x, act):
    """Write the checkpoint of matrix x (bf16, fp16 or fp32; any row stride) into `act`."""
    rows, cols, dev, stride = _input(x, "x", _DTYPES)
    arrays = _checkpoint(act, "act", rows, cols, dev)
    _enqueue("zs_act_pack", dev, x.data_ptr(), _DTYPES[x.dtype], stride, rows, cols, arrays)
    _wrote(act._wrote())
    act._taken_of(x)


def act_unpack(act, out):
    """Read a checkpoint back into matrix `out` (bf16, fp16 or fp32; any row stride), each value
    rounded once; past fp16's range to its largest number."""
    rows, cols, dev, stride = _input(out, "out", _DTYPES)
    arrays = _checkpoint(act, "act", rows, cols, dev)
    _enqueue("zs_act_unpack", dev, arrays, rows, cols, out.data_ptr(), _DTYPES[out.dtype], stride)
    _wrote((out,))


def rmsnorm(x, weight, eps=1e-6, residual=None, h=None, y=None, y8=None, h8=None, rstd=None):
    """h = x + residual, rstd = (mean(h^2) + eps)^-1/2 per row, y = h * rstd * weight, in one
    pass; every output that is given is written: h, y (matrices of x's dtype), y8, h8
    (checkpoints of y and h), rstd (fp32 vector).  h may be x or residual itself."""
    rows, cols, dev, xs = _input(x, "x", HALF)
    dt = x.dtype
    _vector(weight, "weight", (dt,), cols, dev)
    rs = _matrix(residual, "residual", dt, rows, cols, dev) if residual is not None else 0
    hs = _matrix(h, "h", dt, rows, cols, dev) if h is not None else 0
    ys = _matrix(y, "y", dt, rows, cols, dev) if y is not None else 0
    if rstd is not None:
        _vector(rstd, "rstd", (torch.float32,), rows, dev)
    ya = _checkpoint(y8, "y8", rows, cols, dev) if y8 is not None else None
    ha = _checkpoint(h8, "h8", rows, cols, dev) if h8 is not None else None
    _enqueue("zs_rmsnorm", dev, x.data_ptr(), xs, _at(residual), rs, weight.data_ptr(), _DTYPES[dt], rows, cols, eps,
             _at(h), hs, _at(y), ys, ya, ha, _at(rstd))
    wrote = [t for t in (h, y, rstd) if t is not None]
    for act in (y8, h8):
        if act is not None:
            wrote += act._wrote()
    _wrote(wrote)
    if y8 is not None:
        y8._taken_of(y)
    if h8 is not None:
        h8._taken_of(x if h is None and residual is None else h)


def rmsnorm_backward(dy, saved, weight, rstd, dx, dh=None, dweight=None, base=None, workspace=None):
    """Backward of rmsnorm: dx = the gradient of x (and of the residual) from dy and, if it is
    given, dh, the gradient that reaches h by other ways; dweight (bf16, fp16 or fp32) = base +
    the weight's gradient.  `saved` is h or its Act8.  base may be dweight itself: the gradient
    is then added to what is there.  dx may be dy or dh."""
    rows, cols, dev, dys = _input(dy, "dy", HALF)
    dt = dy.dtype
    dxs = _matrix(dx, "dx", dt, rows, cols, dev)
    dhs = _matrix(dh, "dh", dt, rows, cols, dev) if dh is not None else 0
    _vector(weight, "weight", (dt,), cols, dev)
    _vector(rstd, "rstd", (torch.float32,), rows, dev)
    h, hs, h8 = None, 0, None
    if isinstance(saved, Act8):
        h8 = _checkpoint(saved, "saved", rows, cols, dev)
    else:
        h, hs = saved, _matrix(saved, "saved", dt, rows, cols, dev)
    size = 0
    if dweight is not None:
        _vector(dweight, "dweight", tuple(_DTYPES), cols, dev)
        if base is not None:
            _vector(base, "base", (dweight.dtype,), cols, dev)
        workspace, size = _workspace(workspace, A.zs_rmsnorm_workspace(rows, cols), dev)
    elif base is not None:
        raise ValueError("base without dweight")
    _enqueue("zs_rmsnorm_backward", dev, dy.data_ptr(), dys, _at(dh), dhs, _at(h), hs, h8, weight.data_ptr(),
             rstd.data_ptr(), _DTYPES[dt], rows, cols, dx.data_ptr(), dxs, _at(dweight),
             _DTYPES[dweight.dtype] if dweight is not None else A.ZS_FP32, _at(base), _at(workspace), size)
    _wrote((dx, dweight, workspace) if dweight is not None else (dx,))


def act_wgrad(x8, dy, dw, base=None, in_major=False, workspace=None):
    """dw = base + dy^T x: the weight gradient of y = x W^T from the checkpoint of x and the
    gradient dy [rows, outs] of y.  dw is [outs, cols], or [cols, outs] with in_major (weights
    kept as (in, out)), in dy's dtype or fp32; base has dw's dtype, shape and stride and may be
    dw itself: the gradient is then added to what is there.  x8's values take part in dy's dtype:
    exact in bf16, and in fp16 for checkpoints of fp16 values (others are rounded to fp16, past
    its range to its largest number)."""
    rows, outs, dev, dys = _input(dy, "dy", HALF)
    arrays = _checkpoint(x8, "x8", rows, x8.cols, dev)
    shape = (x8.cols, outs) if in_major else (outs, x8.cols)
    if dw.dtype not in (dy.dtype, torch.float32):
        raise ValueError(f"dw is {dw.dtype}, not {dy.dtype} or torch.float32")
    dws = _matrix(dw, "dw", dw.dtype, *shape, dev)
    if base is not None and _matrix(base, "base", dw.dtype, *shape, dev) != dws and shape[0] > 1:
        raise ValueError("base and dw must have the same strides")
    workspace, size = _workspace(workspace, A.zs_act_wgrad_workspace(rows, x8.cols, outs), dev)
    _enqueue("zs_act_wgrad", dev, arrays, rows, x8.cols, dy.data_ptr(), _DTYPES[dy.dtype], dys, outs, dw.data_ptr(),
             _DTYPES[dw.dtype], dws, int(bool(in_major)), _at(base), _at(workspace), size)
    _wrote((dw, workspace))


# ------------------------------------------------------------------------------ autograd

NormOutput = namedtuple("NormOutput", ["y", "h", "y8"])


def _rows(t):
    """A tensor's last dimension as matrix columns, copied only if that takes it: rows that overlap,
    such as a broadcast tensor's, are no matrix that the kernels take."""
    m = t.reshape(-1, t.shape[-1])
    rows, cols = m.shape
    row, col = m.stride()
    return m if (cols == 1 or col == 1) and (rows <= 1 or row >= cols) else m.contiguous()


def _check_grad_into(grad_into, weight):
    if grad_into is None:
        return
    if grad_into.shape != weight.shape or not grad_into.is_contiguous() or grad_into.device != weight.device:
        raise ValueError(f"grad_into must be contiguous with the weight's shape {tuple(weight.shape)} on its device")
    if grad_into.dtype not in (weight.dtype, torch.float32):
        raise ValueError("grad_into has the weight's dtype or fp32")
    if grad_into.requires_grad:
        raise ValueError("grad_into is a plain buffer, without requires_grad")


# Additions to a caller's buffer (grad_into) in a backward pass.  Autograd runs each backward on the
# stream of its forward and orders only the gradients that it is handed; these it never sees.  So
# each addition waits for the one before it to the same storage if that ran on another stream, and
# at the end of a pass the stream that called it waits for the last.  (A pass that fails never
# reports its end: its stream then stays one to wait for, which is harmless.)
class _Adds:
    """The additions to one storage: the stream of the last one, as long as a pass is under way,
    and how many the passes under way have made."""

    __slots__ = ("last", "under_way")

    def __init__(self):
        self.last, self.under_way = None, 0


_adds_lock = threading.RLock()


def _captured(stream):
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _wait_for(stream, last):
    """Let `stream` wait for what `last` holds so far, unless just one of them is being captured
    into a graph, which the wait would end."""
    if last is not None and last != stream and _captured(stream) == _captured(last):
        stream.wait_stream(last)


def _add_in_turn(into, add):
    """Call `add`, which enqueues work that adds to `into`, within a backward pass."""
    device = into.device
    stream = torch.cuda.current_stream(device)
    with _adds_lock:
        adds = into.untyped_storage().__dict__.setdefault("_adds", _Adds())
        _wait_for(stream, adds.last)
        add()
        adds.last = stream
        adds.under_way += 1
    torch.autograd.Variable._execution_engine.queue_callback(lambda: _pass_ended(adds, device))


def _pass_ended(adds, device):
    caller = torch.cuda.current_stream(device)
    with _adds_lock:
        _wait_for(caller, adds.last)
        adds.under_way -= 1
        adds.last = caller if adds.under_way else None


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, save, y8, grad_into):
        ctx.set_materialize_grads(False)
        x2 = _rows(x)
        rows, cols = x2.shape
        # in x's shape from the start: a view made here could not be changed in place afterwards
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        h = torch.empty_like(y) if residual is not None else None
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
        h8 = Act8.empty(rows, cols, save, x.device) if save is not None else None
        rmsnorm(x2, weight, eps, residual=_rows(residual) if residual is not None else None,
                h=h.view(rows, cols) if h is not None else None, y=y.view(rows, cols), y8=y8, h8=h8, rstd=rstd)
        ctx.save, ctx.cols, ctx.grad_into, ctx.two = save, cols, grad_into, residual is not None
        if h8 is not None:
            ctx.save_for_backward(weight, rstd, h8.codes, h8.scales)
        else:
            ctx.save_for_backward(weight, rstd, h if h is not None else x)
        return (y, h) if ctx.two else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        weight, rstd, *kept = ctx.saved_tensors
        if dy is None:
            return dh, dh if ctx.two else None, None, None, None, None, None
        saved = Act8(kept[0], kept[1], ctx.cols, ctx.save) if ctx.save is not None else _rows(kept[0])
        dy2 = _rows(dy)
        dx = torch.empty(dy2.shape, dtype=dy.dtype, device=dy.device)
        into, dweight = ctx.grad_into, None
        if ctx.needs_input_grad[2]:
            dweight = torch.empty_like(weight) if into is None else into
        dh2 = _rows(dh) if dh is not None else None
        if dweight is None or into is None:
            rmsnorm_backward(dy2, saved, weight, rstd, dx, dh=dh2, dweight=dweight)
        else:
            _add_in_turn(into, lambda: rmsnorm_backward(dy2, saved, weight, rstd, dx, dh=dh2, dweight=into, base=into))
        dx = dx.view(dy.shape)
        return (dx, dx if ctx.two else None, dweight if into is None else None, None, None, None, None)


def norm(x, weight, eps=1e-6, residual=None, save="e4m3", y8=None, grad_into=None):
    """rmsnorm under autograd, for x [..., cols]: returns NormOutput(y, h, y8).

    h is x + residual (x itself without one) and carries gradients like y.  save: what backward
    keeps of h: its checkpoint ("e4m3" or "int8"), or None for h in 16 bits.  y8: "e4m3" or
    "int8" writes the checkpoint of y in the same pass, for the linear layers that read y.
    grad_into: a buffer of the weight's shape (its dtype or fp32; with flat_views the weight's
    .grad) that backward adds the weight's gradient to; the weight then receives none from
    autograd.  Additions of one pass from several streams are ordered, and the stream that calls
    backward waits for them, as it does for gradients that autograd accumulates.  Passes called
    from different streams, or host threads, that add to one buffer are the caller's to order.

    To capture forward and backward into a graph, let no eager graph of the same leaves be
    alive: autograd would join their streams in the capture."""
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError("residual must have x's shape and dtype")
    if x.dim() < 1 or x.shape[-1] < 1 or x.dtype not in HALF:
        raise ValueError("x must be a bf16 or fp16 tensor with at least one column")
    _need_gpu(x.device)
    _check_grad_into(grad_into, weight)
    if save is not None and save not in CODES:
        raise ValueError(f"save is 'e4m3', 'int8' or None, not {save!r}")
    cols = x.shape[-1]
    act = Act8.empty(x.numel() // cols, cols, y8, x.device) if y8 is not None else None
    if not (torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, residual, weight))):
        save = None  # no backward will read it
    out = _Norm.apply(x, residual, weight, eps, save, act, grad_into)
    y, h = out if residual is not None else (out, x)
    return NormOutput(y, h, act)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, x8, grad_into):
        ctx.save_for_backward(weight, x8.codes, x8.scales)
        ctx.code, ctx.cols, ctx.grad_into = x8.code, x8.cols, grad_into
        ctx.fills = None if _has_own_version(x8.codes) else _fills(x8.codes)[0]
        return torch.nn.functional.linear(x, weight)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        weight, codes, scales = ctx.saved_tensors
        if ctx.fills is not None and _fills(codes)[0] > ctx.fills:
            raise RuntimeError("the checkpoint of a linear layer's input, needed for its weight's gradient, has been "
                               "modified by an inplace operation: it was filled anew before backward")
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = torch.matmul(dy.contiguous(), weight)
        if ctx.needs_input_grad[1]:
            into, x8, dy2 = ctx.grad_into, Act8(codes, scales, ctx.cols, ctx.code), _rows(dy)
            if into is None:
                dw = torch.empty_like(weight)
                act_wgrad(x8, dy2, dw)
            else:
                _add_in_turn(into, lambda: act_wgrad(x8, dy2, into, base=into))
        return dx, dw, None, None


def linear(x, weight, x8=None, code="e4m3", grad_into=None):
    """y = x W^T under autograd, for x [..., cols] and weight [outs, cols], keeping an 8-bit
    checkpoint of x for the weight's gradient instead of x.

    x8: the checkpoint of x if there is one already (norm's y8: several layers that read one
    tensor share it); otherwise it is taken here, with `code`.  It has to hold what x holds: an x
    changed in place since its checkpoint was taken is refused, any other x (a copy, a result of
    x, a part of a larger tensor) is the caller's to match.  grad_into, and capture into graphs:
    as for norm.  The two products with the weight are the library's; the weight's gradient is
    act_wgrad's."""
    if code not in CODES:
        raise ValueError(f"code is 'e4m3' or 'int8', not {code!r}")
    if x.dim() < 1 or x.dtype not in HALF or weight.dtype != x.dtype or weight.dim() != 2:
        raise ValueError("x and a weight of two dimensions must have one dtype, bf16 or fp16")
    if x.shape[-1] != weight.shape[1] or x.shape[-1] < 1:
        raise ValueError(f"x has {x.shape[-1]} columns, the weight {weight.shape[1]}")
    if not weight.is_contiguous():
        raise ValueError("the weight must be contiguous")
    _need_gpu(x.device)
    if weight.device != x.device:
        raise ValueError(f"the weight lives on {weight.device}, not on {x.device}")
    _check_grad_into(grad_into, weight)
    if x8 is not None:
        _checkpoint(x8, "x8", x.numel() // x.shape[-1], x.shape[-1], x.device)
    if not (weight.requires_grad and torch.is_grad_enabled()) or weight.shape[0] == 0:  # nothing of x is kept
        return torch.nn.functional.linear(x, weight)
    if x8 is None:
        x8 = Act8.of(_rows(x.detach()), code)
    elif x8._outlived(x):
        raise ValueError("x has been changed in place since x8 was taken of it")
    return _Linear.apply(x, weight, x8, grad_into)
