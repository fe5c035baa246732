"""Tensor-level calls of the products (include/zs_product.h) and their autograd form.

    Weight8, weight8_pack        a weight in 8 bits with one scale per 128 x 128 block
    product8                     a linear layer's output, or its input's gradient, from 8-bit operands
    expert_product, expert_wgrad a layer's products where each expert has rows of its own
    Route, route                 the order of tokens' choices by expert
    expert_gather, expert_combine, expert_combine_backward
                                 the rows in that order, and back to their tokens
    linear8, experts, dispatch, combine
                                 the same under autograd

As in the activation operators, the functions work on the current stream of their tensors' device,
write into the tensors they are given, never wait for the GPU, and refuse a wrong type, shape,
stride or device with a ValueError before anything is enqueued.  What a call writes counts as
changed in place for autograd.  The layers have a backward pass and no forward-mode derivative; a
trace records them, and route, as one operation each.
"""

from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _abi as A
from .activations import (_DTYPES, CODES, HALF, Act8, _add_in_turn, _at, _check_grad_into, _checkpoint, _enqueue, _fills,
                          _has_own_version, _input, _matrix, _need_gpu, _rows, _workspace, _wrote, act_wgrad)

BLOCK = 128
_transformed, _traced = torch._C._are_functorch_transforms_active, torch._C._is_tracing


def _blocks(n):
    return -(-n // BLOCK)


class Weight8:
    """A weight [outs, cols] in 8 bits: `codes`, uint8 [outs, cols rounded up to a multiple of 128],
    `scales`, uint8 [blocks of 128 of outs, of cols], and for the input's gradient `codes_t`, uint8
    [cols, outs rounded up to a multiple of 128], or None; contiguous on one GPU.  The codes behind
    each row are zero."""

    __slots__ = ("codes", "codes_t", "scales", "outs", "cols", "device", "arrays", "address", "source")

    def __init__(self, codes, scales, cols, codes_t=None):
        cols = int(cols)
        if cols < 1:
            raise ValueError("cols must be positive")
        if codes.dim() != 2 or codes.shape[0] < 1:
            raise ValueError("codes must be a matrix with at least one row")
        outs = codes.shape[0]
        device = codes.device
        for t, what, shape in ((codes, "codes", (outs, _blocks(cols) * BLOCK)),
                               (scales, "scales", (_blocks(outs), _blocks(cols))),
                               (codes_t, "codes_t", (cols, _blocks(outs) * BLOCK))):
            if t is None and t is codes_t:
                continue
            if t.dtype != torch.uint8 or t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{what} of a weight of {outs} x {cols} must be uint8, contiguous, of shape {shape}, got "
                                 f"{t.dtype} {tuple(t.shape)}")
            if t.device != device:
                raise ValueError(f"codes are on {device}, {what} on {t.device}")
        self.codes, self.codes_t, self.scales, self.outs, self.cols = codes, codes_t, scales, outs, cols
        self.device = device
        self.arrays = A.Weight8Arrays(0, 0, 0)
        self.address = ctypes.addressof(self.arrays)
        self.source = None

    _taken_of = Act8._taken_of
    _outlived = Act8._outlived

    def _wrote(self):
        """The arrays that a write gives a new version; parts of a larger tensor are counted apart, as
        a checkpoint's are."""
        arrays = [t for t in (self.codes, self.codes_t, self.scales) if t is not None]
        if not any(t._is_view() for t in arrays):
            return arrays
        own = [t for t in arrays if _has_own_version(t)]
        for t in arrays[:-1]:
            if not _has_own_version(t):
                _fills(t)[0] += 1
        return own

    @classmethod
    def empty(cls, outs, cols, transposed=True, device="cuda"):
        """A weight with newly allocated, unwritten arrays; `transposed`: with the transposed codes."""
        outs, cols = int(outs), int(cols)

        def array(*shape):
            return torch.empty(shape, dtype=torch.uint8, device=device)

        return cls(array(outs, _blocks(cols) * BLOCK), array(_blocks(outs), _blocks(cols)), cols,
                   array(cols, _blocks(outs) * BLOCK) if transposed else None)

    @classmethod
    def of(cls, w, transposed=True):
        """The 8-bit form of a weight matrix (bf16, fp16 or fp32)."""
        w8 = cls.empty(w.shape[0], w.shape[1], transposed, w.device)
        weight8_pack(w, w8)
        return w8

    @property
    def nbytes(self):
        return self.codes.numel() + self.scales.numel() + (self.codes_t.numel() if self.codes_t is not None else 0)


def _weight8(w8, device):
    if w8.device != device:
        raise ValueError(f"w8 lives on {w8.device}, not on {device}")
    arrays = w8.arrays
    arrays.codes, arrays.scales = w8.codes.data_ptr(), w8.scales.data_ptr()
    arrays.codes_t = w8.codes_t.data_ptr() if w8.codes_t is not None else None
    return w8.address


def weight8_pack(w, w8):
    """Write the 8-bit form of matrix w (bf16, fp16 or fp32; any row stride) into `w8`."""
    outs, cols, dev, stride = _input(w, "w", _DTYPES)
    if (w8.outs, w8.cols) != (outs, cols):
        raise ValueError(f"w8 is a weight of {w8.outs} x {w8.cols}, not of {outs} x {cols}")
    _enqueue("zs_weight8_pack", dev, w.data_ptr(), _DTYPES[w.dtype], stride, outs, cols, _weight8(w8, dev))
    _wrote(w8._wrote())
    w8._taken_of(w)


def product8(x8, w8, y, transposed=False):
    """y = x W^T from the e4m3 checkpoint x8 of x [rows, cols] and the 8-bit weight w8 [outs, cols];
    transposed: y = x W for x [rows, outs], the input's gradient from the checkpoint of the output's.
    y is a bf16 or fp16 matrix of any row stride."""
    rows, n, dev, ys = _input(y, "y", HALF)
    k, wide = (w8.outs, w8.cols) if transposed else (w8.cols, w8.outs)
    if n != wide:
        raise ValueError(f"y has {n} columns, the product {wide}")
    if x8.code != "e4m3":
        raise ValueError("x8 must hold e4m3 codes")
    if transposed and w8.codes_t is None:
        raise ValueError("w8 has no transposed codes")
    arrays = _checkpoint(x8, "x8", rows, k, dev)
    _enqueue("zs_product8", dev, arrays, rows, _weight8(w8, dev), w8.outs, w8.cols, 1 if transposed else 0, y.data_ptr(),
             _DTYPES[y.dtype], ys)
    _wrote((y,))


# ------------------------------------------------------------------------------ experts

def _ends(ends, device, experts=None):
    if ends.dtype != torch.int32 or ends.dim() != 1 or ends.numel() < 1 or not ends.is_contiguous():
        raise ValueError("ends must be a contiguous int32 vector with one element per expert")
    if experts is not None and ends.numel() != experts:
        raise ValueError(f"ends has {ends.numel()} elements for {experts} experts")
    if ends.device != device:
        raise ValueError(f"ends lives on {ends.device}, not on {device}")
    return ends.numel()


def _expert_matrices(t, what, dtypes, experts, rows, cols, device):
    """Check the experts' matrices; returns their row stride and the stride from one to the next."""
    if t.dtype not in dtypes:
        raise ValueError(f"{what} is {t.dtype}, not one of {tuple(dtypes)}")
    if t.shape != (experts, rows, cols):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {(experts, rows, cols)}")
    if t.device != device:
        raise ValueError(f"{what} lives on {t.device}, not on {device}")
    apart, row, col = t.stride()
    if cols > 1 and col != 1:
        raise ValueError(f"{what}: the columns must be consecutive (its stride is {t.stride()})")
    return row, apart


def expert_product(x, w, ends, y, in_major=False, zero_rest=False):
    """y[r] = x[r] W_e^T for each row r of expert e, with w [experts, outs, cols]; in_major: y[r] =
    x[r] W_e with w [experts, cols, outs] (and so, with the same w, the input's gradient from the
    output's).  ends: int32 on the GPU, the row behind each expert's last; the first expert begins
    at row 0, each other behind the one before.  zero_rest writes zeros into the rows of y behind
    the last expert's, which otherwise stay as they were."""
    rows, cols, dev, xs = _input(x, "x", HALF)
    experts = _ends(ends, dev)
    if w.dim() != 3:
        raise ValueError(f"w must have three dimensions, got shape {tuple(w.shape)}")
    outs = w.shape[2 if in_major else 1]
    if outs < 1:
        raise ValueError("w must have at least one row for each expert")
    ws, apart = _expert_matrices(w, "w", (x.dtype,), experts, *((cols, outs) if in_major else (outs, cols)), dev)
    ys = _matrix(y, "y", x.dtype, rows, outs, dev)
    _enqueue("zs_expert_product", dev, x.data_ptr(), xs, w.data_ptr(), ws, apart, _DTYPES[x.dtype], ends.data_ptr(), experts,
             rows, cols, outs, 1 if in_major else 0, y.data_ptr(), ys, 1 if zero_rest else 0)
    _wrote((y,))


def expert_wgrad(x, dy, ends, dw, base=None, in_major=False):
    """dw[e] = base[e] + dy_e^T x_e over the rows of expert e: dw [experts, outs, cols], or [experts,
    cols, outs] with in_major, in x's dtype or fp32.  base has dw's dtype, shape and strides and
    may be dw itself: the gradients are then added to what is there."""
    rows, cols, dev, xs = _input(x, "x", HALF)
    experts = _ends(ends, dev)
    if dy.dim() != 2 or dy.shape[1] < 1:
        raise ValueError(f"dy must be a matrix with at least one column, got shape {tuple(dy.shape)}")
    outs = dy.shape[1]
    dys = _matrix(dy, "dy", x.dtype, rows, outs, dev)
    shape = (cols, outs) if in_major else (outs, cols)
    dws, apart = _expert_matrices(dw, "dw", (x.dtype, torch.float32), experts, *shape, dev)
    if base is not None and base is not dw:
        row, far = _expert_matrices(base, "base", (dw.dtype,), experts, *shape, dev)
        if (row != dws and shape[0] > 1) or (far != apart and experts > 1):
            raise ValueError("base and dw must have the same strides")
    _enqueue("zs_expert_wgrad", dev, x.data_ptr(), xs, dy.data_ptr(), dys, _DTYPES[x.dtype], ends.data_ptr(), experts, rows,
             cols, outs, dw.data_ptr(), _DTYPES[dw.dtype], dws, apart, 1 if in_major else 0, _at(base))
    _wrote((dw,))


# ------------------------------------------------------------------------------ routing

class Route:
    """Where tokens' choices go: `ends`, int32 [experts], the row behind each expert's last; `slot`,
    int32 [tokens * choices], the choice (token * choices + its number) that each row holds, below 0
    for the rows of choices without expert, which lie behind all others; `place`, int32 [tokens,
    choices], the row of each choice, -1 without expert.  Contiguous on one GPU."""

    __slots__ = ("ends", "slot", "place")

    def __init__(self, ends, slot, place):
        if place.dim() != 2 or place.shape[1] < 1:
            raise ValueError(f"place must be [tokens, choices], got shape {tuple(place.shape)}")
        if slot.shape != (place.numel(),):
            raise ValueError(f"slot must have {place.numel()} elements, got shape {tuple(slot.shape)}")
        _ends(ends, place.device)
        for t, what in ((slot, "slot"), (place, "place")):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError(f"{what} must be int32 and contiguous")
            if t.device != place.device:
                raise ValueError(f"{what} lives on {t.device}, not on {place.device}")
        self.ends, self.slot, self.place = ends, slot, place

    @property
    def experts(self):
        return self.ends.numel()

    @property
    def tokens(self):
        return self.place.shape[0]

    @property
    def choices(self):
        return self.place.shape[1]

    @property
    def rows(self):
        return self.slot.numel()


def route(ids, experts, workspace=None):
    """The Route of ids [tokens, choices] (int32 or int64, contiguous): rows ordered by expert, choices
    of one expert in their order.  A number outside 0 .. experts - 1 names no expert."""
    if ids.dim() != 2 or ids.shape[1] < 1:
        raise ValueError(f"ids must be [tokens, choices], got shape {tuple(ids.shape)}")
    if ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
        raise ValueError("ids must be int32 or int64 and contiguous")
    _need_gpu(ids.device)
    if _traced():
        return _route_of(*_Routed.apply(ids, int(experts), workspace))
    return _route(ids, int(experts), workspace)


def _route(ids, experts, workspace):
    device, slots = ids.device, ids.numel()
    own = workspace is None
    workspace, size = _workspace(workspace, A.zs_route_workspace(slots, experts), device)
    ends = torch.empty(experts, dtype=torch.int32, device=device)
    slot = torch.empty(slots, dtype=torch.int32, device=device)
    place = torch.empty(ids.shape, dtype=torch.int32, device=device)
    _enqueue("zs_route", device, ids.data_ptr(), ids.element_size(), slots, experts, ends.data_ptr(), slot.data_ptr(),
             place.data_ptr(), workspace.data_ptr(), size)
    if not own:
        _wrote((workspace,))
    return _route_of(ends, slot, place)


def _route_of(ends, slot, place):
    """A Route of arrays that need no checks."""
    out = Route.__new__(Route)
    out.ends, out.slot, out.place = ends, slot, place
    return out


class _Routed(torch.autograd.Function):
    """route as one operation of a trace."""

    @staticmethod
    def forward(ctx, ids, experts, workspace):
        r = _route(ids, experts, workspace)
        ctx.mark_non_differentiable(r.ends, r.slot, r.place)
        return r.ends, r.slot, r.place

    @staticmethod
    def backward(ctx, *grads):
        return None, None, None


def _routed(route, device):
    place = route.place
    if place.device != device:
        raise ValueError(f"the route lives on {place.device}, not on {device}")
    return place.shape


def _choice_weights(t, what, tokens, choices, device):
    if t.dtype != torch.float32 or t.shape != (tokens, choices) or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous fp32 of shape {(tokens, choices)}")
    if t.device != device:
        raise ValueError(f"{what} lives on {t.device}, not on {device}")


def expert_gather(x, route, out):
    """out[p] = the row of x [tokens, cols] (bf16, fp16 or fp32) whose choice lies at row p of the route;
    zeros in the rows of choices without expert."""
    tokens, cols, dev, xs = _input(x, "x", _DTYPES)
    routed, choices = _routed(route, dev)
    if routed != tokens:
        raise ValueError(f"x has {tokens} rows, the route {routed} tokens")
    outs = _matrix(out, "out", x.dtype, tokens * choices, cols, dev)
    _enqueue("zs_expert_gather", dev, x.data_ptr(), xs, _DTYPES[x.dtype], route.slot.data_ptr(), tokens, choices, cols,
             out.data_ptr(), outs)
    _wrote((out,))


def expert_combine(y, route, out, weights=None):
    """out[t] = the sum over token t's choices of weights[t][j] * the row of y that holds it, in fp32 and
    in the choices' order; weights: fp32 [tokens, choices], or None for ones."""
    tokens, cols, dev, outs = _input(out, "out", _DTYPES)
    routed, choices = _routed(route, dev)
    if routed != tokens:
        raise ValueError(f"out has {tokens} rows, the route {routed} tokens")
    ys = _matrix(y, "y", out.dtype, tokens * choices, cols, dev)
    if weights is not None:
        _choice_weights(weights, "weights", tokens, choices, dev)
    _enqueue("zs_expert_combine", dev, y.data_ptr(), ys, _DTYPES[y.dtype], route.place.data_ptr(), _at(weights), tokens,
             choices, cols, out.data_ptr(), outs)
    _wrote((out,))


def expert_combine_backward(dout, y, route, weights=None, dy=None, dweights=None):
    """Backward of expert_combine: dy[p] = weight * dout[token] for the choice at row p, dweights = the
    choices' dot products of dout and y (fp32 [tokens, choices]); each is written if it is given.  y
    is needed for dweights only."""
    tokens, cols, dev, ds = _input(dout, "dout", _DTYPES)
    routed, choices = _routed(route, dev)
    if routed != tokens:
        raise ValueError(f"dout has {tokens} rows, the route {routed} tokens")
    if dy is None and dweights is None:
        raise ValueError("neither dy nor dweights is given")
    ys = dys = 0
    if dweights is not None:
        _choice_weights(dweights, "dweights", tokens, choices, dev)
        if y is None:
            raise ValueError("dweights needs y")
        ys = _matrix(y, "y", dout.dtype, tokens * choices, cols, dev)
    if weights is not None:
        _choice_weights(weights, "weights", tokens, choices, dev)
    if dy is not None:
        dys = _matrix(dy, "dy", dout.dtype, tokens * choices, cols, dev)
    _enqueue("zs_expert_combine_backward", dev, dout.data_ptr(), ds, _at(y) if dweights is not None else None, ys,
             _DTYPES[dout.dtype], route.slot.data_ptr(), route.place.data_ptr(), _at(weights), tokens, choices, cols,
             _at(dy), dys, _at(dweights))
    _wrote([t for t in (dy, dweights) if t is not None])


# ------------------------------------------------------------------------------ autograd

def _differentiated(*tensors):
    """Whether a layer has to go through its autograd function.  Without a gradient that costs host time
    for nothing, but forward-mode derivatives and function transforms are refused there, and a trace
    records the function (outside of it, the output's allocation alone)."""
    return (torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)
            or forward_ad._current_level >= 0 or _transformed() or _traced())


def _eights(x, weight, x8, w8, turned):
    """The 8-bit forms of a layer's operands that are not given."""
    return (Act8.of(_rows(x)) if x8 is None else x8), (Weight8.of(weight, turned) if w8 is None else w8)


class _Linear8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, x8, w8, grad_into):
        x8, w8 = _eights(x, weight, x8, w8, ctx.needs_input_grad[0])
        y = torch.empty(*x.shape[:-1], w8.outs, dtype=x.dtype, device=x.device)
        product8(x8, w8, y.view(-1, w8.outs))
        ctx.shape, ctx.grad_into = x.shape, grad_into
        kept = [w8.codes, w8.codes_t, w8.scales] if ctx.needs_input_grad[0] else [None] * 3
        kept += [x8.codes, x8.scales] if ctx.needs_input_grad[1] else [None] * 2
        ctx.save_for_backward(*kept)
        # arrays that are parts of a larger tensor have their fills counted (Act8, Weight8)
        ctx.fills = [None if t is None or _has_own_version(t) else _fills(t)[0] for t in kept]
        ctx.like = weight.shape, weight.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        kept = ctx.saved_tensors
        for t, fills, what in zip(kept, ctx.fills, ("weight", "weight", "weight", "input", "input")):
            if fills is not None and _fills(t)[0] > fills:
                raise RuntimeError(f"the 8-bit form of a linear layer's {what}, needed for its gradients, has been modified "
                                   "by an inplace operation: it was filled anew before backward")
        codes, codes_t, scales, x_codes, x_scales = kept
        (outs, cols), dtype = ctx.like
        dy2 = _rows(dy)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = torch.empty(ctx.shape, dtype=dy.dtype, device=dy.device)
            product8(Act8.of(dy2), Weight8(codes, scales, cols, codes_t), dx.view(-1, cols), transposed=True)
        if ctx.needs_input_grad[1]:
            into, x8 = ctx.grad_into, Act8(x_codes, x_scales, cols, "e4m3")
            if into is None:
                dw = torch.empty(outs, cols, dtype=dtype, device=dy.device)
                act_wgrad(x8, dy2, dw)
            else:
                _add_in_turn(into, lambda: act_wgrad(x8, dy2, into, base=into))
        return dx, dw, None, None, None


def linear8(x, weight, w8=None, x8=None, grad_into=None):
    """y = x W^T under autograd in 8 bits, for x [..., cols] and weight [outs, cols]: the output from x's
    and the weight's 8-bit forms, the input's gradient from those of dy and the weight, the
    weight's gradient from x's checkpoint and dy in 16 bits (act_wgrad's).

    x8: the e4m3 checkpoint of x if there is one already (norm's y8); w8: the 8-bit form of the
    weight, with its transposed codes where x needs a gradient: a training program takes it once
    after each optimizer step (weight8_pack), for all micro-steps and passes.  What is not given
    is taken here.  They have to hold what x and the weight hold: a tensor that is known to have
    changed in place since is refused, others (the optimizer's own writes among them) are the
    caller's to match.  grad_into, and capture into graphs: as for norm."""
    if x.dim() < 1 or x.dtype not in HALF or weight.dim() != 2:
        raise ValueError("x must be bf16 or fp16, the weight of two dimensions")
    if weight.dtype != x.dtype:
        raise ValueError(f"the weight is {weight.dtype}, x {x.dtype}")
    outs, cols = weight.shape
    if x.shape[-1] != cols or cols < 1 or outs < 1:
        raise ValueError(f"x has {x.shape[-1]} columns, the weight is {outs} x {cols}")
    _need_gpu(x.device)
    if weight.device != x.device:
        raise ValueError(f"the weight lives on {weight.device}, not on {x.device}")
    _check_grad_into(grad_into, weight)
    rows = x.numel() // cols
    turned = x.requires_grad and torch.is_grad_enabled()
    if x8 is not None:
        if x8.code != "e4m3":
            raise ValueError("x8 must hold e4m3 codes")
        _checkpoint(x8, "x8", rows, cols, x.device)
        if x8._outlived(x):
            raise ValueError("x has been changed in place since x8 was taken of it")
    if w8 is not None:
        if (w8.outs, w8.cols) != (outs, cols) or w8.device != x.device:
            raise ValueError(f"w8 is a weight of {w8.outs} x {w8.cols} on {w8.device}, not of {outs} x {cols} on {x.device}")
        if turned and w8.codes_t is None:
            raise ValueError("w8 has no transposed codes, which the gradient of x needs")
        if w8._outlived(weight):
            raise ValueError("the weight has been changed in place since w8 was taken of it")
    if not _differentiated(x, weight):
        x8, w8 = _eights(x, weight, x8, w8, False)
        y = torch.empty(*x.shape[:-1], outs, dtype=x.dtype, device=x.device)
        product8(x8, w8, y.view(-1, outs))
        return y
    return _Linear8.apply(x, weight, x8, w8, grad_into)


class _Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, ends, in_major, save, grad_into):
        outs = weight.shape[2 if in_major else 1]
        y = torch.empty(x.shape[0], outs, dtype=x.dtype, device=x.device)
        expert_product(x, weight, ends, y, in_major=in_major, zero_rest=True)
        ctx.in_major, ctx.save, ctx.grad_into, ctx.cols = in_major, save, grad_into, x.shape[1]
        kept = []
        if ctx.needs_input_grad[1]:
            if save is not None:
                x8 = Act8.of(x, save)
                kept = [x8.codes, x8.scales]
            else:
                kept = [x]
        ctx.save_for_backward(ends, weight if ctx.needs_input_grad[0] else None, *kept)
        ctx.like = weight.shape, weight.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ends, weight, *kept = ctx.saved_tensors
        dy2 = _rows(dy)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = torch.empty(dy2.shape[0], ctx.cols, dtype=dy.dtype, device=dy.device)
            expert_product(dy2, weight, ends, dx, in_major=not ctx.in_major, zero_rest=True)
        if ctx.needs_input_grad[1]:
            into = ctx.grad_into
            x = kept[0] if ctx.save is None else Act8(kept[0], kept[1], ctx.cols, ctx.save).unpack(dy.dtype)
            if into is None:
                shape, dtype = ctx.like
                dw = torch.empty(shape, dtype=dtype, device=dy.device)
                expert_wgrad(x, dy2, ends, dw, in_major=ctx.in_major)
            else:
                _add_in_turn(into, lambda: expert_wgrad(x, dy2, ends, into, base=into, in_major=ctx.in_major))
        return dx, dw, None, None, None, None


def experts(x, weight, ends, in_major=False, save=None, grad_into=None):
    """expert_product under autograd: y [rows, outs] for x [rows, cols] whose rows are ordered by expert,
    weight [experts, outs, cols] ([experts, cols, outs] with in_major) and ends (a Route's).  Rows
    behind the last expert's are zero in y and in the gradient of x.

    save: what backward keeps of x for the weights' gradient: its checkpoint ("e4m3" or "int8"), or
    None for x itself.  grad_into, a buffer of the weight's shape (its dtype or fp32), and capture
    into graphs: as for norm."""
    if x.dim() != 2 or x.dtype not in HALF or weight.dim() != 3 or weight.dtype != x.dtype:
        raise ValueError("x must be a bf16 or fp16 matrix, the weight of three dimensions in x's dtype")
    _need_gpu(x.device)
    if save is not None and save not in CODES:
        raise ValueError(f"save is 'e4m3', 'int8' or None, not {save!r}")
    _ends(ends, x.device, weight.shape[0])
    _check_grad_into(grad_into, weight)
    if not _differentiated(x, weight):
        y = torch.empty(x.shape[0], weight.shape[2 if in_major else 1], dtype=x.dtype, device=x.device)
        expert_product(_rows(x), weight, ends, y, in_major=in_major, zero_rest=True)
        return y
    return _Experts.apply(_rows(x), weight, ends, bool(in_major), save, grad_into)


def _gathered(x, route):
    out = torch.empty(route.rows, x.shape[1], dtype=x.dtype, device=x.device)
    expert_gather(x, route, out)
    return out


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, *places):
        out = _gathered(x, _route_of(*places))
        ctx.save_for_backward(*places)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        route = _route_of(*ctx.saved_tensors)
        dx = torch.empty(route.tokens, dout.shape[1], dtype=dout.dtype, device=dout.device)
        expert_combine(_rows(dout), route, dx)
        return dx, None, None, None


def dispatch(x, route):
    """expert_gather under autograd: the rows of x [..., cols] (tokens in order) in the route's order."""
    if x.dim() < 1 or x.dtype not in _DTYPES or x.shape[-1] < 1:
        raise ValueError("x must be a bf16, fp16 or fp32 tensor with at least one column")
    if not _differentiated(x):
        return _gathered(_rows(x), route)
    return _Dispatch.apply(_rows(x), route.ends, route.slot, route.place)


def _combined(y, weights, route):
    out = torch.empty(route.tokens, y.shape[1], dtype=y.dtype, device=y.device)
    expert_combine(y, route, out, weights)
    return out


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, *places):
        out = _combined(y, weights, _route_of(*places))
        turn_y, turn_weights = ctx.needs_input_grad[0], weights is not None and ctx.needs_input_grad[1]
        ctx.save_for_backward(*places, weights if turn_y else None, y if turn_weights else None)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        *places, weights, y = ctx.saved_tensors
        route = _route_of(*places)
        dout = _rows(dout)
        dy = dweights = None
        if ctx.needs_input_grad[0]:
            dy = torch.empty(route.rows, dout.shape[1], dtype=dout.dtype, device=dout.device)
        if y is not None:
            dweights = torch.empty(route.tokens, route.choices, dtype=torch.float32, device=dout.device)
        expert_combine_backward(dout, y, route, weights, dy, dweights)
        return dy, dweights, None, None, None


def combine(y, route, weights=None):
    """expert_combine under autograd: the rows of y [rows, cols] back to their tokens, [tokens, cols].
    weights: fp32 [tokens, choices] (the router's), or None for ones."""
    if y.dim() != 2 or y.dtype not in _DTYPES or y.shape[1] < 1:
        raise ValueError("y must be a bf16, fp16 or fp32 matrix with at least one column")
    weights = weights.contiguous() if weights is not None else None
    if not _differentiated(y, weights):
        return _combined(_rows(y), weights, route)
    return _Combine.apply(_rows(y), weights, route.ends, route.slot, route.place)
