"""Plain 64-bit CPU forms of the products, from their definitions (include/zs_product.h): weights in
8 bits with one scale per 128 x 128 block, products of 8-bit operands, products over the experts'
groups of rows with their weight gradients, and the routing of tokens.  Used by tests only."""

from __future__ import annotations

import torch

from . import act_oracle as AO

BLOCK = 128


def weight8(w):
    """Codes, transposed codes and scales (uint8) of a weight matrix."""
    w = w.detach().cpu().double()
    outs, cols = w.shape
    bo, bc = -(-outs // BLOCK), -(-cols // BLOCK)
    wide = torch.zeros(bo * BLOCK, bc * BLOCK, dtype=torch.float64)
    wide[:outs, :cols] = w
    # one row of 128 * 128 elements for each block
    flat = wide.view(bo, BLOCK, bc, BLOCK).permute(0, 2, 1, 3).reshape(bo * bc, BLOCK * BLOCK)
    top = torch.where(torch.isfinite(flat).all(1), flat.abs().amax(1), torch.tensor(float("inf"), dtype=torch.float64))
    b = AO.scale_bytes(top, "e4m3")
    bad = b == 255
    v = torch.where(bad[:, None], torch.zeros_like(flat), flat) / 2.0 ** (b.clamp_max(254) - 127).double()[:, None]
    pos = AO.E4M3[:127]
    m = v.abs()
    hi = torch.searchsorted(pos, m.contiguous()).clamp_max(126)
    lo = (hi - 1).clamp_min(0)
    dlo, dhi = m - pos[lo], pos[hi] - m
    near = torch.where(dlo < dhi, lo, torch.where(dhi < dlo, hi, torch.where(lo % 2 == 0, lo, hi)))
    near = torch.where(pos[hi] == m, hi, near)
    codes = near + 128 * torch.signbit(v).long()
    codes = torch.where(bad[:, None], torch.zeros_like(codes), codes).to(torch.uint8)
    codes = codes.view(bo, bc, BLOCK, BLOCK).permute(0, 2, 1, 3).reshape(bo * BLOCK, bc * BLOCK)
    return codes[:outs].contiguous(), codes.t()[:cols].contiguous(), b.view(bo, bc).to(torch.uint8)


def weight_values(codes, scales, cols):
    """The matrix that an 8-bit weight stands for (float64)."""
    s = 2.0 ** (scales.cpu().double() - 127)
    s = torch.where(scales.cpu() == 255, torch.full_like(s, float("nan")), s)
    s = s.repeat_interleave(BLOCK, 0)[: len(codes)].repeat_interleave(BLOCK, 1)
    return (AO.E4M3[codes.cpu().long()] * s)[:, :cols]


def spans(ends, rows):
    """First and last row of each expert: an end counts as the largest one up to it, within 0 .. rows."""
    out, at = [], 0
    for e in ends.tolist():
        to = max(at, min(max(e, 0), rows))
        out.append((at, to))
        at = to
    return out


def expert_product(x, w, ends, in_major=False):
    """y in float64, with NaN in rows behind the last expert's, and the sums of magnitudes."""
    x, w = x.cpu().double(), w.cpu().double()
    if not in_major:
        w = w.transpose(1, 2)
    y = torch.full((len(x), w.shape[2]), float("nan"), dtype=torch.float64)
    size = torch.zeros_like(y)
    for e, (a, b) in enumerate(spans(ends.cpu(), len(x))):
        y[a:b] = x[a:b] @ w[e].contiguous()
        size[a:b] = x[a:b].abs() @ w[e].abs().contiguous()
    return y, size


def expert_wgrad(x, dy, ends, base=None, in_major=False):
    """dw in float64 and the sums of magnitudes."""
    x, dy = x.cpu().double(), dy.cpu().double()
    a, b = (x, dy) if in_major else (dy, x)
    dw = torch.stack([a[i:j].t() @ b[i:j] for i, j in spans(ends.cpu(), len(x))])
    size = torch.stack([a[i:j].t().abs() @ b[i:j].abs() for i, j in spans(ends.cpu(), len(x))])
    if base is not None:
        dw, size = dw + base.cpu().double(), size + base.cpu().double().abs()
    return dw, size


def route(ids, experts):
    """ends, slot and place as lists become int32 tensors."""
    flat = ids.cpu().reshape(-1).tolist()
    order = [s for e in range(experts) for s in range(len(flat)) if flat[s] == e] if len(flat) * experts < 1 << 16 else None
    if order is None:
        keys = [(f if 0 <= f < experts else experts, s) for s, f in enumerate(flat)]
        order = [s for k, s in sorted(keys) if k < experts]
    lost = [s for s, f in enumerate(flat) if not 0 <= f < experts]
    place = [-1] * len(flat)
    for p, s in enumerate(order):
        place[s] = p
    counts = [0] * experts
    for s in order:
        counts[flat[s]] += 1
    ends = torch.tensor(counts).cumsum(0)
    slot = order + [-1 - s for s in lost]
    as_int = dict(dtype=torch.int32)
    return ends.to(torch.int32), torch.tensor(slot, **as_int), torch.tensor(place, **as_int).view(ids.shape)


def gather(x, slot, choices):
    x = x.cpu()
    out = torch.zeros(len(slot), x.shape[1], dtype=x.dtype)
    for p, s in enumerate(slot.tolist()):
        if 0 <= s < len(slot):
            out[p] = x[s // choices]
    return out


def combine(y, place, weights=None):
    """out in float64 and the sums of magnitudes."""
    y, place = y.cpu().double(), place.cpu()
    out = torch.zeros(len(place), y.shape[1], dtype=torch.float64)
    size = torch.zeros_like(out)
    for t, row in enumerate(place.tolist()):
        for j, p in enumerate(row):
            if 0 <= p < len(y):
                w = 1.0 if weights is None else float(weights[t, j])
                out[t] += w * y[p]
                size[t] += abs(w) * y[p].abs()
    return out, size


def combine_backward(dout, y, slot, choices, weights=None):
    """dy, dweights in float64, and the dot products' sums of magnitudes."""
    dout, y = dout.cpu().double(), y.cpu().double()
    dy = torch.zeros_like(y)
    dweights = torch.zeros(len(dout), choices, dtype=torch.float64)
    size = torch.zeros_like(dweights)
    for p, s in enumerate(slot.tolist()):
        if 0 <= s < len(slot):
            t, j = divmod(s, choices)
            dy[p] = (1.0 if weights is None else float(weights[t, j])) * dout[t]
            dweights[t, j] = dout[t] @ y[p]
            size[t, j] = dout[t].abs() @ y[p].abs()
    return dy, dweights, size
