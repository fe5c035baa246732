"""Plain 64-bit CPU forms of the activation operators, from their definitions (include/zs_act.h):
8-bit codes with power-of-two scales, the root-mean-square norm and its backward, and the weight
gradient.  Used by tests only."""

from __future__ import annotations

import torch

GROUP = 32
QMAX = {"e4m3": 448.0, "int8": 127.0}


def _e4m3_table():
    """Value of each of the 256 bytes: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    out = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        if e == 15 and m == 7:
            v = float("nan")
        else:
            v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append(-v if b & 128 else v)
    return torch.tensor(out, dtype=torch.float64)


E4M3 = _e4m3_table()


def scale_bytes(amax, code):
    """Scale byte of each group from its largest magnitude (float64): the smallest k >= -127 with
    amax <= qmax * 2^k, as k + 127; 255 where amax is not finite."""
    out = torch.zeros(amax.shape, dtype=torch.int64)
    ks = 2.0 ** torch.arange(-127, 128, dtype=torch.float64) * QMAX[code]
    fin = torch.isfinite(amax)
    out[fin] = torch.searchsorted(ks, amax[fin], right=False)
    out[~fin] = 255
    return out


def quantise(x, code):
    """Codes and scales (uint8) of a matrix."""
    x = x.detach().cpu().double()
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    wide = torch.zeros(rows, groups * GROUP, dtype=torch.float64)
    wide[:, :cols] = x
    g = wide.view(rows, groups, GROUP)
    mag = g.abs()
    amax = torch.where(torch.isfinite(g).all(2), mag.amax(2), torch.tensor(float("inf"), dtype=torch.float64)) \
        if g.numel() else mag.new_zeros(rows, groups)
    b = scale_bytes(amax, code)
    bad = (b == 255)[:, :, None].expand_as(g)
    v = torch.where(bad, torch.zeros_like(g), g) / 2.0 ** (b.clamp_max(254) - 127).double()[:, :, None]
    if code == "int8":
        codes = torch.round(v).to(torch.int64) & 255
    else:
        pos = E4M3[:127]
        m = v.abs().clamp_max(448.0)
        hi = torch.searchsorted(pos, m.contiguous(), right=False).clamp_max(126)
        lo = (hi - 1).clamp_min(0)
        dlo, dhi = m - pos[lo], pos[hi] - m
        near = torch.where(dlo < dhi, lo, torch.where(dhi < dlo, hi, torch.where(lo % 2 == 0, lo, hi)))
        near = torch.where(pos[hi] == m, hi, near)
        codes = near + 128 * torch.signbit(v).long()
        codes = torch.where(bad, torch.zeros_like(codes), codes)
    return codes.reshape(rows, groups * GROUP).to(torch.uint8), b.to(torch.uint8)


def values(codes, scales, cols, code):
    """The matrix that a checkpoint stands for (float64)."""
    c = codes.cpu().long()
    v = E4M3[c] if code == "e4m3" else torch.where(c > 127, c - 256, c).double()
    s = 2.0 ** (scales.cpu().double() - 127)
    s = torch.where(scales.cpu() == 255, torch.full_like(s, float("nan")), s)
    rows, groups = scales.shape
    return (v.view(rows, groups, GROUP) * s[:, :, None]).reshape(rows, groups * GROUP)[:, :cols]


def rounded(v, dtype):
    """Round float64 values that fp32 holds exactly to dtype; past fp16's range to its ends."""
    f = v.float()
    if dtype == torch.float16:
        f = torch.where(f.abs() > 65504.0, torch.sign(f) * 65504.0, f)
    return f.to(dtype)


def norm(x, weight, eps, residual=None):
    """Returns (h, rstd, y): h in x's dtype, the others in float64."""
    h = x.cpu().double()
    if residual is not None:
        h = h + residual.cpu().double()
    h = h.to(x.dtype)
    hd = h.double()
    rstd = (hd.square().mean(1) + eps) ** -0.5
    return h, rstd, hd * rstd[:, None] * weight.cpu().double()


def norm_backward(dy, h, weight, rstd, dh=None, base=None):
    """Returns (dx, dweight) in float64; h and rstd as they are taken, in any precision."""
    dy, h, w, r = dy.cpu().double(), h.cpu().double(), weight.cpu().double(), rstd.cpu().double()[:, None]
    xh = h * r
    g = dy * w
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.cpu().double()
    dw = (dy * xh).sum(0)
    return dx, dw if base is None else dw + base.cpu().double()


def wgrad(dy, x, base=None):
    dw = dy.cpu().double().t() @ x.cpu().double()
    return dw if base is None else dw + base.cpu().double()
