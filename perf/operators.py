"""Measured calls of the activation operators: 8-bit activation checkpoints, the root-mean-square
norm that writes them, its backward pass, and the weight gradient taken from them.

`run` computes one call in plain torch operations (`own` false) or through the framework's entry
points (`own` true) on the same inputs.  Matrices are rows (tokens) x cols (features).  A checkpoint
holds one byte per element, in rows padded with zeros to whole groups of 32, and one power-of-two
scale (a biased exponent byte) per group: the smallest that brings the group's largest magnitude
within the code's range.
"""

import math

import torch

own = False

GROUP = 32
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MAX_CODE = {"e4m3": 448.0, "int8": 127.0}


def listed():
    return [
        # one attention input of the two-layer toy list (context 128, hidden 64): latency alone
        {"name": "checkpoint_tiny", "op": "checkpoint", "rows": 128, "cols": 64, "pad": 0, "dtype": "fp16",
         "code": "int8"},
        # a ragged batch with odd sizes, a view into wider rows (no 16-byte alignment anywhere)
        {"name": "checkpoint_ragged", "op": "checkpoint", "rows": 4097, "cols": 1003, "pad": 2, "dtype": "bf16",
         "code": "int8"},
        # the widest activation of a Llama-3-8B-shaped layer, input of its down projection
        {"name": "checkpoint_ffn", "op": "checkpoint", "rows": 16384, "cols": 14336, "pad": 0, "dtype": "bf16",
         "code": "e4m3"},
        # one token through a layer's input norm
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "pad": 0, "dtype": "bf16", "residual": True,
         "keep_h8": False},
        # odd sizes with padded rows
        {"name": "norm_ragged", "op": "norm", "rows": 777, "cols": 1003, "pad": 5, "dtype": "fp16", "residual": True,
         "keep_h8": True},
        # a layer's input norm over a long batch: residual addition, output in 16 and 8 bits, 8-bit checkpoint
        {"name": "norm_block", "op": "norm", "rows": 16384, "cols": 4096, "pad": 0, "dtype": "bf16",
         "residual": True, "keep_h8": True},
        # per-head query norm of a Qwen3-style layer: many short rows
        {"name": "norm_heads", "op": "norm", "rows": 131072, "cols": 128, "pad": 0, "dtype": "bf16",
         "residual": False, "keep_h8": False},
        # the toy list's norm backward from a 16-bit input
        {"name": "norm_backward_tiny", "op": "norm_backward", "rows": 128, "cols": 64, "pad": 0, "dtype": "fp16",
         "saved": "16", "grad": "fp16"},
        # the layer norm's backward from its 8-bit checkpoint, weight gradient added to an fp32 buffer
        {"name": "norm_backward_block", "op": "norm_backward", "rows": 16384, "cols": 4096, "pad": 0,
         "dtype": "bf16", "saved": "e4m3", "grad": "fp32"},
        # the toy list's first feed-forward weight
        {"name": "wgrad_tiny", "op": "wgrad", "rows": 128, "cols": 64, "outs": 256, "dtype": "fp16", "code": "int8",
         "grad": "fp16", "base": False},
        # odd sizes, a long batch and a small weight: the sum over tokens has to be split
        {"name": "wgrad_ragged", "op": "wgrad", "rows": 16381, "cols": 1003, "outs": 517, "dtype": "bf16",
         "code": "int8", "grad": "fp32", "base": False},
        # gate/up projection of a Llama-3-8B-shaped layer, added to the flat bf16 gradient buffer
        {"name": "wgrad_ffn", "op": "wgrad", "rows": 8192, "cols": 4096, "outs": 14336, "dtype": "bf16",
         "code": "e4m3", "grad": "bf16", "base": True},
    ]


def _log_size(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["checkpoint", "norm", "norm_backward", "wgrad"])
    rows = _log_size(rng, 1, 16384)
    cols = _log_size(rng, 33, 14336)
    if rng.random() < 0.5:  # whole groups about half of the time, as model widths are
        cols = max(GROUP, cols // GROUP * GROUP)
    case = {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "fp16"])}
    if op == "wgrad":
        case["outs"] = _log_size(rng, 33, 14336)
        while case["rows"] * case["cols"] * case["outs"] > 8192 * 4096 * 14336:
            case["rows"] = (case["rows"] + 1) // 2
        case.update(code=rng.choice(["e4m3", "int8"]), grad=rng.choice([case["dtype"], "fp32"]),
                    base=rng.random() < 0.5)
        return case
    case["pad"] = rng.choice([0, 0, 8, rng.randint(1, 63)])
    if op == "checkpoint":
        case["code"] = rng.choice(["e4m3", "int8"])
    elif op == "norm":
        case.update(residual=rng.random() < 0.7, keep_h8=rng.random() < 0.5)
    else:
        case.update(saved=rng.choice(["16", "e4m3", "int8"]), grad=rng.choice([case["dtype"], "fp32"]))
    return case


# ------------------------------------------------------------------------------------ inputs

def _activation(g, rows, cols, pad, dtype):
    """Values of unit size with a few features many times larger, as a model's activations are,
    in the first `cols` columns of wider rows."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(cols + pad, generator=g, device="cuda"))
    return x.to(dtype)[:, :cols]


def _gradient(g, rows, cols, pad, dtype):
    # loss-scaled for fp16, as mixed-precision training passes them on
    sigma = 0.05 if dtype == torch.float16 else 1e-3
    return (sigma * torch.randn(rows, cols + pad, generator=g, device="cuda")).to(dtype)[:, :cols]


def _out(rows, cols, dtype):
    return torch.empty(rows, cols, dtype=dtype, device="cuda")


def _checkpoint_buffers(rows, cols):
    groups = -(-cols // GROUP)
    return (torch.empty(rows, groups * GROUP, dtype=torch.uint8, device="cuda"),
            torch.empty(rows, groups, dtype=torch.uint8, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, rows, cols, dtype = case["op"], case["rows"], case["cols"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "checkpoint":
        s["x"] = _activation(g, rows, cols, case["pad"], dtype)
        s["codes"], s["scales"] = _checkpoint_buffers(rows, cols)
        s["back"] = _out(rows, cols, dtype)
    elif op == "norm":
        s["x"] = _activation(g, rows, cols, case["pad"], dtype)
        s["residual"] = _activation(g, rows, cols, case["pad"], dtype) if case["residual"] else None
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dtype)
        s["h"] = _out(rows, cols, dtype) if case["residual"] else None
        s["y"] = _out(rows, cols, dtype)
        s["rstd"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        s["y_codes"], s["y_scales"] = _checkpoint_buffers(rows, cols)
        if case["keep_h8"]:
            s["h_codes"], s["h_scales"] = _checkpoint_buffers(rows, cols)
    elif op == "norm_backward":
        h = _activation(g, rows, cols, case["pad"], dtype)
        s["dy"] = _gradient(g, rows, cols, case["pad"], dtype)
        s["dh"] = _gradient(g, rows, cols, case["pad"], dtype)
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dtype)
        s["rstd"] = torch.rsqrt(h.float().square().mean(1) + EPS)
        if case["saved"] == "16":
            s["h"] = h
        else:
            s["codes"], s["scales"] = _quantise(h.float(), case["saved"])
        grad = DTYPES[case["grad"]]
        s["base"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(grad)
        s["dx"] = _out(rows, cols, dtype)
        s["dweight"] = torch.empty(cols, dtype=grad, device="cuda")
    else:
        outs, grad = case["outs"], DTYPES[case["grad"]]
        s["codes"], s["scales"] = _quantise(_activation(g, rows, cols, 0, dtype).float(), case["code"])
        s["dy"] = _gradient(g, rows, outs, 0, dtype)
        s["base"] = (0.01 * torch.randn(outs, cols, generator=g, device="cuda")).to(grad) if case["base"] else None
        s["dw"] = _out(outs, cols, grad)
    return s


# ------------------------------------------------------------------------------------ plain form

def _quantise(x, code):
    """Codes (bytes) and scale exponents (bytes) of a matrix in 32 bits."""
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    wide = torch.zeros(rows, groups * GROUP, dtype=torch.float32, device=x.device)
    wide[:, :cols] = x
    wide = wide.view(rows, groups, GROUP)
    mantissa, exponent = torch.frexp(wide.abs().amax(2))
    bits = 9 if code == "e4m3" else 7
    over = mantissa > MAX_CODE[code] / 2 ** bits
    byte = (exponent - bits + over + 127).clamp(0, 254)
    byte = torch.where(mantissa == 0, torch.zeros_like(byte), byte)
    scaled = torch.ldexp(wide, (127 - byte)[:, :, None])
    codes = scaled.to(torch.float8_e4m3fn) if code == "e4m3" else torch.round(scaled).to(torch.int8)
    return codes.view(rows, groups * GROUP).view(torch.uint8), byte.to(torch.uint8)


def _values(codes, scales, cols, code):
    """The matrix that a checkpoint stands for, in 32 bits."""
    v = codes.view(torch.float8_e4m3fn if code == "e4m3" else torch.int8).float()
    v = torch.ldexp(v.view(len(v), -1, GROUP), (scales.int() - 127)[:, :, None])
    return v.view(len(v), -1)[:, :cols]


def _seen(codes, scales, code):
    """A checkpoint's two arrays as the numbers that they hold."""
    return codes.view(torch.float8_e4m3fn if code == "e4m3" else torch.int8), scales.view(torch.float8_e8m0fnu)


def _plain_checkpoint(s, c):
    codes, scales = _quantise(s["x"].float(), c["code"])
    return _seen(codes, scales, c["code"]) + (_values(codes, scales, c["cols"], c["code"]).to(s["x"].dtype),)


def _plain_norm(s, c):
    dtype = s["x"].dtype
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dtype)
    v = h.float()
    rstd = 1 / torch.sqrt((v * v).sum(1) / c["cols"] + EPS)
    y = v * rstd[:, None] * s["weight"].float()
    out = [y.to(dtype), rstd, *_seen(*_quantise(y, "e4m3"), "e4m3")]
    if s["h"] is not None:
        out.append(h)
    if c["keep_h8"]:
        out += _seen(*_quantise(v, "e4m3"), "e4m3")
    return out


def _plain_norm_backward(s, c):
    h = s["h"].float() if c["saved"] == "16" else _values(s["codes"], s["scales"], c["cols"], c["saved"])
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = h * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - xhat * ((g * xhat).sum(1, keepdim=True) / c["cols"])) + s["dh"].float()
    dweight = (dy * xhat).sum(0) + s["base"].float()
    return dx.to(s["dy"].dtype), dweight.to(s["base"].dtype)


def _plain_wgrad(s, c):
    dw = s["dy"].float().t() @ _values(s["codes"], s["scales"], c["cols"], c["code"])
    if s["base"] is not None:
        dw = dw + s["base"].float()
    return dw.to(s["dw"].dtype)


# ------------------------------------------------------------------------------------ the framework's calls

def _own_checkpoint(Z, s, c):
    act = Z.Act8(s["codes"], s["scales"], c["cols"], c["code"])
    Z.act_pack(s["x"], act)
    Z.act_unpack(act, s["back"])
    return _seen(s["codes"], s["scales"], c["code"]) + (s["back"],)


def _own_norm(Z, s, c):
    y8 = Z.Act8(s["y_codes"], s["y_scales"], c["cols"], "e4m3")
    h8 = Z.Act8(s["h_codes"], s["h_scales"], c["cols"], "e4m3") if c["keep_h8"] else None
    Z.rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], h=s["h"], y=s["y"], y8=y8, h8=h8, rstd=s["rstd"])
    out = [s["y"], s["rstd"], *_seen(s["y_codes"], s["y_scales"], "e4m3")]
    if s["h"] is not None:
        out.append(s["h"])
    if c["keep_h8"]:
        out += _seen(s["h_codes"], s["h_scales"], "e4m3")
    return out


def _own_norm_backward(Z, s, c):
    saved = s["h"] if c["saved"] == "16" else Z.Act8(s["codes"], s["scales"], c["cols"], c["saved"])
    Z.rmsnorm_backward(s["dy"], saved, s["weight"], s["rstd"], s["dx"], dh=s["dh"], dweight=s["dweight"],
                       base=s["base"])
    return s["dx"], s["dweight"]


def _own_wgrad(Z, s, c):
    Z.act_wgrad(Z.Act8(s["codes"], s["scales"], c["cols"], c["code"]), s["dy"], s["dw"], base=s["base"])
    return s["dw"]


def run(state):
    case = state["case"]
    if own:
        import zero_sharded_mixed_buffer_amd as Z
        call = {"checkpoint": _own_checkpoint, "norm": _own_norm, "norm_backward": _own_norm_backward,
                "wgrad": _own_wgrad}[case["op"]]
        return call(Z, state, case)
    plain = {"checkpoint": _plain_checkpoint, "norm": _plain_norm, "norm_backward": _plain_norm_backward,
             "wgrad": _plain_wgrad}[case["op"]]
    return plain(state, case)


def work(case):
    op, rows, cols = case["op"], case["rows"], case["cols"]
    n = rows * cols
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    eight = rows * (-(-cols // GROUP)) * (GROUP + 1)
    if op == "checkpoint":  # read the source; write codes, scales and the matrix read back
        return {"bytes": 4 * n + eight, "flops": 4 * n}
    if op == "norm":
        tensors = 2 + 2 * case["residual"]  # x and y; the residual and h
        return {"bytes": 2 * n * tensors + eight * (1 + case["keep_h8"]) + 4 * rows + 2 * cols, "flops": 8 * n}
    if op == "norm_backward":
        saved = 2 * n if case["saved"] == "16" else eight
        return {"bytes": 6 * n + saved + 4 * rows + 2 * cols + 2 * cols * size[case["grad"]], "flops": 12 * n}
    outs = case["outs"]
    passes = 2 if case["base"] else 1
    return {"bytes": eight + 2 * rows * outs + passes * outs * cols * size[case["grad"]], "flops": 2 * n * outs}


# ------------------------------------------------------------------------------------ 64 bits

def _exact_codes(x, code):
    """The codes' numbers and the scales of a matrix in 64 bits: the smallest power of two that
    brings each group's largest magnitude within the code's range, found by trying."""
    rows, cols = x.shape
    short = -cols % GROUP
    groups = torch.cat([x, x.new_zeros(rows, short)], 1).reshape(rows, -1, GROUP)
    top = groups.abs().max(2, keepdim=True).values
    k = torch.floor(torch.log2(top.clamp_min(1e-300) / MAX_CODE[code])) - 1
    for _ in range(3):
        k = k + (top > MAX_CODE[code] * torch.exp2(k))
    k = k.clamp(-127, 127)
    scale = torch.exp2(k)
    v = groups / scale
    if code == "int8":
        v = torch.round(v)
    else:
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(1e-300))).clamp_min(-6) - 3)
        v = torch.round(v / step) * step
    return v.reshape(rows, -1), scale.reshape(rows, -1)


def _exact_back(v, scale, cols):
    return (v.reshape(len(v), -1, GROUP) * scale[:, :, None]).reshape(len(v), -1)[:, :cols]


def _number(codes, code):
    return codes.to(torch.int8) if code == "int8" else codes


def _stored(codes, scales, cols, code):
    """The matrix that stored bytes stand for, in 64 bits, decoded from their bit fields."""
    b = codes.long()
    if code == "int8":
        v = torch.where(b >= 128, b - 256, b).double()
    else:
        field, low = (b >> 3) & 15, (b & 7).double()
        v = torch.where(field == 0, low / 512, (1 + low / 8) * torch.exp2(field.double() - 7))
        v = torch.where(b >= 128, -v, v)
    return _exact_back(v, torch.exp2(scales.double() - 127), cols)


def exact(case, seed):
    s = prepare(case, seed)
    op, cols = case["op"], case["cols"]
    if op == "checkpoint":
        v, scale = _exact_codes(s["x"].double(), case["code"])
        return _number(v, case["code"]), scale, _exact_back(v, scale, cols)
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        rstd = (h.pow(2).mean(1) + EPS).pow(-0.5)
        y = h * s["weight"].double() * rstd.unsqueeze(1)
        out = [y, rstd, *_exact_codes(y, "e4m3")]
        if s["h"] is not None:
            out.append(h)
        if case["keep_h8"]:
            out += _exact_codes(h, "e4m3")
        return out
    if op == "norm_backward":
        h = s["h"].double() if case["saved"] == "16" else _stored(s["codes"], s["scales"], cols, case["saved"])
        dy, w, r = s["dy"].double(), s["weight"].double(), s["rstd"].double().unsqueeze(1)
        along = (dy * w * h).mean(1, keepdim=True)
        dx = r * (dy * w) - r.pow(3) * h * along + s["dh"].double()
        return dx, s["base"].double() + (r * dy * h).sum(0)
    dw = torch.mm(s["dy"].double().t().contiguous(), _stored(s["codes"], s["scales"], cols, case["code"]))
    return dw if s["base"] is None else dw + s["base"].double()
