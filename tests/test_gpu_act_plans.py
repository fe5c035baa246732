"""GPU tests of the activation operators at sizes that reach every launch plan: four chunks to a
thread, two rows to a lane, a wave or 512 threads to a row, and the backward passes whose workgroups
go several rounds and leave partial sums.

Tolerances as in test_gpu_act.py: u = 2^-24 for an fp32 operation, eps/2 of the output's type for the
last one, sums by the number of their sequential steps."""

import pytest
import torch

import test_gpu_act as G
from oracle import act_oracle as AO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_mixed_buffer_amd as Z
    Z.lib()
    return Z


def _matrix(rows, cols, dtype, seed, pad=0, sigma=1.0):
    """A matrix inside wider rows whose other columns hold NaN, made on the GPU."""
    wide = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    g = torch.Generator("cuda").manual_seed(seed)
    wide[:, :cols] = (sigma * torch.randn(rows, cols, device="cuda", generator=g)).to(dtype)
    return wide[:, :cols]


def _assert_within(got, want, bound, what):
    over = (got.double() - want).abs() - bound
    assert float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} past its bound"


# ------------------------------------------------------------------------------ checkpoints

@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("cols,pad", [(1003, 5), (1003, 0), (1024, 8), (1024, 0)])
def test_large_checkpoints(Z, cols, pad, dtype, code):
    """More than 2^21 chunks of eight, with gaps between the rows, ragged rows, and neither: packed and
    read back like the same rows a thousand at a time, which are checked against the oracle."""
    rows, step = 17000, 1000
    x = _matrix(rows, cols, dtype, 3, pad)
    act = Z.Act8.empty(rows, cols, code)
    act.codes.fill_(77)
    act.scales.fill_(77)
    Z.act_pack(x, act)
    wide = torch.full((rows, cols + pad), 5.0, dtype=dtype, device="cuda")
    Z.act_unpack(act, wide[:, :cols])
    assert bool((wide[:, cols:] == 5).all())
    for a in range(0, rows, step):
        part = Z.Act8.of(x[a:a + step], code)
        assert torch.equal(act.codes[a:a + step], part.codes) and torch.equal(act.scales[a:a + step], part.scales)
        assert torch.equal(wide[a:a + step, :cols], part.unpack(dtype))
    for rs in (slice(0, 37), slice(rows - 41, rows)):
        codes, scales = AO.quantise(x[rs], code)
        assert torch.equal(act.codes[rs].cpu(), codes) and torch.equal(act.scales[rs].cpu(), scales)
        assert torch.equal(wide[rs, :cols].cpu(), AO.rounded(AO.values(codes, scales, cols, code), dtype))


# ------------------------------------------------------------------------------ norm

# rows and columns that take: a wave to a row, two chunks to a lane; two rows to a lane; 512 threads to a row
# (with a residual); 256 threads of two chunks; 512 of two; 1024 of two
NORMS = [(4097, 1003), (5000, 544), (33001, 100), (33001, 512), (8201, 2600), (8201, 3201), (8201, 4096), (4100, 2049),
         (300, 8191), (300, 16383)]


@pytest.mark.parametrize("with_residual", [True, False])
@pytest.mark.parametrize("dtype,code", [(BF16, "e4m3"), (FP16, "int8"), (FP16, "e4m3")])
@pytest.mark.parametrize("rows,cols", NORMS)
def test_norm(Z, rows, cols, dtype, code, with_residual):
    x = _matrix(rows, cols, dtype, 21, 3)
    r = _matrix(rows, cols, dtype, 22, 6, 3.0) if with_residual else None
    w = _matrix(1, cols, dtype, 23)[0]
    wide_y = torch.full((rows, cols + 7), 9.0, dtype=dtype, device="cuda")
    y, h = wide_y[:, 2:cols + 2], torch.full((rows, cols), 9.0, dtype=dtype, device="cuda")
    y8, h8 = Z.Act8.empty(rows, cols, code), Z.Act8.empty(rows, cols, code)
    for a in (y8, h8):
        a.codes.fill_(77)
        a.scales.fill_(77)
    rstd = torch.empty(rows, device="cuda")
    Z.rmsnorm(x, w, 1e-5, residual=r, h=h, y=y, y8=y8, h8=h8, rstd=rstd)
    h64 = x.double() if r is None else (x.double() + r.double()).to(dtype).double()
    assert torch.equal(h, h64.to(dtype))
    rstd64 = (h64.square().mean(1) + 1e-5) ** -0.5
    _assert_within(rstd, rstd64, rstd64 * (U * 1.001), "rstd")
    y64 = h64 * rstd64[:, None] * w.double()
    tol = 3.1 * U  # rstd, and two products
    half = y64.abs() * (torch.finfo(dtype).eps / 2) + G.TINY[dtype] / 2
    _assert_within(y, y64, half * (1 + tol) + y64.abs() * tol, "y")
    assert bool((wide_y[:, :2] == 9).all()) and bool((wide_y[:, cols + 2:] == 9).all())
    whole = Z.Act8.of(h, code)
    assert torch.equal(h8.codes, whole.codes) and torch.equal(h8.scales, whole.scales)
    for rs in (slice(0, 50), slice(rows - 50, rows)):
        part = Z.Act8(y8.codes[rs].contiguous(), y8.scales[rs].contiguous(), cols, code)
        G._check_codes_near(part, y64[rs].cpu(), 4 * U, code, "y8")
    # every row's y8, within a code's step of y
    _assert_within(y8.unpack(FP32), y64, _code_step(y8, cols, code, y64), "y8")
    assert bool((y8.codes[:, cols:] == 0).all())


def _code_step(act, cols, code, v):
    """Half a step of the code at v (a value known to 4 u), under the scales that act holds."""
    s = (2.0 ** (act.scales.double() - 127))[:, :, None].expand(-1, -1, 32).reshape(len(v), -1)[:, :cols]
    half = s / 2 if code == "int8" else torch.maximum(v.abs() * (1 + 4 * U) * 2.0 ** -4, s * 2.0 ** -10)
    return half + v.abs() * 4 * U


# ------------------------------------------------------------------------------ norm, backward

# rows and columns, rows to a workgroup's round and most workgroups of each plan: all of them go
# several rounds with a last one that some workgroups, or some rows of one, miss
BACKWARDS = [(40003, 128, 32, 512), (20011, 96, 32, 512), (9001, 300, 8, 512), (9005, 1003, 8, 512), (1101, 2048, 2, 512),
             (1201, 1500, 2, 512), (2777, 1025, 2, 512), (5000, 4096, 1, 512), (1300, 2600, 1, 512), (700, 5000, 1, 512),
             (1100, 8192, 1, 512), (601, 16384, 1, 256), (777, 9001, 1, 256)]


@pytest.mark.parametrize("saved", ["16", "e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,cols,per,most", BACKWARDS)
def test_norm_backward(Z, rows, cols, per, most, dtype, saved):
    h = _matrix(rows, cols, dtype, 51, 3)
    dy = _matrix(rows, cols, dtype, 52, 4, 0.01)
    dh = _matrix(rows, cols, dtype, 53, 5, 0.01)
    w = _matrix(1, cols, dtype, 54)[0]
    rstd = ((h.double().square().mean(1) + 1e-5) ** -0.5).float()
    kept, seen = h, h.double()
    if saved != "16":
        kept = Z.Act8.of(h, saved)
        seen = kept.unpack(FP32).double()
    r = rstd.double()[:, None]
    xh, g = seen * r, dy.double() * w.double()
    mean, mean_abs = (g * xh).mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    dx64 = r * (g - xh * mean) + dh.double()
    # a lane adds at most 16 products in sequence before ten tree steps and the waves' sixteen sums
    bound = U * (4 * (r * g).abs() + 45 * (r * xh).abs() * mean_abs + 2 * dx64.abs() + 2 * dh.double().abs()) + 2.0 ** -149
    bound += (dx64.abs() * (torch.finfo(dtype).eps / 2) + G.TINY[dtype] / 2) * 1.01
    products = dy.double() * xh
    mags, sums = products.abs().sum(0), products.sum(0)
    # a lane's sum over its workgroup's rounds, the sum over the rows of a round, and per term xh's
    # roundings (two at most, and its product with dy); workgroups are added in 64 bits
    steps = -(-rows // per)
    assert steps > most
    terms = -(-steps // most) + per + 4
    for grad in (FP32, dtype):
        buffer = torch.full((cols + 9,), 3.0, dtype=grad, device="cuda")
        dweight = buffer[5:cols + 5]
        base = (0.1 * torch.randn(cols, device="cuda", generator=torch.Generator("cuda").manual_seed(55))).to(grad)
        dweight.copy_(base)
        scratch = torch.full((Z.zs_rmsnorm_workspace(rows, cols) // 4,), float("nan"), device="cuda")
        wide = torch.full((rows, cols + 4), 9.0, dtype=dtype, device="cuda")
        dx = wide[:, 1:cols + 1]
        Z.rmsnorm_backward(dy, kept, w, rstd, dx, dh=dh, dweight=dweight, base=dweight, workspace=scratch)
        _assert_within(dx, dx64, bound, "dx")
        want = sums + base.double()
        last = want.abs() * (torch.finfo(grad).eps / 2) + G.TINY[grad] / 2
        _assert_within(dweight, want, U * terms * mags + last * 1.01, "dweight")
        assert bool((buffer[:5] == 3).all()) and bool((buffer[cols + 5:] == 3).all())
        assert bool((wide[:, 0] == 9).all()) and bool((wide[:, cols + 1:] == 9).all())
        again = torch.empty_like(dweight)
        Z.rmsnorm_backward(dy, kept, w, rstd, dy.clone(), dh=dh, dweight=again, base=base)
        assert torch.equal(again, dweight)


# ------------------------------------------------------------------------------ empty batches

@pytest.mark.parametrize("save", ["e4m3", None])
def test_no_rows_under_autograd(Z, save):
    """A batch of no tokens through norm and linear: empty outputs, and gradients of zero."""
    x = torch.zeros(2, 0, 64, dtype=BF16, device="cuda", requires_grad=True)
    r = torch.zeros_like(x, requires_grad=True)
    nw = torch.ones(64, dtype=BF16, device="cuda", requires_grad=True)
    w = torch.ones(24, 64, dtype=BF16, device="cuda", requires_grad=True)
    into = torch.full((24, 64), 2.0, device="cuda")
    out = Z.norm(x, nw, residual=r, save=save, y8="e4m3")
    y = Z.linear(out.y, w, x8=out.y8)
    z = Z.linear(out.y, w, x8=out.y8, grad_into=into)
    assert y.shape == z.shape == (2, 0, 24)
    (y.sum() + z.sum()).backward()
    assert x.grad.shape == r.grad.shape == x.shape
    assert not bool(nw.grad.any()) and not bool(w.grad.any()) and bool((into == 2).all())


# ------------------------------------------------------------------------------ weight gradient

@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_wgrad_rounds_each_value_once(Z, dtype, code):
    """Every code under every scale byte, one row at a time through an identity: a checkpoint's value
    takes part rounded once into dy's type, to nearest even, fp16's subnormal numbers included and
    past fp16's range its largest number.  Below bf16's normal numbers a value may count as zero; scale
    bytes whose codes pass bf16's range are left out (448 * 2^(246 - 127) < 2^128), as an infinity
    times the identity's zeros is NaN."""
    n = 247 if dtype == BF16 else 255
    table = [c for c in range(256) if code == "int8" or c & 127 != 127]
    codes = torch.tensor(table + [0] * (256 - len(table)), dtype=torch.uint8).repeat(n, 1)
    scales = torch.arange(n).to(torch.uint8)[:, None].repeat(1, 8)
    act = Z.Act8(codes.cuda(), scales.cuda(), 256, code)
    dw = torch.empty(n, 256, device="cuda")
    Z.act_wgrad(act, torch.eye(n, dtype=dtype, device="cuda"), dw)
    values = AO.values(codes, scales, 256, code)
    got, want = dw.cpu().double(), AO.rounded(values, dtype).double()
    if dtype == BF16:
        small = values.abs() < 2.0 ** -126
        assert bool((got[small].abs() <= 2.0 ** -126).all())
        got, want = got[~small], want[~small]
    bad = (got != want).nonzero()
    assert len(bad) == 0, (len(bad), bad[0].tolist(), float(got[tuple(bad[0])]), float(want[tuple(bad[0])]))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_wgrad_of_an_fp16_norms_checkpoint(Z, code):
    """fp16 y8, taken from y before its rounding: values that are not on fp16's grid are rounded to it,
    by at most half of fp16's smallest step, and the weight gradient is that of the rounded values."""
    rows, cols, outs = 200, 96, 40
    # small enough that scales go below fp16's smallest step (e4m3's least code is 2^-9 of one)
    x, w = _matrix(rows, cols, FP16, 61), _matrix(1, cols, FP16, 62, sigma=2.0 ** (-9 if code == "e4m3" else -20))[0]
    y8 = Z.Act8.empty(rows, cols, code)
    Z.rmsnorm(x, w, y8=y8)
    dy = _matrix(rows, outs, FP16, 63, sigma=0.1)
    dw = torch.empty(outs, cols, device="cuda")
    Z.act_wgrad(y8, dy, dw)
    values = y8.unpack(FP32).double()
    seen = values.half().double()
    assert float((values - seen).abs().max()) <= 2.0 ** -25
    assert not torch.equal(values, seen)
    want, mags = dy.double().t().contiguous() @ seen, dy.double().abs().t().contiguous() @ seen.abs()
    # sums of 200 terms in fp32, two u a step on the matrix cores
    _assert_within(dw, want, 2 * U * (rows + 8) * mags, "dw")
