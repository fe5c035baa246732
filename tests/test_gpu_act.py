"""GPU tests of the activation operators against their 64-bit oracle.

Checkpoints are compared byte for byte.  Elsewhere the tolerances count roundings, with
u = 2^-24 for an fp32 operation and eps/2 of the output's type for the last one; sums of n
terms are off by at most about n u times the sum of magnitudes (2 u per step on the matrix
cores, whose rounding direction is not assumed)."""

import pytest
import torch

from oracle import act_oracle as AO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF16: 2.0 ** -133, FP16: 2.0 ** -24, FP32: 2.0 ** -149}  # smallest step of each type


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_mixed_buffer_amd as Z
    Z.lib()
    return Z


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _matrix(rows, cols, dtype, seed, pad=0, sigma=1.0, fill=float("nan")):
    """A matrix on the GPU inside wider rows whose other columns hold NaN."""
    wide = torch.full((rows, cols + pad), fill, dtype=dtype)
    wide[:, :cols] = (sigma * torch.randn(rows, cols, generator=_gen(seed))).to(dtype)
    return wide.cuda()[:, :cols]


def _last_rounding(v, dtype):
    return v.abs() * (torch.finfo(dtype).eps / 2) + TINY[dtype] / 2


def _assert_within(got, want, bound, what):
    got = got.detach().cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    ok = ~torch.isnan(want)
    over = ((got - want).abs() - bound)[ok]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} past its bound"


def _same_bytes(act, codes, scales, what):
    assert torch.equal(act.scales.cpu(), scales), f"{what}: scales"
    bad = (act.codes.cpu() != codes).nonzero()
    assert len(bad) == 0, f"{what}: {len(bad)} codes differ, first at {bad[0].tolist()}"


# ------------------------------------------------------------------------------ checkpoints

SHAPES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 64), (7, 100), (1, 4096), (33, 1003), (129, 256), (2, 14336)]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_pack_is_exact(Z, rows, cols, dtype, code):
    for pad in (0, 3, 8):
        x = _matrix(rows, cols, dtype, rows * 7 + cols, pad)
        act = Z.Act8.empty(rows, cols, code)
        act.codes.fill_(77)
        act.scales.fill_(77)
        Z.act_pack(x, act)
        _same_bytes(act, *AO.quantise(x, code), f"{rows}x{cols}+{pad} {dtype} {code}")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_pack_at_the_edges(Z, dtype, code):
    """Zeros of both signs, the range's ends, values next to every border between two scales,
    halves between codes, subnormal numbers, infinities and NaN."""
    top = torch.finfo(dtype).max
    rows = [[0.0] * 5 + [-0.0], [top, -top, 1.0], [TINY[dtype]], [-TINY[dtype] * 5, TINY[dtype] * 3],
            [torch.finfo(dtype).tiny, -1.5 * torch.finfo(dtype).tiny], [float("inf"), 1.0], [-float("inf")],
            [float("nan"), 2.0], [1.0, -float("inf"), float("nan")]]
    for q in (448.0, 127.0, 1.0):
        for k in (-12, -1, 0, 3, 7):
            v = torch.tensor(q * 2.0 ** k).to(dtype)
            for near in (v, torch.nextafter(v, torch.tensor(float("inf"), dtype=dtype)),
                         torch.nextafter(v, torch.tensor(0.0, dtype=dtype))):
                f = float(near)
                rows.append([f, -f, f / 448 * 17, f / 448 * 18.5, f / 127 * 0.5, f / 127 * 1.5, -f / 127 * 2.5])
    x = torch.zeros(len(rows), 96, dtype=dtype)
    for i, r in enumerate(rows):
        x[i, 32:32 + len(r)] = torch.tensor(r, dtype=torch.float64).to(dtype)
        x[i, 0] = 1.0   # neighbours of the group
        x[i, 64] = -3.0
    act = Z.Act8.of(x.cuda(), code)
    _same_bytes(act, *AO.quantise(x, code), f"edges {dtype} {code}")


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_unpack_is_exact(Z, code, dtype):
    """All 256 codes under all 256 scale bytes, into every type."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    act = Z.Act8(codes.cuda(), scales.cuda(), 250, code)
    wide = torch.full((256, 261), 5.0, dtype=dtype, device="cuda")
    Z.act_unpack(act, wide[:, 3:253])
    want = AO.rounded(AO.values(codes, scales, 250, code), dtype)
    got = wide.cpu()[:, 3:253]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    bad = ((got != want) & ~torch.isnan(want)).nonzero()
    assert len(bad) == 0, (len(bad), bad[0].tolist(), float(got[tuple(bad[0])]), float(want[tuple(bad[0])]))
    assert bool((wide.cpu()[:, :3] == 5).all()) and bool((wide.cpu()[:, 253:] == 5).all())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_round_trip(Z, rows, cols, code):
    x = _matrix(rows, cols, BF16, 11, 5)
    act = Z.Act8.of(x, code)
    back = act.unpack(BF16)
    want = AO.values(*AO.quantise(x, code), cols, code)
    assert torch.equal(back.cpu().double(), want)
    step = 2.0 ** -4 if code == "e4m3" else 0.0
    half = x.cpu().double().abs() * step + x.cpu().double().abs().max() / (2 ** 9 if code == "e4m3" else 127)
    assert bool(((back.cpu().double() - x.cpu().double()).abs() <= half).all())


def test_pack_of_no_rows(Z):
    act = Z.Act8.of(torch.empty(0, 40, dtype=BF16, device="cuda"))
    assert act.unpack().shape == (0, 40)


# ------------------------------------------------------------------------------ norm

NORMS = [(1, 1), (1, 64), (5, 33), (17, 128), (3, 129), (9, 512), (2, 1003), (4, 2048), (3, 4095), (2, 4096),
         (700, 96), (2, 5000), (3, 8192), (2, 9001), (1, 16384)]


def _check_codes_near(act, y, tol, code, what):
    """act holds y to the code's rounding, where y itself is only known to +-tol (relative)."""
    cols = y.shape[1]
    groups = act.scales.shape[1]
    wide = torch.zeros(y.shape[0], groups * 32, dtype=torch.float64)
    wide[:, :cols] = y
    amax = wide.view(-1, groups, 32).abs().amax(2)
    lo, hi = AO.scale_bytes(amax * (1 - tol), code), AO.scale_bytes(amax * (1 + tol), code)
    b = act.scales.cpu().long()
    assert bool(((b >= lo) & (b <= hi)).all()), f"{what}: scales"
    s = (2.0 ** (b.double() - 127))[:, :, None].expand(-1, -1, 32).reshape(y.shape[0], -1)[:, :cols]
    got = AO.values(act.codes, act.scales, cols, code)
    half = s / 2 if code == "int8" else torch.maximum(y.abs() * (1 + tol) * 2.0 ** -4, s * 2.0 ** -10)
    over = (got - y).abs() - half - y.abs() * tol
    assert float(over.max()) <= 0, f"{what}: {float(over.max()):.3e}"
    assert bool((act.codes.cpu()[:, cols:] == 0).all())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,cols", NORMS)
def test_norm(Z, rows, cols, dtype, code):
    for pad, with_residual in ((0, True), (5, False), (8, True)):
        x = _matrix(rows, cols, dtype, 21, pad)
        r = _matrix(rows, cols, dtype, 22, pad + 1, 3.0) if with_residual else None
        w = _matrix(1, cols, dtype, 23)[0]
        wide_y = torch.full((rows, cols + 7), 9.0, dtype=dtype, device="cuda")
        y, h = wide_y[:, 2:cols + 2], torch.empty(rows, cols, dtype=dtype, device="cuda")
        y8, h8 = Z.Act8.empty(rows, cols, code), Z.Act8.empty(rows, cols, code)
        rstd = torch.empty(rows, device="cuda")
        Z.rmsnorm(x, w, 1e-5, residual=r, h=h, y=y, y8=y8, h8=h8, rstd=rstd)
        what = f"{rows}x{cols}+{pad} {dtype} {code}"
        h64, rstd64, y64 = AO.norm(x, w, 1e-5, r)
        assert torch.equal(h.cpu(), h64), what
        # the sum in fp64 is exact to 2^-53 per term: what is left is rstd's own rounding
        _assert_within(rstd, rstd64, rstd64 * (U * 1.001), what + " rstd")
        tol = 3.1 * U  # rstd, and two products
        _assert_within(y, y64, _last_rounding(y64, dtype) * (1 + tol) + y64.abs() * tol, what + " y")
        assert bool((wide_y[:, :2] == 9).all()) and bool((wide_y[:, cols + 2:] == 9).all())
        _same_bytes(h8, *AO.quantise(h64, code), what + " h8")
        _check_codes_near(y8, y64, 4 * U, code, what + " y8")


@pytest.mark.parametrize("cols", [96, 128, 300, 512])
def test_norm_of_many_rows(Z, cols):
    """Short rows by the ten thousands, where a lane takes two of them: bit for bit what the same
    rows give a thousand at a time."""
    rows = 33001
    x = torch.randn(rows, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(5)).to(BF16)
    w = _matrix(1, cols, BF16, 6)[0]

    def outputs(n):
        return (torch.empty(n, cols, dtype=BF16, device="cuda"), torch.empty(n, device="cuda"), Z.Act8.empty(n, cols),
                Z.Act8.empty(n, cols, "int8"))

    y, rstd, y8, h8 = outputs(rows)
    Z.rmsnorm(x, w, residual=x, y=y, rstd=rstd, y8=y8, h8=h8)
    for a in range(0, rows, 1000):
        b = min(a + 1000, rows)
        y1, rstd1, y81, h81 = outputs(b - a)
        Z.rmsnorm(x[a:b], w, residual=x[a:b], y=y1, rstd=rstd1, y8=y81, h8=h81)
        assert torch.equal(y[a:b], y1) and torch.equal(rstd[a:b], rstd1)
        for whole, part in ((y8, y81), (h8, h81)):
            assert torch.equal(whole.codes[a:b], part.codes) and torch.equal(whole.scales[a:b], part.scales)


@pytest.mark.parametrize("cols", [2600, 4096])
def test_norm_of_many_wide_rows(Z, cols):
    """Wide rows with a residual by the thousands, where more threads share a row: the rows' sums of
    squares are the same to fp64, so every output is that of the same rows a few at a time."""
    rows = 8200
    x = torch.randn(rows, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(7)).to(BF16)
    r, w = x.flip(0).contiguous(), _matrix(1, cols, BF16, 8)[0]
    y, h, h8 = torch.empty_like(x), torch.empty_like(x), Z.Act8.empty(rows, cols)
    rstd = torch.empty(rows, device="cuda")
    Z.rmsnorm(x, w, residual=r, h=h, y=y, h8=h8, rstd=rstd)
    for a in (0, 4000, rows - 100):
        b = a + 100
        y1, h1, h81, rstd1 = torch.empty_like(x[a:b]), torch.empty_like(x[a:b]), Z.Act8.empty(100, cols), rstd[a:b].clone()
        Z.rmsnorm(x[a:b], w, residual=r[a:b], h=h1, y=y1, h8=h81, rstd=rstd1)
        assert torch.equal(h[a:b], h1) and torch.equal(h8.codes[a:b], h81.codes) and torch.equal(h8.scales[a:b], h81.scales)
        # the order of the fp64 sum differs: rstd may land on the neighbouring fp32 number, and y on
        # the neighbouring bf16 number where it lay between two
        assert float(((rstd[a:b] - rstd1) / rstd1).abs().max()) <= 2 * U
        assert float(((y[a:b].float() - y1.float()).abs() / y1.float().abs().clamp_min(1e-30)).max()) <= 2.0 ** -7


def test_norm_single_outputs(Z):
    """Each output alone, and h in place of x or of the residual."""
    x, r = _matrix(6, 300, BF16, 31), _matrix(6, 300, BF16, 32)
    w = _matrix(1, 300, BF16, 33)[0]
    full = {"h": torch.empty_like(x), "y": torch.empty_like(x), "y8": Z.Act8.empty(6, 300), "h8": Z.Act8.empty(6, 300),
            "rstd": torch.empty(6, device="cuda")}
    Z.rmsnorm(x, w, residual=r, **full)
    for k in full:
        one = Z.Act8.empty(6, 300) if k in ("y8", "h8") else torch.empty_like(full[k])
        Z.rmsnorm(x, w, residual=r, **{k: one})
        if isinstance(one, Z.Act8):
            _same_bytes(one, full[k].codes.cpu(), full[k].scales.cpu(), k)
        else:
            assert torch.equal(one, full[k]), k
    for place in ("x", "residual"):
        a, b = x.clone(), r.clone()
        y = torch.empty_like(x)
        Z.rmsnorm(a, w, residual=b, h=a if place == "x" else b, y=y)
        assert torch.equal(a if place == "x" else b, full["h"]) and torch.equal(y, full["y"])
    with pytest.raises(ValueError):
        Z.rmsnorm(x, w)
    with pytest.raises(ValueError):
        Z.rmsnorm(x, w, h=full["y"], y=full["y"])


def test_norm_of_extreme_rows(Z):
    """Rows of zeros, of the largest and smallest numbers, with an infinity, with a NaN: the
    others do not notice; the sum of squares does not overflow."""
    x = torch.randn(6, 256, generator=_gen(41)).to(BF16)
    x[0] = 0
    x[1] = torch.finfo(BF16).max
    x[2] = 2.0 ** -133
    x[3, 7] = float("inf")
    x[4, 200] = float("nan")
    w = torch.ones(256, dtype=BF16)
    y, rstd, y8 = torch.empty(6, 256, dtype=BF16, device="cuda"), torch.empty(6, device="cuda"), Z.Act8.empty(6, 256)
    Z.rmsnorm(x.cuda(), w.cuda(), 1e-6, y=y, rstd=rstd, y8=y8)
    h64, rstd64, y64 = AO.norm(x, w, 1e-6)
    y, rstd = y.cpu().double(), rstd.cpu().double()
    assert bool((y[0] == 0).all()) and abs(float(rstd[0]) - 1000) < 1e-3
    assert bool((y[1] == 1).all())  # the largest numbers come out as ones
    assert float(rstd[2]) == pytest.approx(1000, rel=1e-6)
    assert float(rstd[3]) == 0 and bool(torch.isnan(y[3, 7])) and bool((y[3, :7] == 0).all())
    assert bool(torch.isnan(y[4]).all())
    assert bool((y8.scales[3].cpu() == torch.tensor([255] + [0] * 7)).all()) and bool((y8.scales[4] == 255).all())
    assert bool(((y[5] - y64[5]).abs() <= _last_rounding(y64[5], BF16) * 1.01 + y64[5].abs() * 4 * U).all())


# ------------------------------------------------------------------------------ norm, backward

def _backward_bounds(dy, h, w, rstd, dh, dx64):
    """dx = rstd (g - xh mean(g xh)) + dh: the products round two to five times, the mean is a
    sum of cols terms of which a lane adds at most 16 in sequence before six to ten tree steps."""
    dy, h, w, r = dy.cpu().double(), h.cpu().double(), w.cpu().double(), rstd.cpu().double()[:, None]
    xh, g = h * r, dy * w
    mean_abs = (g * xh).abs().mean(1, keepdim=True)
    return U * (4 * (r * g).abs() + 45 * (r * xh).abs() * mean_abs + 2 * dx64.abs()
                + (2 * dh.cpu().double().abs() if dh is not None else 0)) + TINY[FP32]


@pytest.mark.parametrize("saved", ["16", "e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,cols", NORMS + [(0, 64), (40, 4096), (1500, 257), (2100, 128)])
def test_norm_backward(Z, rows, cols, dtype, saved):
    for i, (pad, with_dh, grad, with_base) in enumerate(((0, True, FP32, False), (3, False, dtype, True))):
        h = _matrix(rows, cols, dtype, 51, pad)
        dy = _matrix(rows, cols, dtype, 52, pad + 1, 0.01)
        dh = _matrix(rows, cols, dtype, 53, pad + 2, 0.01) if with_dh else None
        w = _matrix(1, cols, dtype, 54)[0]
        rstd = AO.norm(h, w, 1e-5)[1].float().cuda()
        kept, seen = h, h
        if saved != "16":
            kept = Z.Act8.of(h, saved)
            seen = AO.values(kept.codes, kept.scales, cols, saved)
        buffer = torch.full((cols + 9,), 3.0, dtype=grad, device="cuda")  # a gradient buffer's slice, unaligned
        dweight = buffer[5:cols + 5]
        base = dweight if with_base else None
        old = dweight.clone() if with_base else None
        wide = torch.full((rows, cols + 4), 9.0, dtype=dtype, device="cuda")
        dx = wide[:, 1:cols + 1]
        Z.rmsnorm_backward(dy, kept, w, rstd, dx, dh=dh, dweight=dweight, base=base)
        what = f"{rows}x{cols}+{pad} {dtype} {saved}"
        dx64, dw64 = AO.norm_backward(dy, seen, w, rstd, dh, old)
        bound = _backward_bounds(dy, seen, w, rstd, dh, dx64)
        _assert_within(dx, dx64, bound + _last_rounding(dx64, dtype) * 1.01, what + " dx")
        mags = (dy.cpu().double() * seen.cpu().double() * rstd.cpu().double()[:, None]).abs().sum(0)
        terms = min(rows, 64) + 24  # in one lane's sum, and in the folds
        _assert_within(dweight, dw64, U * terms * mags + _last_rounding(dw64, grad) * 1.01, what + " dweight")
        assert bool((buffer[:5] == 3).all()) and bool((buffer[cols + 5:] == 3).all())
        assert bool((wide[:, 0] == 9).all()) and bool((wide[:, cols + 1:] == 9).all())
        again = torch.empty_like(dx)
        Z.rmsnorm_backward(dy, kept, w, rstd, again, dh=dh)  # without the weight's gradient
        assert torch.equal(again, dx)


def test_norm_backward_in_place(Z):
    h, dy, dh = (_matrix(50, 700, BF16, s) for s in (61, 62, 63))
    w = _matrix(1, 700, BF16, 64)[0]
    rstd = AO.norm(h, w, 1e-5)[1].float().cuda()
    want = torch.empty_like(dy)
    Z.rmsnorm_backward(dy, h, w, rstd, want, dh=dh)
    for place in (dy, dh):
        keep = place.clone()
        Z.rmsnorm_backward(dy, h, w, rstd, place, dh=dh)
        assert torch.equal(place, want)
        place.copy_(keep)


def test_norm_backward_marks_a_lost_group(Z):
    """A checkpoint group that stands for NaN makes its row's dx and its 32 columns of the
    weight's gradient NaN, so the step's overflow check sees it; the rest is unharmed."""
    x = _matrix(8, 100, BF16, 71)
    x[3, 70] = float("inf")
    act = Z.Act8.of(x)
    dy, w = _matrix(8, 100, BF16, 72), _matrix(1, 100, BF16, 73)[0]
    rstd = torch.ones(8, device="cuda")
    dx, dweight = torch.empty_like(dy), torch.empty(100, device="cuda")
    Z.rmsnorm_backward(dy, act, w, rstd, dx, dweight=dweight)
    bad = torch.isnan(dx).cpu()
    assert bool(bad[3].all()) and not bool(bad[[0, 1, 2, 4, 5, 6, 7]].any())
    assert torch.isnan(dweight).cpu().nonzero().flatten().tolist() == list(range(64, 96))


# ------------------------------------------------------------------------------ weight gradient

WGRADS = [(1, 1, 1), (1, 64, 48), (2, 33, 5), (31, 32, 128), (32, 40, 129), (33, 256, 64), (100, 130, 127),
          (128, 64, 256), (257, 96, 300), (1000, 513, 70), (4097, 64, 40), (0, 33, 17)]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,cols,outs", WGRADS)
def test_wgrad_of_whole_numbers(Z, rows, cols, outs, dtype, code):
    """Small whole numbers: every sum is exact, so one wrong, missing or doubled term shows."""
    x = torch.randint(-3, 4, (rows, cols), generator=_gen(81)).to(dtype)
    dy = torch.full((rows, outs + 3), float("nan"), dtype=dtype)
    dy[:, :outs] = torch.randint(-2, 3, (rows, outs), generator=_gen(82)).to(dtype)
    dy = dy.cuda()[:, :outs]
    act = Z.Act8.of(x.cuda(), code)
    want = AO.wgrad(dy, x)
    for in_major in (False, True):
        ref = want.t() if in_major else want
        wide = torch.full((ref.shape[0], ref.shape[1] + 5), 7.0, device="cuda")
        dw = wide[:, 2:ref.shape[1] + 2]
        Z.act_wgrad(act, dy, dw, in_major=in_major)
        bad = (dw.cpu().double() != ref).nonzero()
        assert len(bad) == 0, (in_major, len(bad), bad[:3].tolist())
        Z.act_wgrad(act, dy, dw, base=dw, in_major=in_major)
        assert torch.equal(dw.cpu().double(), 2 * ref)
        assert bool((wide[:, :2] == 7).all()) and bool((wide[:, ref.shape[1] + 2:] == 7).all())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("grad", ["own", FP32])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,cols,outs", WGRADS + [(700, 1003, 517), (2048, 512, 640)])
def test_wgrad(Z, rows, cols, outs, dtype, grad, code):
    grad = dtype if grad == "own" else grad
    x = _matrix(rows, cols, dtype, 91)
    dy = _matrix(rows, outs, dtype, 92, 1, 0.01)
    act = Z.Act8.of(x, code)
    seen = AO.values(act.codes, act.scales, cols, code)
    base = _matrix(outs, cols, grad, 93)
    mags = dy.cpu().double().abs().t() @ seen.abs()
    for b in (None, base):
        dw = torch.empty(outs, cols, dtype=grad, device="cuda")
        Z.act_wgrad(act, dy, dw, base=b)
        want = AO.wgrad(dy, seen, b)
        bound = 2 * U * (rows + 8) * mags + 2 * U * want.abs() + _last_rounding(want, grad) * 1.01
        _assert_within(dw, want, bound, f"{rows}x{cols}->{outs} {dtype} {grad} {code}")
        twice = torch.empty_like(dw)
        Z.act_wgrad(act, dy, twice, base=b)
        assert torch.equal(dw, twice)
        turned = torch.empty(cols, outs, dtype=grad, device="cuda")
        Z.act_wgrad(act, dy, turned, base=b.t().contiguous() if b is not None else None, in_major=True)
        assert torch.equal(turned.t(), dw)


# (tokens, cols, outs) that take: one round of large tiles; large tiles with edges; large
# tiles of which the last are split; the same of small tiles; small tiles alone; splits of few
LARGE = [(512, 4096, 4096), (1100, 2051, 4099), (1030, 4097, 4100), (4097, 2051, 4099), (640, 4096, 5000), (9000, 512, 700)]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,cols,outs", LARGE)
def test_wgrad_of_large_weights(Z, rows, cols, outs, dtype, code):
    """Whole numbers again, at sizes that take every tile and split, in both orientations, with
    NaN behind each row of dy; the reference is an exact product in 64 bits on the GPU."""
    g = torch.Generator("cuda").manual_seed(121)
    x = torch.randint(-3, 4, (rows, cols), device="cuda", generator=g).to(dtype)
    wide = torch.full((rows, outs + 9), float("nan"), dtype=dtype, device="cuda")
    wide[:, :outs] = torch.randint(-2, 3, (rows, outs), device="cuda", generator=g).to(dtype)
    dy = wide[:, :outs]
    act = Z.Act8.of(x, code)
    want = dy.double().t().contiguous() @ x.double()
    for in_major in (False, True):
        ref = want.t() if in_major else want
        dw = torch.full(ref.shape, 7.0, device="cuda")
        Z.act_wgrad(act, dy, dw, in_major=in_major)
        assert torch.equal(dw.double(), ref)
        half = torch.zeros(ref.shape, dtype=dtype, device="cuda")
        Z.act_wgrad(act, dy, half, base=half, in_major=in_major)
        assert torch.equal(half, ref.to(dtype))


def test_offsets_past_32_bits(Z):
    """Matrices of more than 2^32 elements (and bytes of codes): their last rows, packed, read
    back, normalised, differentiated and multiplied like the same rows by themselves."""
    rows, cols = 270000, 16000
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(131))
    tail = slice(rows - 300, rows)
    act = Z.Act8.of(x)
    part = Z.Act8.of(x[tail])
    assert torch.equal(act.codes[tail], part.codes) and torch.equal(act.scales[tail], part.scales)
    back = act.unpack()
    assert torch.equal(back[tail], part.unpack())
    del back
    w = _matrix(1, cols, BF16, 132)[0]
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    Z.rmsnorm(x, w, y=y, rstd=rstd)
    y1, rstd1 = torch.empty(300, cols, dtype=BF16, device="cuda"), torch.empty(300, device="cuda")
    Z.rmsnorm(x[tail], w, y=y1, rstd=rstd1)
    assert torch.equal(y[tail], y1) and torch.equal(rstd[tail], rstd1)
    Z.rmsnorm_backward(x, act, w, rstd, y)
    Z.rmsnorm_backward(x[tail], part, w, rstd1, y1)
    assert torch.equal(y[tail], y1)
    # the weight gradient: whole numbers in the last rows, zeros before them
    del y, act
    x.zero_()
    x[tail] = torch.randint(-2, 3, (300, cols), device="cuda").to(BF16)
    other = torch.zeros(rows, 64, dtype=BF16, device="cuda")
    other[tail] = torch.randint(-2, 3, (300, 64), device="cuda").to(BF16)
    for wide, narrow in ((x, other), (other, x)):
        dw = torch.empty(narrow.shape[1], wide.shape[1], device="cuda")
        Z.act_wgrad(Z.Act8.of(wide), narrow, dw)
        assert torch.equal(dw.double(), narrow[tail].double().t().contiguous() @ wide[tail].double())


def test_checkpoint_storage_may_move(Z):
    """A checkpoint whose storage was freed and allocated again is found where it is now; freed
    storage is refused."""
    x = _matrix(40, 64, BF16, 141)
    act = Z.Act8.of(x)
    keep = act.codes.clone()
    storage = act.codes.untyped_storage()
    n = storage.nbytes()
    storage.resize_(0)
    with pytest.raises(ValueError):
        Z.act_unpack(act, x)
    block = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")  # takes the place that was free
    storage.resize_(n)
    act.codes.copy_(keep)
    assert torch.equal(act.unpack().cpu().double(), AO.values(*AO.quantise(x, "e4m3"), 64, "e4m3"))
    del block


def test_wgrad_in_a_gradient_buffer(Z):
    """dw as an unaligned slice of a flat bf16 buffer, added to what is there; the neighbours
    keep their bits."""
    x, dy = _matrix(300, 200, BF16, 101), _matrix(300, 150, BF16, 102)
    flat = torch.randn(150 * 200 + 40, generator=_gen(103)).to(BF16).cuda()
    before = flat.clone()
    dw = flat[13:13 + 150 * 200].view(150, 200)
    act = Z.Act8.of(x)
    Z.act_wgrad(act, dy, dw, base=dw)
    alone = torch.empty(150, 200, device="cuda")
    Z.act_wgrad(act, dy, alone)
    want = (before[13:13 + 150 * 200].view(150, 200).float() + alone).to(BF16)
    assert torch.equal(dw, want)
    assert torch.equal(flat[:13], before[:13]) and torch.equal(flat[13 + 150 * 200:], before[13 + 150 * 200:])


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_wgrad_of_lost_groups(Z, dtype, code):
    """A group that stands for NaN reaches its 32 columns of dw and no others."""
    x = _matrix(100, 128, dtype, 111)
    x[77, 40] = float("nan")
    dw = torch.empty(64, 128, device="cuda")
    Z.act_wgrad(Z.Act8.of(x, code), _matrix(100, 64, dtype, 112), dw)
    bad = torch.isnan(dw).cpu()
    assert bool(bad[:, 32:64].all()) and not bool(bad[:, :32].any()) and not bool(bad[:, 64:].any())


def test_wgrad_at_the_ends_of_fp16(Z):
    """Values that a code rounds past fp16's largest number take part as that number."""
    x = torch.full((4, 32), 65504.0, dtype=FP16)
    x[1] = 2.0 ** -24
    for code in ("e4m3", "int8"):
        act = Z.Act8.of(x.cuda(), code)
        seen = AO.rounded(AO.values(act.codes, act.scales, 32, code), FP16)
        dy = torch.eye(4, dtype=FP16).cuda()
        dw = torch.empty(4, 32, device="cuda")
        Z.act_wgrad(act, dy, dw)
        assert torch.equal(dw.cpu(), seen.float())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_wgrad_takes_every_code(Z, dtype, code):
    """All codes under the scale bytes whose values are normal numbers of the type (or past its
    end), one row at a time through an identity: dw is the checkpoint's values in dy's type."""
    lo, hi = (20, 240) if dtype == BF16 else (127, 255)
    table = [c for c in range(256) if code == "int8" or c & 127 != 127]
    codes = torch.tensor(table + [0] * (256 - len(table)), dtype=torch.uint8).repeat(hi - lo, 1)
    scales = torch.arange(lo, hi).to(torch.uint8)[:, None].repeat(1, 8)
    act = Z.Act8(codes.cuda(), scales.cuda(), 256, code)
    dy = torch.eye(hi - lo, dtype=dtype, device="cuda")
    dw = torch.empty(hi - lo, 256, device="cuda")
    Z.act_wgrad(act, dy, dw)
    want = AO.rounded(AO.values(codes, scales, 256, code), dtype).float()
    assert torch.equal(dw.cpu(), want)


# ------------------------------------------------------------------------------ refusals with GPU tensors

def test_tensor_calls_refuse(Z):
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.zeros(64, dtype=BF16, device="cuda")
    r = torch.zeros(4, device="cuda")
    act = Z.Act8.empty(4, 64)
    bad = [lambda: Z.act_pack(x.t(), act), lambda: Z.act_pack(x[:, ::2], Z.Act8.empty(4, 32)),
           lambda: Z.act_pack(x[:3], act), lambda: Z.act_pack(x.double(), act), lambda: Z.act_pack(x[0], act),
           lambda: Z.act_pack(x[:1].expand(4, 64), act), lambda: Z.act_unpack(act, x[:, :63]),
           lambda: Z.act_pack(x, Z.Act8.empty(4, 64, device="cpu")),
           lambda: Z.rmsnorm(x, w.float(), y=x), lambda: Z.rmsnorm(x.float(), w.float(), y=x.float()),
           lambda: Z.rmsnorm(x, w, y=x.half()), lambda: Z.rmsnorm(x, w[:60], y=x), lambda: Z.rmsnorm(x, w, 0.0, y=x),
           lambda: Z.rmsnorm(x, w, residual=x[:2], y=x), lambda: Z.rmsnorm(x, w, rstd=r.double()),
           lambda: Z.rmsnorm(x, w, rstd=r[:3]), lambda: Z.rmsnorm(x, w, y8=Z.Act8.empty(4, 65)),
           lambda: Z.rmsnorm(torch.zeros(2, 16385, dtype=BF16, device="cuda"),
                             torch.zeros(16385, dtype=BF16, device="cuda"), rstd=r[:2]),
           lambda: Z.rmsnorm_backward(x, x.half(), w, r, x), lambda: Z.rmsnorm_backward(x, x, w, r, x, base=r),
           lambda: Z.rmsnorm_backward(x, x, w, r, x, dweight=w, base=w.float()),
           lambda: Z.rmsnorm_backward(x, x, w, r, x, dweight=w, workspace=torch.zeros(2, device="cuda")),
           lambda: Z.act_wgrad(act, x, torch.zeros(64, 63, device="cuda")),
           lambda: Z.act_wgrad(act, x[:3], torch.zeros(64, 64, device="cuda")),
           lambda: Z.act_wgrad(act, x, torch.zeros(64, 64, device="cuda", dtype=FP16)),
           lambda: Z.act_wgrad(act, x, torch.zeros(64, 64, device="cuda"), base=torch.zeros(64, 80, device="cuda")[:, :64]),
           lambda: Z.act_wgrad(act, x, torch.zeros(64, 64)),
           lambda: Z.norm(x[:, :0], w[:0]), lambda: Z.linear(x[:, :0], torch.zeros(8, 0, dtype=BF16, device="cuda")),
           lambda: Z.linear(x, torch.zeros(8, 64, dtype=BF16, device="cuda"), code="fp8"),
           lambda: Z.norm(x, w, save="fp8"), lambda: Z.norm(x, w, residual=x[:3]),
           lambda: Z.norm(x, w, grad_into=r), lambda: Z.linear(x, torch.zeros(8, 63, dtype=BF16, device="cuda")),
           lambda: Z.linear(x, torch.zeros(8, 64, dtype=BF16, device="cuda"), x8=Z.Act8.empty(3, 64))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")
