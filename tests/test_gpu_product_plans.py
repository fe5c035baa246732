"""Tests of every launch plan of the products: which kernel and tile a call takes goes by its sizes and
alignments, and the sizes here are chosen for the plan that they name.

`plan` states the launch rules a second time, with the thresholds read from the source, so that a
threshold that moves shows on the CPU.  The GPU tests compare all outputs with products in 64 bits; the
tolerances are those of tests/test_gpu_product.py."""

import os
import re

import pytest
import torch

from oracle import act_oracle as AO
from oracle import product_oracle as PO

U = 2.0 ** -24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF16: 2.0 ** -133, FP16: 2.0 ** -24, FP32: 2.0 ** -149}


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_mixed_buffer_amd as Z
    Z.lib()
    return Z


# ------------------------------------------------------------------------------ the launch rules

def _threshold(name):
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(here, "zero_sharded_mixed_buffer_amd", "csrc", "zs_product.hip")) as f:
        return int(re.search(rf"constexpr int64_t {name} = (\d+);", f.read()).group(1))


FEW, LARGE = _threshold("kFewUnits"), _threshold("kLargeUnits")


def _tiles(n, side):
    return -(-n // side)


def _few(m, n, groups, extra):
    """Rows of a, and sixteens of b's rows, to a unit of the kernel for few rows."""
    mf = 1 if m <= 16 * groups else 2
    wide = (_tiles(m, 16 * mf) + extra) * _tiles(n, 32) >= 512
    return f"few {mf} {2 if wide else 1}"


def plan8(m, n):
    if _tiles(m, 32) * _tiles(n, 32) <= FEW:
        return _few(m, n, 1, 0)
    return "large" if _tiles(m, 256) * _tiles(n, 256) >= LARGE else "small"


def plan(m, n, groups, a_by_k, b_by_k, sums, words):
    """words: bases and strides at whole words of 4 bytes."""
    extra = 0 if sums else groups
    if not a_by_k and not b_by_k and (_tiles(m, 32) + extra) * _tiles(n, 32) <= FEW:
        return _few(m, n, groups, extra)
    if not words or (a_by_k and m % 8) or (b_by_k and n % 8):
        return "registers"
    units = groups * _tiles(m, 256) * _tiles(n, 256) if sums else (_tiles(m, 256) + groups) * _tiles(n, 256)
    per_group = m if sums else m // groups
    return "large" if per_group >= 192 and n >= 192 and units >= LARGE else "small"


# ------------------------------------------------------------------------------ the cases

# rows, k, width, plan
PRODUCTS8 = [
    (1, 4500, 600, "few 1 1"), (16, 3460, 16384, "few 1 2"), (64, 4500, 256, "few 2 1"), (512, 2100, 1024, "few 2 2"),
    # one, two, three stages, and what a stage's last groups leave over
    (700, 100, 1000, "small"), (700, 129, 1000, "small"), (700, 384, 1000, "small"),
    # past two segments of scales (sixteen stages each), the last stage whole, or with one to four groups
    (700, 4224, 1000, "small"), (700, 4240, 1000, "small"), (641, 4310, 897, "small"), (700, 4351, 1000, "small"),
    (3000, 100, 4100, "large"), (3000, 256, 4100, "large"), (3000, 300, 4100, "large"),
    (3000, 4224, 4100, "large"), (2817, 4240, 4353, "large"), (3000, 4351, 4100, "large"), (3001, 2049, 4096, "large"),
]

# what the strides and bases are multiples of, in elements of 2 bytes
ALIGNMENTS = ("rows", "words", "odd")
RAGGED = [300, 17, 0, 0, 129, 1]
UNEVEN = [1500, 0, 612]

# in_major, rows of each expert, cols, outs, alignment, plan
EXPERTS = [
    (False, [9] * 16, 1700, 700, "rows", "few 1 2"), (False, [5] * 5, 1700, 96, "odd", "few 1 1"),
    (False, [100, 0, 30], 1130, 200, "words", "few 2 1"), (False, [375, 0, 0, 0], 1130, 1024, "odd", "few 2 2"),
    (False, RAGGED, 64, 808, "rows", "small"), (False, RAGGED, 200, 808, "words", "small"), (False, RAGGED, 1000, 803, "words", "small"),
    (False, RAGGED, 64, 808, "odd", "registers"), (False, RAGGED, 203, 801, "odd", "registers"), (False, RAGGED, 1000, 808, "odd", "registers"),
    (False, UNEVEN, 72, 4096, "rows", "large"), (False, UNEVEN, 200, 4096, "words", "large"), (False, UNEVEN, 1000, 4091, "words", "large"),
    (False, UNEVEN, 333, 4096, "odd", "registers"),
    (True, RAGGED, 64, 136, "rows", "small"), (True, RAGGED, 203, 136, "words", "small"), (True, RAGGED, 1000, 264, "words", "small"),
    (True, RAGGED, 203, 135, "rows", "registers"), (True, RAGGED, 1000, 264, "odd", "registers"), (True, RAGGED, 64, 261, "odd", "registers"),
    (True, UNEVEN, 72, 4096, "rows", "large"), (True, UNEVEN, 200, 4088, "words", "large"), (True, UNEVEN, 1000, 4096, "words", "large"),
    (True, UNEVEN, 333, 4090, "words", "registers"),
]

# in_major, rows of each expert, cols, outs, alignment, plan
GRADIENTS = [
    (False, RAGGED, 64, 136, "words", "small"), (False, RAGGED, 264, 392, "words", "small"), (True, RAGGED, 264, 136, "words", "small"),
    (False, RAGGED, 264, 392, "odd", "registers"), (True, RAGGED, 261, 393, "rows", "registers"), (True, RAGGED, 264, 136, "odd", "registers"),
    (False, [700, 0, 1, 333], 1536, 1800, "rows", "large"), (False, [700, 0, 1, 333], 1536, 1800, "words", "large"),
    (True, [64, 128, 65, 500], 1800, 1352, "words", "large"), (False, [700, 0, 1, 333], 1536, 1800, "odd", "registers"),
]


def _expert_plan(in_major, sizes, cols, outs, alignment):
    return plan(sum(sizes) + 9, outs, len(sizes), False, in_major, False, alignment != "odd")


def _gradient_plan(in_major, sizes, cols, outs, alignment):
    m, n = (cols, outs) if in_major else (outs, cols)
    return plan(m, n, len(sizes), True, True, True, alignment != "odd")


def test_the_cases_take_their_plans():
    for rows, k, width, want in PRODUCTS8:
        assert plan8(rows, width) == want, (rows, k, width)
    for *case, want in EXPERTS:
        assert _expert_plan(*case) == want, case
    for *case, want in GRADIENTS:
        assert _gradient_plan(*case) == want, case
    few = {f"few {m} {n}" for m in (1, 2) for n in (1, 2)}
    assert {c[-1] for c in PRODUCTS8} == few | {"small", "large"}
    for in_major in (False, True):
        want = {"small", "large", "registers"}
        assert {c[-1] for c in EXPERTS if c[0] == in_major} == (want if in_major else want | few)
        assert {c[-1] for c in GRADIENTS if c[0] == in_major} == want


# ------------------------------------------------------------------------------ helpers

def _randn(shape, seed, sigma=1.0):
    return sigma * torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def _stride(cols, alignment):
    """A row stride behind whose columns something else lies."""
    if alignment == "rows":
        return (cols + 15) // 8 * 8
    return cols + 2 + (-cols % 4) if alignment == "words" else cols + 1 + cols % 2


OFFSET = {"rows": 8, "words": 2, "odd": 3}
GAP = {"rows": 8, "words": 2, "odd": 1}


def _placed(values, dtype, alignment, fill=float("nan")):
    """A matrix, or matrices, on the GPU at such an alignment, `fill` around it."""
    stride, offset = _stride(values.shape[-1], alignment), OFFSET[alignment]
    apart = values.shape[-2] * stride + GAP[alignment]
    n = values.shape[0] if values.dim() == 3 else 1
    flat = torch.full((offset + n * apart + stride,), fill, dtype=dtype)
    strides = (apart, stride, 1)[3 - values.dim():]
    if alignment != "rows":
        assert all(s % 4 == 2 if alignment == "words" else s % 2 == 1 for s in strides[-2:-1]) or values.shape[-1] == 1
    flat.as_strided(values.shape, strides, offset).copy_(values.to(dtype))
    flat = flat.cuda()
    return flat, flat.as_strided(values.shape, strides, offset)


def _untouched(flat, view, fill):
    """Whether what lies around a placed matrix still holds `fill`."""
    flat = flat.clone()
    flat.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(fill)
    return bool((flat == fill).all())


def _assert_within(got, want, err, what):
    bound = err + (want.abs() + err) * (torch.finfo(got.dtype).eps / 2) + TINY[got.dtype] / 2
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    over = torch.nan_to_num((got - want).abs() - bound)
    assert float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} past its bound, {int((over > 0).sum())} of {over.numel()}"


# ------------------------------------------------------------------------------ products in 8 bits

def _cut(x, w):
    """What the 8-bit matrix instructions may cut off: 7 * 2^-13 times the largest product of every eight
    elements, summed."""
    pad = -x.shape[1] % 8
    x = torch.nn.functional.pad(x.abs(), (0, pad)).view(len(x), -1, 8)
    w = torch.nn.functional.pad(w.abs(), (0, pad)).view(len(w), -1, 8)
    out = torch.zeros(len(x), len(w), dtype=torch.float64, device=x.device)
    for g in range(x.shape[1]):
        most = torch.zeros_like(out)
        for i in range(8):
            torch.maximum(most, x[:, g, i, None] * w[None, :, g, i], out=most)
        out += most
    return 7 * 2.0 ** -13 * out


@pytest.mark.gpu
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows,k,width,want", PRODUCTS8)
def test_product8(Z, rows, k, width, want, transposed):
    """Scales that differ from group to group and from block to block, then rows and columns that are NaN
    by a scale or a code in the first, the last and a later stage."""
    outs, cols = (k, width) if transposed else (width, k)
    w8 = Z.Weight8.of(_randn((outs, cols), 1).cuda(), transposed)
    x8 = Z.Act8.of(_randn((rows, k), 2).cuda())
    g = torch.Generator().manual_seed(3)
    x8.scales.copy_((x8.scales.cpu().int() + torch.randint(-12, 12, x8.scales.shape, generator=g)).to(torch.uint8))
    w8.scales.copy_((w8.scales.cpu().int() + torch.randint(-12, 12, w8.scales.shape, generator=g)).to(torch.uint8))
    x = AO.values(x8.codes, x8.scales, k, "e4m3").cuda()
    w = PO.weight_values(w8.codes, w8.scales, cols).cuda()
    w = w.t().contiguous() if transposed else w
    exact = x @ w.t()
    err = 2 * k * U * (x.abs() @ w.abs().t()) + _cut(x, w)
    flat = torch.full((rows + 1, width + 5), 7.0, dtype=BF16, device="cuda")
    y = flat[:rows, :width]
    Z.product8(x8, w8, y, transposed=transposed)
    _assert_within(y, exact, err, "y")
    assert bool((flat[rows:] == 7).all()) and bool((flat[:, width:] == 7).all()), "wrote outside"
    again = torch.empty(rows, width, dtype=BF16, device="cuda")
    Z.product8(x8, w8, again, transposed=transposed)
    assert torch.equal(again, y)
    # row -> what of it is NaN; the column block that a weight block makes NaN
    groups, stages = -(-k // 32), -(-k // 128)
    nan_rows = sorted({0, rows // 2, rows - 1})
    for i, r in enumerate(nan_rows):
        if i == 0:
            x8.scales[r, groups - 1] = 255
        elif i == 1:
            x8.codes[r, min(k - 1, 20 * 128 + 5)] = 0x7F
        else:
            x8.scales[r, min(groups - 1, 17 * 4 + 2)] = 255
    block = (stages - 1) if stages < 20 else 18
    last = -(-width // 128) - 1
    w8.scales[(block, last) if transposed else (last, block)] = 255
    Z.product8(x8, w8, y, transposed=transposed)
    exact[nan_rows] = float("nan")
    exact[:, last * 128:] = float("nan")
    _assert_within(y, exact, err, "y beside NaN")


# ------------------------------------------------------------------------------ experts

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("in_major,sizes,cols,outs,alignment,want", EXPERTS)
def test_expert_product(Z, in_major, sizes, cols, outs, alignment, want, dtype):
    rows, n = sum(sizes) + 9, len(sizes)
    _, x = _placed(_randn((rows, cols), 1), dtype, alignment)
    x[sum(sizes):] = float("nan")  # rows that belong to no expert
    _, w = _placed(_randn((n, cols, outs) if in_major else (n, outs, cols), 2, cols ** -0.5), dtype, alignment)
    ends = torch.tensor(sizes).cumsum(0).int().cuda()
    exact, size = torch.full((rows, outs), 7.0, dtype=torch.float64, device="cuda"), torch.zeros(rows, outs, dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(PO.spans(ends.cpu(), rows)):
        we = w[e].double() if in_major else w[e].double().t()
        exact[a:b], size[a:b] = x[a:b].double() @ we, x[a:b].double().abs() @ we.abs()
    for zero_rest in (False, True):
        flat, y = _placed(torch.full((rows, outs), 7.0), dtype, alignment, 7.0)
        Z.expert_product(x, w, ends, y, in_major=in_major, zero_rest=zero_rest)
        if zero_rest:
            exact[sum(sizes):] = 0
        _assert_within(y, exact, 2 * cols * U * size, f"y {zero_rest}")
        assert _untouched(flat, y, 7.0), "wrote outside"
    again = torch.empty(rows, outs, dtype=dtype, device="cuda")
    Z.expert_product(x, w, ends, again, in_major=in_major, zero_rest=True)
    assert torch.equal(again, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (BF16, FP32), (FP16, FP16)])
@pytest.mark.parametrize("in_major,sizes,cols,outs,alignment,want", GRADIENTS)
def test_expert_wgrad(Z, in_major, sizes, cols, outs, alignment, want, dtype, grad):
    rows, n = sum(sizes) + 9, len(sizes)
    _, x = _placed(_randn((rows, cols), 1), dtype, alignment)
    _, dy = _placed(_randn((rows, outs), 2, 0.1), dtype, alignment)
    x[sum(sizes):] = float("nan")
    dy[sum(sizes):] = float("inf")
    ends = torch.tensor(sizes).cumsum(0).int().cuda()
    shape = (n, cols, outs) if in_major else (n, outs, cols)
    exact, size = (torch.zeros(shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for e, (a, b) in enumerate(PO.spans(ends.cpu(), rows)):
        p, q = (x, dy) if in_major else (dy, x)
        p, q = p[a:b].double(), q[a:b].double()
        exact[e], size[e] = p.t() @ q, p.t().abs() @ q.abs()
    for based in (False, True):
        before = _randn(shape, 5) if based else torch.full(shape, 7.0)
        flat, dw = _placed(before, grad, alignment, 7.0)
        plus = dw.double() if based else 0
        Z.expert_wgrad(x, dy, ends, dw, base=dw if based else None, in_major=in_major)
        err = 2 * (max(sizes) + 1) * U * (size + (plus.abs() if based else 0))
        _assert_within(dw, exact + plus, err, f"dw {based}")
        assert _untouched(flat, dw, 7.0), "wrote outside"


# ------------------------------------------------------------------------------ graphs

@pytest.mark.gpu
def test_tiles_in_a_graph(Z):
    """The tiled plans captured together and replayed on changed operands, eager work in between: with more
    LDS than a launch has without asking, each of them sets its kernel's limit in the capture."""
    g = torch.Generator("cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g).to(BF16)

    sizes = [UNEVEN, RAGGED]
    ends = [torch.tensor(s).cumsum(0).int().cuda() for s in sizes]
    x8 = [Z.Act8.empty(3000, 400, device="cuda"), Z.Act8.empty(700, 400, device="cuda")]
    w8, w8s = Z.Weight8.empty(4100, 400), Z.Weight8.empty(1000, 400)
    x = [randn(sum(s), 200) for s in sizes]
    dy = [randn(sum(sizes[0]), 4096), randn(sum(sizes[1]), 808)]
    w = [randn(3, 4096, 200), randn(6, 808, 200)]
    wide = randn(sum(sizes[0]), 4096)

    def everything():
        y8 = [torch.empty(3000, 4100, dtype=BF16, device="cuda"), torch.empty(700, 1000, dtype=BF16, device="cuda")]
        Z.product8(x8[0], w8, y8[0])
        Z.product8(x8[1], w8s, y8[1])
        out = y8
        for i in range(2):
            y, dx = torch.empty_like(dy[i]), torch.empty_like(x[i])
            dw = torch.empty_like(w[i], dtype=FP32)
            Z.expert_product(x[i], w[i], ends[i], y, zero_rest=True)
            Z.expert_product(dy[i], w[i], ends[i], dx, in_major=True, zero_rest=True)
            Z.expert_wgrad(x[i], dy[i], ends[i], dw)
            out += [y, dx, dw]
        dw = torch.empty(3, 4096, 4096, dtype=BF16, device="cuda")
        Z.expert_wgrad(wide, dy[0], ends[0], dw)
        return out + [dw]

    def change():
        for a, rows in zip(x8, (3000, 700)):
            Z.act_pack(randn(rows, 400), a)
        Z.weight8_pack(randn(4100, 400), w8)
        Z.weight8_pack(randn(1000, 400), w8s)
        for t in (*x, *dy, *w, wide):
            t.copy_(randn(*t.shape))

    assert plan8(3000, 4100) == "large" and plan8(700, 1000) == "small"
    assert plan(4096, 4096, 3, True, True, True, True) == "large"
    change()
    everything()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = everything()
    for _ in range(3):
        change()
        for t in got:
            t.fill_(9)
        want = everything()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
