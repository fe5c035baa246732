"""CPU tests of the products, the experts and the routing: the oracle against the definitions, sizes,
and refusals of the C entry points and the tensor-level calls (no kernel runs)."""

import pytest
import torch

from oracle import act_oracle as AO
from oracle import product_oracle as PO

# Addresses that pass the checks and are never read: every call below is refused on the host.
P = 1 << 20
S = 0  # the null stream


@pytest.fixture
def Z():
    import zero_sharded_mixed_buffer_amd as Z
    Z.lib()
    return Z


# ------------------------------------------------------------------------------ the oracle

def test_weight8_oracle_is_the_checkpoints_rule_over_blocks():
    """A weight whose 32-column groups all hold the block's largest magnitude has the checkpoint's codes
    and scales; both orientations hold the same codes; the values are within half a code step."""
    g = torch.Generator().manual_seed(0)
    w = torch.randn(200, 300, generator=g)
    w[:, ::32] = 4.5
    codes, codes_t, scales = PO.weight8(w)
    assert codes.shape == (200, 384) and codes_t.shape == (300, 256) and scales.shape == (2, 3)
    c, s = AO.quantise(w[:, :288], "e4m3")
    assert torch.equal(codes[:, :288], c)
    assert torch.equal(scales.repeat_interleave(128, 0)[:200].repeat_interleave(4, 1)[:, :9], s)
    assert torch.equal(codes_t[:, :200], codes[:, :300].t()) and not codes[:, 300:].any() and not codes_t[:, 200:].any()
    w = torch.randn(130, 140, generator=g) * torch.exp(3 * torch.randn(130, 140, generator=g))
    codes, _, scales = PO.weight8(w)
    v = PO.weight_values(codes, scales, 140)
    step = 2.0 ** (scales.double() - 127)
    step = step.repeat_interleave(128, 0)[:130].repeat_interleave(128, 1)[:, :140]
    assert bool(((v - w.double()).abs() <= w.double().abs() / 16 + step * 2.0 ** -10).all())
    for i in range(2):
        for j in range(2):
            top = float(w[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128].abs().max())
            k = float(step[i * 128, j * 128])
            assert top <= 448 * k and top > 224 * k


def test_weight8_oracle_marks_what_is_not_finite():
    w = torch.ones(130, 260)
    w[3, 200] = float("inf")
    w[129, 0] = float("nan")
    codes, _, scales = PO.weight8(w)
    assert scales.tolist() == [[119, 255, 119], [255, 119, 119]]
    v = PO.weight_values(codes, scales, 260)
    assert bool(torch.isnan(v[:128, 128:256]).all()) and bool(torch.isnan(v[128:, :128]).all())
    assert bool((v[:128, :128] == 1).all()) and bool((v[:, 256:] == 1).all())


def test_spans_of_ends():
    assert PO.spans(torch.tensor([2, 2, 5]), 9) == [(0, 2), (2, 2), (2, 5)]
    assert PO.spans(torch.tensor([4, 1, -3, 7, 2 ** 31 - 1]), 9) == [(0, 4), (4, 4), (4, 4), (4, 7), (7, 9)]


def test_route_oracle():
    ids = torch.tensor([[1, 0], [2, 1], [-1, 1], [0, 5]])
    ends, slot, place = PO.route(ids, 3)
    assert ends.tolist() == [2, 5, 6]
    assert slot.tolist() == [1, 6, 0, 3, 5, 2, -5, -8]
    assert place.tolist() == [[2, 0], [5, 3], [-1, 4], [1, -1]]
    big = torch.randint(-1, 41, (900, 2), generator=torch.Generator().manual_seed(1))
    ends, slot, place = PO.route(big, 40)
    flat = big.reshape(-1)
    order = torch.argsort(torch.where(flat >= 40, -1, flat) % 41, stable=True)  # -1 and 40 become 40: last
    kept = int(ends[-1])
    assert slot[:kept].tolist() == order[:kept].tolist()


def test_combination_oracle_against_autograd():
    """The combination and its backward, and the experts' gradients, against torch's autograd in 64 bits."""
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(-1, 4, (7, 3), generator=g)
    ends, slot, place = PO.route(ids, 4)
    y = torch.randn(21, 5, dtype=torch.float64, generator=g, requires_grad=True)
    w = torch.rand(7, 3, generator=g).requires_grad_()
    dout = torch.randn(7, 5, dtype=torch.float64, generator=g)
    valid = place >= 0
    out = (torch.where(valid, w.double(), 0.0)[:, :, None] * y[place.clamp_min(0).long()]).sum(1)
    out.backward(dout)
    got, _ = PO.combine(y.detach(), place, w.detach())
    assert torch.allclose(got, out.detach(), atol=1e-14)
    dy, dw, _ = PO.combine_backward(dout, y.detach(), slot, 3, w.detach())
    assert torch.allclose(dy, y.grad, atol=1e-14) and torch.allclose(dw.float(), w.grad, atol=1e-6)
    x = torch.randn(6, 4, dtype=torch.float64, generator=g, requires_grad=True)
    weight = torch.randn(2, 3, 4, dtype=torch.float64, generator=g, requires_grad=True)
    ends = torch.tensor([4, 6])
    z = torch.cat([x[:4] @ weight[0].t(), x[4:] @ weight[1].t()])
    dz = torch.randn(6, 3, dtype=torch.float64, generator=g)
    z.backward(dz)
    assert torch.allclose(PO.expert_product(x.detach(), weight.detach(), ends)[0], z.detach())
    assert torch.allclose(PO.expert_product(dz, weight.detach(), ends, in_major=True)[0], x.grad)
    assert torch.allclose(PO.expert_wgrad(x.detach(), dz, ends)[0], weight.grad)
    assert torch.allclose(PO.expert_wgrad(x.detach(), dz, ends, in_major=True)[0], weight.grad.transpose(1, 2))


# ------------------------------------------------------------------------------ sizes

def test_sizes(Z):
    assert Z.zs_weight8_size(1, 1) == (128, 128, 1)
    assert Z.zs_weight8_size(517, 1003) == (517 * 1024, 1003 * 640, 5 * 8)
    for bad in ((0, 1), (1, 0), (-1, 5), (2 ** 23 + 1, 1), (1, 2 ** 40)):
        with pytest.raises(Z.ZsInvalidArgument):
            Z.zs_weight8_size(*bad)
    assert Z.zs_route_workspace(0, 1) >= 16 and Z.zs_route_workspace(1 << 20, 1024) >= 1024 * 1025 * 4
    for bad in ((-1, 4), (2 ** 31, 4), (5, 0), (5, 1025)):
        with pytest.raises(Z.ZsInvalidArgument):
            Z.zs_route_workspace(*bad)


# ------------------------------------------------------------------------------ refusals

def _refused(Z, match, fn, good, **bad):
    with pytest.raises(Z.ZsInvalidArgument, match=match):
        fn(**{**good, **bad}, stream=S)


def test_weight8_and_product8_refusals(Z):
    w8 = Z.Weight8Arrays(P, 2 * P, 3 * P)
    pack = dict(src=P, src_dtype=0, src_stride=64, outs=48, cols=64, w8=w8)
    _refused(Z, "src is NULL", Z.zs_weight8_pack, pack, src=None)
    _refused(Z, "src_dtype", Z.zs_weight8_pack, pack, src_dtype=7)
    _refused(Z, "stride", Z.zs_weight8_pack, pack, src_stride=63)
    _refused(Z, "aligned", Z.zs_weight8_pack, pack, src=P + 1)
    _refused(Z, "outs must be", Z.zs_weight8_pack, pack, outs=0)
    _refused(Z, "cols must be", Z.zs_weight8_pack, pack, cols=0)
    _refused(Z, "at most", Z.zs_weight8_pack, pack, outs=2 ** 23 + 1)
    _refused(Z, "w8 is NULL", Z.zs_weight8_pack, pack, w8=None)
    _refused(Z, "codes or scales", Z.zs_weight8_pack, pack, w8=Z.Weight8Arrays(None, P, P))
    _refused(Z, "16-byte", Z.zs_weight8_pack, pack, w8=Z.Weight8Arrays(P, P + 8, P))
    act = Z.ActArrays(P, 2 * P, 0, 0)
    call = dict(x8=act, rows=4, w8=w8, outs=48, cols=64, transposed=False, y=P, y_dtype=0, y_stride=64)
    _refused(Z, "y_dtype", Z.zs_product8, call, y_dtype=2)
    _refused(Z, "x8 is NULL", Z.zs_product8, call, x8=None)
    _refused(Z, "e4m3", Z.zs_product8, call, x8=Z.ActArrays(P, P, 1, 0))
    _refused(Z, "reserved", Z.zs_product8, call, x8=Z.ActArrays(P, P, 0, 1))
    _refused(Z, "16-byte", Z.zs_product8, call, x8=Z.ActArrays(P + 8, P, 0, 0))
    _refused(Z, "transposed codes", Z.zs_product8, call, w8=Z.Weight8Arrays(P, None, P), transposed=True)
    _refused(Z, "y is NULL", Z.zs_product8, call, y=None)
    _refused(Z, "stride", Z.zs_product8, call, y_stride=47)
    _refused(Z, "stride", Z.zs_product8, call, y_stride=63, transposed=True)
    _refused(Z, "rows is negative", Z.zs_product8, call, rows=-1)
    _refused(Z, "one launch", Z.zs_product8, call, rows=2 ** 31)


def test_expert_refusals(Z):
    call = dict(x=P, x_stride=64, weight=P, w_stride=64, w_expert_stride=64 * 48, dtype=0, ends=P, experts=3, rows=9, cols=64,
                outs=48, in_major=False, y=P, y_stride=48)
    fn = Z.zs_expert_product
    _refused(Z, "dtype", fn, call, dtype=2)
    _refused(Z, "experts must", fn, call, experts=0)
    _refused(Z, "experts must", fn, call, experts=1025)
    _refused(Z, "ends is NULL", fn, call, ends=None)
    _refused(Z, "ends must be aligned", fn, call, ends=P + 2)
    _refused(Z, "x is NULL", fn, call, x=None)
    _refused(Z, "w is NULL", fn, call, weight=None)
    _refused(Z, "y is NULL", fn, call, y=None)
    _refused(Z, "x: the row stride", fn, call, x_stride=63)
    _refused(Z, "w: the row stride", fn, call, w_stride=63)
    _refused(Z, "w: the row stride", fn, call, in_major=True, w_stride=47)
    _refused(Z, "w: the expert stride", fn, call, w_expert_stride=-1)
    _refused(Z, "y: the row stride", fn, call, y_stride=47)
    _refused(Z, "aligned", fn, call, y=P + 1)
    _refused(Z, "cols must", fn, call, outs=0)
    _refused(Z, "cols must", fn, call, cols=0)
    _refused(Z, "2\\^31", fn, call, rows=2 ** 31)
    _refused(Z, "negative", fn, call, rows=-1)
    call = dict(x=P, x_stride=64, dy=P, dy_stride=48, dtype=0, ends=P, experts=3, rows=9, cols=64, outs=48, dw=P, dw_dtype=0,
                dw_stride=64, dw_expert_stride=64 * 48)
    fn = Z.zs_expert_wgrad
    _refused(Z, "dw: the experts' matrices overlap", fn, call, dw_expert_stride=64 * 48 - 1)
    _refused(Z, "dw: the experts' matrices overlap", fn, call, dw_expert_stride=0)
    _refused(Z, "dw: the row stride", fn, call, dw_stride=63)
    _refused(Z, "dw: the row stride", fn, call, in_major=True, dw_stride=47)
    _refused(Z, "dw is NULL", fn, call, dw=None)
    _refused(Z, "dy is NULL", fn, call, dy=None)
    _refused(Z, "dy: the row stride", fn, call, dy_stride=47)
    _refused(Z, "base must be aligned", fn, call, base=P + 1)
    _refused(Z, "dw_dtype", fn, call, dw_dtype=9)
    with pytest.raises(Z.ZsError, match="dw_dtype must be"):
        fn(**{**call, "dw_dtype": 1}, stream=S)


def test_routing_refusals(Z):
    call = dict(ids=P, id_bytes=8, slots=30, experts=4, ends=P, slot=P, place=P, workspace=P, workspace_bytes=1 << 20)
    _refused(Z, "id_bytes", Z.zs_route, call, id_bytes=2)
    _refused(Z, "ids", Z.zs_route, call, ids=None)
    _refused(Z, "ids", Z.zs_route, call, ids=P + 4)
    _refused(Z, "ends", Z.zs_route, call, ends=None)
    _refused(Z, "slot", Z.zs_route, call, slot=None)
    _refused(Z, "place", Z.zs_route, call, place=P + 2)
    _refused(Z, "workspace", Z.zs_route, call, workspace=None)
    _refused(Z, "workspace", Z.zs_route, call, workspace_bytes=15)
    _refused(Z, "experts", Z.zs_route, call, experts=0)
    _refused(Z, "slots", Z.zs_route, call, slots=-1)
    call = dict(x=P, x_stride=64, dtype=0, slot=P, tokens=5, choices=2, cols=64, out=P, out_stride=64)
    _refused(Z, "dtype", Z.zs_expert_gather, call, dtype=5)
    _refused(Z, "choices", Z.zs_expert_gather, call, choices=0)
    _refused(Z, "negative", Z.zs_expert_gather, call, tokens=-1)
    _refused(Z, "cols", Z.zs_expert_gather, call, cols=0)
    _refused(Z, "2\\^31", Z.zs_expert_gather, call, tokens=2 ** 30, choices=4)
    _refused(Z, "x is NULL", Z.zs_expert_gather, call, x=None)
    _refused(Z, "slot is NULL", Z.zs_expert_gather, call, slot=None)
    _refused(Z, "out: the row stride", Z.zs_expert_gather, call, out_stride=60)
    call = dict(y=P, y_stride=64, dtype=0, place=P, weights=None, tokens=5, choices=2, cols=64, out=P, out_stride=64)
    _refused(Z, "y is NULL", Z.zs_expert_combine, call, y=None)
    _refused(Z, "place is NULL", Z.zs_expert_combine, call, place=None)
    _refused(Z, "weights", Z.zs_expert_combine, call, weights=P + 1)
    _refused(Z, "out is NULL", Z.zs_expert_combine, call, out=None)
    call = dict(dout=P, dout_stride=64, y=P, y_stride=64, dtype=0, slot=P, place=P, weights=P, tokens=5, choices=2, cols=64,
                dy=2 * P, dy_stride=64, dweights=P)
    fn = Z.zs_expert_combine_backward
    _refused(Z, "no output", fn, call, dy=None, dweights=None)
    _refused(Z, "y is NULL", fn, call, y=None)
    _refused(Z, "dout is NULL", fn, call, dout=None)
    _refused(Z, "slot is NULL", fn, call, slot=None)
    _refused(Z, "place is NULL", fn, call, place=None)
    _refused(Z, "in place", fn, call, dy=P, dy_stride=96)


def test_tensor_level_refusals(Z):
    """What is wrong with types, shapes, strides and devices is a ValueError, also without a GPU."""
    bf = torch.bfloat16
    u8 = torch.zeros(4, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="scales"):
        Z.Weight8(u8, torch.zeros(2, 1, dtype=torch.uint8), 100)
    with pytest.raises(ValueError, match="codes"):
        Z.Weight8(u8, torch.zeros(1, 2, dtype=torch.uint8), 200)
    with pytest.raises(ValueError, match="codes_t"):
        Z.Weight8(u8, torch.zeros(1, 1, dtype=torch.uint8), 100, codes_t=torch.zeros(100, 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        Z.Weight8(torch.zeros(128, 4, dtype=torch.uint8).t(), torch.zeros(1, 1, dtype=torch.uint8), 100)
    w8 = Z.Weight8(u8, torch.zeros(1, 1, dtype=torch.uint8), 100)
    with pytest.raises(ValueError, match="GPU"):
        Z.weight8_pack(torch.zeros(4, 100, dtype=bf), w8)
    x8 = Z.Act8(torch.zeros(3, 128, dtype=torch.uint8), torch.zeros(3, 4, dtype=torch.uint8), 100)
    with pytest.raises(ValueError, match="GPU"):
        Z.product8(x8, w8, torch.zeros(3, 4, dtype=bf))
    x, w, ends = torch.zeros(6, 8, dtype=bf), torch.zeros(2, 5, 8, dtype=bf), torch.tensor([3, 6], dtype=torch.int32)
    for call in (lambda: Z.expert_product(x, w, ends, torch.zeros(6, 5, dtype=bf)),
                 lambda: Z.expert_wgrad(x, torch.zeros(6, 5, dtype=bf), ends, w),
                 lambda: Z.route(torch.zeros(3, 2, dtype=torch.int64), 4),
                 lambda: Z.experts(x, w, ends), lambda: Z.linear8(x, w[0])):
        with pytest.raises(ValueError, match="GPU"):
            call()
    place = torch.zeros(3, 2, dtype=torch.int32)
    slot = torch.zeros(6, dtype=torch.int32)
    with pytest.raises(ValueError, match="place"):
        Z.Route(ends, slot, place.long())
    with pytest.raises(ValueError, match="slot"):
        Z.Route(ends, slot[:5], place)
    with pytest.raises(ValueError, match="ends"):
        Z.Route(ends.long(), slot, place)
    r = Z.Route(ends, slot, place)
    assert (r.experts, r.tokens, r.choices, r.rows) == (2, 3, 2, 6)
    with pytest.raises(ValueError, match="GPU"):
        Z.expert_gather(torch.zeros(3, 4), r, torch.zeros(6, 4))
    with pytest.raises(ValueError, match="ids"):
        Z.route(torch.zeros(3, 2), 4)


def test_header_is_plain_c(tmp_path):
    """zs_product.h compiles by itself as C99."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "h.c"
    src.write_text('#include "zs_product.h"\nint main(void) { zs_weight8 w = {0, 0, 0}; return w.codes != 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-fsyntax-only", "-I", os.path.join(root, "include"), str(src)],
                   check=True)
