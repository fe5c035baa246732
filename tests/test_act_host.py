"""CPU tests of the activation operators: the oracle against brute force and differences, sizes,
and every refusal of the C entry points and of the tensor-level calls (no kernel runs)."""

import ctypes
import itertools

import pytest
import torch

from oracle import act_oracle as AO


def _z():
    import zero_sharded_mixed_buffer_amd as Z
    try:
        Z.lib()
    except ImportError as e:
        pytest.fail(str(e))
    return Z


# ------------------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_oracle_scale_is_the_smallest_that_holds_the_group(code):
    gen = torch.Generator().manual_seed(1)
    amax = torch.cat([torch.rand(200, generator=gen, dtype=torch.float64) * 2.0 ** torch.randint(-126, 127, (200,), generator=gen),
                      torch.tensor([0.0, 448.0, 449.0, 127.0, 127.5, 2.0 ** -140, 65504.0], dtype=torch.float64)])
    for a, b in zip(amax.tolist(), AO.scale_bytes(amax, code).tolist()):
        assert a <= AO.QMAX[code] * 2.0 ** (b - 127)
        assert b == 0 or a > AO.QMAX[code] * 2.0 ** (b - 128)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_oracle_codes_are_the_nearest(code):
    """Against a search over all 256 codes; ties go to the even code."""
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(3, 64, generator=gen).double()
    x[0, :16] = torch.arange(16).double() / 16 * 2.0 ** -9  # around the smallest steps
    x[0, 16] = 448.0
    codes, scales = AO.quantise(x, code)
    table = AO.E4M3 if code == "e4m3" else torch.arange(256).double() - 256 * (torch.arange(256) > 127)
    for r in range(3):
        for c in range(64):
            s = 2.0 ** (int(scales[r, c // 32]) - 127)
            d = (table * s - x[r, c]).abs()
            d = torch.where(torch.isnan(d), torch.full_like(d, float("inf")), d)
            got = int(codes[r, c])
            assert d[got] == d.min()
            if (d == d.min()).sum() > 1 and float(x[r, c]) != 0:
                assert got % 2 == 0


def test_oracle_norm_backward_against_differences():
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(3, 7, generator=gen, dtype=torch.float64)
    w = torch.randn(7, generator=gen, dtype=torch.float64)
    dy = torch.randn(3, 7, generator=gen, dtype=torch.float64)
    dh = torch.randn(3, 7, generator=gen, dtype=torch.float64)

    def loss(x, w):
        h, _, y = AO.norm(x, w, 1e-5)
        return float((y * dy).sum() + (h * dh).sum())

    _, rstd, _ = AO.norm(x, w, 1e-5)
    dx, dw = AO.norm_backward(dy, x, w, rstd, dh)
    step = 1e-6
    for i, j in itertools.product(range(3), range(7)):
        e = torch.zeros_like(x)
        e[i, j] = step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - float(dx[i, j])) < 1e-7
    for j in range(7):
        e = torch.zeros_like(w)
        e[j] = step
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - float(dw[j])) < 1e-7


def test_oracle_wgrad_against_differences():
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(5, 4, generator=gen, dtype=torch.float64)
    w = torch.randn(3, 4, generator=gen, dtype=torch.float64)
    dy = torch.randn(5, 3, generator=gen, dtype=torch.float64)
    dw = AO.wgrad(dy, x)
    step = 1e-5
    for i, j in itertools.product(range(3), range(4)):
        e = torch.zeros_like(w)
        e[i, j] = step
        diff = float((((x @ (w + e).t()) - (x @ (w - e).t())) * dy).sum() / (2 * step))
        assert abs(diff - float(dw[i, j])) < 1e-8


# ------------------------------------------------------------------------------ C entry points

def test_sizes():
    Z = _z()
    assert Z.zs_act_size(0, 5) == (0, 0)
    assert Z.zs_act_size(3, 32) == (96, 3)
    assert Z.zs_act_size(3, 33) == (192, 6)
    assert Z.zs_act_size(1 << 20, 1 << 20) == (1 << 40, 1 << 35)
    for rows, cols in [(-1, 4), (4, 0), (4, -3), (1 << 40, 1 << 40), (1 << 41, 1)]:
        with pytest.raises(Z._abi.ZsInvalidArgument):
            Z.zs_act_size(rows, cols)


def test_workspaces_grow_with_what_they_hold():
    Z = _z()
    assert Z.zs_rmsnorm_workspace(0, 4096) >= 16
    assert Z.zs_rmsnorm_workspace(1 << 20, 4096) <= 1 << 26
    for cols in (0, 16385):
        with pytest.raises(Z._abi.ZsInvalidArgument):
            Z.zs_rmsnorm_workspace(4, cols)
    with pytest.raises(Z._abi.ZsInvalidArgument):
        Z.zs_rmsnorm_workspace(1 << 34, 128)
    assert Z.zs_act_wgrad_workspace(0, 64, 64) >= 16
    for bad in [(4, 0, 4), (4, 4, 0), (-1, 4, 4), (4, 1 << 31, 4), (4, 1 << 30, 1 << 30)]:
        with pytest.raises(Z._abi.ZsInvalidArgument):
            Z.zs_act_wgrad_workspace(*bad)


# Addresses that pass the checks and are never read: every call below is refused on the host.
P = 1 << 20
S = 0  # the null stream


def _act(code=0, codes=P, scales=P):
    import zero_sharded_mixed_buffer_amd as Z
    return Z.ActArrays(codes, scales, code, 0)


def _refused(fn, *args, **kw):
    import zero_sharded_mixed_buffer_amd as Z
    with pytest.raises(Z._abi.ZsInvalidArgument) as e:
        fn(*args, stream=S, **kw)
    assert len(str(e.value)) > 20
    return str(e.value)


def test_pack_and_unpack_refusals():
    Z = _z()
    ok = dict(src=P, src_dtype=0, src_stride=64, rows=4, cols=64, act=_act())
    for change in [dict(src=None), dict(src=P + 1), dict(src_dtype=3), dict(src_stride=63), dict(rows=-1),
                   dict(cols=0), dict(act=None), dict(act=_act(2)), dict(act=_act(codes=0)), dict(act=_act(scales=0)),
                   dict(act=_act(codes=P + 8)), dict(rows=1 << 36), dict(src_stride=1 << 61),
                   dict(src_dtype=2, src=P + 2)]:
        _refused(Z.zs_act_pack, **{**ok, **change})
    ok = dict(act=_act(), rows=4, cols=64, dst=P, dst_dtype=0, dst_stride=64)
    for change in [dict(dst=None), dict(dst=P + 1), dict(dst_dtype=-1), dict(dst_stride=63), dict(rows=-1),
                   dict(cols=0), dict(act=None), dict(act=_act(-1)), dict(act=_act(codes=P + 4))]:
        _refused(Z.zs_act_unpack, **{**ok, **change})


def test_norm_refusals():
    Z = _z()
    ok = dict(x=P, x_stride=64, residual=P, residual_stride=64, weight=P, dtype=0, rows=4, cols=64, eps=1e-6, h=P,
              h_stride=64, y=P, y_stride=64, y8=_act(), h8=_act(1), rstd=P)
    for change in [dict(x=None), dict(x=P + 1), dict(x_stride=63), dict(residual_stride=1), dict(residual=P + 1),
                   dict(weight=None), dict(weight=P + 1), dict(dtype=2), dict(rows=-1), dict(cols=0), dict(cols=16385),
                   dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-40),
                   dict(h_stride=3), dict(y_stride=3), dict(y=P + 1), dict(y8=_act(7)), dict(h8=_act(codes=P + 2)),
                   dict(rstd=P + 2), dict(rows=1 << 30),
                   dict(h=None, y=None, y8=None, h8=None, rstd=None)]:
        _refused(Z.zs_rmsnorm, **{**ok, **change})


def test_norm_backward_refusals():
    Z = _z()
    ok = dict(dy=P, dy_stride=64, dh=P, dh_stride=64, h=P, h_stride=64, h8=None, weight=P, rstd=P, dtype=1, rows=4,
              cols=64, dx=P, dx_stride=64, dweight=P, dweight_dtype=2, base=P, workspace=P, workspace_bytes=1 << 20)
    for change in [dict(dy=None), dict(dx=None), dict(dy_stride=1), dict(dx_stride=1), dict(dh_stride=1),
                   dict(h_stride=1), dict(h=None), dict(h8=_act()), dict(h=None, h8=_act(9)), dict(weight=None),
                   dict(rstd=None), dict(rstd=P + 1), dict(dtype=2), dict(cols=16385), dict(dweight=None),
                   dict(dweight_dtype=5), dict(dweight=P + 2), dict(base=P + 2), dict(workspace=None),
                   dict(workspace=P + 8), dict(workspace_bytes=15)]:
        _refused(Z.zs_rmsnorm_backward, **{**ok, **change})


def test_wgrad_refusals():
    Z = _z()
    ok = dict(x8=_act(), rows=4, cols=64, dy=P, dy_dtype=0, dy_stride=48, outs=48, dw=P, dw_dtype=0, dw_stride=64,
              in_major=False, base=P, workspace=P, workspace_bytes=1 << 20)
    for change in [dict(x8=None), dict(x8=_act(3)), dict(dy=None), dict(dy=P + 1), dict(dy_dtype=2), dict(dy_stride=47),
                   dict(outs=0), dict(cols=0), dict(rows=-1), dict(dw=None), dict(dw=P + 1), dict(dw_dtype=4),
                   dict(dw_stride=63), dict(in_major=True, dw_stride=47), dict(base=P + 1), dict(workspace=None),
                   dict(workspace=P + 4), dict(workspace_bytes=0), dict(dw_dtype=2, dw=P + 2)]:
        _refused(Z.zs_act_wgrad, **{**ok, **change})
    with pytest.raises(Z.ZsError) as e:
        Z.zs_act_wgrad(**{**ok, "dw_dtype": 1}, stream=S)
    assert e.value.status == -4


# ------------------------------------------------------------------------------ tensor-level calls

def test_checkpoint_arrays_are_checked():
    Z = _z()
    u8 = dict(dtype=torch.uint8)
    good = Z.Act8(torch.zeros(3, 64, **u8), torch.zeros(3, 2, **u8), 40, "int8")
    assert (good.rows, good.cols, good.nbytes) == (3, 40, 198)
    for codes, scales, cols, code in [
            (torch.zeros(3, 64, **u8), torch.zeros(3, 2, **u8), 64, "fp8"),
            (torch.zeros(3, 64), torch.zeros(3, 2, **u8), 64, "e4m3"),
            (torch.zeros(3, 60, **u8), torch.zeros(3, 2, **u8), 60, "e4m3"),
            (torch.zeros(3, 64, **u8), torch.zeros(2, 2, **u8), 64, "e4m3"),
            (torch.zeros(3, 64, **u8), torch.zeros(3, 2, **u8), 0, "e4m3"),
            (torch.zeros(3, 128, **u8)[:, ::2], torch.zeros(3, 2, **u8), 64, "e4m3"),
            (torch.zeros(192, **u8), torch.zeros(3, 2, **u8), 64, "e4m3")]:
        with pytest.raises(ValueError):
            Z.Act8(codes, scales, cols, code)


def test_host_tensors_are_refused():
    """Every tensor-level call refuses host memory before anything else happens."""
    Z = _z()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    r = torch.zeros(4)
    act = Z.Act8.empty(4, 64, "e4m3", "cpu")
    for call in [lambda: Z.act_pack(x, act), lambda: Z.act_unpack(act, x), lambda: Z.rmsnorm(x, w, y=x),
                 lambda: Z.rmsnorm_backward(x, x, w, r, x), lambda: Z.act_wgrad(act, x, torch.zeros(64, 64)),
                 lambda: Z.norm(x, w), lambda: Z.linear(x, torch.zeros(8, 64, dtype=torch.bfloat16)),
                 lambda: Z.Act8.of(x)]:
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_struct_layout_matches_the_header():
    Z = _z()
    assert ctypes.sizeof(Z.ActArrays) == 24
    assert Z.ActArrays.code.offset == 16
