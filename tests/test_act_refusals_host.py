"""CPU tests of refusals of the activation operators' C entry points and tensor-level calls (no
kernel runs)."""

import pytest
import torch

# Addresses that pass the checks and are never read: every call below is refused on the host.
P = 1 << 20
S = 0  # the null stream


@pytest.fixture
def Z():
    import zero_sharded_mixed_buffer_amd as Z
    Z.lib()
    return Z


def _refused(Z, match, fn, *args, **kw):
    with pytest.raises(Z._abi.ZsInvalidArgument, match=match):
        fn(*args, stream=S, **kw)


def test_reserved_field_is_checked(Z):
    """zs_act.reserved is 0, in every call that takes a checkpoint."""
    act = Z.ActArrays(P, P, 0, 1)
    _refused(Z, "reserved", Z.zs_act_pack, P, 0, 64, 4, 64, act)
    _refused(Z, "reserved", Z.zs_act_unpack, act, 4, 64, P, 0, 64)
    _refused(Z, "reserved", Z.zs_rmsnorm, P, 64, None, 0, P, 0, 4, 64, 1e-6, y8=act)
    _refused(Z, "reserved", Z.zs_rmsnorm, P, 64, None, 0, P, 0, 4, 64, 1e-6, h8=act)
    _refused(Z, "reserved", Z.zs_rmsnorm_backward, P, 64, None, 0, None, 0, act, P, P, 0, 4, 64, P, 64)
    _refused(Z, "reserved", Z.zs_act_wgrad, act, 4, 64, P, 0, 48, 48, P, 0, 64, workspace=P, workspace_bytes=1 << 20)


def test_norm_outputs_in_one_place_are_refused(Z):
    """The checkpoint of y and that of h in one pair of arrays, y and h in one matrix: each output would
    overwrite the other."""
    call = dict(x=P, x_stride=64, residual=P, residual_stride=64, weight=P, dtype=0, rows=4, cols=64, eps=1e-6)
    _refused(Z, "y8 and h8", Z.zs_rmsnorm, **call, y8=Z.ActArrays(P, 2 * P, 0, 0), h8=Z.ActArrays(P, 3 * P, 0, 0))
    _refused(Z, "y8 and h8", Z.zs_rmsnorm, **call, y8=Z.ActArrays(P, 2 * P, 0, 0), h8=Z.ActArrays(3 * P, 2 * P, 1, 0))
    _refused(Z, "h and y", Z.zs_rmsnorm, **call, h=2 * P, h_stride=64, y=2 * P, y_stride=64)


def test_in_place_with_another_stride_is_refused(Z):
    """h in x's or the residual's memory, dx in dy's or dh's, has to have its rows where theirs are; one
    row lies the same way at any stride."""
    call = dict(x=P, x_stride=64, residual=2 * P, residual_stride=96, weight=P, dtype=0, rows=4, cols=64, eps=1e-6)
    _refused(Z, "in place", Z.zs_rmsnorm, **call, h=P, h_stride=96)
    _refused(Z, "in place", Z.zs_rmsnorm, **call, h=2 * P, h_stride=64)
    call = dict(dy=P, dy_stride=64, dh=2 * P, dh_stride=96, h=3 * P, h_stride=64, h8=None, weight=P, rstd=P, dtype=0, rows=4,
                cols=64)
    _refused(Z, "in place", Z.zs_rmsnorm_backward, **call, dx=P, dx_stride=96)
    _refused(Z, "in place", Z.zs_rmsnorm_backward, **call, dx=2 * P, dx_stride=64)
