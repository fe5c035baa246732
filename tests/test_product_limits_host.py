"""CPU tests of the sizes that the products' calls take and refuse (no kernel runs: a call whose sizes
pass is refused for a NULL pointer, which is looked at after them)."""

import pytest

P = 1 << 20  # an address that passes the checks and is never read
BF16, FP32 = 0, 2


@pytest.fixture
def Z():
    import zero_sharded_mixed_buffer_amd as Z
    Z.lib()
    return Z


def _lanes(row_bytes):
    """Lanes to a row: one for each 16 bytes, a power of two from 16 to 256."""
    lanes = 16
    while lanes < 256 and lanes * 16 < row_bytes:
        lanes *= 2
    return lanes


WIDTHS = [(1, BF16), (64, FP32), (65, FP32), (128, BF16), (129, BF16), (512, FP32), (513, FP32), (1024, BF16), (1025, BF16), (4096, FP32)]


@pytest.mark.parametrize("cols,dtype", WIDTHS)
def test_rows_of_one_launch(Z, cols, dtype):
    """A launch has whole workgroups of 256 lanes, fewer than 2^32 lanes in all."""
    per_block = 256 // _lanes(cols * (4 if dtype == FP32 else 2))
    most = (2 ** 24 - 1) * per_block
    gather = dict(x_stride=cols, dtype=dtype, slot=P, choices=1, cols=cols, out=P, out_stride=cols, stream=0)
    combine = dict(y_stride=cols, dtype=dtype, place=P, weights=None, cols=cols, out=P, out_stride=cols, stream=0)
    backward = dict(dout_stride=cols, y=P, y_stride=cols, dtype=dtype, slot=P, place=P, weights=P, cols=cols, dy=P, dy_stride=cols,
                    stream=0)
    for tokens, fits in ((most, True), (most + 1, False)):
        with pytest.raises(Z.ZsInvalidArgument, match="x is NULL" if fits else "one launch"):
            Z.zs_expert_gather(None, tokens=tokens, **gather)
        for choices in (1, 7):  # the launches are over the tokens
            with pytest.raises(Z.ZsInvalidArgument, match="y is NULL" if fits else "one launch"):
                Z.zs_expert_combine(None, tokens=tokens, choices=choices, **combine)
            with pytest.raises(Z.ZsInvalidArgument, match="dout is NULL" if fits else "one launch"):
                Z.zs_expert_combine_backward(None, tokens=tokens, choices=choices, **backward)
    with pytest.raises(Z.ZsInvalidArgument, match="x is NULL"):
        Z.zs_expert_gather(None, tokens=most // 7, **{**gather, "choices": 7})
    with pytest.raises(Z.ZsInvalidArgument, match="one launch"):
        Z.zs_expert_gather(None, tokens=most // 7 + 1, **{**gather, "choices": 7})
