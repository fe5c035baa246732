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


def test_outputs_in_an_inputs_place_are_refused(Z):
    """Rows are written while others still read them: an output that begins where an input does is
    refused, but for those that the calls name."""
    def refused(fn, good, **bad):
        with pytest.raises(Z.ZsInvalidArgument, match="same memory|in place of"):
            fn(**{**good, **bad}, stream=0)

    x, w, y = P, 2 * P, 3 * P
    product = dict(x=x, x_stride=64, weight=w, w_stride=64, w_expert_stride=64 * 64, dtype=BF16, ends=P, experts=2, rows=9, cols=64,
                   outs=64, in_major=False, y=y, y_stride=64)
    for in_major in (False, True):
        refused(Z.zs_expert_product, product, y=x, in_major=in_major)
        refused(Z.zs_expert_product, product, y=w, in_major=in_major)
    wgrad = dict(x=x, x_stride=64, dy=w, dy_stride=64, dtype=BF16, ends=P, experts=2, rows=9, cols=64, outs=64, dw=y, dw_dtype=BF16,
                 dw_stride=64, dw_expert_stride=64 * 64)
    refused(Z.zs_expert_wgrad, wgrad, dw=x)
    refused(Z.zs_expert_wgrad, wgrad, dw=w)
    gather = dict(x=x, x_stride=64, dtype=BF16, slot=P, tokens=5, choices=1, cols=64, out=x, out_stride=64)
    refused(Z.zs_expert_gather, gather)
    combine = dict(y=x, y_stride=64, dtype=BF16, place=P, weights=None, tokens=5, choices=1, cols=64, out=x, out_stride=64)
    refused(Z.zs_expert_combine, combine)
    backward = dict(dout=x, dout_stride=64, y=y, y_stride=64, dtype=BF16, slot=P, place=P, weights=P, tokens=5, choices=1, cols=64,
                    dy=x, dy_stride=64)
    refused(Z.zs_expert_combine_backward, backward)
    refused(Z.zs_weight8_pack, dict(src=x, src_dtype=BF16, src_stride=64, outs=48, cols=64, w8=Z.Weight8Arrays(w, w, y)))
    refused(Z.zs_product8, dict(x8=Z.ActArrays(x, w, 0, 0), rows=4, w8=Z.Weight8Arrays(y, None, 4 * P), outs=48, cols=64,
                                transposed=False, y=x, y_dtype=BF16, y_stride=64))
