"""GPU tests of the activation operators' dealings with autograd: what a call writes counts as
changed, and what backward adds to one buffer from several streams is added in order."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_mixed_buffer_amd as Z
    Z.lib()
    return Z


def _randn(shape, dtype, seed, sigma=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (sigma * torch.randn(shape, device="cuda", generator=g)).to(dtype)


# ------------------------------------------------------------------------------ versions

@pytest.mark.parametrize("how", ["act_pack", "y8", "h8"])
def test_refilled_checkpoint_is_noticed(Z, how):
    """A checkpoint filled anew while a layer's backward still needs it is an error there; filled
    anew after the backward, it serves the next pass."""
    xs = [_randn((8, 64), BF16, 1), _randn((8, 64), BF16, 2)]
    nw = torch.ones(64, dtype=BF16, device="cuda")
    w = _randn((16, 64), BF16, 3).requires_grad_()
    act = Z.Act8.empty(8, 64)

    def fill(x):
        if how == "act_pack":
            Z.act_pack(x, act)
        else:
            Z.rmsnorm(x, nw, **{how: act})

    fill(xs[0])
    y = Z.linear(xs[0], w, x8=act)
    fill(xs[1])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    for x in xs:
        fill(x)
        w.grad = None
        dy = _randn((8, 16), BF16, 4)
        Z.linear(x, w, x8=act).backward(dy)
        alone = torch.empty_like(w)
        Z.act_wgrad(act, dy, alone)
        assert torch.equal(w.grad, alone)


def test_overwritten_input_is_noticed(Z):
    x, w = _randn((8, 64), BF16, 5).requires_grad_(), _randn((64,), BF16, 6)
    a = x * 1
    loss = (a * a).sum()
    Z.rmsnorm(a.detach(), w, residual=_randn((8, 64), BF16, 7), h=a.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_mode(Z):
    """Tensors of inference mode, inside and outside of it: the same outputs."""
    x, w = _randn((8, 64), BF16, 8), _randn((64,), BF16, 9)
    y, act = torch.empty_like(x), Z.Act8.empty(8, 64)
    Z.rmsnorm(x, w, y=y, y8=act)
    with torch.inference_mode():
        y2, act2 = torch.empty_like(x), Z.Act8.empty(8, 64)
        Z.rmsnorm(x, w, y=y2, y8=act2)
        out = Z.norm(x, w, y8="e4m3")
    assert torch.equal(y, y2) and torch.equal(act.codes, act2.codes) and torch.equal(out.y, y)
    Z.rmsnorm(x, w, y=y2, y8=act2)
    assert torch.equal(act.unpack(), act2.unpack())
