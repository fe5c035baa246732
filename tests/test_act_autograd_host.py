"""CPU tests of what the activation operators tell autograd and of how they order streams: the
tensor-level calls run on host tensors with the launch itself replaced, so that no kernel runs."""

import pytest
import torch

BF16 = torch.bfloat16


@pytest.fixture
def Z(monkeypatch):
    import zero_sharded_mixed_buffer_amd as Z
    monkeypatch.setattr(Z.activations, "_need_gpu", lambda device: None)
    monkeypatch.setattr(Z.activations, "_enqueue", lambda name, device, *args: None)
    Z.lib()
    return Z


def _randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF16)


def _act(Z, rows, cols, code="e4m3"):
    act = Z.Act8.empty(rows, cols, code, "cpu")
    act.codes.zero_()
    act.scales.zero_()
    return act


# ------------------------------------------------------------------------------ versions

def _versions(*tensors):
    return [t._version for t in tensors]


def test_every_written_tensor_gets_a_new_version(Z):
    """What a call writes is marked as changed, as torch's own writes are; what it reads is not."""
    x, r, w, dy = _randn(4, 64), _randn(4, 64), _randn(64), _randn(4, 24)
    act, other = _act(Z, 4, 64), _act(Z, 4, 64, "int8")
    h, y, dx, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(4)
    flat = torch.zeros(24 * 64 + 64)
    dw, dweight = flat[:24 * 64].view(24, 64), flat[24 * 64:]
    scratch = torch.zeros(1 << 20, dtype=torch.uint8)

    def marks(written, read, call):
        for a in (act, other):
            read = [*read, *(t for t in (a.codes, a.scales) if not any(t is u for u in written))]
        before, still = _versions(*written), _versions(*read)
        call()
        assert all(a > b for a, b in zip(_versions(*written), before))
        assert _versions(*read) == still

    marks([act.codes, act.scales], [x], lambda: Z.act_pack(x, act))
    marks([y], [], lambda: Z.act_unpack(act, y))
    marks([h, y, rstd, act.codes, act.scales, other.codes, other.scales], [x, r, w],
          lambda: Z.rmsnorm(x, w, residual=r, h=h, y=y, y8=act, h8=other, rstd=rstd))
    marks([y], [x, w, h, rstd], lambda: Z.rmsnorm(x, w, y=y))
    marks([r], [x, w], lambda: Z.rmsnorm(x, w, residual=r, h=r))
    marks([dx, dweight, flat, scratch], [x, h, w, rstd],
          lambda: Z.rmsnorm_backward(x, h, w, rstd, dx, dweight=dweight, base=dweight, workspace=scratch))
    marks([dx], [x, w, rstd, flat, scratch],
          lambda: Z.rmsnorm_backward(x, act, w, rstd, dx, workspace=scratch))
    marks([dw, flat, scratch], [dy], lambda: Z.act_wgrad(act, dy, dw, workspace=scratch))


@pytest.mark.parametrize("how", ["act_pack", "y8", "h8"])
def test_refilled_checkpoint_is_noticed(Z, how):
    """A checkpoint that a layer's backward still needs and that is filled anew before it."""
    x, x2, nw = _randn(8, 64), _randn(8, 64, seed=1), _randn(64, seed=2)
    w = _randn(16, 64, seed=3).requires_grad_()
    act = _act(Z, 8, 64)
    Z.act_pack(x, act)
    y = Z.linear(x, w, x8=act)
    if how == "act_pack":
        Z.act_pack(x2, act)
    else:
        Z.rmsnorm(x2, nw, **{how: act})
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_overwritten_input_is_noticed(Z):
    """A tensor that autograd saved and that a norm then writes its sum into."""
    x, w = _randn(8, 64).requires_grad_(), _randn(64)
    a = x * 1
    loss = (a * a).sum()
    Z.rmsnorm(a.detach(), w, residual=_randn(8, 64), h=a.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    b = x * 1
    out = Z.norm(b, w.requires_grad_(), save=None)
    Z.act_unpack(_act(Z, 8, 64), b.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.y.sum().backward()


def test_inference_tensors_are_written(Z):
    """Tensors made in inference mode have no version; the calls take them there and outside."""
    with torch.inference_mode():
        x, w, y = _randn(4, 64), _randn(64), torch.empty(4, 64, dtype=BF16)
        act = _act(Z, 4, 64)
        Z.rmsnorm(x, w, y=y, y8=act)
    Z.rmsnorm(x, w, y=y, y8=act)
    Z.act_unpack(act, y)
