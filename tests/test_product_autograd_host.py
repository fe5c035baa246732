"""CPU tests of what the products' layers tell autograd: the layers run on host tensors with the launch
itself replaced, so that no kernel runs."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

BF16 = torch.bfloat16
pytestmark = pytest.mark.filterwarnings("ignore::torch.jit.TracerWarning")


@pytest.fixture
def Z(monkeypatch):
    import zero_sharded_mixed_buffer_amd as Z
    for module in (Z.activations, Z.products):
        monkeypatch.setattr(module, "_need_gpu", lambda device: None)
        monkeypatch.setattr(module, "_enqueue", lambda name, device, *args: None)
    Z.lib()
    return Z


def _randn(*shape, seed=0, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _route(Z):
    as_int = dict(dtype=torch.int32)
    return Z.Route(torch.tensor([3, 6], **as_int), torch.arange(6, **as_int), torch.arange(6, **as_int).view(3, 2))


# each layer as a function of one of its inputs, and that input
LAYERS = {
    "linear8 of x": lambda Z: (lambda x: Z.linear8(x, _randn(5, 8)), _randn(6, 8)),
    "linear8 of the weight": lambda Z: (lambda w: Z.linear8(_randn(6, 8), w), _randn(5, 8)),
    "experts of x": lambda Z: (lambda x: Z.experts(x, _randn(2, 5, 8), _route(Z).ends), _randn(6, 8)),
    "experts of the weight": lambda Z: (lambda w: Z.experts(_randn(6, 8), w, _route(Z).ends), _randn(2, 5, 8)),
    "dispatch": lambda Z: (lambda x: Z.dispatch(x, _route(Z)), _randn(3, 8)),
    "combine of y": lambda Z: (lambda y: Z.combine(y, _route(Z), torch.ones(3, 2)), _randn(6, 8)),
    "combine of the weights": lambda Z: (lambda w: Z.combine(_randn(6, 8), _route(Z), w), _randn(3, 2, dtype=torch.float32)),
}


# ------------------------------------------------------------------------------ what is kept

def test_experts_keep_the_weight_for_the_inputs_gradient_alone(Z):
    """A weight may change before a backward pass that reads nothing of it, and not before another."""
    x, w = _randn(6, 8), _randn(2, 5, 8).requires_grad_()
    y = Z.experts(x, w, _route(Z).ends)
    with torch.no_grad():
        w.mul_(2)
    y.sum().backward()
    assert w.grad.shape == w.shape and w.grad.dtype == w.dtype
    y = Z.experts(x.requires_grad_(), w, _route(Z).ends)
    with torch.no_grad():
        w.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_combine_keeps_the_weights_for_the_rows_gradient_alone(Z):
    y, weights = _randn(6, 8), torch.ones(3, 2).requires_grad_()
    out = Z.combine(y, _route(Z), weights)
    with torch.no_grad():
        weights.mul_(2)
    out.sum().backward()
    assert weights.grad.shape == (3, 2)
    out = Z.combine(y.requires_grad_(), _route(Z), weights)
    with torch.no_grad():
        weights.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


# ------------------------------------------------------------------------------ other derivatives, traces

@pytest.mark.parametrize("layer", LAYERS)
@pytest.mark.parametrize("requires_grad", [False, True])
def test_forward_mode_is_refused(Z, layer, requires_grad):
    """No layer has a forward-mode derivative: a dual input is refused, as by torch's own functions
    without one, and its tangent does not get lost."""
    f, leaf = LAYERS[layer](Z)
    f(leaf)  # an ordinary one passes
    with fwd.dual_level():
        f(leaf)
        with pytest.raises(NotImplementedError, match="jvp"):
            f(fwd.make_dual(leaf.clone().requires_grad_(requires_grad), torch.ones_like(leaf)))
    with pytest.raises(RuntimeError):
        torch.func.jvp(f, (leaf,), (torch.ones_like(leaf),))


@pytest.mark.parametrize("layer", LAYERS)
@pytest.mark.parametrize("requires_grad", [False, True])
def test_a_trace_holds_the_layer(Z, monkeypatch, layer, requires_grad):
    """What a trace records is the layer's function, and not the allocation of its output alone: each call
    of it enqueues what a call of the layer does."""
    calls = []
    for module in (Z.activations, Z.products):
        monkeypatch.setattr(module, "_enqueue", lambda name, device, *args: calls.append(name))
    f, leaf = LAYERS[layer](Z)
    f(leaf)
    want, calls[:] = list(calls), []
    traced = torch.jit.trace(f, (leaf.requires_grad_(requires_grad),), check_trace=False)
    assert calls == want
    calls.clear()
    traced(leaf.detach())
    assert calls == want


def test_a_trace_routes_anew(Z, monkeypatch):
    """A traced function's route is the one of its present choices, for the layers behind it too."""
    def enqueue(name, device, *args):
        if name == "zs_route":
            routed.append(args[0])  # the choices' address
        elif name == "zs_expert_gather":
            gathered.append(args[3])  # the slots' address

    routed, gathered = [], []
    monkeypatch.setattr(Z.products, "_enqueue", enqueue)

    def f(x, ids):
        r = Z.route(ids, 2)
        return r.slot, Z.dispatch(x, r)

    x = _randn(3, 8)
    traced = torch.jit.trace(f, (x, torch.zeros(3, 2, dtype=torch.int64)), check_trace=False)
    for leaf in (x, x.clone().requires_grad_()):
        ids = torch.ones(3, 2, dtype=torch.int64)
        slot, out = traced(leaf, ids)
        assert routed[-1] == ids.data_ptr() and gathered[-1] == slot.data_ptr() and out.shape == (6, 8)


# ------------------------------------------------------------------------------ strides that mean nothing

def test_base_of_the_experts_gradients_has_the_strides_that_count(Z):
    """With one expert the stride between experts means nothing, with one row that between rows."""
    ends = torch.tensor([6], dtype=torch.int32)
    x, dy = _randn(6, 8), _randn(6, 5)
    dw = torch.empty(1, 5, 8, dtype=BF16)
    Z.expert_wgrad(x, dy, ends, dw, base=torch.empty(4, 5, 8, dtype=BF16)[:1].as_strided((1, 5, 8), (999, 8, 1)))
    one = _randn(6, 1)
    Z.expert_wgrad(x, one, ends, torch.empty(1, 1, 8, dtype=BF16), base=torch.empty(1, 1, 20, dtype=BF16)[:, :, :8])
    two = torch.tensor([2, 6], dtype=torch.int32)
    dw = torch.empty(2, 1, 8, dtype=BF16)
    Z.expert_wgrad(x, one, two, dw, base=torch.empty(2 * 8, dtype=BF16).as_strided((2, 1, 8), (8, 77, 1)))
    with pytest.raises(ValueError, match="same strides"):
        Z.expert_wgrad(x, one, two, dw, base=torch.empty(2, 2, 8, dtype=BF16)[:, :1])
    with pytest.raises(ValueError, match="same strides"):
        Z.expert_wgrad(x, dy, ends, torch.empty(1, 5, 8, dtype=BF16), base=torch.empty(1, 5, 9, dtype=BF16)[:, :, :8])
