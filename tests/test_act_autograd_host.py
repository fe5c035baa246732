"""CPU tests of what the activation operators tell autograd and of how they order streams: the
tensor-level calls run on host tensors with the launch itself replaced, so that no kernel runs."""

import contextlib

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


# ------------------------------------------------------------------------------ streams

class _Stream:
    """A stream that only logs what waits for what."""

    def __init__(self, name, log):
        self.name, self.log = name, log

    def __eq__(self, other):
        return isinstance(other, _Stream) and self.name == other.name

    def __ne__(self, other):
        return not self == other

    def wait_stream(self, other):
        self.log.append((self.name, "waits for", other.name))


class _Streams:
    """torch.cuda's current stream, by name, as the test sets it, and a log of launches and waits."""

    def __init__(self, monkeypatch, Z):
        self.log, self.name, self.capturing = [], "main", ()
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream(self.name, self.log))
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.name in self.capturing)
        monkeypatch.setattr(torch.cuda, "stream", self.entered)
        monkeypatch.setattr(Z.activations, "_enqueue", lambda name, device, *args: self.log.append((self.name, name)))

    @contextlib.contextmanager
    def entered(self, stream):
        outer, self.name = self.name, stream.name
        yield
        self.name = outer


def _node(streams, name, t):
    """t, whose gradient is computed with `name` as the current stream."""
    t.register_hook(lambda g: setattr(streams, "name", name))
    return t


def _ends_on(streams, name):
    """At the end of the pass the engine makes the caller's stream current again."""
    torch.autograd.Variable._execution_engine.queue_callback(lambda: setattr(streams, "name", name))


@pytest.mark.parametrize("what", ["linear", "norm"])
def test_additions_of_two_streams_are_ordered(Z, monkeypatch, what):
    """One buffer that two layers add to, their forwards on two streams: the second addition waits
    for the first, and the stream that called backward for both."""
    streams = _Streams(monkeypatch, Z)
    w = _randn(64, 64).requires_grad_() if what == "linear" else _randn(64).requires_grad_()
    into = torch.zeros_like(w, requires_grad=False)
    x = _randn(4, 64)
    outs = []
    for name in ("s1", "s2"):
        streams.name = name
        if what == "linear":
            outs.append(Z.linear(x, w, x8=_act(Z, 4, 64), grad_into=into))
        else:
            outs.append(Z.norm(x, w, grad_into=into).y)
    for _ in range(2):
        streams.name, streams.log[:] = "main", []
        total = outs[0].sum()
        _node(streams, "s1", outs[0])
        total = total + outs[1].sum()
        _node(streams, "s2", outs[1])
        total.register_hook(lambda g: _ends_on(streams, "main"))
        total.backward(retain_graph=True)
        call = "zs_act_wgrad" if what == "linear" else "zs_rmsnorm_backward"
        first, second = [a for a, b, *_ in streams.log if b == call]
        assert {first, second} == {"s1", "s2"}
        assert streams.log == [(first, call), (second, "waits for", first), (second, call),
                               ("main", "waits for", second)]


def test_one_stream_waits_for_nothing(Z, monkeypatch):
    streams = _Streams(monkeypatch, Z)
    w = _randn(64, 64).requires_grad_()
    into = torch.zeros(64, 64)
    x = _randn(4, 64)
    total = sum(Z.linear(x, w, x8=_act(Z, 4, 64), grad_into=into).sum() for _ in range(3))
    total.backward()
    assert [e for e in streams.log if e[1] != "zs_act_wgrad"] == []


def test_a_failed_pass_leaves_no_harm(Z, monkeypatch):
    """A pass that ends in an error leaves its stream behind as one to wait for, and no more."""
    streams = _Streams(monkeypatch, Z)
    w = _randn(64, 64).requires_grad_()
    into = torch.zeros(64, 64)
    x = _randn(4, 64).requires_grad_()

    def fail(grad):
        raise KeyError("from the test")

    y = x * 1
    y.register_hook(fail)
    streams.name = "s1"
    with pytest.raises(KeyError):
        Z.linear(y, w, x8=_act(Z, 4, 64), grad_into=into).sum().backward()
    for name in ("s2", "s2"):
        streams.name, streams.log[:] = name, []
        Z.linear(x, w, x8=_act(Z, 4, 64), grad_into=into).sum().backward()
        assert (name, "zs_act_wgrad") in streams.log
        assert all(e in (("s2", "waits for", "s1"), ("s2", "zs_act_wgrad")) for e in streams.log)


def test_captured_and_eager_streams_do_not_wait_for_each_other(Z, monkeypatch):
    """A wait between a stream that is being captured and one that is not would end the capture:
    there is none, nor for a stream whose capture has ended since."""
    streams = _Streams(monkeypatch, Z)
    A, into = Z.activations, torch.zeros(4)
    for name, streams.capturing in (("c1", ("c1",)), ("s1", ("c1", "c2")), ("c2", ("c1", "c2")), ("c1", ("c1", "c2")),
                                    ("c2", ("c2",))):
        def add(name=name):
            streams.name = name
            A._add_in_turn(into, lambda: streams.log.append((name, "adds")))
        x = torch.zeros(1, requires_grad=True)
        y = x * 1
        y.register_hook(lambda g: add())
        # the pass fails after its addition, so that its stream stays the last one
        x.register_hook(lambda g: 1 / 0)
        with pytest.raises(ZeroDivisionError):
            y.backward()
    assert streams.log == [("c1", "adds"), ("s1", "adds"), ("c2", "adds"), ("c1", "waits for", "c2"), ("c1", "adds"),
                           ("c2", "adds")]


# ------------------------------------------------------------------------------ checkpoints in a pool

def _pool(Z, layers, rows, cols):
    codes = torch.zeros(layers, rows, cols, dtype=torch.uint8)
    scales = torch.zeros(layers, rows, cols // 32, dtype=torch.uint8)
    return [Z.Act8(codes[i], scales[i], cols) for i in range(layers)]


def test_checkpoints_of_a_pool_are_marked_apart(Z):
    """Checkpoints whose arrays are parts of one tensor share its version: filling one leaves the
    others as they were, filling one anew is noticed by whichever handle it is done."""
    x, nw = _randn(8, 64), _randn(64)
    ws = [_randn(16, 64, seed=i).requires_grad_() for i in range(3)]
    for refill in (None, 0, 1, 2):
        acts = _pool(Z, 3, 8, 64)
        ys = []
        for i, w in enumerate(ws):
            if i == 1:
                Z.rmsnorm(x, nw, y8=acts[i])
            else:
                Z.act_pack(x, acts[i])
            ys.append(Z.linear(x, w, x8=acts[i]))
        if refill is not None:
            Z.act_pack(x, Z.Act8(acts[refill].codes, acts[refill].scales, 64))
        for i, y in enumerate(ys):
            if i == refill:
                with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                    y.sum().backward()
            else:
                y.sum().backward()
    ys = [Z.linear(x, ws[0], x8=acts[0])]
    acts[0].codes.zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        ys[0].sum().backward()


def test_half_pooled_checkpoints(Z):
    """Codes of their own with scales in a pool, and the other way round."""
    x, w = _randn(8, 64), _randn(16, 64).requires_grad_()
    own = [torch.zeros(8, 64, dtype=torch.uint8) for _ in range(2)], [torch.zeros(8, 2, dtype=torch.uint8) for _ in range(2)]
    pool = torch.zeros(2, 8, 64, dtype=torch.uint8), torch.zeros(2, 8, 2, dtype=torch.uint8)
    for codes, scales in ((own[0], pool[1]), (pool[0], own[1])):
        acts = [Z.Act8(codes[i], scales[i], 64) for i in range(2)]
        ys = []
        for act in acts:
            Z.act_pack(x, act)
            ys.append(Z.linear(x, w, x8=act))
        Z.act_pack(x, acts[1])
        ys[0].sum().backward()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            ys[1].sum().backward()


# ------------------------------------------------------------------------------ a checkpoint and its tensor

def _y8(Z, x, nw):
    out = Z.norm(x, nw, y8="e4m3")
    return out.y, out.y8


@pytest.mark.parametrize("how", ["norm", "of", "act_pack", "rmsnorm_y8", "rmsnorm_h8", "rmsnorm_h8_of_x"])
def test_checkpoint_of_a_tensor_changed_since_is_refused(Z, how):
    """linear would multiply by what the tensor holds now and differentiate what it held then."""
    x, nw, w = _randn(2, 4, 64), _randn(64), _randn(8, 64).requires_grad_()
    flat, act = x.view(8, 64), _act(Z, 8, 64)
    t = x
    if how == "norm":
        t, act = _y8(Z, x.requires_grad_(), nw)
    elif how == "of":
        act = Z.Act8.of(flat)
    elif how == "act_pack":
        Z.act_pack(flat, act)
    else:
        t = torch.empty_like(x)
        if how == "rmsnorm_y8":
            Z.rmsnorm(flat, nw, y=t.view(8, 64), y8=act)
        elif how == "rmsnorm_h8":
            Z.rmsnorm(flat, nw, residual=_randn(8, 64), h=t.view(8, 64), h8=act)
        else:
            t = x
            Z.rmsnorm(flat, nw, h8=act)
    for view in (t, t.view(8, 64), t.detach()):
        torch.autograd.grad(Z.linear(view, w, x8=act).sum(), w)
    with torch.no_grad():
        t.mul_(2)
    for view in (t, t.view(8, 64), t.detach()):
        with pytest.raises(ValueError, match="changed"):
            Z.linear(view, w, x8=act)
    with torch.no_grad():
        t.div_(2)
        Z.act_pack(t.view(8, 64), act)  # the checkpoint of what it holds now
    Z.linear(t, w, x8=act).sum().backward()
    frozen = w.detach()
    with torch.no_grad():
        t.mul_(2)
    Z.linear(t, frozen, x8=act)  # nothing is differentiated by the checkpoint


def test_change_through_the_library_is_a_change(Z):
    x, w = _randn(8, 64), _randn(8, 64).requires_grad_()
    act = Z.Act8.of(x)
    Z.act_unpack(_act(Z, 8, 64), x)
    with pytest.raises(ValueError, match="changed"):
        Z.linear(x, w, x8=act)


def test_checkpoints_of_copies_and_plain_arrays_are_taken(Z):
    """What cannot be known is the caller's: a copy, arrays made elsewhere, a tensor without versions,
    one that lies where a freed one lay."""
    x, w = _randn(8, 64), _randn(8, 64).requires_grad_()
    act = Z.Act8.of(x)
    Z.linear(x.clone(), w, x8=act).sum().backward()
    Z.linear(x.data, w, x8=act).sum().backward()
    x.mul_(2)
    Z.linear(x.clone(), w, x8=act).sum().backward()
    Z.linear(x, w, x8=Z.Act8(act.codes, act.scales, 64)).sum().backward()
    act.codes.copy_(act.codes.clone())  # read back from somewhere, for what x holds now
    Z.linear(x, w, x8=act).sum().backward()
    parts = torch.zeros(2, 8, 64, dtype=BF16)
    act = Z.Act8.of(parts[0])
    parts[1].add_(1)
    Z.linear(parts[0], w, x8=act).sum().backward()
    with torch.inference_mode():
        z = _randn(8, 64)
        act = Z.Act8.of(z)
    assert act.unpack().shape == (8, 64)
    x = _randn(8, 64)
    act = Z.Act8.of(x)
    at = x.data_ptr()
    del x
    for _ in range(50):
        again = torch.zeros(8, 64, dtype=BF16)
        again.add_(1)
        Z.linear(again, w, x8=act)
        if again.data_ptr() == at:
            break


def test_checkpoint_does_not_keep_its_tensor(Z):
    import weakref
    x = _randn(8, 64)
    storage = x.untyped_storage()
    act = Z.Act8.of(x)
    alive = weakref.ref(storage)
    del x, storage
    assert alive() is None
    assert act.nbytes == 8 * 66


# ------------------------------------------------------------------------------ empty layers

def test_linear_without_outputs(Z):
    """A weight of no rows: an empty product, whose backward has nothing to add (it was refused in the
    middle of the pass)."""
    x, w = _randn(8, 64).requires_grad_(), torch.zeros(0, 64, dtype=BF16, requires_grad=True)
    for grad_into in (None, torch.zeros(0, 64)):
        y = Z.linear(x, w, grad_into=grad_into)
        assert y.shape == (8, 0)
        y.sum().backward()
        assert x.grad.shape == (8, 64) and not x.grad.any()


def test_buffers_apart_wait_for_nothing(Z, monkeypatch):
    """Additions to two buffers on two streams have no order; two parts of one buffer have."""
    for shared in (False, True):
        streams = _Streams(monkeypatch, Z)
        w = _randn(64, 64).requires_grad_()
        flat = torch.zeros(2, 64, 64)
        intos = [flat[0], flat[1]] if shared else [torch.zeros(64, 64), torch.zeros(64, 64)]
        x = _randn(4, 64)
        outs = [Z.linear(x, w, x8=_act(Z, 4, 64), grad_into=into) for into in intos]
        total = sum(o.sum() for o in outs)
        for o, name in zip(outs, ("s1", "s2")):
            _node(streams, name, o)
        total.register_hook(lambda g: _ends_on(streams, "main"))
        total.backward()
        assert ("s1", "zs_act_wgrad") in streams.log and ("s2", "zs_act_wgrad") in streams.log
        waits = {e for e in streams.log if "waits for" in e}
        if shared:
            assert waits in ({("s2", "waits for", "s1"), ("main", "waits for", "s2")},
                             {("s1", "waits for", "s2"), ("main", "waits for", "s1")})
        else:
            assert waits == {("main", "waits for", "s1"), ("main", "waits for", "s2")}
