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


def test_checkpoint_of_a_tensor_changed_since_is_refused(Z):
    x, nw = _randn((8, 64), BF16, 31).requires_grad_(), torch.ones(64, dtype=BF16, device="cuda")
    w = _randn((16, 64), BF16, 32).requires_grad_()
    out = Z.norm(x, nw, y8="e4m3")
    Z.linear(out.y.view(2, 4, 64), w, x8=out.y8)
    out.y.mul_(2)
    with pytest.raises(ValueError, match="changed"):
        Z.linear(out.y, w, x8=out.y8)
    Z.act_pack(out.y.detach(), out.y8)
    dy = _randn((8, 16), BF16, 33)
    Z.linear(out.y, w, x8=out.y8).backward(dy)
    alone = torch.empty_like(w)
    Z.act_wgrad(Z.Act8.of(out.y.detach()), dy, alone)
    assert torch.equal(w.grad, alone) and x.grad is not None


def test_checkpoints_of_a_pool(Z):
    """Three layers' checkpoints as parts of one allocation, filled in turn: each backward takes its
    own; one filled anew is an error."""
    codes = torch.empty(3, 8, 64, dtype=torch.uint8, device="cuda")
    scales = torch.empty(3, 8, 2, dtype=torch.uint8, device="cuda")
    acts = [Z.Act8(codes[i], scales[i], 64) for i in range(3)]
    xs = [_randn((8, 64), BF16, 41 + i) for i in range(3)]
    ws = [_randn((16, 64), BF16, 51 + i).requires_grad_() for i in range(3)]
    dy = _randn((8, 16), BF16, 61)

    def forward():
        ys = []
        for x, w, act in zip(xs, ws, acts):
            Z.act_pack(x, act)
            ys.append(Z.linear(x, w, x8=act))
        return ys

    for x, w, y in zip(xs, ws, forward()):
        y.backward(dy)
        alone = torch.empty_like(w)
        Z.act_wgrad(Z.Act8.of(x), dy, alone)
        assert torch.equal(w.grad, alone)
    ys = forward()
    Z.act_pack(xs[0], acts[1])
    ys[0].backward(dy)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        ys[1].backward(dy)


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


# ------------------------------------------------------------------------------ streams

def _busy(n=6):
    """A few milliseconds of products on the current stream."""
    a = torch.ones(8192, 8192, dtype=BF16, device="cuda")
    for _ in range(n):
        a = torch.mm(a, a)
    return a


@pytest.mark.parametrize("what", ["linear", "norm"])
@pytest.mark.parametrize("late", [0, 1])
def test_additions_of_two_streams(Z, what, late):
    """One weight, two micro-batches on two streams, one of which is busy when backward begins:
    both gradients are in the buffer when the calling stream reads it, at once, after backward."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    gen = torch.Generator("cuda").manual_seed(11)
    xs = [torch.randint(-3, 4, (64, 96), device="cuda", generator=gen).to(BF16) for _ in range(2)]
    dys = [torch.randint(-2, 3, (64, 96), device="cuda", generator=gen).to(BF16) for _ in range(2)]
    w = torch.ones((96, 96) if what == "linear" else (96,), dtype=BF16, device="cuda", requires_grad=True)
    into = torch.zeros(w.shape, device="cuda")

    def forward(x, buffer):
        if what == "linear":
            return Z.linear(x, w, code="int8", grad_into=buffer)
        return Z.norm(x, w, eps=1e-5, save="int8", grad_into=buffer).y

    parts = []
    for x, dy in zip(xs, dys):
        alone = torch.zeros_like(into)
        forward(x, alone).backward(dy)
        parts.append(alone)
    # the buffer is added to the second part's fp32 sum in one rounding, as here, in either order
    want = parts[0] + parts[1]
    torch.cuda.synchronize()
    for turn in range(4):
        into.zero_()
        ys = []
        for s, x in zip(streams, xs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                ys.append(forward(x, into))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        with torch.cuda.stream(streams[late]):
            _busy()
        if turn % 2:
            torch.autograd.backward(ys, dys)
        else:
            for y, dy in zip(ys, dys):
                y.backward(dy)
        got = into.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, want), turn
        assert w.grad is None
    adds = into.untyped_storage()._adds
    assert adds.last is None and adds.under_way == 0


def test_captured_additions_of_two_streams(Z):
    """The same captured into one graph, replayed with changing gradients."""
    side = torch.cuda.Stream()
    gen = torch.Generator("cuda").manual_seed(12)
    xs = [torch.randint(-3, 4, (64, 96), device="cuda", generator=gen).to(BF16) for _ in range(2)]
    dys = [torch.zeros(64, 40, dtype=BF16, device="cuda") for _ in range(2)]
    w = torch.ones(40, 96, dtype=BF16, device="cuda", requires_grad=True)
    into = torch.zeros(40, 96, device="cuda")

    def run():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        ys = [Z.linear(xs[0], w, code="int8", grad_into=into)]
        with torch.cuda.stream(side):
            ys.append(Z.linear(xs[1], w, code="int8", grad_into=into))
        main.wait_stream(side)
        torch.autograd.backward(ys, dys)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        run()
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for turn in range(4):
        for dy in dys:
            dy.copy_(torch.randint(-2, 3, dy.shape, device="cuda", generator=gen).to(BF16))
        into.zero_()
        graph.replay()
        if turn % 2:
            _busy(1)
        torch.cuda.synchronize()
        want = sum(dy.double().t().contiguous() @ x.double() for x, dy in zip(xs, dys))
        assert torch.equal(into.double(), want), turn


def test_several_host_threads_finish(Z):
    """Four host threads, each with a layer, a stream and a buffer of its own: every one of them ends,
    after all of its rounds, with the gradients that it has alone."""
    import threading
    rounds, count = 8, [0] * 4
    xs = [_randn((64 + 16 * i, 96), BF16, 71 + i) for i in range(4)]
    ws = [_randn((40, 96), BF16, 81 + i).requires_grad_() for i in range(4)]
    intos = [torch.zeros(40, 96, device="cuda") for _ in range(4)]

    def step(i):
        intos[i].zero_()
        Z.linear(xs[i], ws[i], grad_into=intos[i]).float().square().sum().backward()
        return intos[i].clone()

    want = [step(i) for i in range(4)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(rounds):
                got = step(i)
                stream.synchronize()
                if not torch.equal(got, want[i]):
                    wrong.append(i)
                count[i] += 1

    threads = [threading.Thread(target=work, args=(i,), daemon=True) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(30)
    assert not any(t.is_alive() for t in threads)
    assert count == [rounds] * 4 and not wrong


# ------------------------------------------------------------------------------ recomputation

@pytest.mark.parametrize("reentrant", [True, False])
def test_recomputed_layers(Z, reentrant):
    """A norm and two layers under torch's activation checkpointing, alone and one inside the other's
    pass, with gradients in one flat buffer and by autograd: the same gradients as without."""
    from torch.utils.checkpoint import checkpoint
    x0 = _randn((4, 24, 64), BF16, 91)
    nw = (1 + _randn((64,), BF16, 92, 0.1)).requires_grad_()
    ws = [_randn((64, 64), BF16, 93 + i, 0.1).requires_grad_() for i in range(2)]
    flat = torch.zeros(64 + 64 * 64, device="cuda")
    intos = [flat[:64], flat[64:].view(64, 64)]
    dy = _randn((4, 24, 64), BF16, 99)

    def block(x):
        out = Z.norm(x, nw, residual=x, y8="int8", grad_into=intos[0])
        return Z.linear(Z.linear(out.y, ws[0], x8=out.y8, grad_into=intos[1]), ws[1]) + out.h

    def run(wrapped):
        flat.zero_()
        ws[1].grad = None
        x = x0.clone().requires_grad_()
        y = x * 1
        for _ in range(2):
            y = checkpoint(block, y, use_reentrant=reentrant) if wrapped else block(y)
        y.backward(dy)
        assert nw.grad is None and ws[0].grad is None
        return x.grad, ws[1].grad.clone(), flat.clone()

    want = run(False)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(run(True), want))
    adds = flat.untyped_storage()._adds
    assert adds.last is None and adds.under_way == 0
