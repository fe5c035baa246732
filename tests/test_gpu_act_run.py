"""GPU tests of the activation operators as a training program uses them: under autograd, with
gradients in the optimizer's flat buffer, on several streams and captured into graphs."""

import pytest
import torch

from oracle import act_oracle as AO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_mixed_buffer_amd as Z
    Z.lib()
    return Z


def _randn(shape, dtype, seed, sigma=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (sigma * torch.randn(shape, device="cuda", generator=g)).to(dtype)


def _close(got, want, rel, what):
    """Largest error against the largest value: `rel` is a sum of roundings of that size."""
    got, want = got.detach().cpu().double(), want.detach().cpu().double()
    err, top = float((got - want).abs().max()), float(want.abs().max())
    assert err <= rel * top, f"{what}: {err:.3e} of {top:.3e}"


# ------------------------------------------------------------------------------ autograd

@pytest.mark.parametrize("save", ["e4m3", "int8", None])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", [(6, 100), (2, 5, 64), (33, 4096)])
def test_norm_gradients(Z, shape, dtype, save):
    """The gradients of norm are the formula's, on the checkpoint's values where one is kept."""
    x, r = _randn(shape, dtype, 1).requires_grad_(), _randn(shape, dtype, 2).requires_grad_()
    w = _randn((shape[-1],), dtype, 3).requires_grad_()
    out = Z.norm(x, w, eps=1e-5, residual=r, save=save, y8="e4m3")
    dy, dh = _randn(shape, dtype, 4), _randn(shape, dtype, 5)
    torch.autograd.backward([out.y, out.h], [dy, dh])
    h64, rstd64, y64 = AO.norm(x.detach().view(-1, shape[-1]), w.detach(), 1e-5, r.detach().view(-1, shape[-1]))
    eps = torch.finfo(dtype).eps
    assert torch.equal(out.h.detach().cpu().view(-1, shape[-1]), h64)
    _close(out.y.view(-1, shape[-1]), y64, eps / 2 * 1.01, "y")
    assert (out.y8.rows, out.y8.cols, out.y8.code) == (h64.shape[0], shape[-1], "e4m3")
    seen = h64.double() if save is None else AO.values(*AO.quantise(h64, save), shape[-1], save)
    dx64, dw64 = AO.norm_backward(dy.view(-1, shape[-1]), seen, w.detach(), rstd64.float(), dh.view(-1, shape[-1]))
    # one last rounding, and fp32 sums of up to 4096 terms in 45 sequential steps at most
    _close(x.grad.view(-1, shape[-1]), dx64, eps / 2 * 1.01 + 100 * U, "x.grad")
    assert torch.equal(x.grad, r.grad)
    _close(w.grad, dw64, eps / 2 * 1.01 + 100 * U, "w.grad")


def test_norm_partial_gradients(Z):
    """Only y, only h, and no residual."""
    w = torch.ones(64, dtype=BF16, device="cuda", requires_grad=True)
    for use in ("y", "h"):
        x, r = _randn((4, 64), BF16, 11).requires_grad_(), _randn((4, 64), BF16, 12).requires_grad_()
        out = Z.norm(x, w, residual=r)
        g = _randn((4, 64), BF16, 13)
        getattr(out, use).backward(g)
        if use == "h":
            assert torch.equal(x.grad, g) and torch.equal(r.grad, g) and w.grad is None
        else:
            assert x.grad is not None and torch.equal(x.grad, r.grad) and w.grad is not None
        w.grad = None
    x = _randn((4, 64), BF16, 14).requires_grad_()
    out = Z.norm(x, w)
    assert out.h is x and out.y8 is None
    out.y.sum().backward()
    assert x.grad.shape == x.shape


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape,outs", [((5, 40), 24), ((3, 7, 96), 130), ((300, 256), 64)])
def test_linear_gradients(Z, shape, outs, dtype, code):
    x = _randn(shape, dtype, 21).requires_grad_()
    w = _randn((outs, shape[-1]), dtype, 22, 0.1).requires_grad_()
    y = Z.linear(x, w, code=code)
    dy = _randn(y.shape, dtype, 23)
    y.backward(dy)
    flat, dflat = x.detach().view(-1, shape[-1]), dy.view(-1, outs)
    eps = torch.finfo(dtype).eps
    n = flat.shape[0]
    seen = AO.values(*AO.quantise(flat, code), shape[-1], code)
    dw64 = AO.wgrad(dflat, seen)
    mags = float((dflat.cpu().double().abs().t() @ seen.abs()).max())
    err = float((w.grad.cpu().double() - dw64).abs().max())
    assert err <= eps / 2 * 1.01 * float(dw64.abs().max()) + 2 * U * (n + 8) * mags
    # the library's product: one rounding, and sums of at most 256 terms
    _close(y.view(-1, outs), flat.cpu().double() @ w.detach().cpu().double().t(), eps / 2 * 1.01 + 512 * U, "y")
    _close(x.grad.view(-1, shape[-1]), dflat.cpu().double() @ w.detach().cpu().double(), eps / 2 * 1.01 + 512 * U, "dx")


def test_grad_into_accumulates(Z):
    """With grad_into the gradient is added to the buffer, in its type, and autograd gives none."""
    x = _randn((50, 96), BF16, 31)
    w = _randn((40, 96), BF16, 32, 0.1).requires_grad_()
    nw = _randn((96,), BF16, 33).requires_grad_()
    plain, into = [], []
    for _ in range(2):
        out = Z.norm(x, nw, y8="int8")
        Z.linear(out.y, w, x8=out.y8).float().square().sum().backward()
    plain = [w.grad.clone(), nw.grad.clone()]
    w.grad = nw.grad = None
    for buf_dtype in (torch.float32, BF16):
        bw, bn = torch.zeros(40, 96, dtype=buf_dtype, device="cuda"), torch.zeros(96, dtype=buf_dtype, device="cuda")
        for _ in range(2):
            out = Z.norm(x, nw, y8="int8", grad_into=bn)
            Z.linear(out.y, w, x8=out.y8, grad_into=bw).float().square().sum().backward()
        assert w.grad is None and nw.grad is None
        # two bf16 roundings of the gradient and one of the sum, or one sum in fp32
        _close(bw, plain[0], 3 * 2.0 ** -8, "linear")
        _close(bn, plain[1], 3 * 2.0 ** -8, "norm")


def test_broadcast_inputs_and_gradients(Z):
    """Inputs that are one row seen many times, and gradients that arrive that way (from a sum over
    rows), with a residual of the same kind: as their copies give."""
    row, row2 = _randn((1, 96), BF16, 301), _randn((96,), BF16, 302)
    nw, w = _randn((96,), BF16, 303), _randn((24, 96), BF16, 304, 0.1)
    g, gy = _randn((96,), BF16, 305), _randn((24,), BF16, 306)

    def run(copy):
        x, r = row.clone().requires_grad_(), row2.clone().requires_grad_()
        a, b = nw.clone().requires_grad_(), w.clone().requires_grad_()
        wide, wide2 = x.expand(50, 96), r.expand(50, 96)
        if copy:
            wide, wide2 = wide.contiguous(), wide2.contiguous()
        out = Z.norm(wide, a, residual=wide2, y8="int8")
        out.y.sum(0).backward(g, retain_graph=True)
        out.h.sum(0).backward(g, retain_graph=True)
        Z.linear(out.y, b, x8=out.y8).sum(0).backward(gy)
        Z.linear(wide, b).sum(0).backward(gy)
        return [t.grad for t in (x, r, a, b)]

    for p, q in zip(run(False), run(True)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("shape", [(12, 64), (3, 4, 64)])
def test_outputs_may_be_changed_in_place(Z, shape):
    """y and h are tensors of their own: changing them in place is an operation like any other,
    and the saved checkpoint does not notice."""
    x, r = _randn(shape, BF16, 311).requires_grad_(), _randn(shape, BF16, 312).requires_grad_()
    w = _randn((64,), BF16, 313).requires_grad_()
    g = _randn(shape, BF16, 314)
    grads = []
    for in_place in (False, True):
        out = Z.norm(x, w, residual=r)
        if in_place:
            y, h = out.y.mul_(2), out.h.mul_(4)
        else:
            y, h = out.y * 2, out.h * 4
        torch.autograd.backward([y, h], [g, g])
        grads.append([t.grad.clone() for t in (x, r, w)])
        x.grad = r.grad = w.grad = None
    assert all(torch.equal(a, b) for a, b in zip(*grads))


def test_layers_share_a_checkpoint(Z):
    """Two layers read one norm's output and its one checkpoint; a frozen layer keeps nothing; the
    gradients of a sum's two terms are tensors of their own."""
    x, r = _randn((40, 96), BF16, 36).requires_grad_(), _randn((40, 96), BF16, 37).requires_grad_()
    nw = torch.ones(96, dtype=BF16, device="cuda")
    ws = [_randn((24, 96), BF16, 38, 0.1).requires_grad_(), _randn((56, 96), BF16, 39, 0.1).requires_grad_()]
    frozen = _randn((8, 96), BF16, 40, 0.1)
    out = Z.norm(x, nw, residual=r, y8="int8")
    ys = [Z.linear(out.y, w, x8=out.y8) for w in ws] + [Z.linear(out.y, frozen)]
    dys = [_randn(y.shape, BF16, 44 + i) for i, y in enumerate(ys)]
    torch.autograd.backward(ys, dys)
    for w, dy in zip(ws, dys):
        alone = torch.empty_like(w)
        Z.act_wgrad(out.y8, dy, alone)
        assert torch.equal(w.grad, alone)
    assert torch.equal(x.grad, r.grad) and x.grad.data_ptr() != r.grad.data_ptr()
    with torch.no_grad():
        assert torch.equal(Z.linear(out.y, ws[0]), ys[0])
        same = Z.norm(x, nw, residual=r, y8="int8")
        assert torch.equal(same.y, out.y) and torch.equal(same.h, out.h) and torch.equal(same.y8.codes, out.y8.codes)


def test_changed_checkpoint_is_noticed(Z):
    x = _randn((8, 64), BF16, 41)
    w = _randn((16, 64), BF16, 42).requires_grad_()
    act = Z.Act8.of(x)
    y = Z.linear(x, w, x8=act)
    act.codes.zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


# ------------------------------------------------------------------------------ with the optimizer

def _block(Z, x, p, into):
    """Two pre-norm residual layers of one linear each and a last norm: operators in a row, each
    reading the checkpoint that the one before it wrote."""
    g = (lambda i: p[i].grad) if into else (lambda i: None)
    h = x
    branch = None
    for i in (0, 2):
        out = Z.norm(h if branch is None else branch, p[i], residual=None if branch is None else h, y8="int8",
                     save="int8", grad_into=g(i))
        h = out.h
        branch = Z.linear(out.y, p[i + 1], x8=out.y8, grad_into=g(i + 1))
    return Z.norm(branch, p[4], residual=h, save="int8", grad_into=g(4)).y


def _params():
    shapes = [(64,), (64, 64), (64,), (64, 64), (64,)]
    return [torch.nn.Parameter(_randn(s, BF16, 50 + i, 0.2) + (1 if len(s) == 1 else 0)) for i, s in enumerate(shapes)]


def test_training_step_in_the_flat_buffer(Z):
    """Backward writes every weight's gradient into the optimizer's flat buffer, over two
    micro-steps, and the step takes it from there: the same parameters as an optimizer that is
    handed the same gradients as a list."""
    p = _params()
    opt = Z.ZeroShardedAdamW(p, lr=1e-2, flat_views=True)
    q = [t.detach().clone() for t in p]
    ref = Z.ZeroShardedAdamW(q, lr=1e-2)
    for step in range(3):
        opt.zero_grad()
        for micro in range(2):
            x = _randn((4, 32, 64), BF16, 60 + 2 * step + micro)
            _block(Z, x, p, True).float().square().mean().backward()
        grads = [t.grad.clone() for t in p]
        assert all(t.grad.data_ptr() == v.data_ptr() for t, v in zip(p, opt._grad_views))
        assert all(bool(t.abs().max() > 0) for t in grads)
        opt.step()
        ref.step(grads)
        for a, b in zip(p, q):
            assert torch.equal(a.detach(), b)
    assert opt.read_state()["step_t"] == 3
    opt.close()
    ref.close()


def test_block_gradients_against_a_plain_block(Z):
    """The block's gradients beside those of the same block in fp32 with plain autograd.  The
    checkpoints move each by the codes' rounding: int8 of 32 columns is good to 2^-7 of the
    group's largest value, so 2^-5 in all over the five weights' and norms' readings."""
    x = _randn((256, 64), BF16, 71)
    p = _params()
    _block(Z, x, p, False).float().square().mean().backward()

    def rms(v, w):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w

    f = [t.detach().float().requires_grad_() for t in p]
    h = x.float()
    branch = rms(h, f[0]) @ f[1].t()
    h = h + branch
    branch = rms(h, f[2]) @ f[3].t()
    h = h + branch
    rms(h, f[4]).square().mean().backward()
    for i, (a, b) in enumerate(zip(p, f)):
        err = float((a.grad.float() - b.grad).norm() / b.grad.norm())
        assert err <= 2.0 ** -5, (i, err)


def test_an_infinite_activation_skips_the_step(Z):
    """An infinity in an activation reaches the weight's gradient through its checkpoint as NaN,
    and the step is skipped."""
    p = _params()
    opt = Z.ZeroShardedAdamW(p, flat_views=True)
    before = [t.detach().clone() for t in p]
    opt.zero_grad()
    x = _randn((16, 64), BF16, 81)
    x[3, 5] = float("inf")
    act = Z.Act8.of(x)
    Z.act_wgrad(act, _randn((16, 64), BF16, 82), p[1].grad, base=p[1].grad)
    opt.step()
    assert opt.read_state()["overflow"] == 1 and opt.read_state()["step_t"] == 0
    assert all(torch.equal(a.detach(), b) for a, b in zip(p, before))
    opt.close()


# ------------------------------------------------------------------------------ streams and graphs

def _chain(Z, s):
    """One norm with all outputs, its backward and a weight gradient, in the state's buffers."""
    Z.rmsnorm(s["x"], s["w"], residual=s["r"], h=s["h"], y=s["y"], y8=s["y8"], h8=s["h8"], rstd=s["rstd"])
    Z.act_wgrad(s["y8"], s["dy"], s["dw"], base=s["base"], workspace=s["ws1"])
    Z.rmsnorm_backward(s["dn"], s["h8"], s["w"], s["rstd"], s["dx"], dh=s["r"], dweight=s["dweight"],
                       workspace=s["ws2"])
    return [s[k].clone() for k in ("h", "y", "rstd", "dw", "dx", "dweight")] + [s["y8"].codes.clone()]


def _state(Z, seed, rows=700, cols=300, outs=200):
    import zero_sharded_mixed_buffer_amd as zs
    s = {"x": _randn((rows, cols), BF16, seed), "r": _randn((rows, cols), BF16, seed + 1),
         "w": _randn((cols,), BF16, seed + 2), "dy": _randn((rows, outs), BF16, seed + 3),
         "dn": _randn((rows, cols), BF16, seed + 4), "base": _randn((outs, cols), BF16, seed + 5)}
    for k in ("h", "y", "dx"):
        s[k] = torch.empty(rows, cols, dtype=BF16, device="cuda")
    s["rstd"] = torch.empty(rows, device="cuda")
    s["dw"] = torch.empty(outs, cols, dtype=BF16, device="cuda")
    s["dweight"] = torch.empty(cols, device="cuda")
    s["y8"], s["h8"] = zs.Act8.empty(rows, cols), zs.Act8.empty(rows, cols, "int8")
    s["ws1"] = torch.empty(zs.zs_act_wgrad_workspace(rows, cols, outs), dtype=torch.uint8, device="cuda")
    s["ws2"] = torch.empty(zs.zs_rmsnorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    return s


def test_two_streams_at_once(Z):
    """Two chains on two streams, each with its workspaces, and one that allocates its own."""
    states = [_state(Z, 100), _state(Z, 200)]
    want = [_chain(Z, s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for own_workspace in (False, True):
        if own_workspace:
            for s in states:
                s["ws1"] = s["ws2"] = None
        for _ in range(5):
            for i in (0, 1):
                streams[i].wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(streams[i]):
                    got[i] = _chain(Z, states[i])
            for st in streams:
                torch.cuda.current_stream().wait_stream(st)
            torch.cuda.synchronize()
            for i in (0, 1):
                assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_several_host_threads(Z):
    """Four host threads, each with its stream and buffers, run their chains at once."""
    import threading
    states = [_state(Z, 700 + 10 * i, rows=300 + 50 * i) for i in range(4)]
    want = [_chain(Z, s) for s in states]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(10):
                    got = _chain(Z, states[i])
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        bad.append(i)
        except Exception as e:  # reported below, in the test's own thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not bad, bad


def test_captured_and_replayed(Z):
    """Two graphs of chains, replayed several times in turn on changing inputs, with eager calls
    and synchronizations between; every replay against the eager result."""
    states = [_state(Z, 300), _state(Z, 400)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in states:
            _chain(Z, s)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_chain(Z, s))
        graphs.append(g)
    spare = _state(Z, 500)
    for turn in range(4):
        for i in (0, 1):
            for k in ("x", "r", "dy", "dn"):
                states[i][k].copy_(_randn(states[i][k].shape, BF16, 1000 + 10 * turn + i))
        for g in graphs:
            g.replay()
        if turn % 2:
            _chain(Z, spare)
        torch.cuda.synchronize()
        replayed = [[t.clone() for t in o] for o in outs]
        for i in (0, 1):
            want = _chain(Z, states[i])
            assert all(torch.equal(a, b) for a, b in zip(replayed[i], want)), (turn, i)


def test_captured_large_weight_gradient(Z):
    """The large tile's launch, captured and replayed, and the one with split tiles."""
    for rows, cols, outs in ((512, 4096, 4096), (1030, 4097, 4100)):
        x, dy = _randn((rows, cols), BF16, 601), _randn((rows, outs), BF16, 602, 0.01)
        act = Z.Act8.of(x)
        dw, eager = torch.empty(outs, cols, dtype=BF16, device="cuda"), torch.empty(outs, cols, dtype=BF16, device="cuda")
        ws = torch.empty(Z.zs_act_wgrad_workspace(rows, cols, outs), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            Z.act_wgrad(act, dy, dw, workspace=ws)
        for turn in range(3):
            dy.copy_(_randn((rows, outs), BF16, 610 + turn, 0.01))
            graph.replay()
            torch.cuda.synchronize()
            Z.act_wgrad(act, dy, eager)
            assert torch.equal(dw, eager)


def test_captured_training_pass(Z):
    """Forward and backward of the block captured whole, gradients added to the flat buffer: each
    replay adds the same gradient again."""
    p = _params()
    opt = Z.ZeroShardedAdamW(p, flat_views=True)
    x = _randn((64, 64), BF16, 91)

    def run():
        _block(Z, x, p, True).float().square().mean().backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            run()
    torch.cuda.current_stream().wait_stream(side)
    opt.zero_grad()
    run()
    torch.cuda.synchronize()
    once = opt.flat.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        opt.zero_grad()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(opt.flat, once)
    opt.close()


def test_another_devices_tensors_are_refused(Z):
    """A tensor elsewhere than the others (here: in host memory) is a ValueError."""
    x, w = _randn((4, 64), BF16, 1), _randn((64,), BF16, 2)
    for bad in (dict(residual=x.cpu()), dict(y=x.cpu()), dict(rstd=torch.empty(4)),
                dict(y8=Z.Act8.empty(4, 64, device="cpu"))):
        with pytest.raises(ValueError):
            Z.rmsnorm(x, w, **bad)
    with pytest.raises(ValueError):
        Z.rmsnorm(x, w.cpu(), y=x)
