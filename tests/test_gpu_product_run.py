"""GPU tests of the products, the experts and the routing in use: under autograd, in the flat gradient
buffer, on streams, in graphs, at large offsets.

Tolerances as in tests/test_gpu_product.py.  Where a chain of operators is compared with 64 bits as a
whole, each of its r roundings to bf16 changes a tensor by at most 2^-8 of it in norm, and the chain's
result by about r * 2^-8."""

import threading

import pytest
import torch

from oracle import act_oracle as AO
from oracle import product_oracle as PO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_sharded_mixed_buffer_amd as Z
    Z.lib()
    return Z


def _randn(shape, dtype, seed, sigma=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (sigma * torch.randn(shape, device="cuda", generator=g)).to(dtype)


def _near(got, want, size, terms, what, cut=0.0):
    """Within the sum's roundings (and `cut` of the sum of magnitudes) and the last one."""
    err = (2 * terms * U + cut) * size
    got = got.detach().cpu().double()
    bound = err + (want.abs() + err) * (torch.finfo(got_dtype(what)).eps / 2) + 2.0 ** -25
    assert bool(((got - want).abs() <= bound).all()), (what, float(((got - want).abs() - bound).max()))


def got_dtype(what):
    return what[1]


CUT = 7 * 2.0 ** -13  # see tests/test_gpu_product.py


# ------------------------------------------------------------------------------ linear8

@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape,outs", [((5, 64), 48), ((2, 3, 100), 130), ((300, 256), 200), ((1, 33), 1)])
def test_linear8_gradients(Z, shape, outs, dtype, given):
    cols = shape[-1]
    x = _randn(shape, dtype, 1).requires_grad_()
    w = _randn((outs, cols), dtype, 2, 0.1).requires_grad_()
    x8 = Z.Act8.of(x.detach().view(-1, cols)) if given else None
    w8 = Z.Weight8.of(w.detach()) if given else None
    y = Z.linear8(x, w, w8=w8, x8=x8)
    assert y.shape == (*shape[:-1], outs) and y.dtype == dtype
    dy = _randn(y.shape, dtype, 3)
    y.backward(dy)
    xv = AO.values(*AO.quantise(x.view(-1, cols), "e4m3"), cols, "e4m3")
    codes, _, scales = PO.weight8(w)
    wv = PO.weight_values(codes, scales, cols)
    dv = AO.values(*AO.quantise(dy.view(-1, outs), "e4m3"), outs, "e4m3")
    d = dy.view(-1, outs).cpu().double()
    _near(y.view(-1, outs), xv @ wv.t(), xv.abs() @ wv.abs().t(), cols, ("y", dtype), CUT)
    _near(x.grad.view(-1, cols), dv @ wv, dv.abs() @ wv.abs(), outs, ("dx", dtype), CUT)
    _near(w.grad, d.t() @ xv, d.abs().t() @ xv.abs(), len(d), ("dw", dtype))


def test_linear8_partial_gradients_and_none(Z):
    x, w = _randn((40, 64), BF16, 1), _randn((24, 64), BF16, 2)
    plain = Z.linear8(x, w)
    for gx, gw in ((True, False), (False, True)):
        a, b = x.clone().requires_grad_(gx), w.clone().requires_grad_(gw)
        y = Z.linear8(a, b)
        assert torch.equal(y, plain)
        y.backward(_randn(y.shape, BF16, 3))
        assert (a.grad is not None) == gx and (b.grad is not None) == gw
    with torch.no_grad():
        assert torch.equal(Z.linear8(x.clone().requires_grad_(), w), plain)
    with torch.inference_mode():
        assert torch.equal(Z.linear8(x.clone(), w.clone()), plain)


def test_linear8_refuses_what_is_stale(Z):
    x, w = _randn((40, 64), BF16, 1), _randn((24, 64), BF16, 2).requires_grad_()
    x8, w8 = Z.Act8.of(x), Z.Weight8.of(w.detach())
    y = Z.linear8(x, w, w8=w8, x8=x8)
    Z.weight8_pack(_randn((24, 64), BF16, 4), w8)   # the input's gradient is not wanted: only x8 is kept
    y.sum().backward()
    w8 = Z.Weight8.of(w.detach())
    xg = x.clone().requires_grad_()
    y = Z.linear8(xg, w, w8=w8)
    Z.weight8_pack(_randn((24, 64), BF16, 4), w8)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    w8 = Z.Weight8.of(w.detach())
    with torch.no_grad():
        w.mul_(2)
    with pytest.raises(ValueError, match="changed in place since w8"):
        Z.linear8(x, w, w8=w8)
    x8 = Z.Act8.of(x)
    x.mul_(2)
    with pytest.raises(ValueError, match="changed in place since x8"):
        Z.linear8(x, w, x8=x8)
    with pytest.raises(ValueError, match="transposed codes"):
        Z.linear8(xg, w, w8=Z.Weight8.of(w.detach(), transposed=False))
    with pytest.raises(ValueError, match="e4m3"):
        Z.linear8(x, w, x8=Z.Act8.of(x, "int8"))


def test_weights_of_a_pool(Z):
    """8-bit weights whose arrays are parts of one buffer: filling another one does not disturb a pending
    backward pass, filling the same one does."""
    size = [Z.zs_weight8_size(48, 64) for _ in range(2)]
    pool = torch.zeros(2 * (48 * 128 + 64 * 128 + 128), dtype=torch.uint8, device="cuda")

    def part(i):
        at = i * (48 * 128 + 64 * 128 + 128)
        codes = pool[at:at + 48 * 128].view(48, 128)
        codes_t = pool[at + 48 * 128:at + 48 * 128 + 64 * 128].view(64, 128)
        return Z.Weight8(codes, pool[at + 48 * 128 + 64 * 128:][:1].view(1, 1), 64, codes_t)

    assert size[0] == (48 * 128, 64 * 128, 1)
    w = [_randn((48, 64), BF16, i) for i in range(2)]
    w8 = [part(i) for i in range(2)]
    for i in range(2):
        Z.weight8_pack(w[i], w8[i])
    x = _randn((10, 64), BF16, 5).requires_grad_()
    y = Z.linear8(x, w[0], w8=w8[0])
    Z.weight8_pack(w[1], w8[1])
    y.sum().backward()
    y = Z.linear8(x, w[0], w8=w8[0])
    Z.weight8_pack(w[1], w8[0])
    with pytest.raises(RuntimeError, match="filled anew"):
        y.sum().backward()


def test_norm_feeds_linear8(Z):
    """norm's 8-bit output is linear8's input as it is."""
    x, nw = _randn((64, 256), BF16, 1).requires_grad_(), torch.ones(256, dtype=BF16, device="cuda")
    w = _randn((128, 256), BF16, 2, 0.06).requires_grad_()
    into = torch.zeros(128, 256, dtype=FP32, device="cuda")
    out = Z.norm(x, nw, y8="e4m3")
    y = Z.linear8(out.y, w, x8=out.y8, grad_into=into)
    want = torch.empty_like(y)
    Z.product8(out.y8, Z.Weight8.of(w.detach()), want)
    assert torch.equal(y, want)
    dy = _randn(y.shape, BF16, 3)
    y.backward(dy)
    alone = torch.zeros_like(into)
    Z.act_wgrad(out.y8, dy, alone)
    assert torch.equal(into, alone) and w.grad is None and x.grad is not None


# ------------------------------------------------------------------------------ experts

@pytest.mark.parametrize("save", [None, "e4m3", "int8"])
@pytest.mark.parametrize("in_major", [False, True])
@pytest.mark.parametrize("sizes,cols,outs", [([3, 0, 5], 64, 48), ([130, 20, 0, 1], 100, 72)])
def test_experts_gradients(Z, sizes, cols, outs, in_major, save):
    rows, n = sum(sizes) + 4, len(sizes)
    x = _randn((rows, cols), BF16, 1)
    x[sum(sizes):] = float("nan")
    x.requires_grad_()
    w = _randn((n, cols, outs) if in_major else (n, outs, cols), BF16, 2, 0.1).requires_grad_()
    ends = torch.tensor(sizes).cumsum(0).int().cuda()
    y = Z.experts(x, w, ends, in_major=in_major, save=save)
    dy = _randn(y.shape, BF16, 3)
    dy[sum(sizes):] = float("nan")
    y.backward(dy)
    kept = sum(sizes)
    assert bool((y[kept:] == 0).all()) and bool((x.grad[kept:] == 0).all())
    want, size = PO.expert_product(x.detach(), w.detach(), ends, in_major)
    _near(y[:kept], want[:kept], size[:kept], cols, ("y", BF16))
    want, size = PO.expert_product(dy, w.detach(), ends, not in_major)
    _near(x.grad[:kept], want[:kept], size[:kept], outs, ("dx", BF16))
    xv = x.detach().cpu()[:kept]
    if save is not None:
        xv = AO.rounded(AO.values(*AO.quantise(xv, save), cols, save), BF16)
    want, size = PO.expert_wgrad(xv, dy[:kept], ends, in_major=in_major)
    _near(w.grad, want, size, kept, ("dw", BF16))


def test_experts_grad_into(Z):
    x, ends = _randn((50, 64), FP16, 1), torch.tensor([20, 50], dtype=torch.int32, device="cuda")
    w = _randn((2, 40, 64), FP16, 2, 0.1).requires_grad_()
    for grad in (FP16, FP32):
        into = _randn((2, 40, 64), grad, 3)
        want = into.clone()
        for seed in (4, 5):
            dy = _randn((50, 40), FP16, seed)
            Z.experts(x, w, ends, grad_into=into).backward(dy)
            Z.expert_wgrad(x, dy, ends, want, base=want)
        assert torch.equal(into, want) and w.grad is None
    with pytest.raises(ValueError, match="grad_into"):
        Z.experts(x, w, ends, grad_into=torch.zeros(2, 64, 40, dtype=FP16, device="cuda"))
    with pytest.raises(ValueError, match="save"):
        Z.experts(x, w, ends, save="int4")
    with pytest.raises(ValueError, match="ends has"):
        Z.experts(x, w, ends[:1])


def _moe(Z, x, logits, w1, w2, choices, **kw):
    weights, ids = torch.softmax(logits.float(), 1).topk(choices, 1)
    r = Z.route(ids, w1.shape[0])
    h = Z.experts(Z.dispatch(x, r), w1, r.ends, **{k: v[0] for k, v in kw.items()})
    y = Z.experts(torch.nn.functional.silu(h), w2, r.ends, **{k: v[1] for k, v in kw.items()})
    return Z.combine(y, r, weights)


def test_expert_layer_against_64_bits(Z):
    """Router, dispatch, two products and the combination, with all gradients."""
    tokens, hidden, ffn, n, k = 200, 128, 96, 6, 2
    x = _randn((tokens, hidden), BF16, 1).requires_grad_()
    logits = _randn((tokens, n), FP32, 2).requires_grad_()
    w1, w2 = _randn((n, ffn, hidden), BF16, 3, 0.1).requires_grad_(), _randn((n, hidden, ffn), BF16, 4, 0.1).requires_grad_()
    out = _moe(Z, x, logits, w1, w2, k)
    dout = _randn(out.shape, BF16, 5)
    out.backward(dout)

    leaves = [t.detach().cpu().double().requires_grad_() for t in (x, logits, w1, w2)]
    xd, ld, w1d, w2d = leaves
    weights, ids = torch.softmax(ld, 1).topk(k, 1)
    want = torch.zeros(tokens, hidden, dtype=torch.float64)
    rows = []
    for t in range(tokens):
        acc = 0
        for j in range(k):
            e = int(ids[t, j])
            acc = acc + weights[t, j] * (w2d[e] @ torch.nn.functional.silu(w1d[e] @ xd[t]))
        rows.append(acc)
    want = torch.stack(rows)
    want.backward(dout.cpu().double())
    for got, ref, r in ((out, want, 4), (x.grad, xd.grad, 8), (logits.grad, ld.grad, 8), (w1.grad, w1d.grad, 8), (w2.grad, w2d.grad, 8)):
        rel = float((got.detach().cpu().double() - ref.detach()).norm() / ref.detach().norm())
        assert rel <= r * 2.0 ** -8, rel


def test_dispatch_and_combine_differences(Z):
    """Both are linear in their rows, the combination in its weights too: a difference along a direction
    is the gradient's product with it, but for fp32 roundings."""
    tokens, k, n, cols = 30, 3, 5, 40
    r = Z.route(torch.randint(-1, n, (tokens, k), generator=torch.Generator().manual_seed(1)).cuda(), n)
    x, y = _randn((tokens, cols), FP32, 2).requires_grad_(), _randn((tokens * k, cols), FP32, 3).requires_grad_()
    w = _randn((tokens, k), FP32, 4).requires_grad_()
    with torch.no_grad():
        y[int(r.ends[-1]):] = 0
    for leaf, f in ((x, lambda: Z.dispatch(x, r)), (y, lambda: Z.combine(y, r, w)), (w, lambda: Z.combine(y, r, w)),
                    (y, lambda: Z.combine(y, r))):
        out = f()
        g = _randn(out.shape, FP32, 5)
        leaf.grad = None
        out.backward(g)
        d = _randn(leaf.shape, FP32, 6)
        before = (out.detach().double() * g.double()).sum()
        with torch.no_grad():
            leaf += d
        after = (f().detach().double() * g.double()).sum()
        want = (leaf.grad.double() * d.double()).sum()
        scale = float((leaf.grad.double() * d.double()).abs().sum() + (out.detach().double() * g.double()).abs().sum())
        assert abs(float(after - before - want)) <= 16 * U * 4 * scale


def test_expert_layer_trains_in_the_flat_buffer(Z):
    """The experts' gradients land in the flat gradient buffer that the step reads."""
    n, hidden, ffn = 4, 64, 96
    w1 = torch.nn.Parameter(_randn((n, ffn, hidden), BF16, 1, 0.1))
    w2 = torch.nn.Parameter(_randn((n, hidden, ffn), BF16, 2, 0.1))
    opt = Z.ZeroShardedAdamW([w1, w2], lr=1e-3, flat_views=True)
    x, logits = _randn((100, hidden), BF16, 3), _randn((100, n), FP32, 4)
    dout = _randn((100, hidden), BF16, 5)
    opt.zero_grad()
    _moe(Z, x, logits, w1, w2, 2, grad_into=(w1.grad, w2.grad), save=("e4m3", "e4m3")).backward(dout)
    a, b = w1.detach().clone().requires_grad_(), w2.detach().clone().requires_grad_()
    _moe(Z, x, logits, a, b, 2, save=("e4m3", "e4m3")).backward(dout)
    assert torch.equal(w1.grad, a.grad) and torch.equal(w2.grad, b.grad) and float(w1.grad.float().norm()) > 0
    before = w1.detach().clone()
    opt.step()
    assert not torch.equal(before, w1.detach()) and not opt.read_state()["overflow"]
    opt.close()


def test_changed_rows_are_noticed(Z):
    x, w = _randn((20, 64), BF16, 1), _randn((2, 32, 64), BF16, 2).requires_grad_()
    ends = torch.tensor([10, 20], dtype=torch.int32, device="cuda")
    y = Z.experts(x, w, ends)
    x.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = Z.experts(x, w, ends)
    ends.add_(0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_broadcast_rows_and_gradients(Z):
    """Rows that overlap (a broadcast input, the gradient of a sum) are copied first."""
    ends = torch.tensor([3, 8], dtype=torch.int32, device="cuda")
    row = _randn((64,), BF16, 1)
    w = _randn((2, 32, 64), BF16, 2).requires_grad_()
    x = row.expand(8, 64).clone().requires_grad_()
    a = Z.experts(row.expand(8, 64), w, ends)
    b = Z.experts(x, w, ends)
    assert torch.equal(a, b)
    b.sum().backward()
    want, size = PO.expert_product(torch.ones(8, 32, dtype=BF16), w.detach(), ends, True)
    _near(x.grad, want, size, 32, ("dx", BF16))
    y = Z.linear8(row.expand(2, 4, 64), w.detach()[0])
    assert torch.equal(y[0, 0], y[1, 3])


# ------------------------------------------------------------------------------ streams, graphs, threads

def _everything(Z, s):
    """One pass through all operators into the state's buffers; returns the outputs."""
    Z.act_pack(s["x"], s["x8"])
    Z.weight8_pack(s["w"], s["w8"])
    Z.product8(s["x8"], s["w8"], s["y"])
    Z.product8(s["x8t"], s["w8"], s["dx"], transposed=True)
    r = Z.route(s["ids"], 4, s["work"])
    rows = Z.dispatch(s["x"], r)
    Z.expert_product(rows, s["we"], r.ends, s["ye"], zero_rest=True)
    Z.expert_wgrad(rows, s["ye"], r.ends, s["dw"], base=s["base"])
    Z.expert_combine(s["ye"], r, s["out"], s["weights"])
    Z.expert_combine_backward(s["out"], s["ye"], r, s["weights"], s["dy"], s["dweights"])
    return [s[k] for k in ("y", "dx", "ye", "dw", "out", "dy", "dweights")] + [r.ends, r.slot, r.place, rows]


def _state(Z, seed, tokens=300):
    e = lambda *shape, dtype=BF16: torch.empty(shape, dtype=dtype, device="cuda")
    g = torch.Generator("cuda").manual_seed(seed)
    return dict(x=_randn((tokens, 256), BF16, seed), w=_randn((200, 256), BF16, seed + 1), w8=Z.Weight8.empty(200, 256),
                x8=Z.Act8.empty(tokens, 256), x8t=Z.Act8.of(_randn((tokens, 200), BF16, seed + 2)), y=e(tokens, 200), dx=e(tokens, 256),
                ids=torch.randint(-1, 5, (tokens, 2), device="cuda", generator=g), we=_randn((4, 128, 256), BF16, seed + 3),
                ye=e(2 * tokens, 128), dw=e(4, 128, 256, dtype=FP32), base=_randn((4, 128, 256), FP32, seed + 4), out=e(tokens, 128),
                weights=torch.rand(tokens, 2, device="cuda", generator=g), dy=e(2 * tokens, 128), dweights=e(tokens, 2, dtype=FP32),
                work=torch.empty(1 << 16, dtype=torch.uint8, device="cuda"))


def test_two_streams_at_once(Z):
    states = [_state(Z, 10), _state(Z, 20, 333)]
    want = [[t.clone() for t in _everything(Z, s)] for s in states]
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(3):
        for t in (t for s in states for t in (s["y"], s["ye"], s["dw"], s["dy"])):
            t.zero_()
        torch.cuda.synchronize()
        got = []
        for st, s in zip(streams, states):
            with torch.cuda.stream(st):
                got.append(_everything(Z, s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed(Z):
    """Captured with one batch, replayed with others of other routes, eager work in between."""
    s = _state(Z, 30)
    _everything(Z, s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = _everything(Z, s)
    for seed in (40, 50, 60):
        t = _state(Z, seed)
        want = [v.clone() for v in _everything(Z, t)]
        for k in ("x", "w", "ids", "we", "base", "weights"):
            s[k].copy_(t[k])
        s["x8t"].codes.copy_(t["x8t"].codes)
        s["x8t"].scales.copy_(t["x8t"].scales)
        for k in ("y", "dx", "ye", "dw", "out", "dy", "dweights"):
            s[k].fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (seed, i)


def test_captured_training_pass(Z):
    n, hidden, ffn, tokens = 4, 128, 64, 90
    x, logits = _randn((tokens, hidden), BF16, 1), _randn((tokens, n), FP32, 2)
    w1, w2 = _randn((n, ffn, hidden), BF16, 3, 0.1), _randn((n, hidden, ffn), BF16, 4, 0.1)
    wl = _randn((hidden, hidden), BF16, 5, 0.1)
    dout = _randn((tokens, hidden), BF16, 6)

    def one():
        a, b, c = (t.detach().requires_grad_() for t in (w1, w2, wl))
        y = _moe(Z, Z.linear8(x, c), logits, a, b, 2, save=("e4m3", None))
        return torch.autograd.grad(y, (a, b, c), dout)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one()
    for seed in (7, 8, 9):
        x.copy_(_randn(x.shape, BF16, seed))
        logits.copy_(_randn(logits.shape, FP32, seed + 20))
        want = [g.clone() for g in one()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_several_host_threads(Z):
    states = [_state(Z, 70 + 10 * i, 200 + 7 * i) for i in range(4)]
    want = [[t.clone() for t in _everything(Z, s)] for s in states]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got = _everything(Z, states[i])
                torch.cuda.current_stream().synchronize()
                wrong.extend((i, j) for j, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
        assert not t.is_alive()
    assert not wrong


# ------------------------------------------------------------------------------ extremes

def test_offsets_past_32_bits(Z):
    """Matrices whose elements lie further apart than 32 bits of bytes, or of elements."""
    rows, cols, outs = 70000, 64, 72
    wide = torch.zeros(rows, 32768, dtype=BF16, device="cuda")  # 4.6 GB
    x = wide[:, 100:100 + cols]
    x.copy_(_randn((rows, cols), BF16, 1))
    w = _randn((2, outs, cols), BF16, 2)
    ends = torch.tensor([30001, rows], dtype=torch.int32, device="cuda")
    y = wide[:, 30000:30000 + outs]
    Z.expert_product(x, w, ends, y)
    some = torch.tensor([0, 30000, 30001, 66000, rows - 1])
    for i in some.tolist():
        a, b = x[i].cpu().double(), w[int(i >= 30001)].cpu().double()
        _near(y[i], b @ a, b.abs() @ a.abs(), cols, ("y", BF16))
    far = torch.zeros(2 ** 31 + 2 ** 20, dtype=FP32, device="cuda")  # 8.6 GB
    dw = far.as_strided((2, cols, cols), (2 ** 31, cols, 1))
    Z.expert_wgrad(x, x.contiguous(), ends, dw)
    want, size = PO.expert_wgrad(x, x.contiguous(), ends)
    _near(dw, want, size, rows, ("dw", FP32))
    x8 = Z.Act8.empty(rows, 32768 * 2)  # 4.6 GB of codes
    x8.codes.zero_()
    x8.scales.fill_(127)
    x8.codes[-3:, -32:] = 0x38
    w8 = Z.Weight8.of(torch.ones(130, 32768 * 2, dtype=BF16, device="cuda"), transposed=False)
    y = torch.empty(rows, 130, dtype=BF16, device="cuda")
    Z.product8(x8, w8, y)
    assert bool((y[-3:] == 32).all()) and not bool(y[:-3].any())
    few = Z.Act8(x8.codes[-3:], x8.scales[-3:], 32768 * 2)
    y = torch.empty(3, 130, dtype=BF16, device="cuda")
    Z.product8(few, w8, y)
    assert bool((y == 32).all())


@pytest.mark.parametrize("experts", [300, 1024])
def test_many_experts(Z, experts):
    g = torch.Generator().manual_seed(experts)
    sizes = torch.randint(0, 4, (experts,), generator=g)
    sizes[7] = 200
    rows, cols, outs = int(sizes.sum()) + 3, 64, 40
    ends = sizes.cumsum(0).int().cuda()
    x, w, dy = _randn((rows, cols), BF16, 1), _randn((experts, outs, cols), BF16, 2), _randn((rows, outs), BF16, 3)
    y = torch.full((rows, outs), 7.0, dtype=BF16, device="cuda")
    Z.expert_product(x, w, ends, y)
    want, size = PO.expert_product(x, w, ends)
    _near(y[:-3], want[:-3], size[:-3], cols, ("y", BF16))
    assert bool((y[-3:] == 7).all())
    dx = torch.empty(rows, cols, dtype=BF16, device="cuda")
    Z.expert_product(dy, w, ends, dx, in_major=True, zero_rest=True)
    want, size = PO.expert_product(dy, w, ends, True)
    _near(dx[:-3], want[:-3], size[:-3], outs, ("dx", BF16))
    assert not bool(dx[-3:].any())
    dw = torch.empty(experts, outs, cols, dtype=BF16, device="cuda")
    Z.expert_wgrad(x, dy, ends, dw)
    want, size = PO.expert_wgrad(x, dy, ends)
    _near(dw, want, size, 200, ("dw", BF16))


def test_no_rows(Z):
    """Batches of no tokens: empty outputs, weight gradients that are the base or zero."""
    ends = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, w = torch.empty(0, 64, dtype=BF16, device="cuda"), _randn((3, 32, 64), BF16, 1).requires_grad_()
    y = Z.experts(x, w, ends)
    assert y.shape == (0, 32)
    y.sum().backward()
    assert not bool(w.grad.any())
    base = _randn((3, 32, 64), BF16, 2)
    dw = torch.empty_like(base)
    Z.expert_wgrad(x, torch.empty(0, 32, dtype=BF16, device="cuda"), ends, dw, base=base)
    assert torch.equal(dw, base)
    r = Z.route(torch.empty(0, 2, dtype=torch.int64, device="cuda"), 5)
    assert not bool(r.ends.any()) and r.rows == 0
    assert Z.dispatch(x, r).shape == (0, 64) and Z.combine(x, r).shape == (0, 64)
    a, b = x.clone().requires_grad_(), w.detach()[0].clone().requires_grad_()
    for layer in (Z.linear8, Z.linear):
        y = layer(a, b)
        assert y.shape == (0, 32)
        y.sum().backward()
        assert a.grad.shape == (0, 64) and not bool(b.grad.any())


def test_tensor_level_refusals_on_the_gpu(Z):
    x, w = _randn((6, 8), BF16, 1), _randn((2, 5, 8), BF16, 2)
    ends = torch.tensor([3, 6], dtype=torch.int32, device="cuda")
    y = torch.empty(6, 5, dtype=BF16, device="cuda")
    bad = [
        (lambda: Z.expert_product(x.float(), w, ends, y), "x is"),
        (lambda: Z.expert_product(x, w.half(), ends, y), "w is"),
        (lambda: Z.expert_product(x, w, ends.long(), y), "int32"),
        (lambda: Z.expert_product(x, w, ends.cpu(), y), "ends lives"),
        (lambda: Z.expert_product(x, w[:, :, :7], ends, y), "w has shape"),
        (lambda: Z.expert_product(x, w.transpose(1, 2).contiguous().transpose(1, 2), ends, y), "consecutive"),
        (lambda: Z.expert_product(x, w, ends, y[:, :4]), "y has shape"),
        (lambda: Z.expert_product(x.t(), w, ends, y), "consecutive"),
        (lambda: Z.expert_wgrad(x, y, ends, w.float().double()), "dw is"),
        (lambda: Z.expert_wgrad(x, y, ends, w, base=w.float()), "base is"),
        (lambda: Z.expert_wgrad(x, y[:5], ends, w), "dy has shape"),
        (lambda: Z.product8(Z.Act8.of(x), Z.Weight8.of(w[0]), y.float()), "y is"),
        (lambda: Z.product8(Z.Act8.of(x), Z.Weight8.of(w[0]), y[:, :4]), "columns"),
        (lambda: Z.product8(Z.Act8.of(x, "int8"), Z.Weight8.of(w[0]), y), "e4m3"),
        (lambda: Z.product8(Z.Act8.of(y), Z.Weight8.of(w[0], transposed=False), x, transposed=True), "transposed codes"),
        (lambda: Z.weight8_pack(w[0], Z.Weight8.empty(5, 9)), "w8 is a weight of"),
        (lambda: Z.route(ends, 3), "ids must be"),
        (lambda: Z.route(ends.view(2, 1).float(), 3), "ids must be"),
        (lambda: Z.route(ends.view(2, 1), 3, torch.empty(4, dtype=torch.uint8, device="cuda")), "workspace"),
    ]
    r = Z.route(torch.zeros(3, 2, dtype=torch.int32, device="cuda"), 2)
    bad += [
        (lambda: Z.expert_gather(x, r, x), "route"),
        (lambda: Z.expert_combine(x, r, x[:3], weights=torch.ones(3, 2, device="cuda").half()), "weights"),
        (lambda: Z.expert_combine_backward(x[:3], None, r, None, None, torch.empty(3, 2, device="cuda")), "needs y"),
        (lambda: Z.expert_combine_backward(x[:3], x, r), "neither"),
    ]
    for call, match in bad:
        with pytest.raises(ValueError, match=match):
            call()
