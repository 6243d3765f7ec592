"""A training rank's mixture-of-experts block, forward and backward, and a
serving step with adapters, through the owners of the buffers: every stage
against the 64-bit formula on what it was given (bounds as in the stages' own
tests), captured into graphs, on two streams at once, and the owners'
refusals."""
import pytest

import layer_util as lu
from gpu_util import require_gpu, say

torch = pytest.importorskip("torch")

U = 2.0 ** -24
bf16 = torch.bfloat16
mx = lu.mx


class Block:
    """norm -> experts by the router's choice -> two products each -> back onto the residual, and its gradients."""

    def __init__(self, tokens, hidden, inner, choices, experts):
        from lossless_bf16_tensor_exp_amd.codec import ExpertRows, MxLinear, RmsNorm
        rows = tokens * choices
        self.norm = RmsNorm(tokens, hidden)
        self.rows = ExpertRows(tokens, choices, experts)
        self.up = MxLinear(rows, inner, hidden, experts)
        self.down = MxLinear(rows, hidden, inner, experts)

        def new(*shape, dtype=bf16):
            return torch.zeros(*shape, dtype=dtype, device="cuda")

        self.h, self.y, self.out, self.dx, self.dy = (new(tokens, hidden) for _ in range(5))
        self.u, self.du = new(rows, inner), new(rows, inner)
        self.z, self.dz, self.dxs = new(rows, hidden), new(rows, hidden), new(rows, hidden)
        self.dweights = new(tokens, choices, dtype=torch.float32)
        self.dnorm = new(hidden, dtype=torch.float32)
        self.dup, self.ddown = new(experts, inner, hidden), new(experts, hidden, inner)

    def load(self, w1, w2, wn):
        self.up.load(w1)
        self.down.load(w2)
        self.norm.weight.copy_(wn)

    def step(self, x, residual, ids, weights, dout):
        self.norm.forward(x, self.y, residual=residual, h=self.h)
        self.rows.sort(ids)
        at = self.rows.offsets
        self.up.keep_dispatched(self.y, self.rows, self.u)
        self.down.keep(self.u, self.z, at)
        self.rows.combine(self.z, self.out, weights, self.h)
        self.rows.combine_backward(dout, self.z, self.dz, self.dweights, weights)
        self.down.backward(self.dz, self.du, self.ddown, at)
        self.up.backward(self.du, self.dxs, self.dup, at)
        self.rows.dispatch_backward(self.dxs, self.dy)
        self.norm.backward(self.dy, self.h, self.dx, self.dnorm, dh=dout)

    def results(self):
        return [self.h, self.y, self.out, self.dx, self.dy, self.dweights, self.dnorm, self.dup, self.ddown, self.rows.offsets,
                self.rows.place]

    def errors(self):
        return [self.rows.error(), self.up.error(), self.down.error()]


def inputs(gen, tokens, hidden, inner, choices, experts):
    x = (torch.randn(tokens, hidden, generator=gen) * 0.5).to(bf16)
    residual = mx.activations(gen, tokens, hidden)
    ids = lu.choose(gen, tokens, choices, experts)
    weights = torch.softmax(torch.randn(tokens, choices, generator=gen), 1).contiguous()
    dout = (torch.randn(tokens, hidden, generator=gen) * 1e-3).to(bf16)
    w1 = (torch.randn(experts * inner, hidden, generator=gen) * 0.05).to(bf16)
    w2 = (torch.randn(experts * hidden, inner, generator=gen) * 0.05).to(bf16)
    wn = (1 + 0.1 * torch.randn(hidden, generator=gen)).to(bf16)
    return [x, residual, ids, weights, dout], [w1, w2, wn]


def product(got, a, b, half_step=2.0 ** -8):
    """got = a b, an FP32 sum rounded once."""
    size = a.abs() @ b.abs()
    lu.within(got, a @ b, a.shape[1] * U * size, half_step)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden,inner,choices,experts", [(1, 128, 96, 2, 4), (40, 264, 128, 3, 6), (300, 256, 160, 4, 16),
                                                                 (1100, 128, 64, 2, 3)])
def test_block(tokens, hidden, inner, choices, experts):
    require_gpu()
    say(f"block of {tokens} tokens, {choices} of {experts} experts")
    gen = torch.Generator().manual_seed(tokens)
    args, weights = inputs(gen, tokens, hidden, inner, choices, experts)
    x, residual, ids, weight, dout = args
    b = Block(tokens, hidden, inner, choices, experts)
    b.load(*[w.cuda() for w in weights])
    b.step(*[t.cuda() for t in args])
    assert b.errors() == [0, 0, 0]
    w1, w2 = (mx.decode(4, mx.encode(4, w), *w.shape).view(experts, -1, w.shape[1]) for w in weights[:2])
    offsets, place, order = lu.sort(ids, experts)
    assert torch.equal(b.rows.offsets.cpu(), offsets) and torch.equal(b.rows.place.cpu(), place)
    assert torch.equal(b.rows.order.cpu(), order)
    h, s, y = lu.norm(x, residual, weights[2], 1e-6)
    assert torch.equal(b.h.cpu(), h)
    lu.within(b.y, y, 33 * U * y.abs(), 2.0 ** -8)
    used = int(offsets[-1])
    entry = order[:used].long()
    xs = mx.decode(8, mx.encode(8, b.y.cpu()), tokens, hidden)[entry // choices]  # the checkpoint of the dispatched rows
    u, z = b.u.cpu(), b.z.cpu()
    uq = mx.decode(8, mx.encode(8, u), *u.shape)
    dz, du, dxs = b.dz.cpu().double(), b.du.cpu().double(), b.dxs.cpu()
    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        product(u[lo:hi], xs[lo:hi], w1[e].T)
        product(z[lo:hi], uq[lo:hi], w2[e].T)
        product(du[lo:hi], dz[lo:hi], w2[e])
        product(dxs[lo:hi], du[lo:hi], w1[e])
        product(b.ddown[e].cpu(), dz[lo:hi].T, uq[lo:hi])
        product(b.dup[e].cpu(), du[lo:hi].T, xs[lo:hi])
    out, size = lu.combine(z, place, weight, h)
    lu.within(b.out, out, (choices + 2) * U * size, 2.0 ** -8)
    f = weight.view(-1)[entry]
    assert torch.equal(b.dz.cpu()[:used], (f[:, None] * dout[entry // choices].float()).to(bf16))
    terms = dout[entry // choices].double() * z[:used].double()
    got = b.dweights.cpu().view(-1)
    lu.within(got[entry], terms.sum(1), (hidden + 8) * U * terms.abs().sum(1), U)
    assert (got[order[used:].long()] == 0).all()
    dy, size = lu.combine(dxs, place, None, None)
    lu.within(b.dy, dy, (choices + 2) * U * size, 2.0 ** -8)
    hd, sd, dyd = h.double(), b.norm.rstd.cpu().double()[:, None], b.dy.cpu().double()
    g, unit = dyd * weights[2].double(), hd * sd
    m = (g * unit).mean(1, keepdim=True)
    want = sd * (g - unit * m) + dout.double()
    room = U * ((sd * unit).abs() * 64 * (g * unit).abs().mean(1, keepdim=True) + 5 * (sd * g).abs() + 5 * (sd * unit * m).abs() +
                dout.double().abs())
    lu.within(b.dx, want, room, 2.0 ** -8)
    lu.within(b.dnorm, (dyd * unit).sum(0), (tokens + 66) * U * (dyd * unit).abs().sum(0), U)
    # rows of no entry: as they were
    for t in (b.u, b.z, b.dz, b.du, b.dxs):
        assert (t[used:] == 0).all()
    # equal calls, equal bits
    first = [t.clone() for t in b.results()]
    b.step(*[t.cuda() for t in args])
    for one, two in zip(first, b.results()):
        assert torch.equal(one, two)


@pytest.mark.gpu
def test_block_in_a_graph():
    """A captured step sees the inputs, the router's choices among them, that the buffers hold at each replay; another
    step, eager and with buffers of its own, runs between the replays."""
    require_gpu()
    say("block in a graph")
    sizes = (200, 128, 96, 3, 7)
    gen = torch.Generator().manual_seed(1)
    args, weights = inputs(gen, *sizes)
    args, weights = [t.cuda() for t in args], [w.cuda() for w in weights]
    a, b = Block(*sizes), Block(*sizes)
    for block in (a, b):
        block.load(*weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step(*args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(*args)
    for i in range(4):
        new, _ = inputs(gen, *sizes)
        for t, n in zip(args, new):
            t.copy_(n)
        b.step(*args)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for one, two in zip(a.results(), b.results()):
            assert torch.equal(one, two), f"replay {i}"
        assert a.errors() == [0, 0, 0]


@pytest.mark.gpu
def test_blocks_on_two_streams():
    require_gpu()
    say("blocks on two streams")
    sizes = (500, 256, 128, 2, 8)
    cases = [inputs(torch.Generator().manual_seed(10 + i), *sizes) for i in range(2)]
    want = []
    for args, weights in cases:
        b = Block(*sizes)
        b.load(*[w.cuda() for w in weights])
        b.step(*[t.cuda() for t in args])
        want.append([t.clone() for t in b.results()])
    blocks, streams = [Block(*sizes) for _ in cases], [torch.cuda.Stream() for _ in cases]
    given = [[t.cuda() for t in args] for args, _ in cases]
    for b, (_, weights) in zip(blocks, cases):
        b.load(*[w.cuda() for w in weights])
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s, g in zip(blocks, streams, given):
            with torch.cuda.stream(s):
                b.step(*g)
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for one, two in zip(b.results(), w):
            assert torch.equal(one, two)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,n,k,rank,adapters", [(1, 256, 128, 8, 3), (37, 200, 328, 16, 5), (400, 512, 256, 64, 9)])
def test_serving_step_with_adapters(tokens, n, k, rank, adapters):
    """The shared projection in FP32 and the requests' adapters onto it, one plan for two projections, and in a graph."""
    require_gpu()
    say(f"serving step of {tokens} with {adapters} adapters")
    from lossless_bf16_tensor_exp_amd.codec import LowRankAdapters, MxLinear
    gen = torch.Generator().manual_seed(tokens)
    w = (torch.randn(n, k, generator=gen) * 0.05).to(bf16)
    layer = MxLinear(tokens, n, k)
    layer.load(w.cuda())
    one, two = LowRankAdapters(tokens + 5, n, k, rank, adapters), LowRankAdapters(tokens + 5, n, k, rank, adapters)
    for i in range(adapters):
        for which in (one, two):
            r = rank - i % 3 if rank > 3 else rank
            which.load(i, (torch.randn(r, k, generator=gen) * k ** -0.5).to(bf16).cuda(),
                       (torch.randn(n, r, generator=gen) * 0.2).to(bf16).cuda(), 0.5 + i)
    x, ids = torch.empty(tokens, k, dtype=bf16, device="cuda"), torch.empty(tokens, dtype=torch.int64, device="cuda")
    base, y1, y2 = torch.empty(tokens, n, device="cuda"), *(torch.empty(tokens, n, dtype=bf16, device="cuda") for _ in range(2))

    def step():
        one.plan(ids)
        layer.forward(x, base)
        one.add(x, y1, base)
        two.add(x, y2, plan=one)

    def fill():
        x.copy_(mx.activations(gen, tokens, k))
        ids.copy_(torch.randint(-1, adapters, (tokens,), generator=gen))

    def check():
        assert one.error() == 0 and layer.error() == 0
        offsets, _, order = lu.sort(ids.cpu(), adapters)
        for which, y, b in ((one, y1, base.cpu()), (two, y2, torch.zeros(tokens, n))):
            want, size = lu.low_rank(x.cpu(), which.a.cpu(), which.b.cpu(), which.scales.cpu(), offsets, order, b)
            lu.within(y, want, (k + 3 * rank + 4) * U * size + U * want.abs(), 2.0 ** -8)

    fill()
    step()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        fill()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check()


@pytest.mark.gpu
def test_fewer_tokens_than_the_owners_were_made_for():
    require_gpu()
    say("owners with fewer tokens")
    from lossless_bf16_tensor_exp_amd.codec import ExpertRows, RmsNorm
    gen = torch.Generator().manual_seed(3)
    rows, norm = ExpertRows(5000, 4, 9), RmsNorm(5000, 264)
    for tokens in (5000, 1, 0, 1700, 64):
        ids = lu.choose(gen, tokens, 4, 9)
        rows.sort(ids.cuda())
        offsets, place, order = lu.sort(ids, 9)
        assert torch.equal(rows.offsets.cpu(), offsets) and torch.equal(rows.place.cpu(), place.view(tokens, 4))
        assert torch.equal(rows.order.cpu(), order) and rows.rows() == 4 * tokens and rows.error() == 0
        x = torch.randn(tokens, 264, generator=gen).to(bf16).cuda()
        y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(264, device="cuda")
        norm.forward(x, y)
        norm.backward(y, x, dx, dw)
        s = norm.rstd[:tokens].double()
        want = (y.double() * x.double() * s[:, None]).sum(0)
        room = (tokens + 66) * U * (y.double() * x.double() * s[:, None]).abs().sum(0)
        lu.within(dw, want.cpu(), room.cpu(), U)


@pytest.mark.gpu
def test_no_tokens():
    require_gpu()
    say("a block without tokens")
    b = Block(5, 128, 64, 2, 3)
    b.rows.sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert (b.rows.offsets == 0).all() and b.rows.error() == 0
    none, u = torch.empty(0, 128, dtype=bf16, device="cuda"), torch.empty(0, 64, dtype=bf16, device="cuda")
    b.up.load(torch.ones(3, 64, 128, dtype=bf16, device="cuda"))
    b.up.keep_dispatched(none, b.rows, u)
    dw = torch.full((3, 64, 128), 7.0, device="cuda")
    b.up.backward(u, none, dw, b.rows.offsets)
    assert b.up.error() == 0 and (dw == 0).all()
    b.rows.combine(none, none, torch.empty(0, 2, device="cuda"))
    # tokens, none of them with an expert
    b.rows.sort(torch.full((5, 2), -1, dtype=torch.int32, device="cuda"))
    x, z = torch.ones(5, 128, dtype=bf16, device="cuda"), torch.full((10, 128), float("nan"), dtype=bf16, device="cuda")
    out, w = torch.empty_like(x), torch.full((5, 2), float("nan"), device="cuda")
    b.rows.dispatch(x, out=z)
    b.rows.combine(z, out, w, x)
    assert z.isnan().all() and torch.equal(out, x)
    b.rows.combine_backward(x, z, z, w)
    assert z.isnan().all() and (w == 0).all()


@pytest.mark.gpu
def test_a_stream_of_the_caller():
    """Every call goes to the stream it is given: behind what is queued there, whatever the current one does."""
    require_gpu()
    say("calls on a given stream")
    import lossless_bf16_tensor_exp_amd as c
    gen = torch.Generator().manual_seed(2)
    (x, r, ids, weights, dout), _ = inputs(gen, 300, 256, 64, 2, 5)
    x, r, ids, weights, dout = (t.cuda() for t in (x, r, ids, weights, dout))
    a, b = torch.randn(5, 8, 256, generator=gen).to(bf16).cuda(), torch.randn(5, 256, 8, generator=gen).to(bf16).cuda()
    w = torch.ones(256, dtype=bf16, device="cuda")

    def run(x, stream):
        def new(*shape, dtype=bf16):
            return torch.zeros(*shape, dtype=dtype, device="cuda")

        h, y, dx, rows, drows = new(300, 256), new(300, 256), new(300, 256), new(600, 256), new(600, 256)
        s, dw, dweights, out, z = new(300, dtype=torch.float32), new(256), new(300, 2, dtype=torch.float32), new(300, 256), new(300, 256)
        offsets, place, order = new(6, dtype=torch.int64), new(300, 2, dtype=torch.int32), new(300, dtype=torch.int32)
        ws = [new(n, dtype=torch.uint8) for n in (c.rms_norm_workspace_size(300, 256), c.expert_workspace_size(300, 2, 5),
                                                  c.low_rank_workspace_size(300, 256, 256, 8, 5))]
        one = ids[:, 0].contiguous()
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)  # some 10 ms: what went to another stream would read x before it is there
                x.copy_(later)
        c.rms_norm(x, w, y=y, residual=r, h=h, rstd=s, stream=stream)
        c.expert_sort(ids, offsets, place, None, ws[1], stream=stream)
        c.expert_dispatch(y, place, out=rows, stream=stream)
        c.expert_combine(rows, place, out, weights=weights, residual=h, stream=stream)
        c.expert_combine_backward(dout, rows, place, drows, dweights, weights=weights, stream=stream)
        c.rms_norm_backward(out, h, w, s, dx, dw, ws[0], stream=stream)
        c.expert_sort(one, offsets, place.view(-1)[:300], order, ws[1], stream=stream)
        c.low_rank_add(y, a, b, offsets, z, ws[2], base=out, order=order, stream=stream)
        status = [c.ciera_read_error(t, stream) for t in ws]
        torch.cuda.synchronize()
        assert status == [0, 0, 0]
        return [h, y, dx, rows, drows, s, dw, dweights, out, z, offsets, order]

    later = x.clone()
    want = run(x, None)
    early = torch.zeros_like(x)
    for one, two in zip(want, run(early, torch.cuda.Stream())):
        assert torch.equal(one, two)


def test_owners_refuse():
    from lossless_bf16_tensor_exp_amd.codec import ExpertRows, LowRankAdapters, MxLinear, RmsNorm
    for make in (lambda: RmsNorm(4, 0, device="meta"), lambda: RmsNorm(4, 40000, device="meta"), lambda: ExpertRows(4, 0, 3, device="meta"),
                 lambda: ExpertRows(4, 65, 3, device="meta"), lambda: ExpertRows(4, 2, 0, device="meta"),
                 lambda: ExpertRows(2 ** 26, 32, 3, device="meta"), lambda: LowRankAdapters(4, 8, 8, 129, 2, device="meta"),
                 lambda: LowRankAdapters(4, 8, 8, 4, 0, device="meta")):
        with pytest.raises(ValueError):
            make()
    norm, rows = RmsNorm(4, 8, device="cpu"), ExpertRows(4, 2, 3, device="cpu")
    layer, low = MxLinear(8, 16, 8, 3, device="cpu"), LowRankAdapters(4, 16, 8, 4, 2, device="cpu")

    def zeros(*shape):
        return torch.zeros(*shape, dtype=bf16)

    with pytest.raises(ValueError, match="5 rows"):
        norm.forward(zeros(5, 8), zeros(5, 8))
    with pytest.raises(ValueError, match="no forward pass"):
        norm.backward(zeros(4, 8), zeros(4, 8), zeros(4, 8), None)
    for ids in (torch.zeros(5, 2, dtype=torch.int32), torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError, match="made for"):
            rows.sort(ids)
    rows.place, rows.order = rows._place, rows._order
    for x, y, experts in ((zeros(3, 8), zeros(8, 16), rows), (zeros(4, 7), zeros(8, 16), rows), (zeros(4, 8), zeros(7, 16), rows)):
        with pytest.raises(ValueError):
            layer.keep_dispatched(x, experts, y)
    other = ExpertRows(4, 2, 4, device="cpu")
    other.place, other.order = other._place, other._order
    with pytest.raises(ValueError, match="row numbers"):
        layer.keep_dispatched(zeros(4, 8), other, zeros(8, 16))
    assert layer.kept is None
    small = MxLinear(7, 16, 8, 3, device="cpu")
    with pytest.raises(ValueError, match="made for 7"):
        small.keep_dispatched(zeros(4, 8), rows, zeros(8, 16))
    for a, b in ((zeros(5, 8), zeros(16, 5)), (zeros(4, 7), zeros(16, 4)), (zeros(4, 8), zeros(16, 3))):
        with pytest.raises(ValueError):
            low.load(0, a, b)
    low.load(1, zeros(3, 8) + 1, zeros(16, 3) + 2, 0.5)
    assert (low.a[1, :3] == 1).all() and (low.a[1, 3:] == 0).all() and (low.b[1, :, :3] == 2).all() and low.scales[1] == 0.5
