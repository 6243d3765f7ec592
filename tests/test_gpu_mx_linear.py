"""A linear layer's step on microscaled matrices, as a training rank runs it:
weights in 4 bits, the forward pass from an 8-bit checkpoint, both gradients,
and the weights' gradient through the lossless codec, against the 64-bit
formulas (bounds as in test_gpu_mx.py); the layer captured into a graph, and
its refusals."""
import pytest

import mx_util as mx
from gpu_util import require_gpu, say

torch = pytest.importorskip("torch")


def layer_case(gen, tokens, n, k, groups, tail):
    x = mx.activations(gen, tokens, k)
    w = (torch.randn(groups * n, k, generator=gen) * 0.05).to(torch.bfloat16)
    dy = (torch.randn(tokens, n, generator=gen) * 0.01).to(torch.bfloat16)
    offsets = mx.split(gen, tokens, groups, tail=tail) if groups > 1 else None
    return x, w, dy, offsets


def parts(offsets, tokens):
    return enumerate(mx.bounds(offsets, tokens))


def near(got, want, sums, c, half_step, cut=None):
    """|got - want| within an FP32 sum's bound, half a step of the output's type, and what the scaled instructions cut."""
    room = c * 2.0 ** -24 * sums + half_step * (want.abs() + c * 2.0 ** -24 * sums) + 2.0 ** -133
    if cut is not None:
        room = room + cut * (1 + half_step)
    off = (got.double().cpu() - want).abs() - room
    assert (off <= 0).all(), f"off by up to {off.max().item():.3e} more than the bound"


def block_cut(xd, wd):
    """2^-8 of the product of the two blocks' largest values, summed over the blocks of a row pair."""
    blocks = -(-xd.shape[1] // mx.BLOCK)
    xb, wb = (torch.nn.functional.pad(t, (0, blocks * mx.BLOCK - t.shape[1])).view(t.shape[0], blocks, mx.BLOCK).abs().amax(2)
              for t in (xd, wd))
    return xb @ wb.T * 2.0 ** -8


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,n,k,groups,tail", [(1, 96, 200, 1, 0), (70, 256, 128, 1, 0), (300, 160, 320, 5, 7),
                                                    (2100, 128, 256, 1, 0), (1500, 72, 136, 3, 11)])
def test_step_and_gradient_exchange(tokens, n, k, groups, tail):
    require_gpu()
    from lossless_bf16_tensor_exp_amd.codec import MxLinear, Zip3Codec
    say(f"layer {tokens} x {n} x {k} in {groups}")
    gen = torch.Generator().manual_seed(tokens + n)
    x, w, dy, offsets = layer_case(gen, tokens, n, k, groups, tail)
    table = None if offsets is None else offsets.cuda()
    layer = MxLinear(tokens + 3, n, k, groups)
    layer.load(w.cuda().view(groups, n, k))
    mark = 7.0
    y = torch.full((tokens, n), mark, dtype=torch.bfloat16, device="cuda")
    ys = torch.full((tokens, n), mark, device="cuda")
    dx = torch.full((tokens, k), mark, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(groups, n, k, dtype=torch.bfloat16, device="cuda")
    layer.forward(x.cuda(), ys, table)
    assert layer.error() == 0
    layer.keep(x.cuda(), y, table)
    assert layer.error() == 0
    layer.backward(dy.cuda(), dx, dw, table)
    assert layer.error() == 0

    wd = mx.decode(4, mx.encode(4, w), groups * n, k)
    xd = mx.decode(8, mx.encode(8, x), tokens, k)
    live = torch.zeros(tokens, dtype=torch.bool)
    for g, (a, b) in parts(offsets, tokens):
        live[a:b] = True
        wg, xg, xe, dg = wd[g * n:(g + 1) * n], xd[a:b], x[a:b].double(), dy[a:b].double()
        near(ys[a:b], xe @ wg.T, xe.abs() @ wg.abs().T, k, 2.0 ** -24)
        near(y[a:b], xg @ wg.T, xg.abs() @ wg.abs().T, k, 2.0 ** -8, block_cut(xg, wg))
        near(dx[a:b], dg @ wg, dg.abs() @ wg.abs(), n, 2.0 ** -8)
        near(dw[g], dg.T @ xg, dg.abs().T @ xg.abs(), b - a, 2.0 ** -8)
    for t in (y, ys, dx):
        assert (t.cpu()[~live] == mark).all(), "rows of no group were written"

    # the gradient as a rank sends it, on the same stream
    zip3 = Zip3Codec(dw.numel())
    zip3.encode(dw)
    size = zip3.nbytes()
    back = torch.empty_like(dw)
    zip3.decode(zip3.out, size, back)
    assert zip3.error() == 0
    assert torch.equal(back.view(torch.int16), dw.view(torch.int16))

    # a second microbatch on top
    layer.backward(dy.cuda(), None, back, table, accumulate=True)
    for g, (a, b) in parts(offsets, tokens):
        first, more = dw[g].double().cpu(), dy[a:b].double().T @ xd[a:b]
        near(back[g], first + more, dy[a:b].double().abs().T @ xd[a:b].abs() + first.abs(), b - a + 1, 2.0 ** -8)


@pytest.mark.gpu
def test_fewer_rows_than_the_layer_was_made_for():
    """Few rows go through other kernels and parts than many; one layer's workspace serves all."""
    require_gpu()
    from lossless_bf16_tensor_exp_amd.codec import MxLinear
    n, k = 4096, 4224
    gen = torch.Generator().manual_seed(9)
    w = torch.tensor([0.0, 1, -1, 2, -2, 3, 6])[torch.randint(0, 7, (n, k), generator=gen)]
    w[:, ::32] = 6.0
    layer = MxLinear(700, n, k)
    layer.load(w.to(torch.bfloat16).cuda())
    for tokens in (1, 40, 130, 700, 3):
        say(f"layer of 700 with {tokens} rows")
        x, dy = (torch.randint(-8, 9, (tokens, c), generator=gen).to(torch.bfloat16) for c in (k, n))
        y = torch.zeros(tokens, n, device="cuda")
        dx = torch.zeros(tokens, k, device="cuda")
        dw = torch.zeros(n, k, device="cuda")
        layer.keep(x.cuda(), y)
        layer.backward(dy.cuda(), dx, dw)
        assert layer.error() == 0
        # whole numbers below 2^24: FP32 holds every partial sum exactly
        assert torch.equal(y.cpu(), x.float() @ w.t())
        assert torch.equal(dx.cpu(), dy.float() @ w)
        assert torch.equal(dw.cpu(), dy.float().t() @ x.float())


@pytest.mark.gpu
def test_captured_step_takes_new_weights_and_rows():
    """keep and backward in one graph: each replay sees what the buffers hold then, the offsets included."""
    require_gpu()
    from lossless_bf16_tensor_exp_amd.codec import MxLinear
    tokens, n, k, groups = 520, 96, 160, 3
    gen = torch.Generator().manual_seed(5)
    x, w, dy, offsets = [t.cuda() for t in layer_case(gen, tokens, n, k, groups, 4)]
    layer, own = MxLinear(tokens, n, k, groups), MxLinear(tokens, n, k, groups)
    out = [torch.zeros(tokens, n, device="cuda"), torch.zeros(tokens, k, device="cuda"),
           torch.zeros(groups, n, k, device="cuda")]

    def step(which, out):
        which.load(w)
        which.keep(x, out[0], offsets)
        which.backward(dy, out[1], out[2], offsets)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layer, out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(layer, out)
    for i in range(4):
        nx, nw, ndy, noff = layer_case(gen, tokens, n, k, groups, 4)
        for t, new in ((x, nx), (w, nw), (dy, ndy), (offsets, noff)):
            t.copy_(new)
        for t in out:
            t.fill_(float(i))
        want = [torch.full_like(t, float(i)) for t in out]
        step(own, want)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, t in zip(out, want):
            assert torch.equal(got, t), f"replay {i}"
        assert layer.error() == 0


@pytest.mark.gpu
def test_refusals():
    require_gpu()
    from lossless_bf16_tensor_exp_amd.codec import MxLinear
    layer = MxLinear(8, 16, 32, 2)
    x = torch.zeros(8, 32, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([0, 3, 8], device="cuda")
    with pytest.raises(ValueError):
        layer.load(torch.zeros(16, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        layer.forward(x, y)
    with pytest.raises(ValueError):
        layer.keep(x[:, :16], y, offsets)
    with pytest.raises(ValueError):
        layer.keep(torch.zeros(9, 32, dtype=torch.bfloat16, device="cuda"), torch.zeros(9, 16, device="cuda"), offsets)
    with pytest.raises(ValueError):
        layer.backward(y, None, torch.zeros(2, 16, 32, device="cuda"), offsets)  # nothing was kept
    layer.keep(x, y, offsets)
    with pytest.raises(ValueError):
        layer.backward(y[:5], None, torch.zeros(2, 16, 32, device="cuda"), offsets)
    with pytest.raises(ValueError):
        layer.backward(y, x, None, offsets[:2])
    layer.forward(x, y, torch.tensor([0, 9, 8], device="cuda"))
    assert layer.error() == 1  # CIERA_ERR_ARG


def test_sizes_out_of_range():
    from lossless_bf16_tensor_exp_amd.codec import MxLinear
    for args in ((4, 0, 32), (4, 16, 0), (4, 16, 32, 0), (2 ** 31, 16, 32), (4, 2 ** 21, 32, 4096)):
        with pytest.raises(ValueError):
            MxLinear(*args, device="meta")
