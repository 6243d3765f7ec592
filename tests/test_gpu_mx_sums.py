"""The sums of mx4_matmul_mx8.  Operands whose products span many binades and
whose loud parts cancel, so that what an FP32 sum keeps is the whole result:
every product and every partial sum is a whole number of units below 2^24 in
magnitude, so FP32 holds all of them exactly, in any order, and the results
(at most eight significant bits) are exact in BF16 too.  And what the scaled
matrix instructions (scaled=True) may cut of such a sum, and no more."""
import pytest

import mx_util as mx
from gpu_util import require_gpu, say
from test_gpu_mx import lib

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def loud_and_quiet(gen, tokens, n, k, groups):
    """Encoded x and W: in every second block a loud product of 2^9 or -2^9, which the next block's takes away, beside
    quiet ones of 2^-10 .. 2^-6, a handful of them so that their sum has at most eight bits of 2^-10."""
    blocks = k // mx.BLOCK
    x, w = torch.zeros(tokens, blocks, mx.BLOCK), torch.zeros(groups * n, blocks, mx.BLOCK)
    x[:, :, 0] = 128.0
    w[:, 0::2, 0] = 4.0
    w[:, 1::2, 0] = -4.0
    for _ in range(6):
        b, i = (int(torch.randint(0, top, (1,), generator=gen)) for top in (blocks, mx.BLOCK - 1))
        x[:, b, 1 + i] = 2.0 ** -torch.randint(5, 10, (tokens,), generator=gen).float()
        w[:, b, 1 + i] = torch.randint(0, 2, (groups * n,), generator=gen) - 0.5
    x, w = x.view(tokens, k).to(torch.bfloat16), w.view(groups * n, k).to(torch.bfloat16)
    # values as they are: every scale is 1 (the encoder's own would be smaller, and hold them as well)
    def raw(bits, m):
        rows, cols = m.shape
        code = mx._nearest_code(bits, m.double())
        if bits == 4:
            code = code[:, 0::2] | (code[:, 1::2] << 4)
        line, at, size = mx.sections(bits, rows, cols)
        out = torch.zeros(size, dtype=torch.uint8)
        out[:rows * line].view(rows, line)[:, :code.shape[1]] = code.to(torch.uint8)
        out[at:] = 127
        return out
    xq, wq = raw(8, x), raw(4, w)
    assert torch.equal(mx.decode(8, xq, tokens, k), x.double()) and torch.equal(mx.decode(4, wq, groups * n, k), w.double())
    return xq, wq, x.double(), w.double().view(groups, n, k)


SHAPES = [(1, 40, 256, 1), (3, 2048, 512, 1), (40, 4000, 128, 1), (100, 1400, 192, 1), (33, 300, 256, 5), (300, 520, 320, 3),
          (2100, 1100, 192, 1), (6200, 1030, 256, 1), (8200, 2050, 320, 1)]


@pytest.mark.parametrize("tokens,n,k,groups", SHAPES)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_sums_are_fp32_whatever_the_output(tokens, n, k, groups, out):
    say(f"mx8 sums {tokens} x {n} x {k} in {groups} to {out}")
    c = lib()
    gen = torch.Generator().manual_seed(tokens + n)
    xq, wq, x, w = loud_and_quiet(gen, tokens, n, k, groups)
    offsets = mx.split(gen, tokens, groups) if groups > 1 else None
    want = torch.zeros(tokens, n, dtype=torch.float64)
    for g, (a, b) in enumerate(mx.bounds(offsets, tokens)):
        want[a:b] = x[a:b] @ w[g].t()
    assert torch.equal(want.to(out).double(), want) and (want != 0).any()
    y = torch.full((tokens, n), 5.0, dtype=out, device="cuda")
    ws = torch.empty(c.mx_workspace_size(tokens, n, k, groups), dtype=torch.uint8, device="cuda")
    c.mx4_matmul_mx8(xq.cuda(), k, wq.cuda(), y, ws, None if offsets is None else offsets.cuda())
    assert c.ciera_read_error(ws) == 0
    assert torch.equal(y.cpu().double(), want)


@pytest.mark.parametrize("tokens,n,k,groups", SHAPES)
def test_scaled_cuts_no_more_than_documented(tokens, n, k, groups):
    """A quiet product loses less than 2^(E - 13), 2^E being the binade of its block's largest: 2^-4 beside the loud 2^9.
    The loud products cancel across blocks, so nothing larger hides a larger loss; half a step of the output's type is
    2^-8 of the value."""
    say(f"mx8 scaled sums {tokens} x {n} x {k} in {groups}")
    c = lib()
    gen = torch.Generator().manual_seed(tokens + n)
    xq, wq, x, w = loud_and_quiet(gen, tokens, n, k, groups)
    offsets = mx.split(gen, tokens, groups) if groups > 1 else None
    y = torch.zeros(tokens, n, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(c.mx_workspace_size(tokens, n, k, groups), dtype=torch.uint8, device="cuda")
    c.mx4_matmul_mx8(xq.cuda(), k, wq.cuda(), y, ws, None if offsets is None else offsets.cuda(), scaled=True)
    assert c.ciera_read_error(ws) == 0
    for g, (a, b) in enumerate(mx.bounds(offsets, tokens)):
        want = x[a:b] @ w[g].t()
        xb, wb = x[a:b].view(b - a, k // mx.BLOCK, mx.BLOCK), w[g].view(n, k // mx.BLOCK, mx.BLOCK)
        quiet = (xb[:, :, 1:] != 0).double().flatten(1) @ (wb[:, :, 1:] != 0).double().flatten(1).t()
        room = quiet * 2.0 ** -4
        room = room + 2.0 ** -8 * (want.abs() + room)
        assert ((y[a:b].cpu().double() - want).abs() <= room).all(), g


def block_scales(gen, bits, rows, cols):
    """Encoded whole numbers of few bits whose scales differ from block to block, and what they stand for."""
    top, spread = (3, 5) if bits == 8 else (4, 4)
    m = torch.randint(-top, top + 1, (rows, cols), generator=gen).to(torch.bfloat16)
    m[:, ::mx.BLOCK] = top  # so a block's own scale is the same everywhere
    q = mx.encode(bits, m)
    _, at, _ = mx.sections(bits, rows, cols)
    q[at:] += torch.randint(0, spread, q[at:].shape, generator=gen).to(torch.uint8)
    return q, mx.decode(bits, q, rows, cols)


@pytest.mark.parametrize("tokens,n,k,groups", [(1, 40, 260, 1), (40, 4000, 129, 1), (100, 1400, 1100, 1), (300, 520, 1300, 3),
                                               (8200, 1030, 1100, 1), (6600, 2050, 2100, 5)])
def test_every_block_gets_its_own_scale(tokens, n, k, groups):
    """Products of at most 6 bits, 2^6 apart within a block: nothing is cut, and the sums are whole numbers below 2^24
    (12 2^7 k at the most), so they are exact, scaled or not."""
    assert 12 * 2 ** 7 * k < 2 ** 24
    say(f"mx8 block scales {tokens} x {n} x {k} in {groups}")
    c = lib()
    gen = torch.Generator().manual_seed(tokens + k)
    xq, x = block_scales(gen, 8, tokens, k)
    wq, w = block_scales(gen, 4, groups * n, k)
    offsets = mx.split(gen, tokens, groups, empty=0.0) if groups > 1 else None
    want = torch.zeros(tokens, n)
    for g, (a, b) in enumerate(mx.bounds(offsets, tokens)):
        want[a:b] = x[a:b].float() @ w[g * n:(g + 1) * n].t().float()  # exact in FP32 too
    ws = torch.empty(c.mx_workspace_size(tokens, n, k, groups), dtype=torch.uint8, device="cuda")
    for scaled, dtype in ((False, torch.float32), (False, torch.bfloat16), (True, torch.bfloat16)):
        y = torch.zeros(tokens, n, dtype=dtype, device="cuda")
        c.mx4_matmul_mx8(xq.cuda(), k, wq.cuda(), y, ws, None if offsets is None else offsets.cuda(), scaled=scaled)
        assert c.ciera_read_error(ws) == 0
        assert torch.equal(y.cpu(), want.to(dtype)), (scaled, dtype)


def test_scaled_is_for_a_bf16_output():
    c = lib()
    x = torch.zeros(c.mx8_encoded_size(8, 64), dtype=torch.uint8, device="cuda")
    w = torch.zeros(c.mx4_encoded_size(16, 64), dtype=torch.uint8, device="cuda")
    ws = torch.empty(c.mx_workspace_size(8, 16, 64, 1), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        c.mx4_matmul_mx8(x, 64, w, torch.zeros(8, 16, device="cuda"), ws, scaled=True)
    c.mx4_matmul_mx8(x[:0], 64, w, torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda"), ws, scaled=True)
    assert c.ciera_read_error(ws) == 0


def test_layer_chooses():
    """MxLinear's keep: FP32 sums, or the scaled instructions where the layer was made for them and y is BF16."""
    from lossless_bf16_tensor_exp_amd.codec import MxLinear
    say("mx layer, scaled and not")
    c = lib()
    gen = torch.Generator().manual_seed(3)
    tokens, n, k = 70, 96, 320
    x = mx.activations(gen, tokens, k).cuda()
    w = (torch.randn(n, k, generator=gen) * 0.05).to(torch.bfloat16).cuda()
    for scaled in (False, True):
        layer = MxLinear(tokens, n, k, scaled=scaled)
        layer.load(w)
        for dtype in (torch.bfloat16, torch.float32):
            y, want = (torch.zeros(tokens, n, dtype=dtype, device="cuda") for _ in range(2))
            layer.keep(x, y)
            c.mx4_matmul_mx8(layer.xq, k, layer.w, want, layer.ws, scaled=scaled and dtype == torch.bfloat16)
            assert torch.equal(y, want)
            assert layer.error() == 0


def test_values_past_bf16():
    """6 * 2^127 is infinite as BF16, and in the sums of BF16 products; the scaled instructions take it as it is."""
    say("mx8 values past BF16")
    c = lib()
    k = 96
    for tokens, n in ((2, 40), (300, 200)):
        x, w = torch.zeros(tokens, k, dtype=torch.bfloat16), torch.zeros(n, k, dtype=torch.bfloat16)
        x[:, 40], w[:, 40] = 2.0 ** -30, 6.0
        xq, wq = mx.encode(8, x), mx.encode(4, w)
        wq[mx.sections(4, n, k)[1]:] = 254
        ws = torch.empty(c.mx_workspace_size(tokens, n, k, 1), dtype=torch.uint8, device="cuda")
        y = torch.zeros(tokens, n, dtype=torch.bfloat16, device="cuda")
        c.mx4_matmul_mx8(xq.cuda(), k, wq.cuda(), y, ws)
        assert (y == float("inf")).all()
        c.mx4_matmul_mx8(xq.cuda(), k, wq.cuda(), y, ws, scaled=True)
        assert (y == 6 * 2.0 ** 97).all()
