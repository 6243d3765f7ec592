"""The microscaled products at sizes that reach each tile shape, the
contraction in parts, and offsets past 32 bits, on whole-number operands whose
FP32 sums are exact in any order (so are sums of parts); what lies behind a
contraction's end; two captured graphs on one workspace."""
import pytest

import mx_util as mx
from gpu_util import require_gpu, say
from test_gpu_mx import Case, lib, run_all

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("shape", [
    # tokens, n, k, groups, lead, tail: large, middling and small outputs of the products along k ...
    (8200, 2050, 72), (4200, 1600, 100), (2100, 1100, 136), (1500, 1030, 72, 3, 2, 7),
    # ... and along n
    (8200, 72, 2050), (4200, 100, 1600), (2100, 136, 1100, 5, 0, 9), (3000, 40, 1300, 40),
])
def test_tile_shapes(shape):
    say(f"mx products {shape}")
    out = torch.bfloat16 if shape[0] % 200 else torch.float32
    case = Case(sum(shape), *shape)
    run_all(case, out, exact=True)
    run_all(case, torch.float32 if out == torch.bfloat16 else torch.bfloat16, exact=True, ops=("mx8",))


@pytest.mark.parametrize("shape", [(1, 512, 40), (40, 2500, 260), (64, 1030, 127), (100, 1300, 136, 3, 2, 5), (190, 600, 33, 4)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ldw", [(0, 0), (5, 3)])
def test_dx_in_parts(shape, out, ldw):
    """Few rows: n is split; rows of no group and what lies between the rows stay as they were."""
    say(f"mx dx in parts {shape} {out} ld+{ldw}")
    run_all(Case(sum(shape), *shape), out, exact=True, ldw=ldw, ops=("dx",))


@pytest.mark.parametrize("shape", [(9000, 40, 96), (5000, 33, 35, 2, 1, 3), (4099, 300, 130), (1024, 8, 8), (1023, 8, 8)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_wgrad_in_parts(shape, out):
    say(f"mx wgrad in parts {shape} {out}")
    run_all(Case(sum(shape), *shape), out, exact=True, ops=("wgrad",))


def test_infinity_in_the_last_row_of_a_contraction():
    """The steps past a contraction's end repeat nothing: an infinity in its last row stays one, times a non-zero value."""
    c = lib()
    for n, tokens in ((65, 3), (33, 200), (600, 20), (47, 1)):
        say(f"mx infinity n {n} tokens {tokens}")
        k = 70
        gen = torch.Generator().manual_seed(n)
        w = torch.ones(n, k, dtype=torch.bfloat16)
        x = torch.ones(tokens, k, dtype=torch.bfloat16)
        dy = (torch.randint(0, 2, (tokens, n), generator=gen) * 2 - 1).to(torch.bfloat16)
        wq, xq = mx.encode(4, w), mx.encode(8, x)
        _, wat, wsize = mx.sections(4, n, k)
        _, xat, xsize = mx.sections(8, tokens, k)
        wq[wat + (n - 1) * 4 + 1] = 254  # columns 32 .. 63 of the last row: 6 * 2^127
        xq[xat + (tokens - 1) * 4 + 2] = 254  # columns 64 .. 69
        wd, xd = mx.decode(4, wq, n, k), mx.decode(8, xq, tokens, k)
        wd[n - 1, 32:64], xd[tokens - 1, 64:] = float("inf"), float("inf")
        ws = torch.empty(c.mx_workspace_size(tokens, n, k, 1), dtype=torch.uint8, device="cuda")
        dx = torch.zeros(tokens, k, device="cuda")
        dw = torch.zeros(n, k, device="cuda")
        c.mx4_matmul_dx(dy.cuda(), wq.cuda(), dx, ws)
        c.mx8_wgrad(dy.cuda(), xq.cuda(), dw, ws)
        for got, want in ((dx, dy.double() @ wd), (dw, dy.double().t() @ xd)):
            assert torch.equal(got.cpu().double(), want)


def test_offsets_past_32_bits():
    """Rows past 4 GiB of x, of its checkpoint and of dx."""
    c = lib()
    tokens, n, k, base = 2 ** 21 + 77, 24, 2048, 1000
    say(f"mx {tokens} x {n} x {k}")
    case = Case(3, base, n, k)
    at = torch.arange(tokens, device="cuda") % base
    x = case.x.cuda()[at]
    xq = torch.empty(c.mx8_encoded_size(tokens, k), dtype=torch.uint8, device="cuda")
    assert xq.numel() > 2 ** 32
    c.mx8_encode(x, xq)
    back = torch.empty_like(x)
    c.mx8_decode(xq, back)
    assert torch.equal(back, x)  # whole numbers up to 8 are held as they are
    del back
    ws = torch.empty(c.mx_workspace_size(tokens, n, k, 1), dtype=torch.uint8, device="cuda")
    wq = case.wq.cuda()
    want = (case.x.double() @ case.w64[0].t()).float().cuda()[at]
    y = torch.empty(tokens, n, device="cuda")
    c.mx4_matmul(x, wq, y, ws)
    assert torch.equal(y, want)
    c.mx4_matmul_mx8(xq, k, wq, y.zero_(), ws)
    assert torch.equal(y, want)
    del x
    dy = case.dy.cuda()[at]
    dx = torch.empty(tokens, k, dtype=torch.bfloat16, device="cuda")
    c.mx4_matmul_dx(dy, wq, dx, ws)
    want = (case.dy.double() @ case.w64[0]).to(torch.bfloat16).cuda()
    for a in (0, 2 ** 20, tokens - 100000):
        assert torch.equal(dx[a:a + 100000], want[at[a:a + 100000]])
    dy[:tokens - 500] = 0
    dw = torch.empty(n, k, device="cuda")
    c.mx8_wgrad(dy, xq, dw, ws)
    rows = at[tokens - 500:].cpu()
    assert torch.equal(dw.cpu(), (case.dy[rows].double().t() @ case.x[rows].double()).float())


def test_two_graphs_share_a_workspace():
    """Products in parts leave nothing in the workspace that a later one takes."""
    say("mx two graphs")
    c = lib()
    cases = [Case(1, 2100, 40, 96), Case(2, 60, 1100, 72)]
    ws = torch.full((max(c.mx_workspace_size(s.tokens, s.n, s.k, 1) for s in cases),), 0xFF, dtype=torch.uint8, device="cuda")
    held, graphs = [], []
    for s in cases:
        t = dict(dy=s.dy.cuda(), wq=s.wq.cuda(), xq=s.xq.cuda(), dx=torch.zeros(s.tokens, s.k, device="cuda"),
                 dw=torch.zeros(s.n, s.k, device="cuda"))

        def step(t=t):
            c.mx4_matmul_dx(t["dy"], t["wq"], t["dx"], ws)
            c.mx8_wgrad(t["dy"], t["xq"], t["dw"], ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        held.append(t)
        graphs.append(g)
    for turn in range(3):
        for t in held:
            t["dx"].zero_()
            t["dw"].zero_()
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        for s, t in zip(cases, held):
            assert torch.equal(t["dx"].cpu(), (s.dy.double() @ s.w64[0]).float())
            assert torch.equal(t["dw"].cpu(), (s.dy.double().t() @ s.xq64).float())
        assert c.ciera_read_error(ws) == 0
