"""Microscaled matrices on the GPU against a plain 64-bit implementation
(tests/mx_util.py): encoded bytes and decoded values exactly; the products on
whole-number operands, whose FP32 sums are exact in any order, exactly; on
real ones within the bound of an FP32 sum.

That bound: products of two operands are exact in FP32 (8 + 8 significant bits
at most), so a sum of C of them is off by at most C 2^-24 sum |a b|, in any
order; a BF16 output adds half a step, 2^-8 of the value.  mx4_matmul_mx8 to
BF16 may cut, in each block of 32, every product below 2^(E - 13), where 2^E is
the binade of the block's largest: at most 32 * 2^-13 = 2^-8 of the product of
the two blocks' largest values, which is added."""
import pytest

import mx_util as mx
from gpu_util import require_gpu, say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

GUARD = 256


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def lib():
    import lossless_bf16_tensor_exp_amd as ciera
    return ciera


def bits_of(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def strided(t, ld, shift, fill=float("nan")):
    """t on the GPU with rows ld values apart, the first `shift` values into its buffer; `fill` elsewhere."""
    rows, cols = t.shape
    buf = torch.full((shift + rows * ld + 64,), fill, dtype=t.dtype, device="cuda")
    view = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols] if rows else buf[:0].view(0, cols)
    view.copy_(t)
    return buf, view


def same_bytes(got, want):
    got = got.cpu()
    off = (got != want).nonzero().view(-1)
    assert not off.numel(), f"{off.numel()} bytes differ: at {off[:8].tolist()} {got[off[:8]].tolist()} for " \
                            f"{want[off[:8]].tolist()}"


def guarded(nbytes, byte=0xA5):
    return torch.full((nbytes + GUARD,), byte, dtype=torch.uint8, device="cuda")


def mixed(gen, rows, cols):
    """Values of many binades, zeros, subnormals, infinities and NaN among them."""
    x = torch.randn(rows, cols, generator=gen) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=gen).float())
    x = x.to(torch.bfloat16)
    if rows * cols:
        flat = x.view(-1)
        for v in (0.0, -0.0, 1e-39, -3e-40, 9.1e-41, 1e-38, 3.38e38, float("inf"), float("-inf"), float("nan")):
            flat[torch.randint(0, flat.numel(), (1 + flat.numel() // 3000,), generator=gen)] = v
    return x


SHAPES = [(1, 1), (1, 7), (3, 8), (2, 31), (5, 32), (4, 33), (37, 40), (9, 127), (6, 128), (11, 129), (130, 160), (64, 1000),
          (3, 2048), (257, 1408), (1, 8191), (700, 96)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("wider,shift", [(0, 0), (3, 1), (8, 8)])
def test_encode_and_decode(bits, rows, cols, wider, shift):
    say(f"mx{bits} {rows}x{cols} ld+{wider} shift {shift}")
    c = lib()
    gen = torch.Generator().manual_seed(rows * 8192 + cols)
    x = mixed(gen, rows, cols)
    _, xd = strided(x, cols + wider, shift)
    want = mx.encode(bits, x)
    enc, dec = (c.mx8_encode, c.mx8_decode) if bits == 8 else (c.mx4_encode, c.mx4_decode)
    size = (c.mx8_encoded_size if bits == 8 else c.mx4_encoded_size)(rows, cols)
    assert size == want.numel()
    out = guarded(size)
    enc(xd, out[:size])
    same_bytes(out[:size], want)
    assert (out[size:] == 0xA5).all()
    ybuf, y = strided(torch.zeros(rows, cols, dtype=torch.bfloat16), cols + wider, shift, 7.0)
    before = ybuf.clone()
    dec(out[:size], y)
    y64 = mx.decode(bits, want, rows, cols)
    # exact in BF16 unless the rounding took it to 2^128, which is infinity there
    assert torch.equal(torch.nan_to_num(y.cpu().double(), 1e300, 5e300, -5e300),
                       torch.nan_to_num(y64.float().double(), 1e300, 5e300, -5e300))
    assert torch.equal(torch.signbit(y.cpu())[~y64.isnan()], torch.signbit(y64)[~y64.isnan()])
    y.copy_(torch.zeros(rows, cols, dtype=torch.bfloat16))
    assert torch.equal(bits_of(ybuf), bits_of(before)), "a value outside the matrix was written"


@pytest.mark.parametrize("bits", [8, 4])
def test_every_bf16_value(bits):
    say(f"mx{bits} every BF16 value")
    c = lib()
    x = torch.arange(-32768, 32768).to(torch.int16).view(torch.bfloat16)
    for m in (x.view(-1, 32), x.view(32, -1).t().contiguous(), torch.zeros(65536, 32, dtype=torch.bfloat16)):
        if m.shape[0] == 65536:
            m[:, 31] = x
        size = mx.sections(bits, *m.shape)[2]
        out = torch.empty(size, dtype=torch.uint8, device="cuda")
        (c.mx8_encode if bits == 8 else c.mx4_encode)(m.cuda(), out)
        same_bytes(out, mx.encode(bits, m))


def test_nothing_to_encode():
    say("mx empty matrices")
    c = lib()
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    thin = torch.empty(5, 0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((64,), 9, dtype=torch.uint8, device="cuda")
    for enc, dec in ((c.mx8_encode, c.mx8_decode), (c.mx4_encode, c.mx4_decode)):
        for m in (none, thin):
            enc(m, out)
            dec(out, m)
    assert (out == 9).all()


def test_decode_of_a_matrix_made_elsewhere():
    """Scale bytes 1, 254 and 255, every code."""
    say("mx decode, every code and the outer scales")
    c = lib()
    for bits, dec in ((8, c.mx8_decode), (4, c.mx4_decode)):
        line, at, size = mx.sections(bits, 8, 256)
        buf = torch.zeros(size, dtype=torch.uint8)
        codes = torch.arange(256).to(torch.uint8)
        if bits == 8:
            codes[codes % 128 == 127] = 0
        buf[:8 * line] = codes.repeat(8 * line // 256)
        buf[at:] = torch.tensor([1, 2, 127, 130, 253, 254, 255, 120]).to(torch.uint8).repeat(8)
        y = torch.empty(8, 256, dtype=torch.bfloat16, device="cuda")
        dec(buf.cuda(), y)
        want = mx.decode(bits, buf, 8, 256).float().to(torch.bfloat16)
        assert torch.equal(torch.nan_to_num(y.cpu().float(), 7e30), torch.nan_to_num(want.float(), 7e30))


# ------------------------------------------------------------------ products

def whole(gen, rows, cols, most):
    return torch.randint(-most, most + 1, (rows, cols), generator=gen).to(torch.bfloat16)


class Case:
    """Operands of one layer: x, dy, W of `groups` groups, and the rows of each."""

    def __init__(self, seed, tokens, n, k, groups=1, lead=0, tail=0, exact=True, empty=0.3):
        gen = torch.Generator().manual_seed(seed)
        self.tokens, self.n, self.k, self.groups = tokens, n, k, groups
        self.offsets = None
        if groups > 1 or lead or tail:
            self.offsets = mx.split(gen, tokens, groups, empty, lead, tail)
        if exact:  # values that both element types hold under scale 1 (a 6 in every block keeps it there)
            w = torch.tensor([0.0, 1, -1, 2, -2, 3, -3, 4, -4, 6])[torch.randint(0, 10, (groups * n, k), generator=gen)]
            w[:, ::32] = 6.0
            self.w, self.x, self.dy = w.to(torch.bfloat16), whole(gen, tokens, k, 8), whole(gen, tokens, n, 8)
        else:
            self.w = (torch.randn(groups * n, k, generator=gen) * 0.02).to(torch.bfloat16)
            self.x = mx.activations(gen, tokens, k)
            self.dy = mx.activations(gen, tokens, n, 1e-3)
        self.rows = torch.zeros(tokens, dtype=torch.bool)
        for a, b in mx.bounds(self.offsets, tokens):
            self.rows[a:b] = True
        self.x[~self.rows] = float("nan")
        self.dy[~self.rows] = float("nan")
        for g, (a, b) in enumerate(mx.bounds(self.offsets, tokens)):
            if a == b:  # the weights of a group without rows are not used
                self.w[g * n:(g + 1) * n] = float("nan")
        self.wq, self.xq = mx.encode(4, self.w), mx.encode(8, self.x)
        self.w64 = mx.decode(4, self.wq, groups * n, k).view(groups, n, k)
        self.xq64 = mx.decode(8, self.xq, tokens, k)

    def off(self):
        return None if self.offsets is None else self.offsets.cuda()

    def ws(self):
        size = lib().mx_workspace_size(self.tokens, self.n, self.k, self.groups)
        return torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")

    def each(self, op, x):
        """(where, sum, sum of magnitudes, terms) of every group's product in 64 bits."""
        for g, (a, b) in enumerate(mx.bounds(self.offsets, self.tokens)):
            if op == "matmul":
                l, r, at = x[a:b].double(), self.w64[g].t(), slice(a, b)
            elif op == "dx":
                l, r, at = self.dy[a:b].double(), self.w64[g], slice(a, b)
            else:
                l, r, at = self.dy[a:b].double().t(), x[a:b].double(), g
            if a == b and op != "wgrad":
                continue
            yield at, l @ r, l.abs() @ r.abs(), l.shape[1]

    def block_cut(self, at):
        """2^-8 of the sum over blocks of the largest |x| times the largest |w|, for the rows `at` of one group."""
        g = next(i for i, (a, b) in enumerate(mx.bounds(self.offsets, self.tokens)) if (a, b) == (at.start, at.stop))
        tops = []
        for m in (self.xq64[at], self.w64[g]):
            m = torch.nn.functional.pad(m, (0, -self.k % 32)).view(m.shape[0], -1, 32)
            tops.append(m.abs().amax(2))
        return 2.0 ** -8 * tops[0] @ tops[1].t()


def check(case, op, x, out, base, exact, cut=False):
    """out (on the CPU) against the 64-bit product; what belongs to no group still holds `base`."""
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    untouched = torch.ones(out.shape[0], dtype=torch.bool)
    for at, want, mag, terms in case.each(op, x):
        got = out[at]
        if exact:
            assert torch.equal(got, want.to(torch.float32).to(out.dtype)), (op, at)
        else:
            room = terms * 2.0 ** -24 * mag
            if cut:
                room = room + case.block_cut(at)
            room = room + half * (want.abs() + room)
            bad = (got.double() - want).abs() > room
            assert not bad.any() and torch.isfinite(got).all(), (op, at, int(bad.sum()))
        untouched[at] = False
    assert torch.equal(out[untouched], base[untouched])


def run_all(case, out_dtype, exact, ldw=(0, 0), ops=("matmul", "mx8", "dx", "wgrad")):
    """Every product of the case, operands and outputs with rows ldw[0] wider and ldw[1] values into their buffers."""
    c, off = lib(), case.off()
    wq, xq = case.wq.cuda(), case.xq.cuda()
    _, x = strided(case.x, case.k + ldw[0], ldw[1])
    _, dy = strided(case.dy, case.n + ldw[0], ldw[1])
    for op in ops:
        say(f"  {op} tokens {case.tokens} n {case.n} k {case.k} groups {case.groups} {out_dtype} ld+{ldw}")
        ws = case.ws()
        if op == "wgrad":
            for acc in (False, True):
                base = torch.full((case.groups, case.n, case.k), 3.0, dtype=out_dtype)
                buf = torch.full((case.groups * case.n * case.k + 64,), 3.0, dtype=out_dtype, device="cuda")
                dw = buf[:-64].view(case.groups, case.n, case.k)
                c.mx8_wgrad(dy, xq, dw, ws, off, accumulate=acc)
                assert c.ciera_read_error(ws) == 0
                got = dw.cpu()
                if not acc:
                    check(case, op, case.xq64, got, base, exact)
                elif exact:
                    for at, want, _, _ in case.each(op, case.xq64):
                        assert torch.equal(got[at], (want + 3.0).to(torch.float32).to(out_dtype))
                assert (buf[-64:] == 3.0).all()
            continue
        cols = case.k if op == "dx" else case.n
        base = torch.full((case.tokens, cols), 5.0, dtype=out_dtype)
        buf, out = strided(base, cols + ldw[0], ldw[1], 7.0)
        if op == "matmul":
            c.mx4_matmul(x, wq, out, ws, off)
        elif op == "mx8":
            c.mx4_matmul_mx8(xq, case.k, wq, out, ws, off)
        else:
            c.mx4_matmul_dx(dy, wq, out, ws, off)
        assert c.ciera_read_error(ws) == 0
        operand = case.xq64 if op == "mx8" else case.x
        check(case, "dx" if op == "dx" else "matmul", operand, out.cpu(), base, exact,
              cut=op == "mx8" and out_dtype == torch.bfloat16)
        out.fill_(7.0)
        assert (buf == 7.0).all(), "a value outside the output was written"


PRODUCTS = [
    # tokens, n, k, groups, lead, tail
    (1, 1, 1, 1, 0, 0), (1, 16, 128, 1, 0, 0), (1, 64, 40, 1, 0, 0), (2, 17, 129, 1, 0, 0), (16, 48, 256, 1, 0, 0),
    (17, 33, 31, 1, 0, 0), (31, 100, 1000, 1, 0, 0), (33, 130, 200, 1, 0, 0), (64, 128, 64, 1, 0, 0),
    (65, 129, 65, 1, 0, 0), (97, 127, 127, 1, 0, 0), (255, 256, 128, 1, 0, 0), (257, 260, 136, 1, 0, 0),
    (300, 72, 520, 1, 3, 5), (513, 40, 33, 1, 0, 1), (700, 300, 257, 1, 1, 0),
    (40, 50, 96, 7, 2, 3), (64, 96, 128, 64, 0, 0), (90, 130, 70, 3, 0, 9), (500, 80, 100, 70, 0, 0),
    (700, 192, 96, 5, 4, 4), (1200, 64, 72, 3, 0, 11), (130, 20, 40, 130, 0, 0),
]


@pytest.mark.parametrize("shape", PRODUCTS)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_products_of_whole_numbers(shape, out):
    say(f"mx products {shape} {out}")
    run_all(Case(sum(shape), *shape), out, exact=True)


@pytest.mark.parametrize("shape", [PRODUCTS[i] for i in (3, 6, 9, 12, 13, 16, 20)])
@pytest.mark.parametrize("ldw", [(1, 1), (8, 0), (13, 8)])
def test_products_with_strided_rows(shape, ldw):
    say(f"mx products {shape} ld+{ldw}")
    run_all(Case(sum(shape), *shape), torch.bfloat16, exact=True, ldw=ldw)


@pytest.mark.parametrize("shape", [(1, 300, 1408), (37, 256, 2048), (64, 1024, 512, 24), (700, 512, 1000, 4, 0, 9),
                                   (520, 384, 2048), (2100, 256, 96, 2)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_products_of_real_values(shape, out):
    say(f"mx products of real values {shape} {out}")
    run_all(Case(sum(shape), *shape, exact=False), out, exact=False)


def test_a_group_takes_every_row():
    """All rows in one of many groups, first, middle and last."""
    for live in (0, 5, 10):
        say(f"mx products, all rows in group {live} of 11")
        case = Case(live, 600, 70, 90, 11, exact=True, empty=0.0)
        case.offsets = torch.tensor([0] * (live + 1) + [600] * (11 - live))
        run_all(case, torch.float32, exact=True)


def test_no_tokens():
    say("mx products without tokens")
    c = lib()
    wq = mx.encode(4, torch.ones(2 * 40, 64, dtype=torch.bfloat16)).cuda()
    for groups, off in ((1, None), (2, torch.zeros(3, dtype=torch.int64, device="cuda"))):
        ws = torch.full((c.mx_workspace_size(0, 40, 64, groups),), 0x5A, dtype=torch.uint8, device="cuda")
        x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
        y = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
        none = torch.empty(0, dtype=torch.uint8, device="cuda")
        c.mx4_matmul(x, wq, y, ws, off)
        assert c.ciera_read_error(ws) == 0
        c.mx4_matmul_mx8(none, 64, wq, y, ws, off)
        c.mx4_matmul_dx(y, wq, x, ws, off)
        assert c.ciera_read_error(ws) == 0
        dw = torch.ones(groups, 40, 64, device="cuda")
        c.mx8_wgrad(y, none, dw, ws, off, accumulate=True)
        assert (dw == 1).all()
        c.mx8_wgrad(y, none, dw, ws, off)
        assert c.ciera_read_error(ws) == 0 and (dw == 0).all()


@pytest.mark.parametrize("table", [[0, 30, 20, 60], [-1, 20, 40, 60], [0, 20, 40, 61], [60, 40, 20, 0],
                                   [1 << 40, 1 << 41, 0, 60], [-(1 << 62), 1 << 62, 0, 9]])
@pytest.mark.parametrize("n", [40, 200])
def test_offsets_out_of_order_are_reported(table, n):
    """Nothing outside the matrices is touched, and the status says so; the next call is not affected."""
    say(f"mx offsets {table} n {n}")
    c = lib()
    case = Case(1, 60, n, 96, 3, exact=True, empty=0.0)
    off = torch.tensor(table, dtype=torch.int64, device="cuda")
    wq, xq, x, dy, ws = case.wq.cuda(), case.xq.cuda(), case.x.cuda(), case.dy.cuda(), case.ws()
    ybuf, y = strided(torch.zeros(60, n, dtype=torch.bfloat16), n + 8, 8, 7.0)
    xbuf, dx = strided(torch.zeros(60, 96, dtype=torch.bfloat16), 96 + 8, 8, 7.0)
    dw = torch.zeros(3, n, 96, device="cuda")
    for call in (lambda o: c.mx4_matmul(x, wq, y, ws, o), lambda o: c.mx4_matmul_mx8(xq, 96, wq, y, ws, o),
                 lambda o: c.mx4_matmul_dx(dy, wq, dx, ws, o), lambda o: c.mx8_wgrad(dy, xq, dw, ws, o)):
        call(off)
        assert c.ciera_read_error(ws) == c.STATUS_CODES["CIERA_ERR_ARG"]
        call(case.off())
        assert c.ciera_read_error(ws) == 0
    y.fill_(7.0)
    dx.fill_(7.0)
    assert (ybuf == 7.0).all() and (xbuf == 7.0).all()
    run_all(case, torch.float32, exact=True)


def test_non_finite_values_reach_what_depends_on_them():
    """A NaN or an infinity in x, dy or W makes exactly the outputs that use its block (mx) or value NaN or infinite."""
    say("mx products with non-finite values")
    c = lib()
    for tokens in (20, 300):
        case = Case(5, tokens, 150, 200, exact=True)
        wq, ws = case.wq.cuda(), case.ws()
        x, dy = case.x.clone(), case.dy.clone()
        x[7, 199] = float("nan")
        x[11, 0] = float("inf")
        dy[13, 149] = float("nan")
        y = torch.zeros(tokens, 150, device="cuda")
        c.mx4_matmul(x.cuda(), wq, y, ws)
        bad = ~torch.isfinite(y.cpu())
        assert bad[7].all() and bad[11].any() and not bad[[i for i in range(tokens) if i not in (7, 11)]].any()
        xq = mx.encode(8, x).cuda()
        c.mx4_matmul_mx8(xq, 200, wq, y, ws)
        bad = torch.isnan(y.cpu())
        assert bad[7].all() and bad[11].all() and int(bad.any(1).sum()) == 2
        dx = torch.zeros(tokens, 200, device="cuda")
        c.mx4_matmul_dx(dy.cuda(), wq, dx, ws)
        bad = torch.isnan(dx.cpu())
        assert bad[13].all() and int(bad.any(1).sum()) == 1
        dw = torch.zeros(150, 200, device="cuda")
        c.mx8_wgrad(dy.cuda(), xq, dw, ws)
        bad = torch.isnan(dw.cpu())
        cols = torch.zeros(200, dtype=torch.bool)
        cols[192:] = True  # the block of x[7, 199]
        cols[:32] = True   # of x[11, 0]
        want = cols[None, :].expand(150, 200).clone()
        want[149] = True
        assert torch.equal(bad, want)
        w = case.w.clone()
        w[100, 50] = float("nan")
        wq = mx.encode(4, w).cuda()
        c.mx4_matmul(case.x.cuda(), wq, y, ws)
        bad = torch.isnan(y.cpu())
        assert bad[:, 100].all() and int(bad.any(0).sum()) == 1
        c.mx4_matmul_mx8(case.xq.cuda(), 200, wq, y, ws)
        assert torch.equal(torch.isnan(y.cpu()), bad)
        c.mx4_matmul_dx(case.dy.cuda(), wq, dx, ws)
        bad = torch.isnan(dx.cpu())
        assert bad[:, 32:64].all() and int(bad.any(0).sum()) == 32


def test_gradients_against_differences():
    """L = sum(c * y) is linear in x and in W; with whole numbers its
    differences are exact: dx . e = L(x + e) - L(x), dW . e likewise."""
    say("mx gradients against differences")
    c = lib()
    case = Case(9, 90, 60, 70, 4, exact=True)
    gen = torch.Generator().manual_seed(1)
    off, ws = case.off(), case.ws()
    x, dy = torch.nan_to_num(case.x), torch.nan_to_num(case.dy)
    wq = mx.encode(4, torch.nan_to_num(case.w)).cuda()

    def loss(xv, wv):
        y = torch.zeros(90, 60, device="cuda")
        c.mx4_matmul(xv.cuda(), wv, y, ws, off)
        return float((y.cpu().double() * dy.double())[case.rows].sum())

    dx = torch.zeros(90, 70, device="cuda")
    c.mx4_matmul_dx(dy.cuda(), wq, dx, ws, off)
    xq = mx.encode(8, x).cuda()
    dw = torch.zeros(4, 60, 70, device="cuda")
    c.mx8_wgrad(dy.cuda(), xq, dw, ws, off)
    base = loss(x, wq)
    w64 = torch.nan_to_num(case.w).double().view(4, 60, 70)
    for _ in range(4):
        e = whole(gen, 90, 70, 3)
        assert loss(x + e, wq) - base == float((dx.cpu().double() * e.double()).sum())
        move = torch.where(w64.abs() <= 2, torch.randint(-1, 2, w64.shape, generator=gen).double(), 0.0)
        moved = mx.encode(4, (w64 + move).view(240, 70).to(torch.bfloat16)).cuda()
        assert loss(x, moved) - base == float((dw.cpu().double() * move).sum())


def test_calls_repeat_bit_for_bit_and_replay():
    """The same call twice, and replays of a captured layer between eager work, give the same bits."""
    say("mx calls repeated and replayed")
    c = lib()
    for shape in ((24, 96, 256, 5), (900, 200, 264, 3), (400, 256, 256, 1)):
        case = Case(3, *shape, exact=False)
        off = case.off()
        x, dy, wq = torch.nan_to_num(case.x).cuda(), torch.nan_to_num(case.dy).cuda(), case.wq.cuda()
        t, n, k, g = case.tokens, case.n, case.k, case.groups
        xq = torch.zeros(c.mx8_encoded_size(t, k), dtype=torch.uint8, device="cuda")
        outs = [torch.zeros(t, n, device="cuda"), torch.zeros(t, n, device="cuda", dtype=torch.bfloat16),
                torch.zeros(t, k, device="cuda"), torch.zeros(g, n, k, device="cuda")]
        ws = case.ws()

        def layer():
            c.mx8_encode(x, xq)
            c.mx4_matmul(x, wq, outs[0], ws, off)
            c.mx4_matmul_mx8(xq, k, wq, outs[1], ws, off)
            c.mx4_matmul_dx(dy, wq, outs[2], ws, off)
            c.mx8_wgrad(dy, xq, outs[3], ws, off)

        layer()
        first = [bits_of(o).clone() for o in outs]
        layer()
        assert all(torch.equal(bits_of(o), f) for o, f in zip(outs, first))
        x.neg_()
        dy.neg_()
        layer()  # the eager results of the negated operands
        negated = [bits_of(o).clone() for o in outs]
        x.neg_()
        dy.neg_()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph, stream=s):
                layer()
        for i in range(4):
            x.neg_()
            dy.neg_()
            for o in outs:
                o.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for j, (o, f) in enumerate(zip(outs, first if i % 2 else negated)):
                assert torch.equal(bits_of(o), f), (shape, i, j)
            layer()


def test_two_streams_at_once():
    say("mx layers on two streams")
    c = lib()
    case = Case(4, 1500, 320, 256, 6, exact=True)
    sets = []
    for _ in range(2):
        sets.append(dict(x=case.x.cuda(), dy=case.dy.cuda(), w=case.wq.cuda(), xq=case.xq.cuda(), off=case.off(), ws=case.ws(),
                         y=torch.zeros(1500, 320, device="cuda"), dx=torch.zeros(1500, 256, device="cuda"),
                         dw=torch.zeros(6, 320, 256, device="cuda"), s=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(8):
        for d in sets:
            c.mx4_matmul(d["x"], d["w"], d["y"], d["ws"], d["off"], stream=d["s"])
            with torch.cuda.stream(d["s"]):
                c.mx4_matmul_dx(d["dy"], d["w"], d["dx"], d["ws"], d["off"])
            c.mx8_wgrad(d["dy"], d["xq"], d["dw"], d["ws"], d["off"], stream=d["s"])
    torch.cuda.synchronize()
    for d in sets:
        check(case, "matmul", case.x, d["y"].cpu(), torch.zeros(1500, 320), True)
        check(case, "dx", case.x, d["dx"].cpu(), torch.zeros(1500, 256), True)
        check(case, "wgrad", case.xq64, d["dw"].cpu(), torch.zeros(6, 320, 256), True)


def test_binding_refusals():
    say("mx refusals of the binding")
    c = lib()
    case = Case(2, 40, 48, 64, exact=True)
    x, w, xq, ws = case.x.cuda(), case.wq.cuda(), case.xq.cuda(), case.ws()
    y = torch.zeros(40, 48, device="cuda")
    with pytest.raises(ValueError):
        c.mx4_matmul(x, w, torch.zeros(39, 48, device="cuda"), ws)
    with pytest.raises(ValueError):
        c.mx4_matmul(x, w, torch.zeros(48, 40, device="cuda").t(), ws)
    with pytest.raises(TypeError):
        c.mx4_matmul(x, w, y.half(), ws)
    with pytest.raises(TypeError):
        c.mx4_matmul(x.float(), w, y, ws)
    with pytest.raises(ValueError):
        c.mx4_matmul(x, w.cpu(), y, ws)
    with pytest.raises(ValueError):
        c.mx4_matmul(x, w, y, ws, offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        c.mx4_matmul(x, w, y, ws, offsets=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(c.CieraError):
        c.mx4_matmul(x, w[:-1], y, ws)
    with pytest.raises(c.CieraError):
        c.mx4_matmul(x, w, y, ws[:100])
    with pytest.raises(c.CieraError):
        c.mx4_matmul_mx8(xq[:-1], 64, w, y, ws)
    with pytest.raises(ValueError):
        c.mx8_wgrad(y.bfloat16(), xq, torch.zeros(48, 65, device="cuda").t(), ws)
    with pytest.raises(ValueError):
        c.mx8_wgrad(y.bfloat16(), xq, torch.zeros(2, 48, 64, device="cuda"), ws)
    with pytest.raises(c.CieraError):
        c.mx8_encode(x, torch.zeros(100, dtype=torch.uint8, device="cuda"))
