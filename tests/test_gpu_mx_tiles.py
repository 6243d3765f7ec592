"""Every kernel and tile of the microscaled products on a contraction long and
uneven enough to go round its ring of steps, and past the scale bytes that it
holds at a time, more than once; scales differ from block to block.  Operands
are whole numbers whose sums stay below 2^24, so FP32 holds them exactly in any
order.  Without a GPU: the list reaches every choice that the rules can make."""
import pytest

import mx_rules
import mx_util as mx
from gpu_util import require_gpu, say
from test_gpu_mx import Case, check, lib, run_all, strided

torch = pytest.importorskip("torch")

# op, kernel, (tokens, n, k, groups, lead, tail)
TILES = [
    ("bf16", "few16", (40, 300, 2100)), ("bf16", "few16", (90, 130, 1100, 7, 2, 3)),
    ("bf16", "few128", (5, 17000, 1100)), ("bf16", "few128", (70, 1030, 1300, 60, 1, 2)),
    ("bf16", "32x128", (200, 1030, 1500)), ("bf16", "32x128", (900, 520, 1100, 40, 0, 3)),
    ("bf16", "64x128", (2100, 1100, 1300)), ("bf16", "64x128", (3000, 700, 1100, 9, 5, 0)),
    ("bf16", "128x128", (4200, 1600, 1100)), ("bf16", "128x128", (3100, 2050, 1100, 4, 1, 1)),
    ("bf16", "128x256", (8200, 2050, 1100)), ("bf16", "128x256", (7000, 2600, 1100, 6, 0, 7)),
    ("mx8", "few16", (60, 300, 2100)), ("mx8", "few16", (90, 130, 1100, 7, 2, 3)),
    ("mx8", "few128", (5, 17000, 1100)), ("mx8", "few128", (70, 1030, 1300, 60, 1, 2)),
    ("mx8", "64x128", (300, 1030, 1500)), ("mx8", "64x128", (900, 520, 1100, 40, 0, 3)),
    ("mx8", "128x128", (4200, 1600, 1100)), ("mx8", "128x128", (7000, 2600, 1100, 6, 0, 7)),
    ("mx8", "128x256", (8200, 2050, 1100)),
    ("scaled", "32x128", (200, 1030, 1500)), ("scaled", "32x128", (900, 520, 2100, 40, 0, 3)),
    ("scaled", "64x128", (2100, 1100, 1300)), ("scaled", "64x128", (3000, 700, 2100, 9, 5, 0)),
    ("scaled", "128x256", (4200, 1600, 2100)), ("scaled", "128x256", (7000, 1300, 1300, 6, 0, 7)),
    ("dx", "64x128", (2100, 1100, 1030)), ("dx", "64x128", (2000, 1100, 520, 9, 3, 0)),
    ("dx", "32x256", (1000, 600, 1300, 60, 2, 5)), ("dx", "32x256", (1500, 1100, 1030, 90)),
    ("dx", "64x256", (4200, 1100, 2050)), ("dx", "64x256", (5000, 700, 1300, 12, 0, 9)),
    ("dx", "128x256", (8200, 1100, 2050)), ("dx", "128x256", (17000, 600, 3900, 3, 1, 2)),
    ("wgrad", "256x128", (1023, 300, 130)), ("wgrad", "256x128", (1500, 260, 300, 3, 4, 5)),
]
# what each operator's rule can answer, and the contraction values of a step of its kernels
CHOICES = {"bf16": {"few16", "few128", "32x128", "64x128", "128x128", "128x256"}, "mx8": {"few16", "few128", "64x128", "128x128", "128x256"},
           "scaled": {"32x128", "64x128", "128x256"}, "dx": {"64x128", "32x256", "64x256", "128x256"}, "wgrad": {"256x128"}}
STEP = {"bf16": 64, "mx8": 64, "scaled": 128, "dx": 64, "wgrad": 32}
IDS = [f"{op}-{name}-{'x'.join(map(str, s))}" for op, name, s in TILES]


def test_the_list_reaches_every_kernel():
    for op, want in CHOICES.items():
        assert {name for o, name, _ in TILES if o == op} == want, op


@pytest.mark.parametrize("op,name,shape", TILES, ids=IDS)
def test_a_case_reaches_its_kernel(op, name, shape):
    tokens, n, k, groups, lead, tail = (*shape, 1, 0, 0)[:6] if len(shape) == 3 else (*shape, 0, 0)[:6]
    table = groups > 1 or lead > 0 or tail > 0
    if op == "wgrad":
        assert mx_rules.rules().wgrad_parts(tokens, n, k, groups) == 1
        assert tokens // groups // STEP[op] >= 9
        return
    assert mx_rules.kernel(op, tokens, n, k, groups, table) == name
    contraction = n if op == "dx" else k
    if op == "dx":
        assert mx_rules.rules().dx_parts(tokens, n, k, groups) == 1
    assert contraction // STEP[op] >= 9 and contraction % STEP[op]


def test_every_choice_is_known():
    """No sizes choose a kernel that the lists above leave out."""
    sizes = [1, 3, 17, 48, 49, 65, 130, 300, 700, 1030, 2050, 4100, 8200, 20000, 70000]
    for op, known in CHOICES.items():
        if op == "wgrad":
            continue
        for tokens in sizes:
            for n in sizes:
                for k in (64, 1100, 2050, 8200):
                    for groups in (1, 2, 8, 64, 1000):
                        assert mx_rules.kernel(op, tokens, n, k, groups) in known


class Scaled(Case):
    """Whole numbers whose blocks have scales of their own: a block's values are times 1 .. 4 (W) or 1 .. 8 (x)."""

    def __init__(self, seed, *shape):
        super().__init__(seed, *shape, exact=True)
        gen = torch.Generator().manual_seed(seed + 1)
        for bits, buf, rows, spread in ((4, self.wq, self.groups * self.n, 3), (8, self.xq, self.tokens, 4)):
            at = mx.sections(bits, rows, self.k)[1]
            more = torch.randint(0, spread, buf[at:].shape, generator=gen).to(torch.uint8)
            buf[at:] += torch.where(buf[at:] == 255, torch.zeros_like(more), more)
        self.w64 = mx.decode(4, self.wq, self.groups * self.n, self.k).view(self.groups, self.n, self.k)
        self.xq64 = mx.decode(8, self.xq, self.tokens, self.k)
        assert 64 * 24 * self.k < 2 ** 24 and 8 * 24 * self.n < 2 ** 24 and 8 * 64 * self.tokens < 2 ** 24


def run_scaled(case, ldw):
    c = lib()
    base = torch.full((case.tokens, case.n), 5.0, dtype=torch.bfloat16)
    buf, out = strided(base, case.n + ldw[0], ldw[1], 7.0)
    ws = case.ws()
    c.mx4_matmul_mx8(case.xq.cuda(), case.k, case.wq.cuda(), out, ws, case.off(), scaled=True)
    assert c.ciera_read_error(ws) == 0
    # a block's products lie within 2^6 of each other: the instructions cut none of them
    check(case, "matmul", case.xq64, out.cpu(), base, True)
    out.fill_(7.0)
    assert (buf == 7.0).all(), "a value outside the output was written"


@pytest.mark.gpu
@pytest.mark.parametrize("op,name,shape", TILES, ids=IDS)
def test_long_contraction(op, name, shape):
    require_gpu()
    say(f"mx {op} {name} {shape}")
    case = Scaled(sum(shape), *shape)
    strides = [(0, 0), (5, 3)]
    if op == "scaled":
        for ldw in strides:
            run_scaled(case, ldw)
        return
    ops = ({"bf16": "matmul"}.get(op, op),)
    for ldw in strides:
        for out in (torch.bfloat16, torch.float32):
            run_all(case, out, exact=True, ldw=ldw, ops=ops)


@pytest.mark.gpu
@pytest.mark.parametrize("op,name,shape", [t for t in TILES if len(t[2]) == 3],
                         ids=[i for i, t in zip(IDS, TILES) if len(t[2]) == 3])
def test_long_contraction_of_real_values(op, name, shape):
    require_gpu()
    say(f"mx {op} {name} {shape} of real values")
    case = Case(sum(shape), *shape, exact=False)
    if op == "scaled":
        c = lib()
        y = torch.zeros(case.tokens, case.n, dtype=torch.bfloat16, device="cuda")
        ws = case.ws()
        c.mx4_matmul_mx8(case.xq.cuda(), case.k, case.wq.cuda(), y, ws, scaled=True)
        check(case, "matmul", case.xq64, y.cpu(), torch.zeros_like(y, device="cpu"), False, cut=True)
        return
    run_all(case, torch.bfloat16, exact=False, ops=({"bf16": "matmul"}.get(op, op),))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2000, 64, 40), (8000, 16, 33), (100, 16, 1), (200, 3, 7), (70, 1, 5), (65, 1, 1), (129, 130, 2),
                                   (500, 48, 8, 3, 1, 2), (4000, 5, 6, 40), (49, 48, 2048), (90, 1, 2048, 2, 3, 3)])
@pytest.mark.parametrize("ldw", [(0, 0), (3, 1)])
def test_tall_and_narrow(shape, ldw):
    """Many rows of few columns, contractions down to one value."""
    require_gpu()
    say(f"mx tall and narrow {shape} ld+{ldw}")
    case = Case(sum(shape), *shape)
    for out in (torch.float32, torch.bfloat16):
        run_all(case, out, exact=True, ldw=ldw)
