"""rms_norm and rms_norm_backward against the 64-bit formulas.

Bounds, u = 2^-24.  A row's sum of squares (exact products, all positive): at
most 32 additions in a thread, 6 in a wave, 16 over the waves, so 54 u; s = 1 /
sqrt(sum / cols + eps) halves that and adds four roundings of its own, two of
which the root halves: 31 u.  y = h s w: two more, 33 u.  The sum of g u in the
backward pass has three roundings in each term (u, g, the product) besides
those of s itself, which the test takes as given: 57 u of the sum of the
magnitudes, and m two more; dx then adds five of its largest term.  dw: a term
has two roundings, and a sum of that many rows at most rows + 64 additions.
BF16 outputs add half a step, 2^-8."""
import pytest

import layer_util as lu
from gpu_util import require_gpu, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
bf16 = torch.bfloat16
SHAPES = [(1, 1), (3, 7), (2, 8), (5, 31), (4, 33), (9, 128), (130, 160), (7, 1000), (8, 2048), (65, 2049), (3, 4097), (33, 8192),
          (2, 8193), (5, 20001), (3, 32768), (700, 96), (5001, 64)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def lib():
    import lossless_bf16_tensor_exp_amd as ciera
    return ciera


def case(rows, cols, seed=0):
    gen = torch.Generator().manual_seed(rows * 40000 + cols + seed)
    x = (torch.randn(rows, cols, generator=gen) * 0.5).to(bf16)
    r = lu.mx.activations(gen, rows, cols)
    w = (1 + 0.1 * torch.randn(cols, generator=gen)).to(bf16)
    dy = (torch.randn(rows, cols, generator=gen) * 1e-3).to(bf16)
    return x, r, w, dy


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("residual,wider,shift", [(True, 0, 0), (True, 3, 1), (False, 8, 8)])
def test_forward(rows, cols, residual, wider, shift):
    say(f"norm {rows}x{cols} residual {residual} ld+{wider} shift {shift}")
    c = lib()
    x, r, w, _ = case(rows, cols)
    r = r if residual else None
    h64, s64, y64 = lu.norm(x, r, w, 1e-6)
    size = c.mx8_encoded_size(rows, cols)
    ybuf, y = lu.guarded(rows, cols, bf16, wider, shift)
    hbuf, h = lu.guarded(rows, cols, bf16, wider, shift)
    yq = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    rstd = torch.full((rows + 1,), 7.0, device="cuda")
    c.rms_norm(lu.put(x, wider, shift), w.cuda(), y=y, yq=yq[:size], residual=None if r is None else lu.put(r, wider, shift),
               h=h if residual else None, rstd=rstd[:rows])
    if residual:
        assert torch.equal(h.cpu(), h64)
    lu.within(rstd[:rows], s64, 31 * U * s64)
    assert rstd[rows] == 7.0
    lu.within(y, y64, 33 * U * y64.abs(), 2.0 ** -8)
    want = torch.empty(size, dtype=torch.uint8, device="cuda")
    c.mx8_encode(y, want)
    assert torch.equal(yq[:size], want), "yq is not mx8_encode's of y"
    assert (yq[size:] == 0xA5).all()
    lu.untouched(ybuf, y)
    lu.untouched(hbuf, h)
    # each output alone, and the residual stream updated where it is
    y2, yq2 = torch.empty_like(y), torch.empty_like(want)
    c.rms_norm(h if residual else x.cuda(), w.cuda(), y=y2)
    assert torch.equal(y2, y)
    c.rms_norm(h if residual else x.cuda(), w.cuda(), yq=yq2)
    assert torch.equal(yq2, want)
    if residual:
        for which in (0, 1):
            both = [lu.put(x, wider, shift), lu.put(r, wider, shift)]
            c.rms_norm(both[0], w.cuda(), y=y2, residual=both[1], h=both[which])
            assert torch.equal(both[which], h) and torch.equal(y2, y)
    z = lu.put(h.cpu() if residual else x, wider, shift)
    c.rms_norm(z, w.cuda(), y=z)
    assert torch.equal(z, y)


def test_values_at_the_edges():
    """Rows of zeros, subnormals, an infinity, a NaN, and squares past FP32's range, next to ordinary ones."""
    say("norm edges")
    c = lib()
    x = torch.randn(9, 300, generator=torch.Generator().manual_seed(1)).to(bf16)
    x[1] = 0
    x[2] = 1e-39
    x[3, 7] = float("inf")
    x[4, 299] = float("nan")
    x[5, 0] = 3e38
    x[6] = 1e19
    x[7, :] = -0.0
    w = torch.randn(300, generator=torch.Generator().manual_seed(2)).to(bf16)
    y, rstd = torch.empty(9, 300, dtype=bf16, device="cuda"), torch.empty(9, device="cuda")
    yq = torch.empty(c.mx8_encoded_size(9, 300), dtype=torch.uint8, device="cuda")
    c.rms_norm(x.cuda(), w.cuda(), y=y, yq=yq, rstd=rstd)
    _, s, want = lu.norm(x, None, w, 1e-6)
    for i in (0, 1, 2, 8):
        lu.within(rstd[i], s[i], 31 * U * s[i])
        lu.within(y[i], want[i], 33 * U * want[i].abs(), 2.0 ** -8)
    assert rstd[3] == 0 and y[3, 7].isnan() and (y[3, :7] == 0).all() and (y[3, 8:] == 0).all()
    assert y[4].isnan().all() and rstd[4].isnan()
    assert rstd[5] == 0 and (y[5] == 0).all()   # 9e76 is infinite in FP32
    assert rstd[6] == 0 and (y[6] == 0).all()   # 300 * 1e38 too
    assert (y[7] == 0).all()
    enc = torch.empty_like(yq)
    c.mx8_encode(y, enc)
    assert torch.equal(yq, enc)
    # a tiny eps
    c.rms_norm(x.cuda(), w.cuda(), y=y, rstd=rstd, eps=1e-30)
    _, s, want = lu.norm(x, None, w, float(torch.tensor(1e-30)))
    for i in (0, 1, 2):
        lu.within(rstd[i], s[i], 31 * U * s[i])
        lu.within(y[i], want[i], 33 * U * want[i].abs(), 2.0 ** -8)


@pytest.mark.parametrize("cols", [1, 3, 64, 300, 2049, 20001])
@pytest.mark.parametrize("eps", [1e-6, 0.37, 1e-40])
def test_root_of_exact_sums(cols, eps):
    """Whole numbers whose squares' sum is exact (below 2^24): s has the two roundings of mean + eps, halved by the root,
    and its own, so 2 u and what the correction leaves, below 2^-40."""
    say(f"root of exact sums {cols} {eps}")
    c = lib()
    gen = torch.Generator().manual_seed(cols)
    x = torch.randint(-15, 16, (200, cols), generator=gen).to(bf16)
    x[0] = 0
    y, s = torch.empty(200, cols, dtype=bf16, device="cuda"), torch.empty(200, device="cuda")
    c.rms_norm(x.cuda(), torch.ones(cols, dtype=bf16).cuda(), y=y, rstd=s, eps=eps)
    want = 1 / (x.double().square().sum(1) / cols + float(torch.tensor(eps))).sqrt()
    lu.within(s, want, (2 * U + 2.0 ** -40) * want)


@pytest.mark.parametrize("cols", [5, 300, 2048])
def test_infinite_weights(cols):
    """Infinities and NaN of the weight stay in their columns, with the sign that h has there."""
    c = lib()
    gen = torch.Generator().manual_seed(cols)
    x, w = lu.mx.activations(gen, 20, cols), torch.randn(cols, generator=gen).to(bf16)
    x[:, 1:3] = torch.where(x[:, 1:3] == 0, torch.ones((), dtype=bf16), x[:, 1:3])
    y = torch.empty(20, cols, dtype=bf16, device="cuda")
    w[1], w[2], w[4] = float("inf"), float("-inf"), float("nan")
    c.rms_norm(x.cuda(), w.cuda(), y=y)
    _, _, want = lu.norm(x, None, w, 1e-6)
    assert torch.equal(y[:, 1].double().cpu(), want[:, 1]) and torch.equal(y[:, 2].double().cpu(), want[:, 2])
    assert y[:, 4].isnan().all()
    _, _, want = lu.norm(x, None, torch.where(w.isfinite(), w, torch.zeros((), dtype=bf16)), 1e-6)
    keep = w.isfinite()
    lu.within(y.cpu()[:, keep], want[:, keep], 33 * U * want[:, keep].abs(), 2.0 ** -8)


def test_mean_and_eps_past_the_range():
    c = lib()
    x = torch.full((2, 1), 1.8e19, dtype=bf16, device="cuda")
    y, s = torch.empty_like(x), torch.empty(2, device="cuda")
    c.rms_norm(x, torch.ones(1, dtype=bf16, device="cuda"), y=y, rstd=s, eps=2e38)
    assert (s == 0).all() and (y == 0).all()


def backward64(dy, h, w, s, dh):
    hd, s = h.double(), s.double()[:, None]
    g, u = dy.double() * w.double(), hd * s
    m, size = (g * u).mean(1, keepdim=True), (g * u).abs().mean(1, keepdim=True)
    e = torch.zeros_like(g) if dh is None else dh.double()
    room = U * ((s * u).abs() * 64 * size + 5 * (s * g).abs() + 5 * (s * u * m).abs() + e.abs())
    return s * (g - u * m) + e, room, (dy.double() * u).sum(0), (dy.double() * u).abs().sum(0)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("way,wider,shift", [(True, 0, 0), (False, 3, 1)])
@pytest.mark.parametrize("dtype", [bf16, torch.float32])
def test_backward(rows, cols, way, wider, shift, dtype):
    say(f"norm backward {rows}x{cols} dh {way} ld+{wider} {dtype}")
    c = lib()
    x, h, w, dy = case(rows, cols)
    s = lu.norm(h, None, w, 1e-6)[1].float()
    dh = x if way else None
    want, room, dw64, size = backward64(dy, h, w, s, dh)
    dxbuf, dx = lu.guarded(rows, cols, bf16, wider, shift)
    dw = torch.full((cols + 1,), 7.0, dtype=dtype, device="cuda")
    ws = torch.empty(c.rms_norm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    args = [lu.put(dy, wider, shift), lu.put(h, wider, shift), w.cuda(), s.cuda()]
    to = None if dh is None else lu.put(dh, wider, shift)
    c.rms_norm_backward(*args, dx, dw[:cols], ws, dh=to)
    lu.within(dx, want, room, 2.0 ** -8)
    dw_room = (rows + 66) * U * size
    lu.within(dw[:cols], dw64, dw_room, lu.HALF[dtype])
    assert dw[cols] == 7.0
    lu.untouched(dxbuf, dx)
    # on top of what is there
    more = dw.clone()
    c.rms_norm_backward(*args, None, more[:cols], ws, accumulate=True)
    lu.within(more[:cols], dw64 + dw[:cols].double().cpu(), dw_room + U * dw[:cols].double().cpu().abs(), lu.HALF[dtype])
    # dx alone, over dh or dy
    alone = lu.put(dy, wider, shift)
    c.rms_norm_backward(alone, *args[1:], alone, None, dh=to)
    assert torch.equal(alone, dx)
    if way:
        c.rms_norm_backward(*args, to, None, dh=to)
        assert torch.equal(to, dx)


@pytest.mark.parametrize("rows,cols", [(140000, 24), (70001, 100), (17000, 300), (9001, 520), (5003, 1408), (2100, 2056), (1100, 4100),
                                       (1030, 8200)])
def test_more_rows_than_go_at_once(rows, cols):
    """Every shape with workgroups that go round more than once, the last round in part."""
    say(f"norm backward in rounds {rows}x{cols}")
    c = lib()
    gen = torch.Generator(device="cuda").manual_seed(rows)
    h, dy, dh = (torch.randn(rows, cols, generator=gen, device="cuda").to(bf16) for _ in range(3))
    w = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(bf16)
    y, s = torch.empty_like(h), torch.empty(rows, device="cuda")
    c.rms_norm(h, w, y=y, rstd=s)
    _, s64, y64 = lu.norm(h, None, w, 1e-6)
    lu.within(s, s64.cpu(), 31 * U * s64.cpu())
    lu.within(y, y64.cpu(), 33 * U * y64.cpu().abs(), 2.0 ** -8)
    want, room, dw64, size = (t.cpu() for t in backward64(dy, h, w, s, dh))
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(c.rms_norm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    c.rms_norm_backward(dy, h, w, s, dx, dw, ws, dh=dh)
    assert c.ciera_read_error(ws) == 0
    lu.within(dx, want, room, 2.0 ** -8)
    lu.within(dw, dw64, (rows + 66) * U * size, U)
    again = torch.empty_like(dw)
    c.rms_norm_backward(dy, h, w, s, None, again, ws)
    assert torch.equal(again, dw)


def test_backward_against_differences():
    """The formula itself: sum(dy y) moves by dx and dw as h and w move, in 64 bits."""
    gen = torch.Generator().manual_seed(3)
    h, w, dy = (torch.randn(*n, generator=gen, dtype=torch.float64) for n in ((4, 37), (37,), (4, 37)))

    def loss(h, w):
        return (dy * h * ((h.square().mean(1, keepdim=True) + 1e-6) ** -0.5) * w).sum()

    s = (h.square().mean(1) + 1e-6) ** -0.5
    dx, _, dw, _ = backward64(dy, h, w, s, None)
    step = torch.randn(4, 37, generator=gen, dtype=torch.float64) * 1e-5
    assert abs((loss(h + step, w) - loss(h - step, w)) / 2 - (dx * step).sum()) < 1e-12
    step = torch.randn(37, generator=gen, dtype=torch.float64) * 1e-5
    assert abs((loss(h, w + step) - loss(h, w - step)) / 2 - (dw * step).sum()) < 1e-12


def test_no_rows():
    say("norm without rows")
    c = lib()
    none = torch.empty(0, 64, dtype=bf16, device="cuda")
    w = torch.ones(64, dtype=bf16, device="cuda")
    c.rms_norm(none, w, y=none)
    dw = torch.full((64,), 7.0, device="cuda")
    ws = torch.empty(c.rms_norm_workspace_size(0, 64), dtype=torch.uint8, device="cuda")
    c.rms_norm_backward(none, none, w, torch.empty(0, device="cuda"), none, dw, ws, accumulate=True)
    assert (dw == 7).all()
    c.rms_norm_backward(none, none, w, torch.empty(0, device="cuda"), none, dw, ws)
    assert (dw == 0).all()


def test_past_32_bits():
    """Row offsets past 2^32 values: the last rows of a matrix with far-apart rows."""
    say("norm past 32 bits")
    c = lib()
    rows, cols, ld = 1100, 64, 1 << 22
    buf = torch.empty(rows * ld, dtype=bf16, device="cuda")
    x = buf.view(rows, ld)[:, :cols]
    x.copy_(torch.randn(rows, cols, generator=torch.Generator().manual_seed(4)).to(bf16))
    w = torch.ones(cols, dtype=bf16, device="cuda")
    near, y, rstd = x.contiguous(), torch.empty(rows, cols, dtype=bf16, device="cuda"), torch.empty(rows, device="cuda")
    c.rms_norm(near, w, y=y, rstd=rstd)
    dx, dw = torch.empty_like(y), torch.empty(cols, device="cuda")
    ws = torch.empty(c.rms_norm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    c.rms_norm_backward(y, near, w, rstd, dx, dw, ws)
    far = buf.view(rows, ld)[:, 128:128 + cols]
    c.rms_norm(x, w, y=far)
    assert torch.equal(far, y)
    dw2 = torch.empty_like(dw)
    c.rms_norm_backward(far, x, w, rstd, far, dw2, ws)
    assert torch.equal(far, dx) and torch.equal(dw2, dw)


def test_refusals():
    say("norm refusals")
    c = lib()
    m = torch.zeros(4, 64, dtype=bf16, device="cuda")
    w, s = torch.ones(64, dtype=bf16, device="cuda"), torch.ones(4, device="cuda")
    small = torch.empty(c.mx8_encoded_size(4, 64) - 1, dtype=torch.uint8, device="cuda")
    for bad in (lambda: c.rms_norm(m, w),                                  # no output
                lambda: c.rms_norm(m, w, y=m, h=m),                        # h without a residual
                lambda: c.rms_norm(m, w, y=m, eps=0.0),
                lambda: c.rms_norm(m, w, y=m, eps=float("nan")),
                lambda: c.rms_norm(m, w, yq=small)):
        with pytest.raises(c.CieraError):
            bad()
    wide = torch.zeros(1, 32769, dtype=bf16, device="cuda")
    with pytest.raises(c.CieraError):
        c.rms_norm(wide, wide[0], y=wide)
    for bad in (lambda: c.rms_norm(m, w[:63], y=m), lambda: c.rms_norm(m, w, y=m[:3]), lambda: c.rms_norm(m, w, y=m, rstd=s[:3]),
                lambda: c.rms_norm(m, w, y=m, residual=m[:, :63]), lambda: c.rms_norm(m.cpu(), w, y=m),
                lambda: c.rms_norm_backward(m, m[:3], w, s, m, None)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: c.rms_norm(m.float(), w, y=m), lambda: c.rms_norm(m, w.float(), y=m),
                lambda: c.rms_norm(m, w, y=m, rstd=s.to(bf16)), lambda: c.rms_norm_backward(m, m, w, s.double(), m, None)):
        with pytest.raises(TypeError):
            bad()
    ws = torch.empty(c.rms_norm_workspace_size(4, 64) - 256, dtype=torch.uint8, device="cuda")
    for bad in (lambda: c.rms_norm_backward(m, m, w, s, m, s.new_zeros(64)),          # dw without a workspace
                lambda: c.rms_norm_backward(m, m, w, s, m, s.new_zeros(64), ws),      # one that is too small
                lambda: c.rms_norm_backward(m, m, w, s, None, None),
                lambda: c.rms_norm_backward(m, m, w, s, None, s.new_zeros(64), ws, dh=m)):
        with pytest.raises(c.CieraError):
            bad()
