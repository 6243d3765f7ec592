"""Rows of tokens to their experts and back: the sort, the dispatch and drows
exactly; combine and dweights within an FP32 sum's bound (u = 2^-24: a term's
product is rounded or fused, so choices + 2 roundings for combine, and for
dweights cols + 8, any order), and half a step of the output's type."""
import pytest

import layer_util as lu
from gpu_util import require_gpu, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
bf16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def lib():
    import lossless_bf16_tensor_exp_amd as ciera
    return ciera


def sort(ids, experts, order=True):
    c = lib()
    tokens, choices = ids.shape if ids.dim() == 2 else (ids.shape[0], 1)
    offsets = torch.full((experts + 2,), -7, dtype=torch.int64, device="cuda")
    place = torch.full((tokens * choices + 1,), -7, dtype=torch.int32, device="cuda")
    by = torch.full((tokens * choices + 1,), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(c.expert_workspace_size(tokens, choices, experts), dtype=torch.uint8, device="cuda")
    c.expert_sort(ids, offsets[:-1], place[:-1].view(ids.shape), by[:-1] if order else None, ws)
    assert offsets[-1] == -7 and place[-1] == -7 and by[-1] == -7
    return offsets[:-1], place[:-1].view(ids.shape), by[:-1], c.ciera_read_error(ws)


@pytest.mark.parametrize("tokens,choices,experts", [(1, 1, 1), (1, 8, 64), (8, 8, 64), (63, 3, 5), (64, 1, 2), (1000, 6, 66),
                                                    (4096, 2, 128), (2500, 8, 64), (5000, 1, 4096), (300, 64, 64), (4001, 4, 1023),
                                                    (3000, 2, 1024), (70000, 1, 3), (33000, 8, 64), (6143, 1, 7), (1536, 4, 7), (6145, 1, 300),
                                                    (66000, 8, 5), (20000, 4, 4096)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(tokens, choices, experts, dtype):
    say(f"sort {tokens} x {choices} of {experts} {dtype}")
    gen = torch.Generator().manual_seed(tokens + experts)
    ids = torch.randint(-1, experts, (tokens, choices), generator=gen)
    ids[tokens // 2:tokens // 2 + 70] = experts - 1  # a stretch of one expert
    want = lu.sort(ids, experts)
    got = sort(ids.to(dtype).cuda(), experts)
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w.to(g.dtype))
    assert got[3] == 0
    place = sort(ids.to(dtype).cuda(), experts, order=False)[1]
    assert torch.equal(place.cpu(), want[1])


@pytest.mark.parametrize("value", [-1, 0, 5])
def test_all_entries_alike(value):
    say(f"sort, all entries {value}")
    for tokens in (0, 1, 64, 1000, 20000):
        ids = torch.full((tokens,), value, dtype=torch.int32)
        got, want = sort(ids.cuda(), 6), lu.sort(ids, 6)
        for g, w in zip(got, want):
            assert torch.equal(g.cpu(), w.to(g.dtype))
        assert got[3] == 0


@pytest.mark.parametrize("tokens", [3, 5000])
@pytest.mark.parametrize("bad", [6, -2, 2 ** 31 - 1, -2 ** 31])
def test_numbers_of_no_expert(tokens, bad):
    say(f"sort with {bad} among {tokens}")
    ids = torch.randint(0, 6, (tokens, 2), generator=torch.Generator().manual_seed(1), dtype=torch.int64)
    ids[tokens - 1, 1] = bad
    want = lu.sort(ids, 6)
    for t in (ids.to(torch.int32), ids):
        got = sort(t.cuda(), 6)
        for g, w in zip(got, want):
            assert torch.equal(g.cpu(), w.to(g.dtype))
        assert got[3] == 1  # CIERA_ERR_ARG
    ids[tokens - 1, 1] = bad * 2 ** 32 + 3  # not 3
    assert sort(ids.cuda(), 6)[3] == 1


SHAPES = [(1, 1, 1, 1), (1, 8, 64, 2048), (5, 3, 4, 7), (9, 2, 3, 31), (64, 6, 66, 33), (130, 8, 16, 128), (70, 1, 9, 520),
          (33, 5, 8, 2049), (20, 9, 12, 1000), (3, 64, 64, 96), (6, 4, 8, 8200), (2, 2, 2, 20001), (1500, 4, 7, 24)]


def case(tokens, choices, experts, cols):
    gen = torch.Generator().manual_seed(tokens * 7 + cols)
    ids = lu.choose(gen, tokens, choices, experts, 0.15 if tokens > 1 else 0.0)
    offsets, place, _ = lu.sort(ids, experts)
    x = lu.mx.activations(gen, tokens, cols)
    weights = torch.softmax(torch.randn(tokens, choices, generator=gen), 1).contiguous()
    return gen, place, int(offsets[-1]), x, weights


@pytest.mark.parametrize("tokens,choices,experts,cols", SHAPES)
@pytest.mark.parametrize("wider,shift", [(0, 0), (3, 1), (8, 8)])
def test_dispatch(tokens, choices, experts, cols, wider, shift):
    say(f"dispatch {tokens} x {choices} of {experts}, {cols} ld+{wider}")
    c = lib()
    _, place, used, x, _ = case(tokens, choices, experts, cols)
    rows = tokens * choices
    want = torch.full((rows, cols), 7.0, dtype=bf16)
    has = place.view(-1) >= 0
    want[place.view(-1)[has].long()] = x[torch.arange(rows)[has] // choices]
    buf, out = lu.guarded(rows, cols, bf16, wider, shift)
    c.expert_dispatch(lu.put(x, wider, shift), place.cuda(), out=out)
    assert torch.equal(out.cpu(), want)
    lu.untouched(buf, out)
    # in 8 bits: the bytes that the dispatched rows have there, rows of no entry as they were
    size, kp = c.mx8_encoded_size(rows, cols), lu.mx.pitch(cols)
    outq = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    c.expert_dispatch(lu.put(x, wider, shift), place.cuda(), outq=outq[:size])
    enc = torch.full((size,), 0xA5, dtype=torch.uint8)
    line, at, _ = lu.mx.sections(8, rows, cols)
    if used:
        full = lu.mx.encode(8, want)
        enc[:used * kp] = full[:used * kp]
        enc[at:at + used * kp // 32] = full[at:at + used * kp // 32]
    assert torch.equal(outq[:size].cpu(), enc)
    assert (outq[size:] == 0xA5).all()
    # both at once
    out.fill_(7.0)
    outq.fill_(0xA5)
    c.expert_dispatch(lu.put(x, wider, shift), place.cuda(), out=out, outq=outq[:size])
    assert torch.equal(out.cpu(), want) and torch.equal(outq[:size].cpu(), enc)
    # fewer rows than places: what lies behind is left out
    if rows > 1:
        few = rows // 2
        buf, out = lu.guarded(few, cols, bf16, wider, shift)
        c.expert_dispatch(lu.put(x, wider, shift), place.cuda(), out=out)
        assert torch.equal(out.cpu(), want[:few])
        lu.untouched(buf, out)


def test_dispatch_non_finite():
    say("dispatch of non-finite values")
    c = lib()
    x = torch.randn(5, 96, generator=torch.Generator().manual_seed(1)).to(bf16)
    x[1, 40], x[3, 0] = float("nan"), float("-inf")
    place = torch.tensor([[4], [2], [0], [1], [3]], dtype=torch.int32)
    out, outq = torch.empty(5, 96, dtype=bf16, device="cuda"), torch.empty(c.mx8_encoded_size(5, 96), dtype=torch.uint8, device="cuda")
    c.expert_dispatch(x.cuda(), place.cuda(), out=out, outq=outq)
    want = x[torch.tensor([2, 3, 1, 4, 0])]
    assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))
    assert torch.equal(outq.cpu(), lu.mx.encode(8, want))


@pytest.mark.parametrize("tokens,choices,experts,cols", SHAPES)
@pytest.mark.parametrize("dtype,to,wider,shift", [(bf16, bf16, 0, 0), (bf16, torch.float32, 3, 1), (torch.float32, bf16, 3, 1),
                                                  (torch.float32, torch.float32, 8, 8)])
def test_combine_and_backward(tokens, choices, experts, cols, dtype, to, wider, shift):
    say(f"combine {tokens} x {choices} of {experts}, {cols} {dtype} to {to}")
    c = lib()
    gen, place, used, x, weights = case(tokens, choices, experts, cols)
    n = tokens * choices
    rows = (torch.randn(n, cols, generator=gen) * 0.5).to(dtype)
    rows[used:] = float("nan")  # of no expert: not read
    weights[place < 0] = float("nan")
    dout = (torch.randn(tokens, cols, generator=gen) * 1e-3).to(bf16)
    rd, pd, wd = lu.put(rows, wider, shift), place.cuda(), weights.cuda()
    for w, r in ((weights, x), (weights, None), (None, x), (None, None)):
        want, size = lu.combine(rows, place, w, r)
        buf, out = lu.guarded(tokens, cols, to, wider, shift)
        c.expert_combine(rd, pd, out, weights=None if w is None else wd, residual=None if r is None else lu.put(r, wider, shift))
        lu.within(out, want, (choices + 2) * U * size, lu.HALF[to])
        lu.untouched(buf, out)
    if to is bf16:  # onto the residual itself
        own = lu.put(x, wider, shift)
        c.expert_combine(rd, pd, own, weights=wd, residual=own)
        want, size = lu.combine(rows, place, weights, x)
        lu.within(own, want, (choices + 2) * U * size, 2.0 ** -8)

    buf, drows = lu.guarded(n, cols, bf16, wider, shift)
    dw = torch.full((tokens * choices + 1,), 7.0, device="cuda")
    for w in (weights, None):
        drows.fill_(7.0)
        dw.fill_(7.0)
        c.expert_combine_backward(lu.put(dout, wider, shift), rd, pd, drows, dw[:-1].view(tokens, choices),
                                  weights=None if w is None else wd)
        wr = torch.full((n, cols), 7.0, dtype=bf16)
        has = place.view(-1) >= 0
        token, at = torch.arange(n)[has] // choices, place.view(-1)[has].long()
        f = torch.ones(len(at)) if w is None else w.view(-1)[has]
        wr[at] = (f[:, None] * dout[token].float()).to(bf16)
        assert torch.equal(drows.cpu(), wr)
        terms = dout[token].double() * rows[at].double()
        want, size = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
        want[has], size[has] = terms.sum(1), terms.abs().sum(1)
        lu.within(dw[:-1], want, (cols + 8) * U * size, U)
        assert dw[-1] == 7.0
        lu.untouched(buf, drows)
    # either gradient alone
    d2, w2 = torch.full_like(drows, 7.0), torch.empty(tokens, choices, device="cuda")
    c.expert_combine_backward(dout.cuda(), rd, pd, d2, None)
    c.expert_combine_backward(dout.cuda(), rd, pd, None, w2)
    assert torch.equal(d2.cpu(), wr) and torch.equal(w2.view(-1), dw[:-1])


def test_dispatch_and_its_gradient_are_transposes():
    """<dispatch(x), d> = <x, combine(d)> on whole numbers, exactly."""
    say("dispatch and its gradient")
    c = lib()
    gen = torch.Generator().manual_seed(8)
    place = lu.sort(lu.choose(gen, 50, 4, 9), 9)[1].cuda()
    x, d = (torch.randint(-3, 4, (n, 40), generator=gen).to(bf16).cuda() for n in (50, 200))
    out, dx = torch.zeros_like(d), torch.empty(50, 40, device="cuda")
    c.expert_dispatch(x, place, out=out)
    c.expert_combine(d, place, dx)
    assert (out.double() * d.double()).sum() == (x.double() * dx.double()).sum()


def test_non_finite_rows_reach_only_their_tokens():
    say("combine of non-finite rows")
    c = lib()
    place = torch.tensor([[0, 1], [2, 3], [4, -1]], dtype=torch.int32, device="cuda")
    rows = torch.ones(6, 24, dtype=bf16, device="cuda")
    rows[2, 5], rows[3, 6], rows[5] = float("inf"), float("nan"), float("nan")
    out = torch.empty(3, 24, device="cuda")
    weights = torch.tensor([[0.5, 0.25], [1.0, 1.0], [2.0, float("inf")]], device="cuda")
    c.expert_combine(rows, place, out, weights=weights)
    assert (out[0] == 0.75).all() and (out[2] == 2).all()
    assert out[1, 5] == float("inf") and out[1, 6].isnan() and (out[1, 7:] == 2).all()


def test_past_32_bits():
    say("experts past 32 bits")
    c = lib()
    rows, cols, ld = 1100, 64, 1 << 22
    buf = torch.empty(rows * ld, dtype=bf16, device="cuda")
    far = buf.view(rows, ld)[:, :cols]
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(rows, cols, generator=gen).to(bf16).cuda()
    place = torch.randperm(rows, generator=gen).to(torch.int32).view(rows, 1).cuda()
    c.expert_dispatch(x, place, out=far)
    assert torch.equal(far[place.view(-1).long()], x)
    out, dw = torch.empty_like(x), torch.empty(rows, 1, device="cuda")
    c.expert_combine(far, place, out)
    assert torch.equal(out, x)
    d = buf.view(rows, ld)[:, 128:128 + cols]
    c.expert_combine_backward(x, far, place, d, dw)
    assert torch.equal(d, far)
    assert torch.allclose(dw.view(-1).double(), x.double().square().sum(1), rtol=72 * U)
    # tokens' rows far apart
    c.expert_dispatch(far, place, out=out)
    assert torch.equal(out[place.view(-1).long()], far)
    # an mx8 matrix whose scales lie past 2^32 bytes
    rows, cols = 40000, 1 << 17
    size = c.mx8_encoded_size(rows, cols)
    outq = torch.zeros(size, dtype=torch.uint8, device="cuda")
    x = torch.randn(2, cols, generator=gen).to(bf16)
    c.expert_dispatch(x.cuda(), torch.tensor([[39999], [33333]], dtype=torch.int32, device="cuda"), outq=outq, rows=rows)
    enc = lu.mx.encode(8, x)
    for i, at in enumerate((39999, 33333)):
        assert torch.equal(outq[at * cols:(at + 1) * cols].cpu(), enc[i * cols:(i + 1) * cols])
        s = rows * cols + at * cols // 32
        assert torch.equal(outq[s:s + cols // 32].cpu(), enc[2 * cols + i * cols // 32:2 * cols + (i + 1) * cols // 32])


def test_refusals():
    say("experts refusals")
    c = lib()
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    offsets, order = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    place, m = torch.zeros_like(ids), torch.zeros(4, 64, dtype=bf16, device="cuda")
    ws = torch.empty(c.expert_workspace_size(4, 2, 3), dtype=torch.uint8, device="cuda")
    w, r = torch.ones(4, 2, device="cuda"), torch.zeros(8, 64, dtype=bf16, device="cuda")
    with pytest.raises(c.CieraError):
        c.expert_sort(ids, offsets, place, order, ws[:256])
    for bad in (lambda: c.expert_sort(ids, offsets[:1], place, order, ws), lambda: c.expert_sort(ids, offsets, place[:3], order, ws),
                lambda: c.expert_sort(ids, offsets, place, order[:7], ws), lambda: c.expert_sort(ids.t(), offsets, place, order, ws),
                lambda: c.expert_sort(ids.cpu(), offsets, place, order, ws), lambda: c.expert_dispatch(m[:3], place, out=r),
                lambda: c.expert_dispatch(m, place, out=r[:, :63]), lambda: c.expert_combine(r, place, m[:3]),
                lambda: c.expert_combine(r, place, m, weights=w[:, :1].contiguous()),
                lambda: c.expert_combine(r, place, m, residual=m[:, :60]),
                lambda: c.expert_combine_backward(m, r, place, r[:7], w), lambda: c.expert_combine_backward(m, r, place, r, w[:3])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: c.expert_sort(ids.float(), offsets, place, order, ws), lambda: c.expert_sort(ids, offsets.int(), place, order, ws),
                lambda: c.expert_sort(ids, offsets, place.long(), order, ws), lambda: c.expert_dispatch(m.float(), place, out=r),
                lambda: c.expert_combine(r, place, m, weights=w.to(bf16)), lambda: c.expert_combine(r.double(), place, m)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: c.expert_dispatch(m, place), lambda: c.expert_combine_backward(m, r, place, None, None),
                lambda: c.expert_dispatch(m, place, outq=ws[:100].contiguous()),
                lambda: c.expert_dispatch(m, torch.zeros(4, 65, dtype=torch.int32, device="cuda"), out=r)):
        with pytest.raises(c.CieraError):
            bad()
