"""low_rank_add against the 64-bit formula: exactly on whole numbers whose sums
FP32 holds, and on real ones within its bound.  u = 2^-24: the inner values
have k roundings (products of BF16 are exact) and that of the scale; three
parts hold them whole, so the outer sum has 3 ranks of exact products; ranks
are filled up to 128 at most with zeros, which add nothing; base adds one.
So (k + 3 rank + 4) u of the sum of the magnitudes, u of y, and half a step of
the output's type."""
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


def workspace(tokens, n, k, rank, adapters):
    return torch.empty(lib().low_rank_workspace_size(tokens, n, k, rank, adapters), dtype=torch.uint8, device="cuda")


def case(tokens, n, k, rank, adapters, none=0.2, whole=False):
    gen = torch.Generator().manual_seed(tokens * 3 + n + k + rank)
    ids = torch.randint(0, adapters, (tokens,), generator=gen)
    ids[torch.rand(tokens, generator=gen) < none] = -1
    offsets, _, order = lu.sort(ids, adapters)
    if whole:
        x = torch.randint(-3, 4, (tokens, k), generator=gen).to(bf16)
        a = torch.randint(-2, 3, (adapters, rank, k), generator=gen).to(bf16)
        b = torch.randint(-1, 2, (adapters, n, rank), generator=gen).to(bf16)
        base = torch.randint(-100, 101, (tokens, n), generator=gen).float()
        return x, a, b, None, offsets, order, base
    x = lu.mx.activations(gen, tokens, k)
    a = (torch.randn(adapters, rank, k, generator=gen) * k ** -0.5).to(bf16)
    b = (torch.randn(adapters, n, rank, generator=gen) * 0.2).to(bf16)
    return x, a, b, torch.rand(adapters, generator=gen) * 2 - 0.5, offsets, order, torch.randn(tokens, n, generator=gen)


SHAPES = [(1, 8, 8, 1, 1), (1, 2048, 2048, 16, 4), (7, 96, 200, 3, 5), (64, 130, 64, 16, 70), (33, 520, 1000, 17, 3), (200, 65, 72, 32, 9),
          (150, 1025, 129, 40, 2), (40, 700, 2049, 64, 6), (90, 48, 513, 100, 4), (17, 1000, 96, 128, 2), (600, 128, 31, 8, 130),
          (5, 33, 7, 5, 64), (1000, 256, 256, 64, 1)]


@pytest.mark.parametrize("tokens,n,k,rank,adapters", SHAPES)
@pytest.mark.parametrize("base_type,to,wider,shift", [(bf16, bf16, 0, 0), (torch.float32, torch.float32, 3, 1),
                                                      (torch.float32, bf16, 8, 8), (bf16, torch.float32, 3, 1)])
def test_adapters(tokens, n, k, rank, adapters, base_type, to, wider, shift):
    say(f"adapters {tokens} x {n} x {k} rank {rank} of {adapters} {base_type} to {to}")
    c = lib()
    x, a, b, scales, offsets, order, base = case(tokens, n, k, rank, adapters)
    base = base.to(base_type)
    ws = workspace(tokens, n, k, rank, adapters)
    dev = [lu.put(x, wider, shift), a.cuda(), b.cuda(), offsets.cuda()]
    want, size = lu.low_rank(x, a, b, scales, offsets, order, base)
    room = (k + 3 * rank + 4) * U * size + U * want.abs()
    buf, y = lu.guarded(tokens, n, to, wider, shift)
    bd = lu.put(base, wider, shift)
    c.low_rank_add(*dev, y, ws, base=bd, order=order.cuda(), scales=scales.cuda())
    assert c.ciera_read_error(ws) == 0
    lu.within(y, want, room, lu.HALF[to])
    lu.untouched(buf, y)
    if to is base_type:  # onto the projection's result itself
        c.low_rank_add(*dev, bd, ws, base=bd, order=order.cuda(), scales=scales.cuda())
        assert torch.equal(bd, y)
    # rows that lie sorted, without scales, without base: rows of no adapter become zeros
    at = order.long()
    want, size = lu.low_rank(x[at], a, b, None, offsets, None, torch.zeros(tokens, n))
    y.fill_(7.0)
    c.low_rank_add(lu.put(x[at], wider, shift), *dev[1:], y, ws)
    lu.within(y, want, (k + 3 * rank + 4) * U * size + U * want.abs(), lu.HALF[to])
    assert (y[int(offsets[-1]):] == 0).all()


@pytest.mark.parametrize("tokens,n,k,rank,adapters", SHAPES)
def test_whole_numbers(tokens, n, k, rank, adapters):
    say(f"adapters on whole numbers {tokens} x {n} x {k} rank {rank}")
    c = lib()
    x, a, b, _, offsets, order, base = case(tokens, n, k, rank, adapters, whole=True)
    y = torch.empty(tokens, n, device="cuda")
    c.low_rank_add(x.cuda(), a.cuda(), b.cuda(), offsets.cuda(), y, workspace(tokens, n, k, rank, adapters), base=base.cuda(),
                   order=order.cuda())
    assert torch.equal(y.double().cpu(), lu.low_rank(x, a, b, None, offsets, order, base)[0])


@pytest.mark.parametrize("tokens,n,k,rank,adapters", [(3, 8200, 130, 16, 2), (20, 5000, 8200, 33, 3), (18, 3333, 5000, 128, 2),
                                                      (9, 512, 511, 64, 8), (2000, 1100, 72, 20, 1500), (4500, 600, 64, 12, 2)])
@pytest.mark.parametrize("y_type", [bf16, torch.float32])
def test_slabs_and_long_contractions(tokens, n, k, rank, adapters, y_type):
    """Few tiles, whose columns go in slabs; contractions of many steps; more lists than a wave counts at once."""
    say(f"adapters in slabs {tokens} x {n} x {k} rank {rank} of {adapters}")
    c = lib()
    x, a, b, scales, offsets, order, base = case(tokens, n, k, rank, adapters)
    y = torch.empty(tokens, n, dtype=y_type, device="cuda")
    ws = workspace(tokens, n, k, rank, adapters)
    c.low_rank_add(x.cuda(), a.cuda(), b.cuda(), offsets.cuda(), y, ws, base=base.cuda(), order=order.cuda(), scales=scales.cuda())
    assert c.ciera_read_error(ws) == 0
    want, size = lu.low_rank(x, a, b, scales, offsets, order, base)
    lu.within(y, want, (k + 3 * rank + 4) * U * size + U * want.abs(), lu.HALF[y_type])


def test_inner_values_keep_24_bits():
    """Inner values of 24 significant bits, picked out one by one: nothing of them is lost."""
    say("adapters, inner values whole")
    c = lib()
    gen = torch.Generator().manual_seed(6)
    for rank in (16, 32, 128):
        # v_r = 2^16 p + 2^8 q + r: three products of whole numbers of 8 bits
        parts = torch.randint(128, 256, (5, 3), generator=gen)
        x = (parts * torch.tensor([2 ** 16, 2 ** 8, 1])).to(bf16)
        a = torch.zeros(1, rank, 3)
        a[0, :, :] = torch.randint(0, 2, (rank, 3), generator=gen).float() * 2 - 1
        b = torch.zeros(1, 48, rank)
        b[0, torch.arange(48), torch.randint(0, rank, (48,), generator=gen)] = 1
        a, b = a.to(bf16), b.to(bf16)
        offsets = torch.tensor([0, 5])
        y = torch.empty(5, 48, device="cuda")
        c.low_rank_add(x.cuda(), a.cuda(), b.cuda(), offsets.cuda(), y, workspace(5, 48, 3, rank, 1))
        assert torch.equal(y.double().cpu(), lu.low_rank(x, a, b, None, offsets, None, torch.zeros(5, 48))[0])


def test_no_tokens_and_no_adapter():
    say("adapters without tokens, without adapters")
    c = lib()
    a, b = torch.ones(2, 4, 16, dtype=bf16, device="cuda"), torch.ones(2, 24, 4, dtype=bf16, device="cuda")
    ws = workspace(8, 24, 16, 4, 2)
    none = torch.empty(0, 16, dtype=bf16, device="cuda")
    c.low_rank_add(none, a, b, torch.zeros(3, dtype=torch.int64, device="cuda"), torch.empty(0, 24, device="cuda"), ws)
    assert c.ciera_read_error(ws) == 0
    x, base = torch.ones(40, 16, dtype=bf16, device="cuda"), torch.randn(40, 24, device="cuda")
    for table in ([0, 0, 0], [40, 40, 40], [17, 17, 17]):
        y = torch.full((40, 24), 7.0, device="cuda")
        c.low_rank_add(x, a, b, torch.tensor(table, device="cuda"), y, ws, base=base)
        assert torch.equal(y, base)
    # rows before the first list and behind the last
    y = torch.full((40, 24), 7.0, device="cuda")
    c.low_rank_add(x, a, b, torch.tensor([3, 20, 36], device="cuda"), y, ws, base=base)
    want = base.clone()
    want[3:36] += 64
    assert torch.equal(y, want)


def test_offsets_out_of_order():
    """Nothing outside the matrices is touched, and the status says so."""
    say("adapters, offsets out of order")
    c = lib()
    a, b = torch.ones(3, 4, 16, dtype=bf16, device="cuda"), torch.ones(3, 24, 4, dtype=bf16, device="cuda")
    ws = workspace(20, 24, 16, 4, 3)
    x = torch.ones(20, 16, dtype=bf16, device="cuda")
    for table in ([0, 9, 5, 20], [0, 5, 9, 21], [-1, 5, 9, 20], [0, 20, 0, 20], [5, 2 ** 40, 9, 20]):
        buf, y = lu.guarded(20, 24, torch.float32)
        c.low_rank_add(x, a, b, torch.tensor(table, device="cuda"), y, ws)
        assert c.ciera_read_error(ws) == 1
        lu.untouched(buf, y)
    # an order that leaves the matrix
    buf, y = lu.guarded(20, 24, torch.float32)
    order = torch.arange(20, dtype=torch.int32)
    order[4], order[11] = 2 ** 30, -5
    c.low_rank_add(x, a, b, torch.tensor([0, 10, 15, 20], device="cuda"), y, ws, order=order.cuda())
    lu.untouched(buf, y)
    live = torch.ones(20, dtype=torch.bool)
    live[[4, 11]] = False
    assert (y[live] == 64).all()


def test_non_finite_values_stay_in_their_rows():
    say("adapters, non-finite values")
    c = lib()
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(20, 64, generator=gen).to(bf16)
    a, b = torch.randn(2, 8, 64, generator=gen).to(bf16), torch.randn(2, 40, 8, generator=gen).to(bf16)
    base = torch.randn(20, 40, generator=gen)
    offsets = torch.tensor([0, 9, 18])
    x[2, 5], x[11, 0], x[19, 3], base[4, 7] = float("nan"), float("inf"), float("nan"), float("-inf")
    want, size = lu.low_rank(x, a, b, None, offsets, None, base)
    y = torch.empty(20, 40, device="cuda")
    c.low_rank_add(x.cuda(), a.cuda(), b.cuda(), offsets.cuda(), y, workspace(20, 40, 64, 8, 2), base=base.cuda())
    fine = [i for i in range(20) if i not in (2, 11)]
    lu.within(y[fine], want[fine], (64 + 24 + 4) * U * torch.nan_to_num(size[fine]) + U * torch.nan_to_num(want[fine]).abs(), U)
    assert y[2].isnan().all() and not torch.isfinite(y[11]).any()
    # an adapter's NaN reaches its own rows alone
    a[1, 3, 9] = float("nan")
    c.low_rank_add(x.cuda(), a.cuda(), b.cuda(), offsets.cuda(), y, workspace(20, 40, 64, 8, 2), base=base.cuda())
    assert torch.isfinite(y[[0, 1, 3, 5, 8]]).all() and y[9:18].isnan().all() and torch.isfinite(y[18:]).all()
    # values next to BF16's largest
    x = torch.full((1, 1), 3.38e38).to(bf16)
    one = torch.ones(1, 1, 1, dtype=bf16)
    y = torch.empty(1, 1, device="cuda")
    c.low_rank_add(x.cuda(), one.cuda(), one.cuda(), torch.tensor([0, 1], device="cuda"), y, workspace(1, 1, 1, 1, 1))
    assert y.item() == x.item()


def test_past_32_bits():
    say("adapters past 32 bits")
    c = lib()
    tokens, n, k, ld = 1100, 40, 64, 1 << 22
    buf = torch.empty(tokens * ld, dtype=bf16, device="cuda")
    x, y = buf.view(tokens, ld)[:, :k], buf.view(tokens, ld)[:, 128:128 + n]
    gen = torch.Generator().manual_seed(3)
    x.copy_(torch.randint(-3, 4, (tokens, k), generator=gen).to(bf16))
    y.copy_(torch.randint(-3, 4, (tokens, n), generator=gen).to(bf16))
    a = torch.randint(-1, 2, (3, 8, k), generator=gen).to(bf16).cuda()
    b = torch.randint(-1, 2, (3, n, 8), generator=gen).to(bf16).cuda()
    offsets, ws = torch.tensor([0, 400, 1000, 1100], device="cuda"), workspace(tokens, n, k, 8, 3)
    want = torch.empty(tokens, n, dtype=bf16, device="cuda")
    c.low_rank_add(x.contiguous(), a, b, offsets, want, ws, base=y.contiguous())
    c.low_rank_add(x, a, b, offsets, y, ws, base=y)
    assert torch.equal(y, want)
    # an adapter whose weights lie past 2^32 bytes
    adapters, rank, k = 1100, 128, 16400
    a = torch.empty(adapters, rank, k, dtype=bf16, device="cuda")
    b = torch.empty(adapters, 8, rank, dtype=bf16, device="cuda")
    a[-1] = torch.randint(-1, 2, (rank, k), generator=gen).to(bf16)
    b[-1] = torch.randint(-1, 2, (8, rank), generator=gen).to(bf16)
    x = torch.randint(-1, 2, (2, k), generator=gen).to(bf16)
    offsets = torch.zeros(adapters + 1, dtype=torch.int64)
    offsets[-1] = 2
    y = torch.empty(2, 8, device="cuda")
    c.low_rank_add(x.cuda(), a, b, offsets.cuda(), y, workspace(2, 8, k, rank, adapters))
    assert torch.equal(y.double().cpu(), (x.double() @ a[-1].double().cpu().T) @ b[-1].double().cpu().T)


def test_refusals():
    say("adapters refusals")
    c = lib()
    x, y = torch.zeros(4, 16, dtype=bf16, device="cuda"), torch.zeros(4, 24, dtype=bf16, device="cuda")
    a, b = torch.zeros(2, 8, 16, dtype=bf16, device="cuda"), torch.zeros(2, 24, 8, dtype=bf16, device="cuda")
    offsets, ws = torch.tensor([0, 2, 4], device="cuda"), workspace(4, 24, 16, 8, 2)
    order = torch.arange(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: c.low_rank_add(x, a[0], b, offsets, y, ws), lambda: c.low_rank_add(x, a, b[:1], offsets, y, ws),
                lambda: c.low_rank_add(x, a, b, offsets[:2], y, ws), lambda: c.low_rank_add(x, a, b, offsets, y[:, :23], ws),
                lambda: c.low_rank_add(x, a, b, offsets, y, ws, base=y[:3]), lambda: c.low_rank_add(x, a, b, offsets, y, ws, order=order[:3]),
                lambda: c.low_rank_add(x, a, b, offsets, y, ws, scales=torch.ones(3, device="cuda")),
                lambda: c.low_rank_add(x, a.transpose(1, 2).contiguous().transpose(1, 2), b, offsets, y, ws)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: c.low_rank_add(x.float(), a, b, offsets, y, ws), lambda: c.low_rank_add(x, a.float(), b, offsets, y, ws),
                lambda: c.low_rank_add(x, a, b, offsets.int(), y, ws), lambda: c.low_rank_add(x, a, b, offsets, y, ws, order=order.long())):
        with pytest.raises(TypeError):
            bad()
    big = torch.zeros(2, 129, 16, dtype=bf16, device="cuda")
    with pytest.raises(c.CieraError):
        c.low_rank_add(x, big, torch.zeros(2, 24, 129, dtype=bf16, device="cuda"), offsets, y, ws)
    with pytest.raises(c.CieraError):
        c.low_rank_add(x, a, b, offsets, y, ws[:256])
    wide = torch.zeros(4, 40, dtype=bf16, device="cuda")
    with pytest.raises(c.CieraError):  # y itself at another stride
        c.low_rank_add(x, a, b, offsets, wide[:, :24], ws, base=wide.view(-1)[:96].view(4, 24))
