"""low_rank_add with infinities in B against the 64-bit formula: an infinity
times an inner value is an infinity of their sign, NaN where the inner value is
zero or an infinity of the other sign is added; all other columns, rows and
adapters keep their bits."""
import pytest

import layer_util as lu
from gpu_util import require_gpu, say
from test_gpu_low_rank import U, bf16, case, lib, workspace

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("tokens,n,k,rank,adapters", [(5, 40, 24, 1, 2), (40, 200, 64, 8, 3), (64, 130, 72, 16, 3), (33, 1100, 256, 17, 2),
                                                      (50, 72, 40, 32, 4), (150, 700, 129, 40, 2), (90, 65, 64, 64, 3), (48, 640, 96, 100, 2),
                                                      (200, 1025, 64, 128, 2)])
@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("kind", [bf16, torch.float32])
def test_infinities_in_b(tokens, n, k, rank, adapters, whole, kind):
    say(f"adapters, infinities in b {tokens} x {n} x {k} rank {rank} of {adapters} {'whole' if whole else 'real'} {kind}")
    c = lib()
    x, a, b, scales, offsets, order, base = case(tokens, n, k, rank, adapters, whole=whole)
    base = base.to(kind)
    if whole:
        x[::7] = 0  # inner values of zero: NaN in the columns of an infinity

    def run(b, onto):
        ws = workspace(tokens, n, k, rank, adapters)
        y = base.cuda() if onto else torch.full((tokens, n), 7.0, dtype=kind, device="cuda")
        c.low_rank_add(x.cuda(), a.cuda(), b.cuda(), offsets.cuda(), y, ws, base=y if onto else base.cuda(), order=order.cuda(),
                       scales=None if scales is None else scales.cuda())
        assert c.ciera_read_error(ws) == 0
        return y

    plain = run(b, False)
    inf, at = float("inf"), {}
    b = b.clone()
    at[0] = [2, n // 2, n - 1, n - 3]
    b[0, 2, 0], b[0, n // 2, rank // 2], b[0, n - 1, rank - 1] = inf, -inf, inf
    b[0, n - 3, 0], b[0, n - 3, rank - 1] = inf, -inf  # both signs, from 2 ranks on
    if adapters > 2:
        at[2] = [0, n - 2]
        b[2, 0, rank // 3], b[2, n - 2] = -inf, float("nan")
    y = run(b, False)
    assert torch.equal(torch.nan_to_num(run(b, True).float(), 1.0, 2.0, 3.0), torch.nan_to_num(y.float(), 1.0, 2.0, 3.0))
    want, size = lu.low_rank(x, a, b, scales, offsets, order, base)
    same = torch.ones(tokens, n, dtype=torch.bool)
    for g, columns in at.items():
        for row in order[int(offsets[g]):int(offsets[g + 1])].tolist():
            same[row, columns] = False
    assert torch.equal(y.cpu()[same], plain.cpu()[same])
    size = torch.nan_to_num(size, 0.0, 0.0)
    lu.within(y, want, (k + 3 * rank + 4) * U * size + U * torch.nan_to_num(want, 0.0, 0.0, 0.0).abs(), lu.HALF[kind])


@pytest.mark.parametrize("rank", [1, 16, 20, 64, 128])
def test_infinite_inner_values(rank):
    """Infinities on both sides, and of x alone."""
    say(f"adapters, infinite inner values, rank {rank}")
    c = lib()
    x = torch.tensor([[1.0, 0.0], [float("inf"), 0.0], [-1.0, 0.0], [float("-inf"), 1.0]], dtype=bf16)
    a = torch.zeros(1, rank, 2)
    a[0, :, 0], a[0, :, 1] = 1.0, 1.0
    b = torch.ones(1, 5, rank)
    b[0, 1, 0], b[0, 2], b[0, 3] = float("inf"), float("-inf"), 0.0
    b[0, 4] = -2.0
    a, b = a.to(bf16), b.to(bf16)
    y = torch.empty(4, 5, device="cuda")
    c.low_rank_add(x.cuda(), a.cuda(), b.cuda(), torch.tensor([0, 4], device="cuda"), y, workspace(4, 5, 2, rank, 1))
    want, _ = lu.low_rank(x, a, b, None, torch.tensor([0, 4]), None, torch.zeros(4, 5))
    lu.within(y, want, torch.zeros_like(want))
