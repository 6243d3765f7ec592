"""LowRankAdapters.load on the stream of the calls that read the adapter."""
import pytest

import layer_util as lu
from gpu_util import require_gpu, say

torch = pytest.importorskip("torch")

U = 2.0 ** -24
bf16 = torch.bfloat16


def test_every_write_is_on_the_given_stream(monkeypatch):
    from lossless_bf16_tensor_exp_amd.codec import LowRankAdapters
    low = LowRankAdapters(4, 16, 8, 4, 2, device="cpu")
    low.load(1, torch.ones(4, 8, dtype=bf16), torch.ones(16, 4, dtype=bf16))
    seen = []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def state(self):
            return [t.clone() for t in (low.a, low.b, low.scales)]

        def __enter__(self):
            seen.append((self.stream, self.state()))

        def __exit__(self, *_):
            seen.append((self.stream, self.state()))

    before = On(None).state()
    monkeypatch.setattr(torch.cuda, "stream", On)
    low.load(1, torch.full((2, 8), 3.0, dtype=bf16), torch.full((16, 2), 5.0, dtype=bf16), 0.5, stream="s")
    after = On(None).state()
    assert [s for s, _ in seen] == ["s", "s"]
    assert all(torch.equal(a, b) for a, b in zip(before, seen[0][1])) and all(torch.equal(a, b) for a, b in zip(after, seen[1][1]))
    assert (low.a[1, :2] == 3).all() and (low.a[1, 2:] == 0).all() and (low.b[1, :, :2] == 5).all() and (low.b[1, :, 2:] == 0).all()
    assert low.scales.tolist() == [1.0, 0.5] and (low.a[0] == 0).all()


@pytest.mark.gpu
def test_an_adapter_replaced_between_two_steps():
    """A step, a load and a step queued on one stream behind a wait: the first sees the adapter as it was, the second as
    it is then, whatever the current stream does."""
    require_gpu()
    say("an adapter replaced between two steps on a given stream")
    from lossless_bf16_tensor_exp_amd.codec import LowRankAdapters
    gen = torch.Generator().manual_seed(4)
    tokens, n, k, rank, adapters = 70, 264, 200, 16, 4
    low = LowRankAdapters(tokens, n, k, rank, adapters)

    def adapter(r):
        return (torch.randn(r, k, generator=gen) * k ** -0.5).to(bf16), (torch.randn(n, r, generator=gen) * 0.2).to(bf16)

    for i in range(adapters):
        a, b = adapter(rank)
        low.load(i, a.cuda(), b.cuda(), 1.0 + i)
    x = lu.mx.activations(gen, tokens, k)
    ids = torch.randint(-1, adapters, (tokens,), generator=gen)
    ids[:3] = 2
    given, on = x.cuda(), ids.cuda()
    new = [t.cuda() for t in adapter(rank - 3)]
    y1, y2 = torch.zeros(tokens, n, device="cuda"), torch.zeros(tokens, n, device="cuda")
    was = [t.cpu() for t in (low.a, low.b, low.scales)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)  # some 10 ms: a write on another stream would come before the first step
    low.plan(on, stream)
    low.add(given, y1, stream=stream)
    low.load(2, *new, 0.5, stream=stream)
    low.add(given, y2, stream=stream)
    assert low.error(stream) == 0
    torch.cuda.synchronize()
    now = [t.cpu() for t in (low.a, low.b, low.scales)]
    assert (now[0][2, rank - 3:] == 0).all() and torch.equal(now[0][2, :rank - 3], new[0].cpu()) and now[2][2] == 0.5
    offsets, _, order = lu.sort(ids, adapters)
    for y, (a, b, scales) in ((y1, was), (y2, now)):
        want, size = lu.low_rank(x, a, b, scales, offsets, order, torch.zeros(tokens, n))
        lu.within(y, want, (k + 3 * rank + 4) * U * size + U * want.abs(), U)


def test_trained_parameters_leave_no_graph():
    """Adapters as a training loop holds them: the buffers take their values and keep nothing of them."""
    from lossless_bf16_tensor_exp_amd.codec import LowRankAdapters
    low = LowRankAdapters(4, 16, 8, 4, 2, device="cpu")
    a = torch.nn.Parameter(torch.full((3, 8), 2.0, dtype=bf16))
    b = torch.nn.Parameter(torch.full((16, 3), 3.0, dtype=bf16))
    scale = torch.nn.Parameter(torch.tensor(0.25))
    for _ in range(2):
        low.load(1, a * 2, b, scale)
        for t in (low.a, low.b, low.scales):
            assert not t.requires_grad and t.grad_fn is None
    assert (low.a[1, :3] == 4).all() and (low.b[1, :, :3] == 3).all() and low.scales[1] == 0.25
    assert torch.is_grad_enabled()
