"""What an owner's ``error`` says: of calls that were made, and CIERA_OK where
none was, whatever its memory held before.  Without a GPU the library's reading
of a workspace is replaced by one of a tensor in host memory."""
import pytest

torch = pytest.importorskip("torch")
from gpu_util import require_gpu, say  # noqa: E402

bf16 = torch.bfloat16
HEAD, SLOTS, ARG = 256, 8, 1  # bytes before the status words, and where among them their number lies


def owners(device):
    """An owner of each kind, and the name of the call that reads its workspace."""
    from lossless_bf16_tensor_exp_amd.codec import CieraCodec, ExpertRows, LowRankAdapters, MxLinear, Zip3Codec
    zip3, ciera = Zip3Codec(5000, device=device), CieraCodec(5000, 64, device=device)
    made = [(zip3, "error"), (ciera, "error"), (ciera, "decode_error"), (MxLinear(8, 16, 32, 3, device=device), "error"),
            (ExpertRows(8, 2, 3, device=device), "error"), (LowRankAdapters(8, 16, 32, 4, 3, device=device), "error")]
    return made


def read_on_the_host(ws, stream=None):
    """ciera_read_error of a workspace in host memory."""
    slots = int(ws[SLOTS:SLOTS + 8].view(torch.int64))
    assert 0 <= slots and HEAD + 4 * slots <= ws.numel(), f"{slots} status words in a workspace of {ws.numel()} bytes"
    return int(ws[HEAD:HEAD + 4 * slots].view(torch.int32).max()) if slots else 0


@pytest.fixture
def used_memory(monkeypatch):
    """Memory comes with something in it, as on a device where tensors were before."""
    from lossless_bf16_tensor_exp_amd import codec
    empty = torch.empty

    def used(*shape, **kw):
        t = empty(*shape, **kw)
        t.view(torch.uint8).fill_(1)
        return t

    monkeypatch.setattr(torch, "empty", used)
    monkeypatch.setattr(codec, "ciera_read_error", read_on_the_host)


def test_no_call_no_error(used_memory):
    for owner, error in owners("cpu"):
        assert getattr(owner, error)() == 0, type(owner).__name__


@pytest.fixture
def on_the_host(used_memory, monkeypatch):
    """A sort and an add that leave a status in the workspaces they are given, as their kernels do: CIERA_ERR_ARG of a
    number of no expert, and of offsets out of order."""
    from lossless_bf16_tensor_exp_amd import codec

    def leave(ws, ok):
        ws[SLOTS:SLOTS + 8].view(torch.int64).fill_(1)
        ws[HEAD:HEAD + 4].view(torch.int32).fill_(0 if ok else ARG)

    def sort(ids, offsets, place, order, ws, stream=None):
        leave(ws, bool((ids < offsets.numel() - 1).all()))

    def add(x, a, b, offsets, y, ws, base=None, order=None, scales=None, stream=None):
        leave(ws, bool((offsets.diff() >= 0).all()))

    monkeypatch.setattr(codec, "expert_sort", sort)
    monkeypatch.setattr(codec, "low_rank_add", add)


def check_shared_plan(device):
    """Owners whose adds take another's plan: each error is that of the plan its own last add took, and of the add."""
    from lossless_bf16_tensor_exp_amd.codec import LowRankAdapters
    planner, user, idle = (LowRankAdapters(8, 16, 32, 4, 3, device=device) for _ in range(3))
    x, y = torch.ones(5, 32, dtype=bf16, device=device), torch.zeros(5, 16, dtype=bf16, device=device)
    good = torch.tensor([0, 2, -1, 1, 2], device=device)
    bad = torch.tensor([0, 2, 3, 1, 2], device=device)  # of three adapters
    planner.plan(good)
    assert planner.error() == 0  # it planned and added nothing
    user.add(x, y, plan=planner)
    assert user.error() == planner.error() == idle.error() == 0
    planner.plan(bad)
    user.add(x, y, plan=planner)
    assert user.error() == planner.error() == ARG and idle.error() == 0
    # a plan of its own does not hide what its add took, and the next add takes its own
    user.plan(good)
    assert user.error() == ARG
    user.add(x, y)
    assert user.error() == 0 and planner.error() == ARG
    # its own last plan, of which no add has been made
    user.plan(bad)
    assert user.error() == ARG
    planner.plan(good)
    user.add(x, y, plan=planner)
    assert user.error() == ARG
    user.plan(good)
    assert user.error() == planner.error() == 0
    # an add of offsets out of order
    planner.rows.offsets.copy_(torch.tensor([0, 4, 2, 5]))
    user.add(x, y, plan=planner)
    assert user.error() == ARG and planner.error() == 0


def test_shared_plan(on_the_host):
    check_shared_plan("cpu")


@pytest.mark.gpu
def test_shared_plan_on_the_gpu():
    require_gpu()
    say("the status of adds by another's plan")
    check_shared_plan("cuda")


@pytest.mark.gpu
def test_no_call_no_error_on_the_gpu():
    require_gpu()
    say("the status of owners that made no call")
    for n in (256, 512, 768, 1024, 4096, 1 << 16, 1 << 20):  # what the owners' buffers are then made from
        full = [torch.full((n,), 1, dtype=torch.uint8, device="cuda") for _ in range(32)]
        del full
    torch.cuda.synchronize()
    for owner, error in owners("cuda"):
        assert getattr(owner, error)() == 0, type(owner).__name__
