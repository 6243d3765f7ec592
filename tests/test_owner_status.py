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
