"""ciera_read_error of a workspace on another device than the current one: it
waits for the stream of the workspace's device, where the calls on it went.
The devices are stand-ins."""
import contextlib
import types

import pytest

pytest.importorskip("torch")


@pytest.fixture
def two_devices(monkeypatch):
    """Two devices, the first of them current, and what the C function was called with."""
    import lossless_bf16_tensor_exp_amd as ciera
    seen, current = [], [0]

    @contextlib.contextmanager
    def device(d):
        was, current[0] = current[0], d
        yield
        current[0] = was

    def current_stream(d=None):
        return types.SimpleNamespace(cuda_stream=100 + (current[0] if d is None else d))

    def read(ws, stream):
        seen.append((current[0], stream.value))
        return 0

    monkeypatch.setattr(ciera, "_torch", lambda: types.SimpleNamespace(
        cuda=types.SimpleNamespace(device=device, current_stream=current_stream)))
    monkeypatch.setattr(ciera, "_check_bytes", lambda ws, name: None)
    monkeypatch.setattr(ciera, "load_library", lambda: types.SimpleNamespace(ciera_read_error=read))
    return ciera, seen, current


def workspace(device):
    return types.SimpleNamespace(device=device, data_ptr=lambda: 4096, numel=lambda: 512)


def test_the_workspaces_own_device(two_devices):
    ciera, seen, current = two_devices
    assert ciera.ciera_read_error(workspace(0)) == ciera.ciera_read_error(workspace(1)) == 0
    assert seen == [(0, 100), (1, 101)] and current == [0]


def test_a_given_stream(two_devices):
    ciera, seen, current = two_devices
    ciera.ciera_read_error(workspace(1), types.SimpleNamespace(cuda_stream=7))
    assert seen == [(1, 7)] and current == [0]
