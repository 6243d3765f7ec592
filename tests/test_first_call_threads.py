"""First calls of several threads at once: each finds every C function bound."""
import sys
import threading

import pytest

pytest.importorskip("torch")


def test_a_first_call_while_another_thread_binds(monkeypatch):
    """At every step of one thread's binding but the first another makes its first call."""
    from lossless_bf16_tensor_exp_amd import layers
    monkeypatch.setattr(layers, "_functions", {})
    library, seen, missing = layers.load_library(), [], []

    def first_call():
        table = layers._bind()
        missing.extend(n for n in ("rms_norm_workspace_size", "rms_norm", "expert_sort", "low_rank_add") if n not in table)
        missing.extend(n for n in ("rms_norm", "low_rank_add") if n not in layers._functions)

    class Slow:
        def __getattr__(self, name):
            if threading.current_thread() is not threading.main_thread():
                return getattr(library, name)
            if seen:
                other = threading.Thread(target=first_call)
                other.start()
                other.join(10)
                assert not other.is_alive(), name
            seen.append(name)
            return getattr(library, name)

    slow = Slow()
    monkeypatch.setattr(layers, "load_library", lambda: slow)
    assert "low_rank_add" in layers._bind()
    assert seen and not missing, missing


def test_first_calls_of_four_threads(monkeypatch):
    from lossless_bf16_tensor_exp_amd import layers
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    failed = []
    try:
        for _ in range(300):
            monkeypatch.setattr(layers, "_functions", {})
            gate = threading.Barrier(4)

            def call():
                gate.wait()
                try:
                    assert layers.low_rank_workspace_size(4, 64, 64, 8, 2) > 0
                    layers._functions["low_rank_add"]
                except KeyError as e:
                    failed.append(str(e))

            threads = [threading.Thread(target=call) for _ in range(4)]
            for t in threads:
                t.start()
            for t in threads:
                t.join()
    finally:
        sys.setswitchinterval(interval)
    assert not failed, f"{len(failed)} calls found no {sorted(set(failed))}"
