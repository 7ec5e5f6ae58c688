"""The row-wise operators' first call from two threads at once, on the host."""
import threading

import pytest

import edge_message_passing_b200 as emp

torch = pytest.importorskip("torch")


def test_first_calls_of_two_threads(monkeypatch):
    """A second thread comes while the first is still at the set-up: it has to find the types all the same."""
    inside, go = threading.Event(), threading.Event()

    class Slow(dict):
        def update(self, *a, **k):
            inside.set()
            go.wait(10)
            super().update(*a, **k)

    monkeypatch.setattr(emp, "_torch", lambda: torch)          # (which wants a device)
    monkeypatch.setattr(emp, "_T", None)
    monkeypatch.setattr(emp, "_stream_of", emp._stream_of)
    monkeypatch.setattr(emp, "_CODES", Slow())
    seen = []

    def second():
        emp._row_torch()
        seen.append(emp._CODES.get(torch.bfloat16))

    first = threading.Thread(target=emp._row_torch)
    first.start()
    assert inside.wait(10)
    late = threading.Thread(target=second)
    late.start()
    late.join(0.5)                     # it comes back with a type's code, or waits in the same set-up
    go.set()
    first.join(10)
    late.join(10)
    assert seen == [1] and emp._CODES[torch.float32] == 0
