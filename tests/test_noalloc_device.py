"""noalloc_status asks the library for the status word of its own device, with
that device current (CPU only: the calls are recorded, not made)."""
import contextlib

import torch

from learned_bit_lut_b200 import _lib


def test_status_word_of_another_device(monkeypatch):
    events = []

    @contextlib.contextmanager
    def device(dev):
        events.append(("enter", torch.device(dev).index))
        yield
        events.append(("leave", torch.device(dev).index))

    def status_word(_):
        events.append(("query",))
        return 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev: events.append(("synchronize", torch.device(dev).index)))
    monkeypatch.setattr(_lib.lib, "any4_noalloc_status_word", status_word)
    monkeypatch.setattr(_lib, "_DeviceWord", lambda ptr: [0])
    monkeypatch.setattr(torch, "as_tensor", lambda word, device: torch.zeros(1, dtype=torch.int32))
    assert _lib.noalloc_status(torch.device("cuda", 3)) == 0
    assert events == [("enter", 3), ("query",), ("synchronize", 3), ("leave", 3)]
