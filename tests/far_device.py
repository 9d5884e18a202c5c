"""A stand-in for a second GPU: CPU tensors that say they are on cuda:1 while
cuda:0 is current, and a library that records the device that was current when
an entry was called. What the binding does around its calls needs no GPU."""
import contextlib

import torch


class Far(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))

    def get_device(self):
        return 1


def far(t):
    return t.as_subclass(Far)


class Machine:
    """The current device and the calls made: (entry, current device, arguments)."""

    def __init__(self):
        self.current, self.calls = 0, []

    def __getattr__(self, entry):
        def fn(*args):
            self.calls.append((entry, self.current, args))
            return 0
        return fn


def install(monkeypatch):
    """Puts a Machine in place of the library and the CUDA runtime."""
    from newton_schulz_gram_gb300 import _lib, block
    m = Machine()

    @contextlib.contextmanager
    def device(index):
        before, m.current = m.current, torch.device("cuda", index).index if isinstance(index, int) else index.index
        try:
            yield
        finally:
            m.current = before

    empty = torch.empty

    def far_empty(*shape, dtype=None, device=None):
        assert torch.device(device if not isinstance(device, int) else f"cuda:{device}").index == 1
        return far(empty(*shape, dtype=dtype))

    class Stream:
        cuda_stream = 0

    monkeypatch.setattr(_lib, "_LIB", m)
    monkeypatch.setattr(_lib, "_current_device", lambda: m.current, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: m.current)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    monkeypatch.setattr(torch, "empty", far_empty)
    monkeypatch.setattr(block, "_empty", far_empty)
    monkeypatch.setattr(block, "_raw_stream", lambda index: 0)
    return m
