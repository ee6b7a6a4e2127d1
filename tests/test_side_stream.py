"""What a call allocates for itself when it is given another stream than the current one: made_on
with stand-ins for the streams, on the CPU."""
import contextlib

import torch

from speculative_decoding_verification_41_gb300 import binding


class _Tensor(torch.Tensor):
    """A tensor that notes the streams it was recorded on."""

    def record_stream(self, stream):
        self.__dict__.setdefault("seen", []).append(stream)


def _patched(monkeypatch):
    now = ["current"]

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    return now


class _Side:
    device = torch.device("cpu")


class _Buffers:
    def __init__(self, where):
        self.B = 3
        self.where = where
        self.a = torch.zeros(2).as_subclass(_Tensor)
        self.none = None


def test_without_a_stream_nothing_changes(monkeypatch):
    now = _patched(monkeypatch)
    b = binding.made_on(None, lambda: _Buffers(now[-1]))
    assert b.where == "current" and not hasattr(b.a, "seen")


def test_allocated_on_the_call_s_stream_and_kept_for_the_current_one(monkeypatch):
    now = _patched(monkeypatch)
    side = _Side()
    b = binding.made_on(side, lambda: _Buffers(now[-1]))
    assert b.where is side and b.a.seen == ["current"] and now == ["current"]
    made = []
    t = binding.made_on(side, lambda: made.append(now[-1]) or torch.zeros(1).as_subclass(_Tensor))
    assert made == [side] and t.seen == ["current"]
