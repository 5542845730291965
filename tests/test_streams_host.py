"""CPU checks of the stream that a call's own memory belongs to."""
import contextlib

import torch

from adam_ob_compress_amd import _native as nat


class Stream:
    cuda_stream = 7


def test_a_new_workspace_is_the_streams(monkeypatch):
    """Memory that torch gives out on one stream may still be in use there, so a call on another takes its own on that one."""
    current = []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    s = Stream()
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda number, device: (number, device))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: list(current))   # what it is given out on
    assert nat._workspace(None, 8, "cuda:0", s) == [s]
    assert nat._workspace(None, 8, "cuda:0", 9) == [(9, "cuda:0")]
    assert nat._workspace(None, 8, "cuda:0", None) == []
    assert nat._workspace("given", 8, "cuda:0", s) == "given"
