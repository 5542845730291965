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


def test_one_bit_steps_make_their_clips_before_the_first_step(monkeypatch):
    """What a step allocates and fills on the current stream is not ordered with a step on another, and cannot be captured."""
    from adam_ob_compress_amd import schedule

    made, calls = [], []

    class Clip:
        def __init__(self, params, *, max_norm, grad_dtype):
            made.append((params[0].numel(), max_norm, grad_dtype))
            self.norms = torch.zeros(2)

        def __call__(self, grads, stream):
            calls.append((grads[0].dtype, stream))
            return self.norms[-1:]

    class Plan:
        n, num_chunks = 64, 1

    monkeypatch.setattr(schedule, "GradClip", Clip)
    for name in ("ob_adam_warmup_step", "ob_adam_compress_step"):
        monkeypatch.setattr(nat, name, lambda *a: calls.append(a[-1]))
    guards = []
    monkeypatch.setattr(nat, "ob_plan_set_guard", lambda plan, norm: guards.append((norm is not None, len(calls))))
    opt = schedule.OneBitAdam(Plan(), *(torch.zeros(64) for _ in range(4)), lr=1.0, freeze_step=1, max_norm=2.0)
    assert sorted(made, key=str) == [(64, 2.0, torch.bfloat16), (64, 2.0, torch.float32)]
    s = Stream()
    for dtype in (torch.float32, torch.bfloat16):
        opt.step(torch.zeros(64, dtype=dtype), stream=s)
    assert len(made) == 2 and [c[0] for c in calls if isinstance(c, tuple)] == [torch.float32, torch.bfloat16]
    assert all(c[1] is s for c in calls if isinstance(c, tuple))
    # each step looks at its norm, behind its clipping, and the plan's later calls at none
    assert guards == [(True, 1), (False, 2), (True, 3), (False, 4)]
    for bad, error in ((torch.zeros(64, dtype=torch.float16), TypeError), (torch.zeros(32), ValueError)):
        before = len(calls)
        try:
            opt.step(bad)
        except error:
            assert len(calls) == before   # what the step refuses is not clipped
        else:
            raise AssertionError("not refused")
    monkeypatch.setattr(nat, "ob_adam_compress_step", lambda *a: 1 / 0)
    guards.clear()
    try:
        opt.step(torch.zeros(64))
    except ZeroDivisionError:
        assert [g[0] for g in guards] == [True, False]
    made.clear()
    schedule.OneBitAdam(Plan(), *(torch.zeros(64) for _ in range(4)), lr=1.0)
    assert not made


def test_guard_refusals():
    lib = nat.lib()
    assert lib.ob_plan_set_guard(None, None) == 1
