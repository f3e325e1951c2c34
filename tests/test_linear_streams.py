"""Where the wrappers' own tensors come from when a stream is given, without a device: their allocation happens while
that stream is the current one, and every one of them is held for the stream that the caller goes on with."""
import contextlib
import types

import pytest
import torch

import async_stage_tile_amd as pt
from async_stage_tile_amd import linear


class Recorder:
    """Stands for a tensor and for what allocates it."""

    def __init__(self, log):
        self.log = log

    def new_empty(self, shape, dtype):
        self.log.append(("new", self.log.current))
        return self

    def record_stream(self, stream):
        self.log.append(("held", stream))


class Log(list):
    current = "caller's"


@pytest.fixture
def log(monkeypatch):
    log = Log()

    @contextlib.contextmanager
    def on(stream):
        before, log.current = log.current, stream
        yield
        log.current = before

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: log.current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return log


def test_tensors_of_a_given_stream(log):
    linear._setup()
    like, made = Recorder(log), []
    for shape in ((4, 64), (4,), (1024,)):
        linear._make(made, "given", like, shape, torch.float32)
    assert log == [("new", "given")] * 3 and len(made) == 3
    log.clear()
    side = types.SimpleNamespace(device=types.SimpleNamespace(index=0), cuda_stream=77)
    linear._call(lambda *args: 0 if args == (1, 77) else 1, "name", 0, side, made, 1)
    assert log == [("held", "caller's")] * 3


def test_tensors_of_the_current_stream(log):
    like, made = Recorder(log), []
    linear._make(made, None, like, (4, 64), torch.float32)
    pt._hold_for(None, 0, *made)
    pt._hold_for("caller's", 0, *made)
    assert log == [("new", "caller's")]
