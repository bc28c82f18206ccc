"""examples/decoder_layer.py without a GPU: the order of its work on streams."""
import importlib.util
import os
import sys
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Streams:
    """What main() asks of torch.cuda, written down as it comes."""

    def __init__(self):
        self.log, self.at = [], ["main"]

    def stream(self, name):
        return types.SimpleNamespace(name=name, wait_stream=lambda other: self.log.append((name, "waits for", other.name)))

    def within(self, name):
        import contextlib

        @contextlib.contextmanager
        def change():
            self.at.append(name)
            yield
            self.at.pop()
        return change()

    def did(self, what):
        self.log.append((self.at[-1], what))


@pytest.fixture
def example():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_first_steps_wait_for_the_set_up_on_the_other_stream(example, monkeypatch):
    import torch
    s = Streams()

    class Layer:
        def __init__(self, *a):
            s.did("set-up")
            self.x, self.status, self.seq_lens = self, 0, torch.zeros(1)

        def normal_(self):
            s.did("x")

        def step(self):
            s.did("step")

        def float(self):
            return torch.ones(1)

    class Event:
        def __init__(self, **kw):
            pass

        def record(self):
            pass

        def elapsed_time(self, other):
            return 1.0

    monkeypatch.setattr(example, "DecoderLayer", Layer)
    monkeypatch.setattr(sys, "argv", ["decoder_layer.py", "--steps", "3"])
    for name, value in (("Stream", lambda: s.stream("side")), ("current_stream", lambda: s.stream(s.at[-1])),
                        ("stream", lambda stream: s.within(stream.name)), ("Event", Event), ("synchronize", lambda: None),
                        ("CUDAGraph", lambda: types.SimpleNamespace(replay=lambda: s.did("replay"))),
                        ("graph", lambda graph: s.within("capture"))):
        monkeypatch.setattr(torch.cuda, name, value)
    example.main()
    set_up = max(i for i, e in enumerate(s.log) if e in (("main", "set-up"), ("main", "x")))
    first = s.log.index(("side", "step"))
    assert ("side", "waits for", "main") in s.log[set_up + 1:first], s.log
    after = max(i for i, e in enumerate(s.log) if e == ("side", "step"))
    assert ("main", "waits for", "side") in s.log[after + 1:s.log.index(("main", "replay"))]
