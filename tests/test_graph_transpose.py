"""The sender transpose that a Graph keeps: calls on other streams wait for it, threads never see half of it, and one
made inside a capture is not kept.  Streams and the transpose itself are stand-ins; no GPU needed."""
import pytest
import torch


class Stream:
    def __init__(self, name, log):
        self.name, self.log = name, log

    def record_event(self):
        self.log.append(("record", self.name))
        return "event of " + self.name

    def wait_event(self, event):
        self.log.append(("wait", self.name, event))


class Tensor:
    def __init__(self, log, name):
        self.log, self.name = log, name

    def record_stream(self, stream):
        self.log.append(("used", self.name, stream.name))


@pytest.fixture
def world(monkeypatch):
    from equivariant_tensor_product_b200 import autograd
    log, now = [], dict(stream=None, capturing=False)
    made = lambda *a: log.append(("transpose", now["stream"].name)) or (Tensor(log, "colptr"), Tensor(log, "perm"))
    monkeypatch.setattr(autograd, "tp_csr_transpose", made)
    monkeypatch.setattr(autograd, "stream_of", lambda index: now["stream"].name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    graph = autograd.Graph(torch.tensor([0, 1, 2]), torch.tensor([1, 0]))
    return graph, now, log, Stream("a", log), Stream("b", log)


def test_another_stream_waits(world):
    graph, now, log, a, b = world
    now["stream"] = a
    first = graph.transpose()
    assert graph.transpose() == first and log == [("transpose", "a"), ("record", "a")]
    now["stream"] = b
    assert graph.transpose() == first
    assert log[2:] == [("wait", "b", "event of a"), ("used", "colptr", "b"), ("used", "perm", "b")]


def test_what_a_capture_makes_is_its_own(world):
    graph, now, log, a, b = world
    now.update(stream=a, capturing=True)
    first = graph.transpose()
    assert graph._colptr is None and graph.transpose() != first
    now["capturing"] = False
    kept = graph.transpose()
    assert log == [("transpose", "a")] * 3 + [("record", "a")]
    now.update(stream=b, capturing=True)
    assert graph.transpose() == kept and log[4:] == []         # no wait for an event outside the capture


def test_both_arrays_are_there_when_the_first_is(world):
    graph, now, log, a, _ = world
    now["stream"] = a
    seen = []

    class Watch(type(graph)):
        def __setattr__(self, name, value):
            if name == "_colptr" and value is not None:
                seen.append((self._perm, self._built))
            super().__setattr__(name, value)
    graph.__class__ = Watch
    graph.transpose()
    assert len(seen) == 1 and None not in seen[0]
