"""How a call on another stream is ordered against the current one, and that
its tensors are kept for it (CPU, with stand-ins for torch's streams)."""
import contextlib
import types

import pytest

from selective_state_space_51_b200._launch import launch


class Torch:
    """What launch() uses of torch, with a record of what it does."""

    def __init__(self):
        outer = self
        self.did = []
        self.device = types.SimpleNamespace(index=0)
        self.captured = set()

        class Stream:
            def __init__(self, handle, device=None):
                self.cuda_stream, self.device = handle, device or outer.device

            def wait_stream(self, other):
                outer.did.append(("wait", self.cuda_stream,
                                  other.cuda_stream))

        class Tensor:
            def record_stream(self, stream):
                outer.did.append(("keep", stream.cuda_stream))

        self.Stream, self.Tensor = Stream, Tensor
        self.current = Stream(0)
        self.cuda = types.SimpleNamespace(
            ExternalStream=lambda handle, device: Stream(handle, device),
            current_device=lambda: 0,
            current_stream=lambda device: self.current,
            device=lambda device: contextlib.nullcontext(),
            stream=self.on,
            is_current_stream_capturing=lambda: (
                self.current.cuda_stream in self.captured))
        self._C = types.SimpleNamespace(
            _cuda_getCurrentRawStream=lambda i: self.current.cuda_stream)

    @contextlib.contextmanager
    def on(self, stream):
        was, self.current = self.current, stream
        yield
        self.current = was

    def call(self, s, *args):
        self.did.append(("call", s, self.current.cuda_stream))
        return "result"

    def launch(self, stream, *args):
        self.did.clear()
        assert launch(self, self.device, stream, self.call,
                      *args) == "result"
        return self.did


@pytest.fixture
def torch():
    return Torch()


def test_the_current_stream(torch):
    t = torch.Tensor()
    assert torch.launch(None, t, 3) == [("call", 0, 0)]
    assert torch.launch(torch.Stream(0), t) == [("call", 0, 0)]
    assert torch.launch(0, t) == [("call", 0, 0)]
    torch.current = torch.Stream(7)
    assert torch.launch(None, t) == [("call", 7, 7)]
    assert torch.launch(torch.Stream(7), t) == [("call", 7, 7)]


def test_another_stream_waits_and_keeps_the_tensors(torch):
    a, b = torch.Tensor(), torch.Tensor()
    assert torch.launch(torch.Stream(5), a, None, 0.5, b, (1, 2)) == [
        ("wait", 5, 0), ("call", 5, 5), ("keep", 5), ("keep", 5)]


def test_a_raw_stream_waits(torch):
    assert torch.launch(5, torch.Tensor()) == [("wait", 5, 0), ("call", 5, 5)]


def test_captured_calls(torch):
    torch.captured = {5}
    assert ("wait", 5, 0) not in torch.launch(torch.Stream(5))
    torch.current = torch.Stream(6)
    assert ("wait", 5, 6) not in torch.launch(torch.Stream(5))
    torch.captured = {5, 6}          # one capture, forked
    assert ("wait", 5, 6) in torch.launch(torch.Stream(5))
    torch.captured = {6}             # forks here
    assert ("wait", 5, 6) in torch.launch(torch.Stream(5))


def test_another_devices_stream_is_refused(torch):
    far = torch.Stream(5, types.SimpleNamespace(index=1))
    with pytest.raises(ValueError):
        launch(torch, torch.device, far, torch.call)
