"""Host side of the prepared norm calls and of calls on a given stream (no GPU
needed): the device, the streams and the library are stand-ins that record
what they are told."""
import types

import pytest
import torch

from zero_sharded_optimizer_flatten_gb300 import train_ops as T


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle
        self.waited = []

    def wait_event(self, event):
        self.waited.append(event)


@pytest.fixture
def cpu_calls(monkeypatch):
    """Prepared calls over host tensors: device 0 with current stream 7, a
    library that records its calls, and a list of (stream, tensor) records."""
    seen = types.SimpleNamespace(device=0, current=7, calls=[], kept=[], capturing=False,
                                 streams={7: FakeStream(7), 9: FakeStream(9)})

    def record(*args):
        seen.calls.append(args)
        return 0

    def size(tensors, n, out):
        out._obj.value = 64
        return 0

    monkeypatch.setattr(T, "_lib", types.SimpleNamespace(
        zero_grad_norm=record, zero_clip_grad_norm=record, zero_grad_norm_workspace_bytes=size))
    monkeypatch.setattr(T, "_device", lambda: seen.device)
    monkeypatch.setattr(T, "_raw_stream", lambda device: seen.current)
    monkeypatch.setattr(T, "_grad_tensor", lambda t, what: T._type(t, what))
    monkeypatch.setattr(T, "_keep_for", lambda stream, *tensors: seen.kept.extend(
        (getattr(stream, "cuda_stream", stream), t.data_ptr()) for t in tensors))
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: seen.streams[seen.current])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: seen.capturing)
    monkeypatch.setattr(torch.cuda, "Event", lambda: types.SimpleNamespace(record=lambda *a: None))
    return seen


def prepared(kind):
    grads = [torch.ones(8), torch.ones(3)]
    return T.GradNorm(grads) if kind == "norm" else T.ClipGradNorm(grads, 1.0)


@pytest.mark.parametrize("kind", ["norm", "clip"])
def test_prepared_call_keeps_its_buffers_for_another_stream(cpu_calls, kind):
    """The object may be dropped right after a call on a stream that its
    buffers were not allocated on: both are recorded there, whether the stream
    is given or current."""
    call = prepared(kind)
    own = {call.result.data_ptr(), call._workspace.data_ptr()}
    call()
    assert cpu_calls.kept == [] and cpu_calls.calls[-1][-1] == 7   # its own stream
    for given in (cpu_calls.streams[9], 9):
        cpu_calls.kept.clear()
        call(given)
        assert cpu_calls.calls[-1][-1] == 9
        assert {t for s, t in cpu_calls.kept if s == 9} == own
    cpu_calls.kept.clear()
    cpu_calls.current = 9
    call()
    assert cpu_calls.calls[-1][-1] == 9
    assert {t for s, t in cpu_calls.kept if s == 9} == own


@pytest.mark.parametrize("kind", ["norm", "clip"])
def test_prepared_call_refuses_another_current_device(cpu_calls, kind):
    """Launches go to the current device: with another one than the buffers'
    nothing is called."""
    call = prepared(kind)
    cpu_calls.device = 1
    for stream in (None, cpu_calls.streams[9]):
        with pytest.raises(ValueError, match="current device"):
            call(stream)
    assert cpu_calls.calls == []
    cpu_calls.device = 0
    call()
    assert len(cpu_calls.calls) == 1


class FakeTensor:
    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


def test_handles_of_the_default_stream_are_recorded_as_that_stream(monkeypatch):
    """0 and 1 are the default stream's handles; a stream object made from
    handle 0 would be a new stream of its own."""
    made = []
    default = object()
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: default)
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device=None: made.append(handle) or ("external", handle))
    t, given = FakeTensor(), FakeStream(9)
    T._keep_for(0, t, None)
    T._keep_for(1, t)
    T._keep_for(64, t)
    T._keep_for(given, t)
    T._keep_for(None, t)
    assert t.streams == [default, default, ("external", 64), given] and made == [64]
