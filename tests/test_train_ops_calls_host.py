"""Host side of the prepared norm calls and of calls on a given stream (no GPU
needed): the device, the streams and the library are stand-ins that record
what they are told."""
import contextlib
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
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: seen.streams[handle])
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


def order_of(tokens, topk, n_experts):
    i32 = dict(dtype=torch.int32)
    return T.ExpertOrder(torch.zeros(n_experts + 1, **i32), torch.zeros(tokens, topk, **i32),
                         torch.zeros(tokens * topk, **i32), n_experts, tokens, topk)


def test_calls_on_a_given_stream_make_their_buffers_there(monkeypatch):
    """Whatever a call allocates or fills, it does with the given stream
    current; what it returns is recorded for the caller's stream too."""
    class Made(FakeTensor):
        def __init__(self):
            super().__init__()
            self.made_on = current[-1]

    caller, side = FakeStream(7), FakeStream(9)
    current = [caller]

    class Use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *error):
            current.pop()

    def make(n):
        return lambda *a: tuple(Made() for _ in range(n)) if n > 1 else Made()

    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    fast = types.SimpleNamespace(
        block_join=make(3), block_join_backward=lambda *a: {"dx": Made(), "dw_pre": Made(), "db": None},
        block_join_workspace_bytes=lambda *a: 64, expert_sort=make(3), expert_dispatch=make(1),
        expert_dispatch_backward=make(1), expert_combine=make(1), expert_combine_backward=make(2))
    monkeypatch.setattr(T, "_fast", fast)
    x, ids, order = torch.ones(4, 8), torch.zeros(4, 2, dtype=torch.int32), order_of(4, 2, 3)

    def outputs(stream):
        sort = T.zero_expert_sort(ids, 3, stream=stream)
        grads = T.zero_block_join_backward(x, x, x, None, None, stream=stream)
        return [*T.zero_block_join(x, x, stream=stream), grads["dx"], grads["dw_pre"],
                sort.offsets, sort.rows, sort.pairs, T.zero_expert_dispatch(x, order, stream=stream),
                T.zero_expert_dispatch_backward(x, order, stream=stream),
                T.zero_expert_combine(x, x, order, stream=stream),
                *T.zero_expert_combine_backward(x, x, x, order, stream=stream)]

    for t in outputs(side):
        assert t.made_on is side and caller in t.streams
    for t in outputs(None):
        assert t.made_on is caller and t.streams == []
    assert current == [caller]


@pytest.mark.parametrize("kind", ["norm", "clip"])
def test_first_call_on_another_stream_waits_for_the_buffers(cpu_calls, kind, monkeypatch):
    """The memory of the buffers may have queued work of the stream it came
    from; another stream waits for that once, but not while it is captured
    (capture begins with the device idle, and may not wait on outside work)."""
    marks = []
    monkeypatch.setattr(torch.cuda, "Event", lambda: types.SimpleNamespace(
        record=lambda *a: marks.append(cpu_calls.current)))
    side = cpu_calls.streams[9]
    call = prepared(kind)
    assert marks == [7]
    call()
    assert not cpu_calls.streams[7].waited
    cpu_calls.capturing = True
    call(side)
    assert side.waited == []
    cpu_calls.capturing = False
    for _ in range(3):
        call(side)
    assert len(side.waited) == 1
    cpu_calls.current = 9
    call()
    assert len(side.waited) == 1 and not cpu_calls.streams[7].waited


def test_a_call_prepared_inside_a_capture_waits_for_nothing(cpu_calls):
    cpu_calls.capturing = True
    call = prepared("norm")
    cpu_calls.capturing = False
    call(cpu_calls.streams[9])
    assert cpu_calls.streams[9].waited == [] and cpu_calls.calls[-1][-1] == 9
