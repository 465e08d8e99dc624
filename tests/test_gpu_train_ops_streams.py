"""The training-step operators on streams other than the current one: memory
that a call makes stays its own until that stream is done with it."""
import gc
import math

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z

pytestmark = pytest.mark.gpu

BUSY = 200_000_000   # cycles a stream is kept busy: some 100 ms


@pytest.fixture(autouse=True)
def _cuda_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.synchronize()
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(BUSY)


@pytest.mark.parametrize("given", [True, False])
def test_prepared_norm_dropped_right_after_its_call(given):
    """The workspace of an object that is gone is not handed out while the
    other stream still needs it."""
    grads = [torch.full((300_000,), 2.0, device="cuda"), torch.full((77,), 1.0, device="cuda")]
    want = math.sqrt(4 * 300_000 + 77)
    size = Z.zero_grad_norm_workspace_bytes(grads)
    side = torch.cuda.Stream()
    for make in (lambda: Z.GradNorm(grads), lambda: Z.ClipGradNorm(grads, 1e9)):
        make()(stream=side)   # the kernels' first use takes its time
        torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        call = make()
        at = call._workspace.data_ptr()
        busy(side)
        if given:
            norm = call(stream=side)
        else:
            with torch.cuda.stream(side):
                norm = call()
        del call
        held = []
        for _ in range(4):
            held.append(torch.full((size,), 255, dtype=torch.uint8, device="cuda"))
            assert held[-1].data_ptr() != at or side.query()
        side.synchronize()
        assert abs(float(norm) - want) <= 1e-5 * want


def small_join(rows=3000, hidden=1024):
    g = torch.Generator(device="cuda").manual_seed(3)
    x, b = (torch.randn(rows, hidden, device="cuda", generator=g).bfloat16() for _ in range(2))
    w = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
    return x, b, w


def test_gradients_of_an_unused_output_are_zero_on_the_given_stream():
    """While the current stream is busy, a consumer on the given stream sees
    the zeros of dw_pre and dbias_pre."""
    x, b, w = small_join()
    side = torch.cuda.Stream()
    how = dict(w_post=w, bias_post=w, w_pre=w, bias_pre=w, kind="layer")
    _, _, stats = Z.zero_block_join(x, b, want_stats=True, **how)
    d_o = torch.ones_like(x)
    torch.cuda.synchronize()
    for _ in range(3):
        dirty = torch.full((64, 1024), 5.0, device="cuda", dtype=torch.bfloat16)
        del dirty
        busy(torch.cuda.current_stream())
        g = Z.zero_block_join_backward(x, b, d_o, None, stats, stream=side, **how)
        with torch.cuda.stream(side):
            seen = g["dw_pre"].clone(), g["dbias_pre"].clone()
        side.synchronize()
        assert not seen[0].any() and not seen[1].any()
        torch.cuda.synchronize()


def test_calls_on_a_given_stream_leave_freed_memory_of_the_current_one_alone():
    """Memory freed on the current stream may still be read by its queued
    work; a call on another stream does not get it."""
    x, b, w = small_join()
    ids = torch.randint(0, 8, (3000, 2), device="cuda", dtype=torch.int32)
    weights = torch.rand(3000, 2, device="cuda")
    order = Z.zero_expert_sort(ids, 8)
    ys = Z.zero_expert_dispatch(x, order)
    _, _, stats = Z.zero_block_join(x, b, w_post=w, w_pre=w, want_stats=True)
    side = torch.cuda.Stream()
    grads = [torch.ones(100_000, device="cuda")]
    torch.cuda.synchronize()
    calls = [
        lambda: Z.zero_block_join(x, b, w_post=w, w_pre=w, want_stats=True, stream=side),
        lambda: Z.zero_block_join_backward(x, b, x, x, stats, w_post=w, w_pre=w, stream=side).values(),
        lambda: (Z.zero_expert_dispatch(x, order, stream=side),),
        lambda: (Z.zero_expert_dispatch_backward(ys, order, stream=side),),
        lambda: (Z.zero_expert_combine(ys, weights, order, stream=side),),
        lambda: Z.zero_expert_combine_backward(x, ys, weights, order, stream=side),
        lambda: vars(Z.zero_expert_sort(ids, 8, stream=side)).values(),
        lambda: (Z.zero_grad_norm(grads, stream=side),),
    ]
    for call in calls:
        plain = [t for t in call() if isinstance(t, torch.Tensor)]
        torch.cuda.synchronize()
        sizes = [(t.shape, t.dtype) for t in plain]
        want = [t.clone() for t in plain]
        del plain
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        freed = [torch.full(s, 3, dtype=d, device="cuda") for s, d in sizes]
        at = {t.untyped_storage().data_ptr() for t in freed}
        busy(torch.cuda.current_stream())
        del freed
        got = [t for t in call() if isinstance(t, torch.Tensor)]
        assert not at & {t.untyped_storage().data_ptr() for t in got}
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_results_of_a_given_stream_are_held_for_the_caller():
    """Dropped while the caller's stream still reads it, a result is not
    handed to the stream that made it."""
    x, b, w = small_join()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, _, _ = Z.zero_block_join(x, b, w_post=w, stream=side)
    at = o.data_ptr()
    torch.cuda.current_stream().wait_stream(side)
    busy(torch.cuda.current_stream())
    copy = o.clone()
    want_first = o[0].clone()
    del o
    for _ in range(3):
        again, _, _ = Z.zero_block_join(x, b, w_post=w, scale=9.0, stream=side)
        assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(copy[0], want_first)


def test_prepared_norm_on_another_stream_waits_for_its_memory():
    """The workspace takes over memory that queued work still reads: the call
    on another stream runs after it."""
    grads = [torch.full((300_000,), 2.0, device="cuda")]
    size = Z.zero_grad_norm_workspace_bytes(grads)
    side = torch.cuda.Stream()
    Z.GradNorm(grads)(stream=side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.full((size + 1024,), 3, dtype=torch.uint8, device="cuda")
    at = before.data_ptr()
    copy = torch.empty_like(before)
    torch.cuda.synchronize()
    busy(torch.cuda.current_stream())
    copy.copy_(before)
    del before
    call = Z.GradNorm(grads)
    assert at <= call._workspace.data_ptr() < at + 1024
    norm = call(stream=side)
    side.synchronize()
    assert abs(float(norm) - math.sqrt(4 * 300_000)) <= 1e-2
    assert bool((copy == 3).all())


def test_prepared_clip_captured_and_called_elsewhere():
    """One object: called, captured on the capture's stream, replayed, called
    on a third stream; and one prepared inside the capture."""
    g = [torch.full((5000,), 2.0, device="cuda")]
    call = Z.ClipGradNorm(g, 1.0)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        inside = Z.GradNorm(g)
        inside()
    g[0].fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(call._norm) - 3 * math.sqrt(5000)) <= 1e-3
    assert abs(float(inside._norm) - 1.0) <= 1e-4
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = inside(stream=side)
    side.synchronize()
    assert abs(float(norm) - 1.0) <= 1e-4
