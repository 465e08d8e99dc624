"""The training-step operators on streams other than the current one: memory
that a call makes stays its own until that stream is done with it."""
import gc
import math

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z

pytestmark = pytest.mark.gpu

BUSY = 100_000_000   # cycles a stream is kept busy: some 50 ms


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
    torch.cuda.synchronize()
    for make in (lambda: Z.GradNorm(grads), lambda: Z.ClipGradNorm(grads, 1e9)):
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
            assert held[-1].data_ptr() != at
        side.synchronize()
        assert abs(float(norm) - want) <= 1e-5 * want
