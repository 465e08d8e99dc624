"""Gradients of every token's own loss: what one token's does to the others'.
Tolerances as in tests/test_gpu_loss.py; rows of dx by a reference of the row
alone."""
import gc

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z
from tests.test_gpu_loss import inputs, near, reference

pytestmark = pytest.mark.gpu

H16, B16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _cuda_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def gradients(x, w, targets, d, **how):
    ce = Z.zero_linear_cross_entropy(x, w, targets)
    return Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, reduction="none", **how)


@pytest.mark.parametrize("dtype", [H16, B16], ids=str)
@pytest.mark.parametrize("hidden", [64, 61])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")], ids=str)
def test_an_infinite_gradient_stays_in_its_row(dtype, hidden, value):
    x, w, targets = inputs(70, hidden, 300, dtype, left_out=0.1)
    targets[3] = 7
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    d = torch.rand(70, device="cuda", generator=g) + 0.5
    d[3] = d.min()
    want, _ = gradients(x, w, targets, d)
    d[3] = value
    dx, dw = gradients(x, w, targets, d)
    rest = torch.arange(70, device="cuda") != 3
    assert torch.equal(dx[rest], want[rest]) and bool(dx[rest].any())
    assert not bool(dx[3].isfinite().any()) and not bool(dw.isfinite().any())
    only = gradients(x, w, targets, d, want=("dx",))[0]
    assert torch.equal(only[rest], want[rest]) and not bool(only[3].isfinite().any())


@pytest.mark.parametrize("dtype", [H16, B16], ids=str)
def test_only_infinite_gradients(dtype):
    x, w, targets = inputs(9, 64, 300, dtype, left_out=0.0)
    dx, dw = gradients(x, w, targets, torch.full((9,), float("inf"), device="cuda"))
    assert not bool(dx.isfinite().any()) and not bool(dw.isfinite().any())
