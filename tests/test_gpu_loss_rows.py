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


def check_rows(x, w, targets, d, dx, dw, dw_dtype=None, scale=1.0):
    """dx row by row, each with what its own gradient is rounded with."""
    V, H = w.shape
    flat, at = dx.reshape(-1, H).double(), targets.reshape(-1)
    for t in range(at.numel()):
        ref = reference(x[t:t + 1], w, at[t:t + 1], scale, d[t:t + 1], "none")
        past = (ref["dx"].abs() >= 65520.0 + ref["off_dx"]) & (flat[t:t + 1] == ref["dx"].sign() * float("inf"))
        got, want = dx[t:t + 1].clone(), ref["dx"].clone()   # past binary16's largest number: infinity
        if dx.dtype == H16:
            got[past], want[past] = 0.0, 0.0
        near(got, want, ref["off_dx"], f"dx of token {t}")
    if dw is not None:
        ref = reference(x, w, targets, scale, d, "none", dw_dtype)
        near(dw, ref["dw"], ref["off_dw"], "dw")


@pytest.mark.parametrize("dtype", [H16, B16], ids=str)
@pytest.mark.parametrize("shape", [(90, 64, 700), (41, 61, 300), (300, 72, 1003), (20, 512, 9000)], ids=str)
@pytest.mark.parametrize("dw_dtype", [None, F32], ids=str)
def test_gradients_of_very_different_tokens(shape, dtype, dw_dtype):
    """From 2^10 down to 2^-20, and one of 2^40 that passes fp16's end by itself."""
    T, H, V = shape
    x, w, targets = inputs(T, H, V, dtype, left_out=0.1)
    d = 2.0 ** torch.linspace(10.0, -20.0, T, device="cuda")
    dx, dw = gradients(x, w, targets, d, dw_dtype=dw_dtype)
    check_rows(x, w, targets, d, dx, dw, dw_dtype)
    only = gradients(x, w, targets, d, want=("dx",))[0]
    assert torch.equal(only, dx)
    only = gradients(x, w, targets, d, want=("dw",), dw_dtype=dw_dtype)[1]
    assert torch.equal(only, dw)
    d[2] = 2.0 ** 40
    dx, _ = gradients(x, w, targets, d, dw_dtype=dw_dtype)
    check_rows(x, w, targets, d, dx, None)


def test_own_scales_in_several_pieces_of_the_vocabulary():
    """4096 tokens twice over in fp16: three pieces of 32768 columns and less."""
    x, w, targets = inputs(4096, 64, 70000, H16, left_out=0.1)
    d = 2.0 ** torch.linspace(10.0, -20.0, 4096, device="cuda")
    for dw_dtype in (None, F32):
        dx, dw = gradients(x, w, targets, d, dw_dtype=dw_dtype)
        few = torch.arange(0, 4096, 137, device="cuda")
        check_rows(x[few], w, targets[few], d[few], dx[few], None)
        ref = reference(x, w, targets, 1.0, d, "none", dw_dtype)
        near(dw, ref["dw"], ref["off_dw"], "dw")


def test_workspace_is_enough_for_every_reduction():
    x, w, targets = inputs(50, 64, 3000, H16)
    n = Z.zero_linear_cross_entropy_workspace_bytes(x, w, targets, backward=True)
    guard = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
    ce = Z.zero_linear_cross_entropy(x, w, targets)
    for reduction in ("none", "sum", "mean"):
        d = torch.ones(50 if reduction == "none" else (), device="cuda")
        got = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, reduction=reduction, workspace=guard[:n])
        assert bool((guard[n:] == 77).all())
        for p, q in zip(got, Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, reduction=reduction)):
            assert torch.equal(p, q)
