"""A bounded wait that gave up never leaves results that look right: from the
device error word that one raised on purpose (on a barrier that nothing completes,
after a millisecond) until zero_sync reports it, the cross entropy's kernels take
their own flag as raised, and write NaN."""
import gc

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z
from tests.test_gpu_loss import inputs
from zero_sharded_optimizer_flatten_gb300.zero import ZERO_ERR_TIMEOUT

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


# sizes: few tokens (one launch less), many, rows that the products write and that they do not, split sums, pieces
CASES = [(40, 64, 300, B16, None), (40, 61, 300, H16, None), (1500, 128, 700, B16, F32), (8, 512, 9000, H16, F32),
         (1100, 61, 1003, B16, F32), (4096, 64, 70000, H16, None)]


def results(x, w, targets, dw_dtype, reduction, want, ce=None):
    ce = ce or Z.zero_linear_cross_entropy(x, w, targets)
    d = torch.ones(targets.shape if reduction == "none" else (), device="cuda")
    return ce, *Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, reduction=reduction, dw_dtype=dw_dtype,
                                                     want=want)


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("reduction", ["none", "mean"])
def test_nan_until_it_is_reported(case, reduction):
    T, H, V, dtype, dw_dtype = case
    x, w, targets = inputs(T, H, V, dtype, left_out=0.2)
    targets[0], targets[1] = 5, -1
    gone = (targets < 0) | (targets >= V)
    Z.zero_sync()
    clean = {want: results(x, w, targets, dw_dtype, reduction, want) for want in (("dx", "dw"), ("dx",), ("dw",))}
    fine = clean[("dx", "dw")][0]
    Z.zero_selftest_wait_timeout(1_000_000)
    for want in clean:
        for before in (None, fine):   # a forward call in the same state, and one from before
            ce, dx, dw = results(x, w, targets, dw_dtype, reduction, want, before)
            if before is None:
                for t in (ce.losses, ce.lse, ce.rest):
                    assert bool(t[~gone].isnan().all()) and not bool(t[gone].any())
                assert bool(ce.total[:2].isnan().all()) and float(ce.total[2]) == float((~gone).sum())
            if dx is not None:
                assert bool(dx[~gone].isnan().all()) and not bool(dx[gone].any())
            if dw is not None:
                assert bool(dw.isnan().all())
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_sync()
    assert e.value.status == ZERO_ERR_TIMEOUT
    for want, (ce, dx, dw) in clean.items():
        again, *grads = results(x, w, targets, dw_dtype, reduction, want)
        for a, b in zip((ce.losses, ce.lse, ce.rest, ce.total, dx, dw),
                        (again.losses, again.lse, again.rest, again.total, *grads)):
            assert (a is None and b is None) or torch.equal(a, b)
    Z.zero_sync()
