"""The cross entropy of tokens whose target stands far above the other scores:
small losses and their gradients, relative to themselves.

The scores are exact: every product and partial sum is a multiple of 1/16 below
2^12.  In base 2 they are rounded once, and their constant once (2^-23 of them
together), the difference of two and the logarithm of a sum are rounded after
that; a sum of exponentials is off by less than 400 * 2^-24 of itself.  All of it
is relative in the others' probability, which is what a small loss is:
REL = 2 * 1.45 * |z| 2^-23 + 400 * 2^-24 + 2^-20.

Gradients: dz is g (p - [target]) rounded to the inputs' type (fp16: or by 2^-25
of its scale, 2^14 / g), the others' p off by 2^-21 (|lse| + |z|) besides; products
and sums of dx over V and of dw over T columns as in the tests of the cross
entropy: (V/16 + 2) 2^-22 + 80 2^-24 of the sum of their sizes.
"""
import gc

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z

pytestmark = pytest.mark.gpu

H16, B16, F32 = torch.float16, torch.bfloat16, torch.float32
UNIT = {F32: 2.0 ** -24, H16: 2.0 ** -11, B16: 2.0 ** -8}
TINY = {F32: 2.0 ** -126, H16: 2.0 ** -25, B16: 2.0 ** -126}


@pytest.fixture(autouse=True)
def _cuda_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def near(got, ref, slack, what):
    bound = slack + ref.abs() * UNIT[got.dtype] * 1.001 + TINY[got.dtype]
    if got.dtype == H16:
        # 65504 is binary16's largest number and 32 half its step: from 65520 on nearest is infinity, of the same sign
        past = (ref.abs() >= 65520.0 + slack) & (got.double() == ref.sign() * float("inf"))
        got, ref = torch.where(past, torch.zeros_like(got), got), torch.where(past, torch.zeros_like(ref), ref)
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{float(got[bad][0])} for {float(ref[bad][0])}")


def confident(T, V, margins, dtype, lift=0.0, H=64):
    """x [T, H + T + 1], w, targets: the target's score is `margin` above what the
    first H channels make, and all scores `lift` above that."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + V)
    x = torch.zeros(T, H + T + 1, device="cuda")
    w = torch.zeros(V, H + T + 1, device="cuda")
    x[:, :H] = torch.randint(-1, 2, (T, H), device="cuda", generator=g).float()
    w[:, :H] = torch.randint(-3, 4, (V, H), device="cuda", generator=g).float() / 16
    targets = torch.randint(0, V, (T,), device="cuda", generator=g)
    at = torch.arange(T, device="cuda")
    x[at, H + at] = 1.0
    w[targets, H + at] = torch.tensor(margins, device="cuda").repeat(-(-T // len(margins)))[:T]
    x[:, H + T], w[:, H + T] = 1.0, lift
    return x.to(dtype), w.to(dtype), targets


def reference(x, w, targets):
    """(losses, lse, the others' probability, its relative bound), in 64 bits and without cancellation."""
    z = x.double() @ w.double().t()
    at = targets[:, None]
    zt = z.gather(1, at)
    others = z.scatter(1, at, -float("inf"))
    d = (torch.logsumexp(others, 1, keepdim=True) - zt)[:, 0]
    losses = torch.nn.functional.softplus(d, threshold=1e9)
    rel = 2 * 1.45 * z.abs().max(dim=1).values * 2.0 ** -23 + 400 * 2.0 ** -24 + 2.0 ** -20
    return losses, zt[:, 0] + losses, torch.sigmoid(d), rel


CASES = [(48, 1000, (20.0, 22.5, 25.0, 30.0, 34.25, 40.0), 0.0), (48, 1000, (10.0, 12.5, 15.0, 18.0), 20.0),
         (300, 5003, (8.0, 16.0, 24.0, 36.0), -30.0), (7, 2, (20.0, 40.0), 0.0), (5, 1, (3.0,), 0.0),
         (40, 30000, (-40.0, 5.0, 28.0), 10.0)]


@pytest.mark.parametrize("dtype", [H16, B16], ids=str)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_small_losses(case, dtype):
    T, V, margins, lift = case
    x, w, targets = confident(T, V, margins, dtype, lift)
    ce = Z.zero_linear_cross_entropy(x, w, targets)
    losses, lse, rest, rel = reference(x, w, targets)
    near(ce.losses, losses, losses * rel, "losses")
    near(ce.lse, lse, rel + lse.abs() * 2.0 ** -23, "lse")
    near(ce.total[1:2], losses.sum()[None], (losses * rel).sum() + losses.sum() * 2.0 ** -20, "total")


def test_small_losses_of_long_rows():
    """More than 2048 channels: z from several accumulators."""
    x, w, targets = confident(30, 700, (20.0, 30.0, 40.0), B16, 0.0, H=2500)
    ce = Z.zero_linear_cross_entropy(x, w, targets)
    losses, lse, rest, rel = reference(x, w, targets)
    near(ce.losses, losses, losses * rel, "losses")


def test_scores_that_are_not_finite():
    """An infinite score of the target, of another column, of all."""
    x = torch.zeros(4, 64, device="cuda", dtype=B16)
    w = torch.zeros(300, 64, device="cuda", dtype=B16)
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = 1.0, 1.0, 1.0, 1.0
    targets = torch.tensor([7, 8, 9, 10], device="cuda")
    w[7, 0] = float("inf")      # its target: inf - inf
    w[200, 1] = float("inf")    # another column
    w[9, 2] = float("-inf")     # its target: probability 0
    w = torch.where(w.isnan(), torch.zeros_like(w), w)
    ce = Z.zero_linear_cross_entropy(x, w, targets)
    # inf * 0 is NaN in the other rows' products with those channels
    assert not bool(ce.losses.isfinite()[:3].any()) and not bool(ce.total[:2].isfinite().any())


@pytest.mark.parametrize("dtype", [H16, B16], ids=str)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradients_of_confident_tokens(case, dtype):
    T, V, margins, lift = case
    x, w, targets = confident(T, V, margins, dtype, lift)
    ce = Z.zero_linear_cross_entropy(x, w, targets)
    losses, lse, rest, rel = reference(x, w, targets)
    near(ce.rest, rest, rest * rel, "rest")
    d = torch.full((), 2.0 ** 12, device="cuda")
    xd, wd = x.double(), w.double()
    z = xd @ wd.t()
    p = torch.exp(z - lse[:, None])
    dz = p.scatter(1, targets[:, None], -rest[:, None]) * float(d)
    off = dz.abs() * (UNIT[dtype] * 1.001 + 2.0 ** -20 + 2.0 ** -21 * (lse.abs() + z.abs().amax(1))[:, None])
    off = off + (float(d) * 2.0 ** -13 * 2.0 ** -25 if dtype == H16 else 0.0)
    refs = {"dx": dz @ wd, "dw": dz.t() @ xd}
    slack = {"dx": (off + dz.abs() * ((V / 16 + 2) * 2.0 ** -22 + 80 * 2.0 ** -24)) @ wd.abs(),
             "dw": (off + dz.abs() * ((T / 16 + 2) * 2.0 ** -22)).t() @ xd.abs()}
    dx, dw = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, reduction="sum")
    near(dx, refs["dx"], slack["dx"], "dx")
    near(dw, refs["dw"], slack["dw"], "dw")
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    (Z.linear_cross_entropy(a, b, targets, reduction="sum") * d).backward()
    assert torch.equal(a.grad, dx) and torch.equal(b.grad, dw)


def test_gradients_of_changed_losses_and_without_rest():
    """What a caller makes of the losses does not enter; without `rest` the
    gradient of ordinary tokens is the same but for roundings."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn(90, 64, device="cuda", generator=g).to(B16)
    w = (torch.randn(400, 64, device="cuda", generator=g) / 8).to(B16)
    targets = torch.randint(-1, 400, (90,), device="cuda", generator=g)
    ce = Z.zero_linear_cross_entropy(x, w, targets)
    one = torch.ones((), device="cuda")
    dx, dw = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one)
    assert bool((ce.rest[targets < 0] == 0).all())
    ce.losses.mul_(3.0)
    again = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    a = x.clone().requires_grad_()
    out = Z.linear_cross_entropy(a, w, targets, reduction="none")
    out.mul_(2.0)
    out.sum().backward()
    assert bool(a.grad.isfinite().all()) and bool(a.grad.any())
    ce.rest = None
    less = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one)
    # at most a rounding step of dz's largest entries apart
    assert float((less[0].double() - dx.double()).abs().max()) <= 2.0 ** -7 * float(dx.abs().max())
    assert float((less[1].double() - dw.double()).abs().max()) <= 2.0 ** -7 * float(dw.abs().max())
