"""The linear softmax cross entropy and its gradients against 64-bit
implementations.

Tolerances.  u(T) is the half spacing of the type an output is rounded to.

* z: products of 16-bit numbers are exact in binary32; the tensor cores add 16
  of them and the sum so far at a time, cutting what falls below the largest
  one's last place: at most 2^-22 of the absolute sum a step, H/16 + 2 steps.
  dz = (H/16 + 2) 2^-22 scale sum |x||w| bounds it (the largest over a row).
* lse: the exponentials' exponents are off by dz and their own rounding, |z|
  2^-22; ex2 and the sums over 256 columns, the tiles and the threads are off by
  less than 400 * 2^-24 relative in all, which is absolute in the logarithm; a
  loss is off by that and dz twice.
* dx: dz is off by its rounding, u(type) relative (fp16: 2^-25 of its scale
  below the normal range, the scale being at most 2^14 / the largest gradient),
  and by p's relative error, twice that of lse.  Its products are added as
  above, over the vocabulary; split sums add at most 80 * 2^-24 more.  dw the
  same over the tokens; for a binary32 one dz is two numbers, off by u(type)^2.
"""
import gc
import math

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z

pytestmark = pytest.mark.gpu

H16, B16, F32 = torch.float16, torch.bfloat16, torch.float32
UNIT = {F32: 2.0 ** -24, H16: 2.0 ** -11, B16: 2.0 ** -8}
TINY = {F32: 2.0 ** -149, H16: 2.0 ** -25, B16: 2.0 ** -134}


@pytest.fixture(autouse=True)
def _cuda_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def inputs(T, H, V, dtype, seed=0, left_out=0.2, ids=torch.int64, pad=0):
    """x, w and targets; rows `pad` elements apart from one another."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + T * 977 + H * 31 + V)
    targets = torch.randint(0, V, (T,), device="cuda", generator=g)
    gone = torch.rand(T, device="cuda", generator=g) < left_out
    far = torch.tensor([-1, -100, V, V + 7], device="cuda")
    targets = torch.where(gone, far[targets % 4], targets).to(ids)
    w = torch.randn(V, H + pad, device="cuda", generator=g) * (1.5 / math.sqrt(H))
    x = torch.randn(T, H + pad, device="cuda", generator=g)
    return x.to(dtype)[:, :H], w.to(dtype)[:, :H], targets


def near(got, ref, slack, what):
    """|got - ref| <= slack + the rounding to got's type."""
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} for {tuple(ref.shape)}"
    if not got.numel():
        return
    g = got.double()
    bound = slack + ref.abs() * UNIT[got.dtype] * 1.001 + TINY[got.dtype]
    bad = ~((g - ref).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, "
                           f"worst {float((g - ref).abs()[bad].max())} against bound "
                           f"{float((bound + torch.zeros_like(g))[bad].min())}")


def reference(x, w, targets, scale, d=None, reduction="mean", dw_dtype=None):
    """Losses and gradients in 64 bits, with the bounds on what they are off by."""
    V, H = w.shape
    kept = ((targets >= 0) & (targets < V)).nonzero()[:, 0]
    T = targets.numel()
    xd, wd = x[kept].double(), w.double()
    at = targets[kept].long()[:, None]
    z = xd @ wd.t() * scale
    lse = torch.logsumexp(z, dim=1)
    step = abs(scale) * (H / 16 + 2) * 2.0 ** -22
    off = step * (xd.abs() @ wd.abs().t()).max(dim=1).values if kept.numel() else xd.new_zeros(0)
    off = off + (z.abs().max(dim=1).values * 2.0 ** -22 if kept.numel() else 0)
    off_lse = off + 400 * 2.0 ** -24
    zero = torch.zeros(T, dtype=torch.float64, device="cuda")
    r = {"losses": zero.clone(), "lse": zero.clone(), "off_lse": zero.clone(), "off_loss": zero.clone()}
    r["losses"][kept], r["lse"][kept] = lse - z.gather(1, at)[:, 0], lse
    r["off_lse"][kept], r["off_loss"][kept] = off_lse + lse.abs() * 2.0 ** -23, off_lse * 2 + lse.abs() * 2.0 ** -22
    n = kept.numel()
    r["total"] = torch.stack([r["losses"].sum() / max(1, n), r["losses"].sum(), zero.new_tensor(float(n))])
    slack = r["off_loss"].sum() + r["losses"].abs().sum() * 2.0 ** -20
    r["off_total"] = torch.stack([slack / max(1, n), slack, slack * 0])
    if d is None:
        return r
    g = d.double()
    g = g[kept] if reduction == "none" else (g / max(1, n) if reduction == "mean" else g).expand(n)
    g = g[:, None]
    p = torch.exp(z - lse[:, None])
    dz = p.clone()
    dz.scatter_add_(1, at, torch.full_like(lse[:, None], -1.0))
    dz = dz * g
    fine = UNIT[x.dtype] * 1.001 + 2.0 ** -22
    fine_dw = UNIT[x.dtype] ** 2 * 1.01 + 2.0 ** -22 if dw_dtype == F32 else fine
    tiny = (float(g.abs().max()) * 2.0 ** -13 if n else 0.0) * (2.0 ** -25 if x.dtype == H16 else 0.0)
    rest = p * g.abs() * (2.1 * off_lse[:, None] + 2.0 ** -20) + tiny
    err, err_dw = dz.abs() * fine + rest, dz.abs() * fine_dw + rest
    s = abs(scale)
    r["dx"] = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    r["dx"][kept] = scale * (dz @ wd)
    r["off_dx"] = torch.zeros_like(r["dx"])
    r["off_dx"][kept] = s * ((err + dz.abs() * ((V / 16 + 2) * 2.0 ** -22 + 80 * 2.0 ** -24)) @ wd.abs())
    r["dw"] = scale * (dz.t() @ xd)
    steps = (n / 16 + 2) * (2 if dw_dtype == F32 else 1)
    r["off_dw"] = s * ((err_dw + dz.abs() * steps * 2.0 ** -22).t() @ xd.abs())
    return r


def check(T, H, V, dtype, *, scale=1.0, reduction="mean", d_value=1.0, dw_dtype=None, **how):
    x, w, targets = inputs(T, H, V, dtype, **how)
    if reduction == "none":
        d = torch.rand(T, device="cuda") * d_value
    else:
        d = torch.full((), d_value, device="cuda")
    ce = Z.zero_linear_cross_entropy(x, w, targets, scale=scale)
    ref = reference(x, w, targets, scale, d, reduction, dw_dtype)
    near(ce.losses, ref["losses"], ref["off_loss"], "losses")
    near(ce.lse, ref["lse"], ref["off_lse"], "lse")
    near(ce.total, ref["total"], ref["off_total"], "total")
    dx, dw = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, reduction=reduction, scale=scale,
                                                  dw_dtype=dw_dtype)
    assert dw.dtype == (dw_dtype or dtype)
    near(dx, ref["dx"], ref["off_dx"], "dx")
    near(dw, ref["dw"], ref["off_dw"], "dw")
    return x, w, targets, ce, d, dx, dw


SIZES = [(1, 64, 256), (1, 1, 1), (3, 8, 5), (5, 16, 255), (128, 64, 512), (129, 72, 257), (256, 256, 256),
         (257, 264, 1000), (300, 513, 777), (700, 1001, 1003), (2, 4096, 2000), (40, 5120, 600),
         (1000, 520, 5003)]


@pytest.mark.parametrize("dtype", [H16, B16], ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_loss_and_gradients(size, dtype):
    check(*size, dtype, d_value=1024.0 if dtype == H16 else 1.0)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("dw_dtype", [None, F32], ids=str)
@pytest.mark.parametrize("scale", [1.0, -0.3, 2.5])
def test_reductions_types_and_scales(reduction, dw_dtype, scale):
    check(333, 136, 901, H16, scale=scale, reduction=reduction, d_value=64.0, dw_dtype=dw_dtype)
    check(70, 99, 301, B16, scale=scale, reduction=reduction, d_value=0.25, dw_dtype=dw_dtype)
