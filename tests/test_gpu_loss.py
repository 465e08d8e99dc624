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
    terms = 2 if dw_dtype == F32 else 1
    fine_dw = UNIT[x.dtype] ** terms * 1.01 + 2.0 ** -22
    tiny = (float(g.abs().max()) * 2.0 ** -13 if n else 0.0) * (2.0 ** -25 if x.dtype == H16 else 0.0)
    rest = p * g.abs() * (2.1 * off_lse[:, None] + 2.0 ** -20) + tiny
    err, err_dw = dz.abs() * fine + rest, dz.abs() * fine_dw + rest
    s = abs(scale)
    r["dx"] = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    r["dx"][kept] = scale * (dz @ wd)
    r["off_dx"] = torch.zeros_like(r["dx"])
    r["off_dx"][kept] = s * ((err + dz.abs() * ((V / 16 + 2) * 2.0 ** -22 + 80 * 2.0 ** -24)) @ wd.abs())
    r["dw"] = scale * (dz.t() @ xd)
    steps = (n / 16 + 2) * terms
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


@pytest.mark.parametrize("dtype", [H16, B16], ids=str)
def test_narrow_tiles_and_split_sums(dtype):
    """Few rows against many columns: tiles narrower than 256, dx in parts."""
    check(8, 512, 32000, dtype, d_value=64.0)
    check(130, 264, 30522, dtype, left_out=0.0)
    check(300, 1000, 9000, dtype, left_out=0.9, dw_dtype=F32)


@pytest.mark.parametrize("dw_dtype", [None, F32], ids=str)
def test_several_pieces_of_the_vocabulary(dw_dtype):
    """dz takes more than the half GB that a piece may: 4096 x 70000 (two pieces, or three for a binary32 dw),
    hidden sizes whose rows the products write and whose rows they do not."""
    check(4096, 64, 70000, B16, dw_dtype=dw_dtype, left_out=0.1)
    check(4096, 37, 70001, H16, dw_dtype=dw_dtype, left_out=0.5, d_value=256.0)


@pytest.mark.parametrize("pad", [1, 3, 8, 40])
@pytest.mark.parametrize("hidden", [64, 65])
def test_strides_and_starts(hidden, pad):
    check(290, hidden, 530, B16, pad=pad)
    x, w, targets = inputs(290, hidden + 9, 530, H16)
    for at in (0, 1, 8, 9):
        a, b = x[:, at:at + hidden], w[:, at:at + hidden]
        ce = Z.zero_linear_cross_entropy(a, b, targets)
        one = torch.ones((), device="cuda")
        got = Z.zero_linear_cross_entropy_backward(a, b, targets, ce, one)
        a, b = a.contiguous(), b.contiguous()
        same = Z.zero_linear_cross_entropy(a, b, targets)
        assert torch.equal(ce.losses, same.losses) and torch.equal(ce.lse, same.lse)
        for p, q in zip(got, Z.zero_linear_cross_entropy_backward(a, b, targets, same, one)):
            assert torch.equal(p, q)


def test_outputs_that_start_anywhere_and_only_what_is_wanted():
    for H in (64, 61):
        x, w, targets, ce, d, dx, dw = check(100, H, 300, B16)
        flat = torch.full((100 * H + 300 * H + 32,), 3.0, dtype=B16, device="cuda")
        for a in (1, 3, 8):
            out_x, out_w = flat[a:a + 100 * H].view(100, H), flat[100 * H + 16 + a:][:300 * H].view(300, H)
            got = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, dx=out_x, dw=out_w)
            assert got[0] is out_x and got[1] is out_w
            assert torch.equal(out_x, dx) and torch.equal(out_w, dw)
            assert bool((flat[:a] == 3).all()) and bool((flat[100 * H + a:100 * H + 16 + a] == 3).all())
            assert bool((flat[100 * H + 16 + a + 300 * H:] == 3).all())
            flat.fill_(3.0)
        only = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, want=("dx",))
        assert only[1] is None and torch.equal(only[0], dx)
        only = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, want=("dw",))
        assert only[0] is None and torch.equal(only[1], dw)


def test_int32_targets_shapes_and_own_workspace():
    x, w, targets = inputs(240, 72, 500, B16, ids=torch.int32)
    ws = torch.empty(Z.zero_linear_cross_entropy_workspace_bytes(x, w, targets) + 256, dtype=torch.uint8, device="cuda")
    a = Z.zero_linear_cross_entropy(x.view(4, 60, 72), w, targets.view(4, 60), workspace=ws)
    b = Z.zero_linear_cross_entropy(x, w, targets.long())
    assert a.losses.shape == (4, 60)
    assert torch.equal(a.losses.view(-1), b.losses) and torch.equal(a.total, b.total)
    n = Z.zero_linear_cross_entropy_workspace_bytes(x, w, targets, backward=True, dw_dtype=F32)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    one = torch.ones((), device="cuda")
    dx, dw = Z.zero_linear_cross_entropy_backward(x.view(4, 60, 72), w, targets.view(4, 60), a, one, dw_dtype=F32,
                                                  workspace=ws)
    assert dx.shape == (4, 60, 72) and dw.dtype == F32
    with pytest.raises(ValueError):
        Z.zero_linear_cross_entropy_backward(x, w, targets, b, one, dw_dtype=F32, workspace=ws[:n - 256])


def test_nothing_kept_and_no_tokens():
    x, w, targets = inputs(70, 40, 99, H16)
    for x, targets in ((x, torch.full_like(targets, -1)), (x[:0], targets[:0])):
        ce = Z.zero_linear_cross_entropy(x, w, targets)
        assert ce.total.tolist() == [0.0, 0.0, 0.0] and not bool(ce.losses.any()) and not bool(ce.lse.any())
        for reduction in ("mean", "sum", "none"):
            d = torch.ones(targets.shape if reduction == "none" else (), device="cuda")
            dx, dw = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, reduction=reduction)
            assert dx.shape == x.shape and not bool(dx.any()) and not bool(dw.any())


def test_nothing_of_left_out_rows_is_read():
    """NaN and infinities in the rows of left-out tokens, in what lies between
    rows and in the gradients of their losses stay where they are."""
    for H in (64, 63):
        x, w, targets, ce, d, dx, dw = check(300, H, 400, B16, reduction="none")
        gone = (targets < 0) | (targets >= 400)
        store = torch.full((300, H + 8), float("nan"), dtype=B16, device="cuda")
        store[:, :H] = x
        store[gone] = float("inf")
        d = torch.where(gone, torch.full_like(d, float("nan")), d)
        again = Z.zero_linear_cross_entropy(store[:, :H], w, targets)
        assert torch.equal(again.losses, ce.losses) and torch.equal(again.total, ce.total)
        got = Z.zero_linear_cross_entropy_backward(store[:, :H], w, targets, again, d, reduction="none")
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


def test_not_finite_rows_stay_in_their_losses():
    x, w, targets = inputs(40, 64, 300, H16, left_out=0.0)
    clean = Z.zero_linear_cross_entropy(x, w, targets)
    x = x.clone()
    x[7, 3] = float("nan")
    ce = Z.zero_linear_cross_entropy(x, w, targets)
    assert bool(ce.losses[7].isnan()) and bool(ce.total[:2].isnan().all())
    rest = torch.arange(40, device="cuda") != 7
    assert torch.equal(ce.losses[rest], clean.losses[rest])
    dx, dw = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, torch.ones((), device="cuda"))
    assert bool(dx[7].isnan().all()) and not bool(dx[rest].isnan().any()) and bool(dw.isnan().all())


@pytest.mark.parametrize("d_value", [0.0, 1e-30, 1e30, float("inf")])
def test_gradients_of_any_size(d_value):
    """The scale that dz is rounded with follows the gradient; 0 gives 0."""
    x, w, targets = inputs(50, 64, 200, B16, left_out=0.0)
    ce = Z.zero_linear_cross_entropy(x, w, targets)
    d = torch.full((), d_value, device="cuda")
    dx, dw = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, d, reduction="sum")
    if d_value == 0.0:
        assert not bool(dx.any()) and not bool(dw.any())
    elif math.isinf(d_value):
        assert not bool(dx.isfinite().any())
    else:
        ref = reference(x, w, targets, 1.0, d, "sum")
        near(dx, ref["dx"], ref["off_dx"], "dx")
        near(dw, ref["dw"], ref["off_dw"], "dw")


def test_same_bits_each_time():
    for T, H, V in ((1500, 128, 4000), (40, 2000, 30000)):
        x, w, targets = inputs(T, H, V, B16)
        one = torch.ones((), device="cuda")
        ce = Z.zero_linear_cross_entropy(x, w, targets)
        grads = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one)
        for _ in range(3):
            again = Z.zero_linear_cross_entropy(x, w, targets)
            assert torch.equal(again.losses, ce.losses) and torch.equal(again.total, ce.total)
            for p, q in zip(grads, Z.zero_linear_cross_entropy_backward(x, w, targets, again, one)):
                assert torch.equal(p, q)


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_autograd_and_differences(reduction):
    """The gradient along a direction against a difference of the 64-bit loss:
    the step's own error is h^2 / 6 times a third derivative (below 1 a token
    along a direction that changes logits by h at most), the kernel's the bounds
    of its gradients."""
    x, w, targets = inputs(120, 80, 300, B16)
    x, w = x.clone().requires_grad_(), w.clone().requires_grad_()
    out = Z.linear_cross_entropy(x, w, targets, scale=0.8, reduction=reduction)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    weight = torch.rand(out.shape, device="cuda", generator=g)
    (out * weight).sum().backward()
    vx, vw = torch.randn(120, 80, device="cuda", generator=g).double(), torch.randn(300, 80, device="cuda",
                                                                                      generator=g).double() / 9
    kept = ((targets >= 0) & (targets < 300))
    n = int(kept.sum())
    at = targets.clamp(0, 299)[:, None]

    def f(h):
        z = (x.detach().double() + h * vx) @ (w.detach().double() + h * vw).t() * 0.8
        losses = torch.where(kept, torch.logsumexp(z, 1) - z.gather(1, at)[:, 0], torch.zeros_like(z[:, 0]))
        if reduction == "none":
            return float((losses * weight).sum())
        return float(losses.sum() * weight / (n if reduction == "mean" else 1))
    h = 1e-4
    diff = (f(h) - f(-h)) / (2 * h)
    got = float((x.grad.double() * vx).sum() + (w.grad.double() * vw).sum())
    ref = reference(x.detach(), w.detach(), targets, 0.8, weight, reduction)
    unit = UNIT[B16]
    slack = float(((ref["off_dx"] + ref["dx"].abs() * unit) * vx.abs()).sum()
                  + ((ref["off_dw"] + ref["dw"].abs() * unit) * vw.abs()).sum())
    assert abs(diff - got) <= slack + 1e-5 * n


def test_autograd_of_one_input_and_of_expanded_gradients():
    x, w, targets = inputs(60, 64, 100, B16)
    for which in (0, 1):
        a = [x.clone(), w.clone()]
        a[which].requires_grad_()
        Z.linear_cross_entropy(*a, targets).backward()
        assert a[which].grad is not None and a[1 - which].grad is None
    a = x.clone().requires_grad_()
    Z.linear_cross_entropy(a, w, targets, reduction="none").sum().backward()   # an expanded gradient
    b = x.clone().requires_grad_()
    Z.linear_cross_entropy(b, w, targets, reduction="sum").backward()
    assert torch.equal(a.grad, b.grad)


def test_captured_and_replayed_beside_another_graph():
    """Two graphs with their own memory, replayed in turn on other inputs."""
    made = []
    for T, H, V in ((300, 128, 1000), (40, 72, 9000)):
        x, w, targets = inputs(T, H, V, B16)
        one = torch.ones((), device="cuda")
        ce = Z.zero_linear_cross_entropy(x, w, targets)
        Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ce = Z.zero_linear_cross_entropy(x, w, targets)
            grads = Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one)
        made.append((graph, x, w, targets, one, ce, grads))
    for seed in (1, 2):
        for graph, x, w, targets, one, ce, grads in made:
            T, H, V = x.shape[0], x.shape[1], w.shape[0]
            for to, new in zip((x, w, targets), inputs(T, H, V, B16, seed=seed, left_out=0.3 * seed)):
                to.copy_(new)
        for graph, *_ in made:
            graph.replay()
        for graph, x, w, targets, one, ce, grads in made:
            same = Z.zero_linear_cross_entropy(x, w, targets)
            assert torch.equal(ce.losses, same.losses) and torch.equal(ce.total, same.total)
            for p, q in zip(grads, Z.zero_linear_cross_entropy_backward(x, w, targets, same, one)):
                assert torch.equal(p, q)


def test_two_streams_at_once():
    cases = [inputs(700, 256, 5000, B16, seed=k) for k in range(2)]
    one = torch.ones((), device="cuda")
    want = []
    for x, w, targets in cases:
        ce = Z.zero_linear_cross_entropy(x, w, targets)
        want.append((ce.losses, *Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(5):
        for (x, w, targets), s, out in zip(cases, streams, got):
            ce = Z.zero_linear_cross_entropy(x, w, targets, stream=s)
            out.append((ce.losses, *Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one, stream=s)))
    torch.cuda.synchronize()
    for outs, ref in zip(got, want):
        for out in outs:
            assert all(torch.equal(p, q) for p, q in zip(out, ref))


def test_refusals_on_the_device():
    x, w, targets = inputs(10, 64, 100, B16)
    for bad in (lambda: Z.zero_linear_cross_entropy(x, w[:, :60], targets),
                lambda: Z.zero_linear_cross_entropy(x, w, targets[:9]),
                lambda: Z.zero_linear_cross_entropy(x.t(), w, targets),
                lambda: Z.zero_linear_cross_entropy(x, w, targets.cpu()),
                lambda: Z.zero_linear_cross_entropy(x, w[:, ::2], targets),
                lambda: Z.zero_linear_cross_entropy(x, w, targets[::2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: Z.zero_linear_cross_entropy(x.float(), w.float(), targets),
                lambda: Z.zero_linear_cross_entropy(x, w.half(), targets),
                lambda: Z.zero_linear_cross_entropy(x, w, targets.float())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(Z.ZeroError):
        Z.zero_linear_cross_entropy(x, w, targets, scale=0.0)
    ce = Z.zero_linear_cross_entropy(x, w, targets)
    one = torch.ones((), device="cuda")
    with pytest.raises(ValueError):
        Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one, reduction="none")
    with pytest.raises(ValueError):
        Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one, want=("dx",), dw=torch.empty_like(w))
    with pytest.raises(TypeError):
        Z.zero_linear_cross_entropy_backward(x, w, targets, ce, one, dw_dtype=H16)
