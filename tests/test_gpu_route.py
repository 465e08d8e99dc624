"""The experts' router and its gradient against 64-bit implementations.

Tolerances.  An exponent z - top (or z - lse) in base 2 is off by 2^-22 of the
row's largest magnitude; ex2 by 2^-22 relative; a row's sum by 48 * 2^-24: p and
the weights by REL = 2^-22 |z|max + 2^-21 + 2^-18 relative at most, lse by the
same absolutely.  The sums of p over the tokens add a strand of at most
T / 4864 + 32 + 152 + 32 values.  The gradient is a difference of products of
these with sums over the experts: 4 REL of the terms' absolute sums.
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


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def scores(T, E, dtype, seed=0, barred=0.0, padded=0.0, scale=1.0):
    g = gen(seed * 7919 + T * 31 + E)
    z = torch.randn(T, E, device="cuda", generator=g) * scale + torch.linspace(0, 1, E, device="cuda")
    z[torch.rand(T, E, device="cuda", generator=g) < barred] = -math.inf
    z[torch.rand(T, device="cuda", generator=g) < padded] = -math.inf
    return z.to(dtype)


def near(got, ref, slack, what):
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} for {tuple(ref.shape)}"
    g = got.double()
    bound = slack + ref.abs() * UNIT[got.dtype] * 1.001 + TINY[got.dtype]
    bad = ~((g - ref).abs() <= bound) & ~(g.isnan() & ref.isnan())
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{float(g[bad][0])} for {float(ref[bad][0])}")


def forward64(z, chosen, kept, K, normalize):
    """weights, balance, zloss, lse in 64 bits for the given choices."""
    there = (z > -math.inf).any(dim=1, keepdim=True)
    safe = torch.where(there, z, torch.zeros_like(z))
    lse = torch.where(there, torch.logsumexp(safe, 1, keepdim=True), torch.zeros_like(safe[:, :1]))
    p = torch.where(there, torch.exp(z - lse), torch.zeros_like(z))
    w = torch.where(kept, p.gather(1, chosen), torch.zeros((), dtype=z.dtype, device=z.device))
    if normalize:
        w = torch.where(there, w / torch.where(there, w.sum(1, keepdim=True), torch.ones_like(lse)), w)
    T, E = z.shape
    n = max(1, int(there.sum()))
    counts = torch.bincount(chosen[kept], minlength=E)
    balance = (counts.double() * p.sum(0)).sum() * E / (K * n * n)
    return w, balance, lse.square().sum() / n, lse[:, 0], p, counts, n


def reference(z, K):
    order = torch.sort(z.float(), dim=1, descending=True, stable=True)
    chosen, kept = order.indices[:, :K], order.values[:, :K] > -math.inf
    return chosen, kept


def rel_of(z):
    zf = z.double()
    most = torch.where(zf.isinf(), torch.zeros_like(zf), zf).abs().max(dim=1, keepdim=True).values
    return most * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -18


def check(z, K, normalize, d_weights=True, d_losses=True):
    T, E = z.shape
    r = Z.zero_expert_route(z, K, normalize=normalize)
    chosen, kept = reference(z, K)
    assert torch.equal(r.ids, torch.where(kept, chosen, torch.full_like(chosen, -1)).to(torch.int32))
    z64 = z.double().requires_grad_()
    w, balance, zloss, lse, p, counts, n = forward64(z64, chosen, kept, K, normalize)
    assert torch.equal(r.counts, counts.to(torch.int32))
    rel = rel_of(z)
    near(r.weights, w, w * rel * 2, "weights")
    near(r.stats[:T], lse, rel[:, 0] + lse.abs() * 2.0 ** -23, "lse")
    assert float(r.stats[T]) == float((z > -math.inf).any(dim=1).sum())
    strand = (T / 4864 + 220) * 2.0 ** -24
    worst = float(rel.max()) if T else 0.0
    near(r.losses, torch.stack([balance, zloss]),
         torch.stack([balance * (worst + strand + 2.0 ** -21),
                      zloss * (strand + 2.0 ** -21) + (2 * lse.abs() * rel[:, 0]).sum() / n + worst ** 2]), "losses")
    g = gen(E)
    dw = torch.randn(T, K, device="cuda", generator=g) if d_weights else None
    dl = torch.tensor([0.7, -0.2], device="cuda") * 10 if d_losses else None
    got = Z.zero_expert_route_backward(z, r, dw, dl)
    assert got.dtype == z.dtype
    loss = 0
    if d_weights:
        loss = loss + (w * dw.double()).sum()
    if d_losses:
        loss = loss + (balance * dl[0].double() + zloss * dl[1].double())
    grad, = torch.autograd.grad(loss, z64)
    grad = torch.nan_to_num(grad)
    with torch.no_grad():
        load = counts.double() * E / (K * n * n) * (abs(float(dl[0])) if d_losses else 0)
        size = p * (load + (p * load).sum(1, keepdim=True) + 2 / n * (abs(float(dl[1])) if d_losses else 0) * lse.abs()[:, None])
        if d_weights:
            wd = (w * dw.double().abs())
            size = size + p * (0 if normalize else wd.sum(1, keepdim=True))
            size = size.scatter_add(1, chosen, (wd + (w * wd.sum(1, keepdim=True) if normalize else 0)) * kept)
    # where terms cancel (normalised weights and an expert that was not chosen) the 64-bit reference has the
    # rounding of its own terms, below 2^-44 of the sum of all |gradients| in the row (1.6e-18 seen)
    near(got, grad, size * 4 * rel + 2.0 ** -44 * (size.sum(1, keepdim=True)), "d_logits")
    return r, got


@pytest.mark.parametrize("dtype", [H16, B16, F32], ids=str)
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 8, 2), (5, 2, 1), (7, 17, 3), (33, 31, 31), (64, 32, 32), (100, 33, 4),
                                   (999, 64, 6), (50, 100, 8), (300, 128, 8), (70, 200, 5), (513, 256, 8), (20, 257, 1),
                                   (40, 512, 8), (9, 700, 10), (12, 1024, 32), (6000, 8, 2)], ids=str)
@pytest.mark.parametrize("normalize", [True, False])
def test_route(shape, dtype, normalize):
    T, E, K = shape
    check(scores(T, E, dtype), K, normalize)
    check(scores(T, E, dtype, 1, barred=0.4, padded=0.2), K, normalize)


@pytest.mark.parametrize("have", [(True, False), (False, True)])
def test_one_gradient_alone(have):
    for normalize in (True, False):
        check(scores(200, 40, F32), 4, normalize, *have)


def test_ties_go_to_the_lowest_expert():
    for E in (3, 32, 64, 300, 1024):
        z = torch.zeros(40, E, device="cuda")
        z[::2] = -0.0  # equal to 0
        z[1, : E // 2] = -0.0
        K = min(E, 8)
        r = Z.zero_expert_route(z, K)
        assert r.ids.tolist() == [list(range(K))] * 40
        assert torch.equal(r.weights, torch.full((40, K), 1.0, device="cuda") / K)
        z = scores(500, E, F32).round()  # few different values
        check(z, K, True)


def test_every_token_left_out_and_no_tokens():
    z = torch.full((9, 20), -math.inf, device="cuda", dtype=B16)
    r, d = check(z, 3, True)
    assert bool((r.ids == -1).all()) and bool((r.weights == 0).all()) and r.losses.tolist() == [0.0, 0.0]
    assert bool((d == 0).all())
    r = Z.zero_expert_route(z[:0], 3)
    assert r.ids.shape == (0, 3) and r.counts.tolist() == [0] * 20 and r.losses.tolist() == [0.0, 0.0]
    assert Z.zero_expert_route_backward(z[:0], r, r.weights, r.losses).shape == (0, 20)


def test_fewer_experts_left_than_choices():
    z = torch.full((4, 50), -math.inf, device="cuda")
    z[:, 7], z[1, 3], z[2, 49] = 1.0, 5.0, -9.0
    r, _ = check(z, 4, True)
    assert r.ids.tolist() == [[7, -1, -1, -1], [3, 7, -1, -1], [7, 49, -1, -1], [7, -1, -1, -1]]


def test_nan_and_infinite_scores_stay_in_their_row():
    z = scores(6, 40, F32)
    clean = Z.zero_expert_route(z, 4)
    z[2, 5], z[4, 9] = math.nan, math.inf
    r = Z.zero_expert_route(z, 4)
    assert int(r.ids[2, 0]) == 5 and int(r.ids[4, 0]) == 9
    assert bool(r.weights[[2, 4]].isnan().any()) and bool(r.losses.isnan().all())
    rows = [0, 1, 3, 5]
    assert torch.equal(r.ids[rows], clean.ids[rows]) and torch.equal(r.weights[rows], clean.weights[rows])
    d = Z.zero_expert_route_backward(z, r, torch.ones(6, 4, device="cuda"))
    assert not bool(d[rows].isnan().any())


def test_large_scores_and_strides():
    check(scores(300, 48, F32, scale=30.0), 5, True)
    store = torch.randn(100, 300, device="cuda", generator=gen(0))
    for z in (store[:, :256], store[:, 1:257], store[::2, 4:68], store[:1, :256]):
        check(z, 8, False)


def test_same_bits_each_time_and_large_batches():
    for T, E, dtype in ((70_000, 64, B16), (30_000, 256, F32)):
        z = scores(T, E, dtype)
        a, da = check(z, 8, True)
        b, db = check(z, 8, True)
        assert torch.equal(a.losses, b.losses) and torch.equal(a.weights, b.weights) and torch.equal(da, db)


def test_autograd_and_differences():
    """The kernel's gradient against differences of the 64-bit function, away
    from borders between choices."""
    z = scores(50, 24, F32).requires_grad_()
    K, h = 3, 1e-5
    chosen, kept = reference(z.detach(), K)
    g = gen(9)
    dw = torch.randn(50, K, device="cuda", generator=g)
    for normalize in (True, False):
        ids, weights, counts, losses = Z.expert_route(z, K, normalize=normalize)
        assert not ids.requires_grad and not counts.requires_grad
        loss = (weights * dw).sum() + 3.0 * losses[0] + 0.1 * losses[1]
        grad, = torch.autograd.grad(loss, z)
        v = torch.randn(50, 24, device="cuda", generator=g).double()

        def f(t):
            w, balance, zloss, *_ = forward64(t, chosen, kept, K, normalize)
            return float((w * dw.double()).sum() + 3.0 * balance + 0.1 * zloss)
        base = z.detach().double()
        diff = (f(base + h * v) - f(base - h * v)) / (2 * h)
        # h^2 times third derivatives (below 10 |v|^3 a term), 64-bit noise 1e-15 / h, and the kernel's own 1e-5
        size = float((grad.double().abs() * v.abs()).sum())
        assert abs(diff - float((grad.double() * v).sum())) <= 1e-5 * size + 1e-6
    ids, weights, counts, losses = Z.expert_route(z, K)
    grad, = torch.autograd.grad(losses[0], z)  # the weights take no part
    r = Z.zero_expert_route(z.detach(), K)
    assert torch.equal(grad, Z.zero_expert_route_backward(z.detach(), r, None, torch.tensor([1.0, 0.0], device="cuda")))


def test_captured_and_replayed():
    z = scores(300, 64, F32)
    dw, dl = torch.ones(300, 4, device="cuda"), torch.ones(2, device="cuda")
    r = Z.zero_expert_route(z, 4)
    Z.zero_expert_route_backward(z, r, dw, dl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = Z.zero_expert_route(z, 4)
        d = Z.zero_expert_route_backward(z, r, dw, dl)
    for seed in range(3):
        z.copy_(scores(300, 64, F32, seed, barred=0.3, padded=0.1))
        graph.replay()
        e = Z.zero_expert_route(z, 4)
        for k in ("ids", "weights", "counts", "losses", "stats"):
            assert torch.equal(getattr(r, k), getattr(e, k)), k
        assert torch.equal(d, Z.zero_expert_route_backward(z, e, dw, dl))


def test_route_sort_and_combine_together():
    """The router's ids and weights through the sort, dispatch and combine."""
    z = scores(200, 16, F32, padded=0.1)
    r = Z.zero_expert_route(z, 2)
    order = Z.zero_expert_sort(r.ids, 16)
    assert torch.equal(order.offsets[1:] - order.offsets[:-1], r.counts)
    x = torch.randn(200, 64, device="cuda", generator=gen(1))
    y = Z.zero_expert_combine(Z.zero_expert_dispatch(x, order), r.weights, order)
    kept = (r.ids[:, :1] >= 0).double()
    near(y, x.double() * kept, x.double().abs() * 2.0 ** -21, "y")
