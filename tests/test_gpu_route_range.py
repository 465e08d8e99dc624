"""The router and its gradient on rows of scores of any size, against the
definition in 64 bits.

Tolerances.  They do not grow with the scores.  A difference z - top is rounded
once, its product with log2(e) twice (the constant as well): an exponent in base
2 is off by at most |z - top| 1.45 * 3 * 2^-24, and |z - top| is at most 104
where exp does not vanish in binary32.  ex2 is off by 2^-22 relative, a row's
sum of up to 1024 by 48 * 2^-24 and its reciprocal by 2^-23, so p and the
weights by REL = 104 * 4.4 * 2^-24 + 2^-18 < 2^-15 relative and 2^-126 absolutely
(ex2 flushes what is smaller).  lse is top and a logarithm below 7 (off by 2^-22 of itself),
rounded: 2^-23 of it and REL.  Sums of p over the tokens add (T / 4864 + 220) 2^-24, the
gradient's sums over the experts 4 REL of the terms' absolute sums.
"""
import gc
import math

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z

pytestmark = pytest.mark.gpu

H16, B16, F32 = torch.float16, torch.bfloat16, torch.float32
UNIT = {F32: 2.0 ** -24, H16: 2.0 ** -11, B16: 2.0 ** -8}
TINY = {F32: 2.0 ** -126, H16: 2.0 ** -25, B16: 2.0 ** -126}
REL = 2.0 ** -15


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
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{float(got[bad][0])} for {float(ref[bad][0])}")


def definition(z, K, normalize):
    """(chosen, kept, weights, balance, zloss, lse, p, counts, n) in 64 bits; z requires a gradient."""
    order = torch.sort(z.detach(), dim=1, descending=True, stable=True)
    chosen, kept = order.indices[:, :K], order.values[:, :K] > -math.inf
    there = kept[:, :1]
    top = torch.where(there, order.values[:, :1], torch.zeros_like(order.values[:, :1]))
    e = torch.exp(z - top)   # differences first: exact enough at any size in 64 bits
    total = torch.where(there, e.sum(1, keepdim=True), torch.ones_like(top))
    p = e / total
    lse = torch.where(there, top + total.log(), torch.zeros_like(top))[:, 0]
    # top is a constant above; d lse / dz is p all the same
    w = torch.where(kept, p.gather(1, chosen), torch.zeros_like(p[:, :1]))
    if normalize:
        w = torch.where(there, w / torch.where(there, w.sum(1, keepdim=True), torch.ones_like(top)), w)
    T, E = z.shape
    n = max(1, int(there.sum()))
    counts = torch.bincount(chosen[kept], minlength=E)
    return chosen, kept, w, (counts.double() * p.sum(0)).sum() * E / (K * n * n), lse.square().sum() / n, lse, p, counts, n


def rows(E, dtype, bases, seed=0):
    """Two rows for each size: all scores equal, and scores a few steps of the
    type below it; between them ordinary rows."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + E)
    z = []
    for base in bases:
        flat = torch.full((E,), base, device="cuda", dtype=torch.float64).to(dtype)
        near_it = (flat.double() - torch.rand(E, device="cuda", generator=g) * 9).to(dtype)
        z += [flat, near_it, torch.randn(E, device="cuda", generator=g).to(dtype)]
    return torch.stack(z)


SIZES = {F32: (-1e4, 1e4, -1e6, 1e6, -1e9, 1e9, -2e9, 3e9, -3e38, 3e38, torch.finfo(F32).min, torch.finfo(F32).max),
         B16: (-1e4, 1e4, -1e9, 1e9, -3e9, 3e9, -3e38, 3e38, torch.finfo(B16).min, torch.finfo(B16).max),
         H16: (-1e4, 1e4, torch.finfo(H16).min, torch.finfo(H16).max)}


@pytest.mark.parametrize("dtype", list(SIZES), ids=str)
@pytest.mark.parametrize("experts", [8, 17, 64, 256, 1000])
@pytest.mark.parametrize("normalize", [True, False])
def test_rows_of_any_size(experts, dtype, normalize):
    K = 3
    z = rows(experts, dtype, SIZES[dtype])
    T = z.shape[0]
    r = Z.zero_expert_route(z, K, normalize=normalize)
    chosen, kept, w, balance, zloss, lse, p, counts, n = definition(z.double(), K, normalize)
    assert torch.equal(r.ids, chosen.to(torch.int32)) and torch.equal(r.counts, counts.to(torch.int32))
    near(r.weights, w, w * 2 * REL, "weights")
    near(r.stats[:T], lse, lse.abs() * 2.0 ** -23 + REL, "lse")
    near(r.losses[:1], balance[None], balance[None] * (REL + (T / 4864 + 220) * 2.0 ** -24), "balance")
    if float(zloss) < 1e38:
        near(r.losses[1:], zloss[None], zloss[None] * 2.0 ** -16 + 2 * REL * lse.abs().mean(), "z loss")
    else:
        assert float(r.losses[1]) == math.inf   # as a binary32 number


@pytest.mark.parametrize("dtype", [B16, F32], ids=str)
def test_a_padded_token_under_a_mask_of_the_lowest_value(dtype):
    """The usual mask of a padded token leaves the others' losses alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    z = torch.randn(500, 64, device="cuda", generator=g).to(dtype)
    z[::5] = torch.finfo(dtype).min
    z[1::5, ::2] = torch.finfo(dtype).min   # and experts barred so
    r = Z.zero_expert_route(z, 4)
    assert bool(r.weights.isfinite().all()) and bool(r.losses[:1].isfinite().all())
    assert torch.equal(r.weights[::5], torch.full((100, 4), 0.25, device="cuda"))
    balance = definition(z.double(), 4, True)[3]
    near(r.losses[:1], balance[None], balance[None] * REL, "balance")


def gradient(z, K, normalize, dw, dl):
    """In 64 bits, with the size of its terms."""
    z64 = z.double().requires_grad_()
    chosen, kept, w, balance, zloss, lse, p, counts, n = definition(z64, K, normalize)
    loss = (w * dw.double()).sum() + dl[0].double() * balance + dl[1].double() * zloss
    grad, = torch.autograd.grad(loss, z64)
    grad = torch.nan_to_num(grad)
    with torch.no_grad():
        E = z.shape[1]
        load = counts.double() * E / (K * n * n) * abs(float(dl[0]))
        wd = w * dw.double().abs()
        direct = wd + w * wd.sum(1, keepdim=True) if normalize else wd
        size = p * (load + (p * load).sum(1, keepdim=True) + 2 / n * abs(float(dl[1])) * lse.abs()[:, None])
        if not normalize:
            size = size + p * wd.sum(1, keepdim=True)
        size = size.scatter_add(1, chosen, direct * kept)
    return grad, size


@pytest.mark.parametrize("dtype", list(SIZES), ids=str)
@pytest.mark.parametrize("experts", [8, 17, 64, 256, 1000])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_of_rows_of_any_size(experts, dtype, normalize):
    K = 3
    z = rows(experts, dtype, SIZES[dtype])
    g = torch.Generator(device="cuda")
    g.manual_seed(experts)
    dw = torch.randn(z.shape[0], K, device="cuda", generator=g)
    r = Z.zero_expert_route(z, K, normalize=normalize)
    for dl in (torch.tensor([7.0, 0.0], device="cuda"), torch.tensor([0.0, 0.0], device="cuda"),
               torch.tensor([7.0, 1e-3], device="cuda")):
        if float(dl[1]) and dtype == F32:
            continue   # lse as a factor: past binary32's end for the largest rows
        got = Z.zero_expert_route_backward(z, r, dw, dl)
        grad, size = gradient(z, K, normalize, dw, dl)
        near(got, grad, size * 4 * REL + 2.0 ** -44 * size.sum(1, keepdim=True), "d_logits")


def test_a_token_masked_with_a_large_value_gets_the_gradient_of_equal_choices():
    """Scores that are all -1e9: probabilities 1/8, so the gradient of the
    balance loss is that of any token with equal scores."""
    z = torch.zeros(6, 8, device="cuda")
    z[2:] = -1e9
    dl = torch.tensor([1.0, 0.0], device="cuda")
    d = Z.zero_expert_route_backward(z, Z.zero_expert_route(z, 2), None, dl)
    assert torch.equal(d[2:], d[:1].expand(4, 8)) and bool((d != 0).any())


@pytest.mark.parametrize("experts", [4, 40, 256])
@pytest.mark.parametrize("normalize", [True, False])
def test_the_same_experts_in_another_order_token_after_token(experts, normalize):
    """The same few experts are every token's choices, in turning order, so that
    one expert's place is cleared for a token and taken for the next by another
    thread; several tokens a warp."""
    T, K = 40_000, 4
    turn = (torch.arange(T, device="cuda")[:, None] // 9728 + torch.arange(K, device="cuda")) % K
    z = torch.full((T, experts), -9.0, device="cuda")
    z.scatter_(1, turn, torch.linspace(2.0, 0.5, K, device="cuda").expand(T, K).contiguous())
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    dw, dl = torch.randn(T, K, device="cuda", generator=g), torch.zeros(2, device="cuda")
    r = Z.zero_expert_route(z, K, normalize=normalize)
    assert torch.equal(r.ids, turn.to(torch.int32))
    got = Z.zero_expert_route_backward(z, r, dw, dl)
    grad, size = gradient(z, K, normalize, dw, dl)
    near(got, grad, size * 4 * REL + 2.0 ** -44 * size.sum(1, keepdim=True), "d_logits")
    for _ in range(3):
        assert torch.equal(got, Z.zero_expert_route_backward(z, r, dw, dl))


def test_lse_of_equal_scores():
    """The sum of E ones is exact, and so is 0 + log(E) but for the base-2
    logarithm's 2^-22 and its product with log(2), 2^-24 and 2^-25 for the
    constant."""
    for experts in range(1, 1025):
        if experts > 64 and experts % 37 and experts & (experts - 1):
            continue
        r = Z.zero_expert_route(torch.zeros(2, experts, device="cuda"), 1)
        want = math.log(experts)
        assert abs(float(r.stats[0].double()) - want) <= want * 1.376 * 2.0 ** -22, experts
