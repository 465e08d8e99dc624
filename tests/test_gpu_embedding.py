"""The token embedding and its table's gradient against 64-bit implementations.

Tolerances.  u(T) is the half spacing of the type an output is rounded to.  y is
one binary32 product (2^-24, and 2^-24 for the factor's own rounding) before
that.  A row of the gradient adds a chunk of 8 to 32 rows one by one, then the
chunks' sums: a quarter of them one by one, then four: at most
50 + c / 32 additions of 2^-24 of the absolute sum for an id of c tokens, and
two roundings for the factor.
"""
import gc

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


def near(got, ref, slack, what):
    """|got - ref| <= slack + the rounding to got's type, NaN meets NaN."""
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} for {tuple(ref.shape)}"
    g = got.double()
    bound = slack + ref.abs() * UNIT[got.dtype] * 1.001 + TINY[got.dtype]
    bad = ~((g - ref).abs() <= bound) & ~(g.isnan() & ref.isnan())
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def ids_of(kind, T, V, g):
    if kind == "texts":  # the k-th id about 1/k as often as the first
        u = torch.rand(T, device="cuda", generator=g, dtype=torch.float64)
        return ((V + 1.0) ** u - 1).long().clamp_(0, V - 1)
    if kind == "one":
        return torch.full((T,), V // 2, dtype=torch.int64, device="cuda")
    if kind == "none":
        return torch.tensor([-1, V, -2 ** 40, 2 ** 40], device="cuda")[torch.arange(T, device="cuda") % 4]
    ids = torch.randint(0, V, (T,), device="cuda", generator=g)
    far = torch.tensor([-1, -100, V, 2 ** 40 + 1], device="cuda")
    gone = torch.rand(T, device="cuda", generator=g) < 0.3
    return torch.where(gone, far[ids % 4], ids)


def exact_rows(ids, table, scale):
    kept = (ids >= 0) & (ids < table.shape[0])
    y = torch.zeros(*ids.shape, table.shape[1], dtype=torch.float64, device="cuda")
    y[kept] = table.double()[ids[kept].long()] * scale
    return y


def exact_gradient(dy, ids, V, scale, base=None):
    """The gradient and its slack."""
    H = dy.shape[-1]
    kept = (ids >= 0) & (ids < V)
    at, d = ids[kept].long(), dy.double()[kept]
    out = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, at, d) * scale
    size = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, at, d.abs()) * abs(scale)
    count = torch.bincount(at, minlength=V).double()[:, None]
    slack = size * (52 + count / 32) * 2.0 ** -24
    if base is not None:
        out = out + base.double()
        slack = slack + (out.abs() + base.double().abs()) * 2.0 ** -24
    return out, slack


PAIRS = [(H16, H16), (H16, F32), (B16, B16), (B16, F32), (F32, F32)]
BACK = PAIRS + [(F32, H16), (F32, B16)]


@pytest.mark.parametrize("types", PAIRS, ids=str)
@pytest.mark.parametrize("hidden", [1, 7, 8, 64, 129, 768, 1001, 4096, 8200])
def test_lookup(hidden, types):
    g = gen(hidden)
    table = torch.randn(517, hidden, device="cuda", generator=g).to(types[0])
    for T in (1, 3, 1000):
        ids = ids_of("some", T, 517, g)
        for scale in (1.0, 0.3, -27.0):
            y = Z.zero_embedding(ids, table, scale=scale, dtype=types[1])
            ref = exact_rows(ids, table, scale)
            assert y.dtype == types[1]
            near(y, ref, ref.abs() * 2.0 ** -23, "y")
    assert torch.equal(Z.zero_embedding(ids.clamp(0, 516).to(torch.int32), table), table[ids.clamp(0, 516)])


def test_lookup_shapes_strides_and_outputs():
    g = gen(1)
    store = torch.randn(100, 80, device="cuda", generator=g).to(B16)
    ids = torch.randint(-1, 100, (3, 5, 7), device="cuda", generator=g)
    for table in (store[:, :64], store[:, 3:20], store[::2, 8:72], store[:1, :9], store[5:5 + 3]):
        y = Z.zero_embedding(ids % table.shape[0], table)
        assert y.shape == (3, 5, 7, table.shape[1])
        assert torch.equal(y, table[ids % table.shape[0]])
    out = torch.full((3, 5, 7, 64), 9.0, dtype=B16, device="cuda")
    assert Z.zero_embedding(ids, store[:, :64], out=out) is out
    near(out, exact_rows(ids, store[:, :64], 1.0), 0, "out")
    shifted = torch.empty(3 * 5 * 7 * 64 + 1, dtype=B16, device="cuda")[1:].view(3, 5, 7, 64)
    Z.zero_embedding(ids, store[:, :64], out=shifted)
    assert torch.equal(shifted, out)
    assert Z.zero_embedding(ids[:0], store).shape == (0, 5, 7, 80)
    inf = torch.full((4, 8), float("inf"), dtype=H16, device="cuda")
    assert bool((Z.zero_embedding(torch.tensor([-1, 4], device="cuda"), inf) == 0).all())


@pytest.mark.parametrize("types", BACK, ids=str)
@pytest.mark.parametrize("hidden", [1, 7, 8, 64, 129, 768, 1001, 4096])
@pytest.mark.parametrize("kind", ["some", "texts", "one", "none"])
def test_gradient(kind, hidden, types):
    g = gen(hidden)
    for T, V in ((1, 1), (31, 40), (32, 3), (33, 1000), (64, 5), (1000, 129), (4099, 30522)):
        if V * hidden > 1 << 25:
            V = 257
        dy = torch.randn(T, hidden, device="cuda", generator=g).to(types[0])
        ids = ids_of(kind, T, V, g)
        for scale in (1.0, -0.37):
            got = Z.zero_embedding_backward(dy, ids, V, scale=scale, dtype=types[1])
            assert got.dtype == types[1]
            near(got, *exact_gradient(dy, ids, V, scale), f"T {T} V {V} scale {scale}")
        base = torch.randn(V, hidden, device="cuda", generator=g).to(types[1])
        out = base.clone()
        assert Z.zero_embedding_backward(dy, ids.to(torch.int32), V, scale=0.5, out=out, accumulate=True) is out
        ids32 = ids.to(torch.int32)
        near(out, *exact_gradient(dy, ids32, V, 0.5, base), f"accumulate T {T} V {V}")
        untouched = torch.ones(V, dtype=torch.bool, device="cuda")
        untouched[ids32[(ids32 >= 0) & (ids32 < V)].long()] = False
        assert torch.equal(out[untouched], base[untouched])


@pytest.mark.parametrize("T,V,hidden", [(40_000, 131_072, 16), (70_001, 32_000, 8), (3000, 1 << 22, 2),
                                        (20_000, 500, 520)])
@pytest.mark.parametrize("kind", ["some", "texts", "one"])
def test_gradient_of_many_tokens_and_ids(T, V, hidden, kind):
    g = gen(T)
    dy = torch.randn(T, hidden, device="cuda", generator=g)
    ids = ids_of(kind, T, V, g)
    got = Z.zero_embedding_backward(dy, ids, V)
    near(got, *exact_gradient(dy, ids, V, 1.0), kind)
    assert torch.equal(got, Z.zero_embedding_backward(dy, ids, V))  # the same bits


def test_gradient_strides_and_offsets():
    g = gen(3)
    store = torch.randn(300, 100, device="cuda", generator=g).to(H16)
    ids = ids_of("some", 300, 70, g)
    for dy in (store[:, :64], store[:, 5:70], store[:, 8:72]):
        got = Z.zero_embedding_backward(dy, ids, 70)
        near(got, *exact_gradient(dy, ids, 70, 1.0), "strided")
        flat = torch.full((70 * dy.shape[1] + 9,), 5.0, dtype=H16, device="cuda")
        for at in (1, 4, 8):
            out = flat[at:at + got.numel()].view(got.shape)
            Z.zero_embedding_backward(dy, ids, 70, out=out)
            assert torch.equal(out, got)
            assert bool((flat[:at] == 5).all()) and bool((flat[at + got.numel():] == 5).all())
            flat.fill_(5.0)
    one = Z.zero_embedding_backward(store[:1].expand(1, 100), ids[:1], 70)
    near(one, *exact_gradient(store[:1], ids[:1], 70, 1.0), "one token")


def test_nothing_of_left_out_rows_is_read():
    ids = torch.tensor([0, -1, 1, 99, 0, -5], device="cuda")
    dy = torch.ones(6, 24, device="cuda")
    dy[[1, 3, 5]] = float("nan")
    got = Z.zero_embedding_backward(dy, ids, 3)
    assert got[:, 0].tolist() == [2.0, 1.0, 0.0] and not bool(got.isnan().any())
    dy[0] = float("inf")
    assert Z.zero_embedding_backward(dy, ids, 3)[:, 0].tolist() == [float("inf"), 1.0, 0.0]


def test_autograd_and_differences():
    g = gen(5)
    ids = ids_of("some", 60, 20, g).view(3, 20)
    table = torch.randn(20, 40, device="cuda", generator=g).requires_grad_()
    d = torch.randn(3, 20, 40, device="cuda", generator=g)
    y = Z.embedding(ids, table, scale=3.0)
    (y * d).sum().backward()
    v = torch.randn(20, 40, device="cuda", generator=g)

    def loss(t):
        return float((exact_rows(ids, t, 3.0) * d.double()).sum())
    # linear in the table: the difference is the derivative up to binary32's part in the gradient
    base = table.detach().double()
    diff = (loss(base + v.double()) - loss(base - v.double())) / 2
    slack = exact_gradient(d, ids, 20, 3.0)[1] + table.grad.double().abs() * 2.0 ** -23
    assert abs(diff - float((table.grad.double() * v.double()).sum())) <= float((slack * v.abs()).sum()) + 1e-9
    # a broadcast gradient, and a 16-bit table onto a binary32 stream
    half = table.detach().to(B16).requires_grad_()
    y = Z.embedding(ids, half, dtype=F32)
    assert y.dtype == F32
    y.sum().backward()
    near(half.grad, *exact_gradient(torch.ones(3, 20, 40, device="cuda"), ids, 20, 1.0), "broadcast")


def test_captured_and_replayed_with_other_ids():
    g = gen(6)
    table = torch.randn(500, 64, device="cuda", generator=g).to(H16)
    ids = ids_of("some", 333, 500, g)
    dy = torch.randn(333, 64, device="cuda", generator=g).to(H16)
    Z.zero_embedding(ids, table)
    Z.zero_embedding_backward(dy, ids, 500)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = Z.zero_embedding(ids, table)
        d = Z.zero_embedding_backward(dy, ids, 500)
    for kind in ("texts", "one", "none", "some"):
        ids.copy_(ids_of(kind, 333, 500, g))
        dy.normal_(generator=g)
        graph.replay()
        near(y, exact_rows(ids, table, 1.0), 0, kind)
        near(d, *exact_gradient(dy, ids, 500, 1.0), kind)


def test_calls_on_a_given_stream():
    g = gen(7)
    table = torch.randn(500, 64, device="cuda", generator=g).to(H16)
    ids = ids_of("texts", 2000, 500, g)
    dy = torch.randn(2000, 64, device="cuda", generator=g).to(H16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = Z.zero_embedding(ids, table, stream=side)
    d = Z.zero_embedding_backward(dy, ids, 500, stream=side.cuda_stream)
    side.synchronize()
    near(y, exact_rows(ids, table, 1.0), 0, "y")
    near(d, *exact_gradient(dy, ids, 500, 1.0), "dtable")
