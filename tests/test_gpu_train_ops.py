"""The training-step operators against plain 64-bit implementations.

Tolerances.  u(T) is the half spacing of the type an output is rounded to
(2^-24, 2^-11, 2^-8 relative; 2^-25 absolute below fp16's normal range).  All
arithmetic before that rounding is binary32 (2^-24 an operation):

* norm: at most 72 squares are added in binary32 before they join a sum held
  as two binary32 numbers, so the sum is off by at most 74 * 2^-24 = 4.4e-6 relative and the norm
  by half of it, 2.3e-6 with its own rounding.
* join: a row sum of H terms is a strand of at most H/32 + 40 additions; for
  the H used here (at most 8200) that is 300 * 2^-24 = 1.8e-5 of the terms'
  absolute sum in the worst case, and the sums' errors add up in the square
  root of the strand for rounding that is not all one way.  E = 2e-5 of the
  row's largest magnitude bounds both; gradients pass through two such sums
  and the statistics: 3 E.  Column sums over rows: 3 E of the sum of absolute
  terms.
* experts: topk <= 8 products and sums: (8 + 2) * 2^-24 of the absolute sum;
  a dot over H: as the join's row sums, of the terms' absolute sum.
"""
import gc
import math

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z

pytestmark = pytest.mark.gpu

H16, B16, F32 = torch.float16, torch.bfloat16, torch.float32
UNIT = {F32: 2.0 ** -24, H16: 2.0 ** -11, B16: 2.0 ** -8}
TINY = {F32: 2.0 ** -149, H16: 2.0 ** -25, B16: 2.0 ** -134}
NORM_TOL = 2.3e-6
E = 2e-5


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


def close(got, ref, slack, what):
    """|got - ref| <= slack + the rounding to got's type, NaN meets NaN."""
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} for {tuple(ref.shape)}"
    if not got.numel():
        return
    g, r = got.double(), ref.double()
    assert torch.equal(torch.isnan(g), torch.isnan(r)), f"{what}: NaN positions"
    bound = slack + r.abs() * UNIT[got.dtype] * 1.001 + TINY[got.dtype]
    bad = ((g - r).abs() > bound) & ~torch.isnan(r)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((g - r).abs()[bad].max())} against "
                           f"{float(r.abs()[bad].max())}")


# ---------------------------------------------------------------------------
# gradient norm and clipping


def exact_norm(grads, kind="l2"):
    if kind == "inf":
        return max([float(g.double().abs().max()) for g in grads if g.numel()], default=0.0)
    return math.sqrt(sum(float(g.double().pow(2).sum()) for g in grads))


def grads_of(sizes, dtypes, seed, scale=1e-2):
    g = gen(seed)
    return [(torch.randn(n, device="cuda", generator=g) * scale).to(dt)
            for n, dt in zip(sizes, dtypes)]


SIZES = [
    [1], [7], [8], [4095], [4096], [4097], [12289], [0, 5, 0], [1, 2, 3, 4, 5, 6, 7, 8, 9],
    [100_003, 17, 65536, 1, 4096 * 5 + 3],
]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("dtype", [H16, B16, F32])
@pytest.mark.parametrize("kind", ["l2", "inf"])
def test_norm(sizes, dtype, kind):
    grads = grads_of(sizes, [dtype] * len(sizes), sum(sizes) + len(sizes))
    norm = float(Z.zero_grad_norm(grads, kind))
    ref = exact_norm(grads, kind)
    assert abs(norm - ref) <= (0 if kind == "inf" else NORM_TOL) * ref


@pytest.mark.parametrize("src", [H16, B16, F32])
@pytest.mark.parametrize("dst", [H16, B16, F32])
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
def test_clip_into_views_at_any_offset(src, dst, offset):
    """Sources and destinations that start anywhere, of any pair of types."""
    sizes = [5, 4096, 8191, 3, 20000, 1, 12288]
    g = gen(offset)
    store = (torch.randn(sum(sizes) + 64, device="cuda", generator=g) * 0.1).to(src)
    flat = torch.full((sum(sizes) + 64,), 7.0, dtype=dst, device="cuda")
    grads, out, at = [], [], 0
    for k, n in enumerate(sizes):
        grads.append(store[at + (offset * k) % 9:][:n].clone() if k % 2 else store[at + offset:at + offset + n])
        out.append(flat[at + offset:at + offset + n])
        at += n
    for max_norm in (1e9, 1.5, 0.0):
        norm = float(Z.zero_clip_grad_norm(grads, max_norm, out=out))
        ref = exact_norm(grads)
        assert abs(norm - ref) <= NORM_TOL * ref
        factor = min(1.0, max_norm / (ref + 1e-6))
        for k, (a, b) in enumerate(zip(grads, out)):
            want = a.double() * factor
            close(b, want, want.abs() * (NORM_TOL + 2.0 ** -23), f"tensor {k}")
    assert bool((flat[:offset] == 7).all()) and bool((flat[at + offset:] == 7).all())


@pytest.mark.parametrize("kind", ["l2", "inf"])
@pytest.mark.parametrize("n", [63, 65, 257, 1000, 1001, 2500])
def test_clip_many_tensors_in_place(n, kind):
    """Over one launch's table: several launches, the same factor for all."""
    rng = np.random.default_rng(n)
    sizes = [int(x) for x in rng.integers(0, 3000, n)]
    kinds = [(F32, B16, H16)[k % 3] for k in range(n)]
    grads = grads_of(sizes, kinds, n)
    before = [g.double() for g in grads]
    norm = float(Z.zero_clip_grad_norm(grads, 0.25, kind))
    ref = exact_norm(before, kind)
    assert abs(norm - ref) <= NORM_TOL * ref
    factor = min(1.0, 0.25 / (ref + 1e-6))
    for k in range(n):
        close(grads[k], before[k] * factor, (before[k] * factor).abs() * (NORM_TOL + 2.0 ** -23),
              f"tensor {k}")


def test_norm_range_and_nonfinite():
    # squares outside binary32's range, alone and mixed
    for values in ([3e30, 4e30], [3e-25, 4e-25], [3e30, 1.0], [1e20, 1e-20, 5.0], [0.0, 0.0],
                   [65504.0] * 5000, [2.0 ** 20, 2.0 ** 20 - 1]):
        g = [torch.tensor(values, dtype=F32, device="cuda")]
        ref = exact_norm(g)
        assert abs(float(Z.zero_grad_norm(g)) - ref) <= NORM_TOL * ref, values
    for bad in (float("inf"), float("-inf"), float("nan")):
        for dtype in (H16, B16, F32):
            for at in (0, 9, 5000):
                for kind in ("l2", "inf"):
                    g = [torch.ones(10, dtype=dtype, device="cuda"),
                         torch.ones(6000, dtype=dtype, device="cuda")]
                    g[1][at] = bad
                    keep = [t.clone() for t in g]
                    call = Z.ClipGradNorm(g, 0.5, kind)
                    norm = float(call())
                    r = call.read()
                    assert r.nonfinite == 1 and r.coef == 1.0
                    assert math.isnan(norm) if math.isnan(bad) else norm == float("inf")
                    assert all(torch.equal(torch.nan_to_num(a, 5.0), torch.nan_to_num(b, 5.0))
                               for a, b in zip(g, keep))


def test_empty_lists_and_none():
    assert float(Z.zero_grad_norm([])) == 0.0
    assert float(Z.zero_grad_norm([None, torch.empty(0, device="cuda")])) == 0.0
    assert float(Z.zero_clip_grad_norm([], 1.0)) == 0.0
    g = torch.full((10,), 2.0, device="cuda")
    assert abs(float(Z.zero_clip_grad_norm([None, g, None], 1.0)) - math.sqrt(40)) < 1e-5
    assert abs(float(g.double().pow(2).sum()) - 1.0) < 1e-5


def test_prepared_call_sees_new_values_and_order_of_elements():
    a = torch.randn(300, 70, device="cuda", generator=gen(1))
    b = torch.randn(64, 33, device="cuda", generator=gen(2)).to(B16).t()   # dense, transposed
    out = [torch.empty_like(a), torch.empty(64, 33, dtype=F32, device="cuda").t()]
    call = Z.ClipGradNorm([a, b], 1.0, out=out)
    for scale in (1.0, 3.0, 1e-3):
        a.mul_(scale)
        ref = exact_norm([a, b])
        assert abs(float(call()) - ref) <= NORM_TOL * ref
        f = min(1.0, 1.0 / (ref + 1e-6))
        close(out[0], a.double() * f, (a.double() * f).abs() * 3e-6, "a")
        close(out[1], b.double() * f, (b.double() * f).abs() * 3e-6, "b")


def test_norm_is_the_same_every_time_and_on_another_stream():
    grads = grads_of([1_000_003, 77, 500_001], [B16, F32, H16], 5)
    first = float(Z.zero_grad_norm(grads))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        assert float(Z.zero_grad_norm(grads)) == first
        with torch.cuda.stream(side):
            inner = Z.zero_grad_norm(grads)
        given = Z.zero_grad_norm(grads, stream=side)
        side.synchronize()
        assert float(inner) == first and float(given) == first


def test_norm_past_32_bits():
    n = (1 << 31) + 12345
    g = torch.full((n,), 0.5, dtype=H16, device="cuda")
    norm = float(Z.zero_clip_grad_norm([g], 1.0))
    ref = 0.5 * math.sqrt(n)
    assert abs(norm - ref) <= NORM_TOL * ref
    want = torch.tensor(0.5 / (ref + 1e-6), dtype=torch.float64)
    for at in (0, 1 << 30, (1 << 31) - 1, 1 << 31, n - 1):
        assert abs(float(g[at]) - float(want)) <= 2.0 ** -25 + float(want) * 1e-3


# ---------------------------------------------------------------------------
# block join


def join_inputs(R, H, act, res, par, gate, post, pre, layer, seed, b=True, pad=0):
    g = gen(seed)

    def t(*shape, dtype, scale, shift=0.0):
        if pad and len(shape) == 2 and shape[1] > 1:
            wide = torch.randn(shape[0], shape[1] + pad, device="cuda", generator=g)
            return (wide * scale + shift).to(dtype)[:, :shape[1]]
        return (torch.randn(*shape, device="cuda", generator=g) * scale + shift).to(dtype)

    shape = {"none": None, "channel": (H,), "row": (R, 1), "full": (R, H)}[gate]
    return dict(
        x=t(R, H, dtype=res, scale=2.0), b=t(R, H, dtype=act, scale=0.5, shift=0.1) if b else None,
        gate=None if shape is None or not b else t(*shape, dtype=act, scale=0.3, shift=0.5),
        w_post=t(H, dtype=par, scale=0.1, shift=1.0) if post and b else None,
        bias_post=t(H, dtype=par, scale=0.1) if post and layer and b else None,
        w_pre=t(H, dtype=par, scale=0.1, shift=1.0) if pre else None,
        bias_pre=t(H, dtype=par, scale=0.1) if pre and layer else None)


def join_exact(v, kind, scale, eps):
    """(o, n) in 64 bits; v: the inputs as double tensors."""
    def norm(t, w, bias):
        if kind == "layer":
            t = t - t.mean(-1, keepdim=True)
        t = t / torch.sqrt(t.pow(2).mean(-1, keepdim=True) + eps) * w
        return t if bias is None else t + bias

    o = v["x"]
    if v["b"] is not None:
        u = v["b"] if v["w_post"] is None else norm(v["b"], v["w_post"], v["bias_post"])
        o = o + scale * (u if v["gate"] is None else u * v["gate"])
    return o, None if v["w_pre"] is None else norm(o, v["w_pre"], v["bias_pre"])


def top(t):
    """Largest magnitude of every row."""
    return t.double().abs().amax(-1, keepdim=True) if t.numel() else t.double()


def check_join(v, kind, scale=0.7, eps=1e-6, use_o=True, use_n=True):
    double = {k: None if t is None else t.double().detach().requires_grad_(True)
              for k, t in v.items()}
    o, n = join_exact(double, kind, scale, eps)
    params = {k: t for k, t in v.items() if k not in ("x", "b")}
    got_o, got_n, stats = Z.zero_block_join(v["x"], v["b"], kind=kind, scale=scale, eps=eps,
                                            want_stats=True, **params)
    with torch.no_grad():
        size = top(v["x"]) + (0 if v["b"] is None else top(o - double["x"]))
        close(got_o, o, E * size, "o")
        if n is not None:
            # errors of o enter n through its 1/deviation
            dev = torch.sqrt(((o - (o.mean(-1, keepdim=True) if kind == "layer" else 0)) ** 2)
                             .mean(-1, keepdim=True) + eps)
            amp = size / dev * v["w_pre"].double().abs().max() if n.numel() else 0
            close(got_n, n, E * (amp + top(n)), "n")
    if n is None:
        use_n = False
    g = gen(99)
    d_o = torch.randn(o.shape, device="cuda", generator=g).to(v["x"].dtype) if use_o else None
    act = got_n.dtype if got_n is not None else None
    d_n = torch.randn(o.shape, device="cuda", generator=g).to(act) if use_n else None
    if not use_o and not use_n:
        return
    loss = 0
    if use_o:
        loss = loss + (o * d_o.double()).sum()
    if use_n:
        loss = loss + (n * d_n.double()).sum()
    loss.backward()
    got = Z.zero_block_join_backward(v["x"], v["b"], d_o, d_n, stats, kind=kind, scale=scale,
                                     eps=eps, **params)
    with torch.no_grad():
        # the size of what adds up in a row's gradient: do and the norm's
        # terms, each at most sqrt(H) times the row's root mean square
        ref = {"d" + k: t.grad for k, t in double.items() if t is not None and t.grad is not None}
        grow = top(ref["dx"])
        if use_n:
            dev = torch.sqrt(((o - (o.mean(-1, keepdim=True) if kind == "layer" else 0)) ** 2)
                             .mean(-1, keepdim=True) + eps)
            grow = grow + 4 * top(d_n.double() * v["w_pre"].double()) / dev * (1 + size / dev)
        close(got["dx"], ref["dx"], 3 * E * grow, "dx")
        if v["b"] is None:
            assert got["db"] is None
        else:
            gate = scale if v["gate"] is None else scale * v["gate"].double()
            du = (ref["dx"] * gate)
            dgrow = grow * (abs(scale) if v["gate"] is None else (scale * v["gate"].double()).abs())
            u = v["b"].double()
            if v["w_post"] is not None:
                b = v["b"].double()
                c = b - (b.mean(-1, keepdim=True) if kind == "layer" else 0)
                dev = torch.sqrt(c.pow(2).mean(-1, keepdim=True) + eps)
                hat = c / dev
                u = hat * v["w_post"].double()
                if v["bias_post"] is not None:
                    u = u + v["bias_post"].double()
                sized = top(b) / dev
                q = top(dgrow.expand_as(b)) * v["w_post"].double().abs().max()
                close(got["db"], ref["db"], 12 * E * q / dev * (1 + sized), "db")
                close(got["dw_post"], ref["dw_post"],
                      3 * E * (dgrow.expand_as(b) * (1 + sized + hat.abs())).sum(0), "dw_post")
                if v["bias_post"] is not None:
                    close(got["dbias_post"], ref["dbias_post"],
                          3 * E * dgrow.expand_as(b).sum(0), "dbias_post")
            else:
                close(got["db"], ref["db"], 3 * E * dgrow, "db")
            if v["gate"] is not None:
                slack = 6 * E * abs(scale) * grow * (u.abs() + top(u))
                if v["gate"].shape != u.shape:
                    slack = slack.sum(0) if v["gate"].dim() == 1 else slack.sum(1, keepdim=True)
                close(got["dgate"], ref["dgate"], slack, "dgate")
        if use_n:
            hat = (n - (0 if v["bias_pre"] is None else v["bias_pre"].double())) / v["w_pre"].double()
            amp = 1 + size / dev if v["b"] is None or v["w_post"] is None else 1 + size / torch.sqrt(
                ((o - (o.mean(-1, keepdim=True) if kind == "layer" else 0)) ** 2)
                .mean(-1, keepdim=True) + eps)
            dn = d_n.double().abs()
            close(got["dw_pre"], ref["dw_pre"], 3 * E * (dn * (amp + hat.abs())).sum(0), "dw_pre")
            if v["bias_pre"] is not None:
                close(got["dbias_pre"], ref["dbias_pre"], 3 * E * dn.sum(0), "dbias_pre")
        elif v["w_pre"] is not None:
            assert not got["dw_pre"].any()


TYPES = [(H16, H16, H16), (B16, B16, F32), (B16, F32, B16), (H16, F32, F32), (F32, F32, F32)]


@pytest.mark.parametrize("act,res,par", TYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
def test_join_types_gates_and_norms(act, res, par, kind, gate):
    for post, pre in ((True, True), (True, False), (False, True), (False, False)):
        for R, H in ((37, 768), (5, 1000), (3, 61)):
            check_join(join_inputs(R, H, act, res, par, gate, post, pre, kind == "layer",
                                   R * H + post), kind)


HIDDENS = [1, 2, 7, 8, 31, 32, 33, 64, 100, 255, 256, 257, 264, 512, 1021, 1024, 2048, 2056, 4096,
           4104, 5120, 8192, 8200]


@pytest.mark.parametrize("H", HIDDENS)
@pytest.mark.parametrize("act,res,par", [(B16, B16, B16), (F32, F32, F32), (H16, F32, F32)],
                         ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_join_hidden_sizes(H, act, res, par, kind):
    check_join(join_inputs(11, H, act, res, par, "channel", True, True, kind == "layer", H), kind,
               eps=1e-3)


@pytest.mark.parametrize("R", [0, 1, 2, 3, 151, 152, 153, 700, 5000])
@pytest.mark.parametrize("H", [256, 1024, 250])
def test_join_row_counts(R, H):
    v = join_inputs(R, H, B16, B16, F32, "channel", True, True, True, R)
    if R:
        check_join(v, "layer")
        return
    o, n, stats = Z.zero_block_join(v["x"], v["b"], kind="layer", want_stats=True,
                                    **{k: v[k] for k in v if k not in ("x", "b")})
    assert o.shape == n.shape == (0, H) and stats.shape == (0, 4)
    got = Z.zero_block_join_backward(v["x"], v["b"], o, n, stats, kind="layer",
                                     **{k: v[k] for k in v if k not in ("x", "b")})
    for k in ("dw_post", "dbias_post", "dw_pre", "dbias_pre", "dgate"):
        assert got[k].shape == (H,) and not got[k].any()


@pytest.mark.parametrize("pad", [1, 8, 24])
@pytest.mark.parametrize("H", [512, 768, 509])
def test_join_strided_rows(H, pad):
    check_join(join_inputs(40, H, B16, B16, B16, "full", True, True, False, pad, pad=pad), "rms")
    check_join(join_inputs(40, H, H16, F32, F32, "row", False, True, True, pad, pad=pad), "layer")


@pytest.mark.parametrize("use_o,use_n", [(True, False), (False, True)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_join_one_gradient_only(use_o, use_n, kind):
    for H in (512, 300):
        check_join(join_inputs(9, H, B16, B16, F32, "channel", True, True, kind == "layer", 3), kind,
                   use_o=use_o, use_n=use_n)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_alone(kind):
    for R, H, act in ((20, 768, B16), (6, 333, F32), (1, 4096, H16)):
        check_join(join_inputs(R, H, act, act, act, "none", False, True, kind == "layer", H, b=False),
                   kind)
    # an fp32 stream normed for 16-bit parameters gives 16 bits
    v = join_inputs(8, 256, B16, F32, B16, "none", False, True, False, 1, b=False)
    o, n, _ = Z.zero_block_join(v["x"], w_pre=v["w_pre"])
    assert o is v["x"] and n.dtype == B16


def test_join_rows_of_zeros_large_values_and_nonfinite_rows():
    """A row's values stay in the row: zeros, huge values, NaN and infinity."""
    for H in (512, 259):
        v = join_inputs(8, H, B16, F32, F32, "channel", True, True, True, 4)
        v["b"][1] = 0
        v["x"][1] = 0
        v["x"][2] *= 1e12
        v["b"][3, 5] = float("nan")
        v["x"][4, 7] = float("inf")
        params = {k: t for k, t in v.items() if k not in ("x", "b")}
        o, n, stats = Z.zero_block_join(v["x"], v["b"], kind="layer", want_stats=True, **params)
        d = {k: None if t is None else t.double() for k, t in v.items()}
        ro, rn = join_exact(d, "layer", 1.0, 1e-6)
        fine = [0, 1, 2, 5, 6, 7]
        close(o[fine], ro[fine], E * top(ro[fine]), "o")
        close(n[fine], rn[fine], 20 * E * (1 + top(rn[fine])), "n")
        assert torch.isnan(n[3]).all() and torch.isnan(o[3]).all()
        assert torch.isnan(n[4]).all() and int(torch.isfinite(o[4]).sum()) == H - 1


def test_join_in_place():
    for H in (1024, 77):
        v = join_inputs(12, H, B16, B16, B16, "channel", True, True, False, 8)
        params = {k: t for k, t in v.items() if k not in ("x", "b")}
        o, n, _ = Z.zero_block_join(v["x"], v["b"], **params)
        x, b = v["x"].clone(), v["b"].clone()
        Z.zero_block_join(x, b, o=x, n=b, **params)
        assert torch.equal(x, o) and torch.equal(b, n)


def test_join_same_bits_every_time_on_streams_and_in_a_graph():
    v = join_inputs(3000, 1024, B16, B16, B16, "channel", True, True, False, 6)
    params = {k: t for k, t in v.items() if k not in ("x", "b")}
    d_o, d_n = torch.randn_like(v["x"]), torch.randn_like(v["x"])

    def both(stream=None):
        o, n, stats = Z.zero_block_join(v["x"], v["b"], want_stats=True, stream=stream, **params)
        g = Z.zero_block_join_backward(v["x"], v["b"], d_o, d_n, stats, stream=stream, **params)
        return [o, n] + [t for t in g.values() if t is not None]

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again = both(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["channel", "row", "full"])
@pytest.mark.parametrize("H", [96, 45])
def test_join_gradient_against_differences(kind, gate, H):
    """Central differences of the forward call along random directions.  In
    binary32 the loss (64-bit sums of R H products near 1) is off by about
    sqrt(R H) 2^-24 * 4 = 7e-6; over 2h = 2e-2 that is 4e-4, and the third
    derivative leaves h^2 = 1e-4 of terms near the gradient's size."""
    v = join_inputs(6, H, F32, F32, F32, gate, True, True, kind == "layer", H)
    g = gen(7)
    leaves = {k: None if t is None else t.clone().requires_grad_(True) for k, t in v.items()}
    c1, c2 = (torch.randn(6, H, device="cuda", generator=g) for _ in range(2))

    def loss(w):
        w = dict(w)
        o, n = Z.block_join(w.pop("x"), w.pop("b"), kind=kind, scale=0.6, **w)
        return (o.double() * c1).sum() + (n.double() * c2).sum()

    loss(leaves).backward()
    for k, t in v.items():
        if t is None:
            continue
        for _ in range(3):
            step = torch.randn(t.shape, device="cuda", generator=g)
            step /= step.norm()
            h = 1e-2
            up = loss({**v, k: t + h * step})
            down = loss({**v, k: t - h * step})
            want = float(up - down) / (2 * h)
            have = float((leaves[k].grad.double() * step).sum())
            assert abs(want - have) <= 1e-3 + 5e-3 * abs(have) + 1e-3 * float(leaves[k].grad.norm()), k


def test_join_autograd_wiring():
    """Unused outputs, frozen inputs, expanded gradients, more dimensions."""
    v = join_inputs(24, 64, F32, F32, F32, "channel", True, True, False, 2)
    x, b = v["x"].reshape(2, 3, 4, 64).requires_grad_(True), v["b"].reshape(2, 3, 4, 64)
    w = v["w_pre"].clone().requires_grad_(True)
    o, n = Z.block_join(x, b, w_post=v["w_post"], w_pre=w, gate=v["gate"])
    assert o.shape == n.shape == (2, 3, 4, 64)
    o.sum().backward()
    assert torch.allclose(x.grad, torch.ones_like(x)) and w.grad is None or not w.grad.any()
    x.grad = None
    n2 = Z.block_join(x, w_pre=w)[1]
    n2.sum().backward()
    ref = x.detach().clone().double().requires_grad_(True)
    (ref / torch.sqrt(ref.pow(2).mean(-1, keepdim=True) + 1e-6) * w.double()).sum().backward()
    close(x.grad, ref.grad, 3 * E * 10, "dx")


def test_join_past_32_bits():
    R, H = 530_000, 4096   # 2.17e9 elements
    x = torch.zeros(R, H, dtype=B16, device="cuda")
    b = torch.empty(R, H, dtype=B16, device="cuda").fill_(1.0)
    b[-1] = torch.linspace(-1, 1, H, device="cuda").to(B16)
    w = torch.ones(H, dtype=B16, device="cuda")
    o, n, stats = Z.zero_block_join(x, b, w_post=w, w_pre=w, scale=0.5, want_stats=True)
    last = b[-1].double()
    u = last / torch.sqrt(last.pow(2).mean() + 1e-6)
    close(o[-1], 0.5 * u, E * 2, "o")
    assert bool((n[-2] == 1).all()) and bool((o[R // 2] == 0.5).all())
    g = Z.zero_block_join_backward(x, b, o, None, stats, w_post=w, scale=0.5,
                                   want={"db", "dw_post"})
    # rows of ones: du = 0.25, bh = 1 (1/sqrt(1 + 1e-6)): every column sums to
    # (R-1)/4 but for the last row, and db vanishes
    want = (R - 1) * 0.25
    assert float((g["dw_post"].double() - want).abs().max()) <= want * 2 * UNIT[B16]
    assert float(g["db"][:-1].abs().max()) <= 1e-5


# ---------------------------------------------------------------------------
# expert permutation


def sorted_pairs(ids, n_experts):
    """(offsets, rows, pairs) by lists."""
    T, K = ids.shape
    flat = ids.reshape(-1).tolist()
    members = [[] for _ in range(n_experts)]
    for p, e in enumerate(flat):
        if 0 <= e < n_experts:
            members[e].append(p)
    offsets = np.concatenate([[0], np.cumsum([len(m) for m in members])])
    order = [p for m in members for p in m]
    rows = np.full(T * K, -1, np.int64)
    rows[order] = np.arange(len(order))
    pairs = np.full(T * K, -1, np.int64)
    pairs[:len(order)] = order
    return offsets, rows.reshape(T, K), pairs


def choose(T, K, n_experts, seed, drop=0.0, dtype=torch.int32):
    g = gen(seed)
    ids = torch.randint(0, n_experts, (T, K), device="cuda", generator=g)
    if drop:
        ids[torch.rand(T, K, device="cuda", generator=g) < drop] = -1
    return ids.to(dtype)


SORTS = [(0, 2, 4), (1, 1, 1), (1, 8, 8), (5, 3, 2), (31, 1, 7), (33, 1, 7), (16, 2, 64),
         (1000, 2, 8), (4096, 2, 64), (2999, 3, 17), (20000, 8, 256), (8192, 1, 1),
         (65536, 6, 512), (3000, 4, 1023), (5000, 2, 4096), (100, 2, 4096), (40000, 1, 3)]


@pytest.mark.parametrize("T,K,n_experts", SORTS)
@pytest.mark.parametrize("dtype,drop", [(torch.int32, 0.0), (torch.int64, 0.3)])
def test_sort(T, K, n_experts, dtype, drop):
    ids = choose(T, K, n_experts, T + K + n_experts, drop, dtype)
    order = Z.zero_expert_sort(ids, n_experts)
    offsets, rows, pairs = sorted_pairs(ids.cpu(), n_experts)
    assert np.array_equal(order.offsets.cpu().numpy(), offsets)
    assert np.array_equal(order.rows.cpu().numpy(), rows)
    assert np.array_equal(order.pairs.cpu().numpy(), pairs)


def test_sort_odd_ids():
    """All dropped; all of one expert; ids far outside, of both widths."""
    for ids, n_experts in ((torch.full((100, 2), -1, device="cuda"), 5),
                           (torch.full((5000, 3), 4, device="cuda"), 5),
                           (torch.tensor([[1 << 40, -(1 << 40)], [(1 << 32) + 1, 2]],
                                         device="cuda"), 3),
                           (torch.tensor([[5, 4], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32,
                                         device="cuda"), 5)):
        order = Z.zero_expert_sort(ids, n_experts)
        offsets, rows, pairs = sorted_pairs(ids.cpu(), n_experts)
        assert np.array_equal(order.offsets.cpu().numpy(), offsets)
        assert np.array_equal(order.rows.cpu().numpy(), rows)
        assert np.array_equal(order.pairs.cpu().numpy(), pairs)


def check_rows(T, K, n_experts, Hd, dtype, wtype, drop, pad=0, seed=0):
    g = gen(seed + T)
    ids = choose(T, K, n_experts, seed, drop)
    order = Z.zero_expert_sort(ids, n_experts)
    M = int(order.offsets[-1])
    x, dy = ((torch.randn(T, Hd + pad, device="cuda", generator=g)).to(dtype)[:, :Hd]
             for _ in range(2))
    ys, dxs = (torch.randn(T * K, Hd, device="cuda", generator=g).to(dtype) for _ in range(2))
    ys[M:], dxs[M:] = float("nan"), float("nan")   # never read
    w = torch.rand(T, K, device="cuda", generator=g).to(wtype)
    pairs = order.pairs[:M].long()
    token = pairs // K

    xs = Z.zero_expert_dispatch(x, order)
    assert torch.equal(xs[:M], x[token]) and not xs[M:].any()
    y = Z.zero_expert_combine(ys, w, order)
    wd = w.double().reshape(-1)[pairs][:, None]
    terms = wd * ys[:M].double()

    def back(rows):
        return torch.zeros(T, Hd, dtype=torch.float64, device="cuda").index_add_(0, token, rows)

    step = 10 * 2.0 ** -24
    close(y, back(terms), step * back(terms.abs()), "y")
    dx = Z.zero_expert_dispatch_backward(dxs, order)
    close(dx, back(dxs[:M].double()), step * back(dxs[:M].double().abs()), "dx")
    dys, dw = Z.zero_expert_combine_backward(dy, ys, w, order)
    close(dys[:M], wd * dy[token].double(), step * (wd * dy[token].double()).abs(), "dys")
    assert not dys[M:].any()
    ref, size = (torch.zeros(T * K, dtype=torch.float64, device="cuda") for _ in range(2))
    prod = dy[token].double() * ys[:M].double()
    ref[pairs], size[pairs] = prod.sum(1), prod.abs().sum(1)
    close(dw.reshape(-1), ref, E * size, "dweights")


@pytest.mark.parametrize("dtype,wtype", [(B16, F32), (B16, B16), (H16, H16), (F32, F32)],
                         ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("T,K,n_experts,Hd", [(1, 1, 1, 8), (7, 2, 4, 4096), (300, 3, 9, 1001),
                                              (129, 8, 33, 768), (500, 2, 64, 64), (40, 1, 5, 1),
                                              (33, 6, 16, 2056), (10, 2, 3, 8192), (0, 2, 3, 16)])
def test_rows(T, K, n_experts, Hd, dtype, wtype):
    for drop in (0.0, 0.4):
        check_rows(T, K, n_experts, Hd, dtype, wtype, drop, seed=Hd)


def test_rows_strided_and_all_dropped():
    check_rows(50, 2, 4, 256, B16, F32, 0.1, pad=8)
    check_rows(50, 2, 4, 256, B16, F32, 0.1, pad=3)
    check_rows(50, 2, 4, 255, F32, F32, 0.1, pad=1)
    check_rows(64, 3, 4, 256, B16, F32, 1.1)


def test_dropped_and_zero_weight_rows_with_nonfinite_values():
    """A dropped choice's weight is not used, whatever it holds."""
    ids = torch.tensor([[0, -1], [1, 0], [-1, -1]], dtype=torch.int32, device="cuda")
    order = Z.zero_expert_sort(ids, 2)
    w = torch.tensor([[1.0, float("nan")], [2.0, 3.0], [float("inf"), float("nan")]], device="cuda")
    ys = torch.arange(1.0, 7.0, device="cuda")[:, None].expand(6, 16).contiguous()
    y = Z.zero_expert_combine(ys, w, order)
    # rows: (t0,k0) 0, (t1,k1) 1, (t1,k0) 2
    assert y[:, 0].tolist() == [1.0, 2.0 * 3.0 + 3.0 * 2.0, 0.0]
    dys, dw = Z.zero_expert_combine_backward(torch.ones(3, 16, device="cuda"), ys, w, order)
    assert dys[:, 0].tolist() == [1.0, 3.0, 2.0, 0.0, 0.0, 0.0]
    assert dw.tolist() == [[16.0, 0.0], [48.0, 32.0], [0.0, 0.0]]


def test_experts_gradients_against_differences():
    """The pass x -> dispatch -> scale by expert -> combine is linear in x and
    in the weights: differences are exact up to rounding (2^-24 sqrt(terms) /
    h of sums near 30)."""
    T, K, n_experts, Hd = 20, 3, 5, 24
    ids = choose(T, K, n_experts, 3, 0.2)
    order = Z.zero_expert_sort(ids, n_experts)
    g = gen(4)
    x = torch.randn(T, Hd, device="cuda", generator=g)
    w = torch.rand(T, K, device="cuda", generator=g)
    c = torch.randn(T, Hd, device="cuda", generator=g)
    by_row = torch.randn(T * K, 1, device="cuda", generator=g)

    def loss(x, w):
        return (Z.expert_combine(Z.expert_dispatch(x, order) * by_row, w, order).double() * c).sum()

    lx, lw = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    loss(lx, lw).backward()
    for t, leaf, at in ((x, lx, 0), (w, lw, 1)):
        for _ in range(4):
            step = torch.randn(t.shape, device="cuda", generator=g)
            h = 0.25
            args = [[x, w], [x, w]]
            args[0][at], args[1][at] = t + h * step, t - h * step
            want = float(loss(*args[0]) - loss(*args[1])) / (2 * h)
            have = float((leaf.grad.double() * step).sum())
            assert abs(want - have) <= 1e-4 * (1 + float(leaf.grad.norm()) * float(step.norm()))


def test_experts_on_a_stream_and_in_a_graph():
    ids = choose(700, 2, 16, 1, 0.1)
    x = torch.randn(700, 256, device="cuda").to(B16)
    w = torch.rand(700, 2, device="cuda")

    def run(stream=None):
        order = Z.zero_expert_sort(ids, 16, stream=stream)
        xs = Z.zero_expert_dispatch(x, order, stream=stream)
        return [order.rows, xs, Z.zero_expert_combine(xs, w, order, stream=stream)]

    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))


def test_experts_past_32_bits():
    T, K, Hd = 66_000, 8, 4096   # 2.16e9 elements of sorted rows
    ids = choose(T, K, 64, 2)
    order = Z.zero_expert_sort(ids, 64)
    x = torch.arange(T, device="cuda").remainder(251).to(B16)[:, None].expand(T, Hd).contiguous()
    xs = Z.zero_expert_dispatch(x, order)
    pairs = order.pairs.long()
    for at in (0, T * K // 2, T * K - 2, T * K - 1):
        assert bool((xs[at] == x[pairs[at] // K]).all())
    dx = Z.zero_expert_dispatch_backward(xs, order)
    assert torch.equal(dx[::977], (x[::977].float() * K).to(B16))


# ---------------------------------------------------------------------------
# refusals


def test_refusals():
    x = torch.ones(4, 16, device="cuda")
    b = torch.ones(4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    for bad in (dict(w_post=w[:8]), dict(w_post=w.to(B16), w_pre=w), dict(gate=torch.ones(3, device="cuda")),
                dict(kind="other"), dict(eps=0.0), dict(eps=float("nan")), dict(scale=float("inf")),
                dict(bias_pre=w), dict(w_pre=w, bias_pre=w), dict(w_pre=w.cpu()), dict(n=x)):
        with pytest.raises((ValueError, TypeError, Z.ZeroError)):
            Z.zero_block_join(x, b, **bad)
    for bad in ((x.double(), b), (x.cpu(), b), (x, b[:, :8]), (x.to(B16), b), (x, b.to(torch.int32)),
                (torch.ones(16, 4, device="cuda").t(), b), (x[:1].expand(4, 16), b)):
        with pytest.raises((ValueError, TypeError, Z.ZeroError)):
            Z.zero_block_join(*bad)
    with pytest.raises(Z.ZeroError):   # a post norm needs the forward's statistics
        Z.zero_block_join_backward(x, b, x, None, None, w_post=w)
    with pytest.raises(Z.ZeroError):
        Z.zero_block_join_backward(x, b, None, None, None)
    with pytest.raises(TypeError):
        Z.zero_block_join_backward(x, b, x.to(B16), None, None)

    g = torch.ones(100, device="cuda")
    for bad in ([g.double()], [g.cpu()], [torch.ones(10, 10, device="cuda")[:, :3]], [3.0],
                [g.expand(5, 100)]):
        with pytest.raises((ValueError, TypeError)):
            Z.zero_grad_norm(bad)
    for max_norm in (-1.0, float("nan"), float("inf")):
        with pytest.raises(Z.ZeroError):
            Z.zero_clip_grad_norm([g], max_norm)
    for grads, out in (([g, g], None), ([g[:60], g[50:]], None), ([g], [g[:50]]), ([g], [g, g]),
                       ([g[:50]], [g[25:75]]), ([g[:50], g[50:]], [torch.ones(50, device="cuda"), g[:50]])):
        with pytest.raises(ValueError):
            Z.zero_clip_grad_norm(grads, 1.0, out=out)
    with pytest.raises(ValueError):
        Z.zero_grad_norm([g], "l1")
    assert bool((g == 1).all())

    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    order = Z.zero_expert_sort(ids, 3)
    for bad in ((ids.float(), 3), (ids[0], 3), (ids.t(), 3), (ids.cpu(), 3), (ids[:, :0], 3)):
        with pytest.raises((ValueError, TypeError)):
            Z.zero_expert_sort(*bad)
    for n_experts in (0, -1, 4097):
        with pytest.raises(Z.ZeroError):
            Z.zero_expert_sort(ids, n_experts)
    weights = torch.ones(4, 2, device="cuda")
    for bad in (lambda: Z.zero_expert_dispatch(x[:3], order),
                lambda: Z.zero_expert_dispatch(x.double(), order),
                lambda: Z.zero_expert_dispatch(x, order, out=x),
                lambda: Z.zero_expert_combine(x, weights, order),
                lambda: Z.zero_expert_combine(torch.ones(8, 16, device="cuda"), weights[:, :1], order),
                lambda: Z.zero_expert_combine(torch.ones(8, 16, device="cuda"), weights.to(B16), order),
                lambda: Z.zero_expert_combine_backward(x.to(B16), torch.ones(8, 16, device="cuda"),
                                                       weights, order),
                lambda: Z.zero_expert_dispatch_backward(torch.ones(7, 16, device="cuda"), order)):
        with pytest.raises((ValueError, TypeError, Z.ZeroError)):
            bad()


# ---------------------------------------------------------------------------
# rows and tensors that start anywhere


def shifted(t, by):
    """The same values in memory that starts `by` elements after an allocation."""
    if t is None:
        return None
    store = torch.full((t.numel() + by + 16,), float("nan"), dtype=t.dtype, device="cuda")
    view = store[by:by + t.numel()].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("by", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("R,H", [(7, 512), (33, 96), (1, 4096), (160, 61), (12, 1536)])
@pytest.mark.parametrize("act,res,gate_type", [(B16, B16, B16), (H16, H16, F32), (B16, F32, F32),
                                               (F32, F32, F32)], ids=lambda t: str(t)[6:])
def test_join_tensors_that_start_anywhere(by, R, H, act, res, gate_type):
    """Every tensor a view at an odd offset; values past the views are NaN,
    so a read that strays shows."""
    v = join_inputs(R, H, act, res, F32, "full", True, True, True, by)
    v["gate"] = v["gate"].to(gate_type)
    check_join({k: shifted(t, by) for k, t in v.items()}, "layer")
    v = join_inputs(R, H, act, res, act, "channel", True, True, False, by)
    check_join({k: shifted(t, by) for k, t in v.items()}, "rms")


@pytest.mark.parametrize("H", [100, 128, 1000, 1024, 4001])
def test_join_aligned_and_shifted_rows_agree(H):
    """Whole and single accesses of the same rows: the same sums in another
    order, so equal within 2 E of a row's size."""
    v = join_inputs(50, H, F32, F32, F32, "row", True, True, False, H)
    params = {k: t for k, t in v.items() if k not in ("x", "b")}
    o, n, _ = Z.zero_block_join(v["x"], v["b"], **params)
    o2, n2, _ = Z.zero_block_join(shifted(v["x"], 1), shifted(v["b"], 3), **params)
    close(o2, o.double(), 2 * E * top(o), "o")
    close(n2, n.double(), 2 * E * top(n), "n")


@pytest.mark.parametrize("by", [1, 3, 8])
def test_expert_rows_that_start_anywhere(by):
    T, K, n_experts = 60, 3, 7
    for Hd, dtype in ((256, B16), (255, B16), (130, F32), (64, H16)):
        order = Z.zero_expert_sort(choose(T, K, n_experts, by, 0.2), n_experts)
        g = gen(by)
        x = torch.randn(T, Hd, device="cuda", generator=g).to(dtype)
        ys = torch.randn(T * K, Hd, device="cuda", generator=g).to(dtype)
        w = torch.rand(T, K, device="cuda", generator=g)
        xs = Z.zero_expert_dispatch(shifted(x, by), order)
        assert torch.equal(xs, Z.zero_expert_dispatch(x, order))
        y, y2 = (Z.zero_expert_combine(t, w, order) for t in (ys, shifted(ys, by)))
        close(y2, y.double(), 2 * UNIT[dtype] * y.double().abs() + 1e-6, "y")
        dys, dw = Z.zero_expert_combine_backward(x, ys, w, order)
        dys2, dw2 = Z.zero_expert_combine_backward(shifted(x, by), shifted(ys, by), w, order)
        assert torch.equal(dys, dys2)
        close(dw2, dw.double(), E * float((x.double().abs().max() * ys.double().abs().max()) * Hd), "dw")


@pytest.mark.parametrize("dtype", [H16, B16, F32])
def test_grads_that_start_anywhere_stay_in_bounds(dtype):
    """Neighbours of every view are NaN and stay so."""
    sizes = [1, 7, 8, 9, 15, 16, 17, 31, 1023, 1025, 8191, 8192, 8193, 8199, 16385, 25000]
    g = gen(1)
    for by in range(8):
        grads = [shifted((torch.randn(n, device="cuda", generator=g)).to(dtype), by) for n in sizes]
        for out_by in (0, 1, 5):
            out = [shifted(torch.zeros(n, device="cuda").to(B16), out_by) for n in sizes]
            norm = float(Z.zero_clip_grad_norm(grads, 2.0, out=out))
            ref = exact_norm(grads)
            assert abs(norm - ref) <= NORM_TOL * ref
            f = min(1.0, 2.0 / (ref + 1e-6))
            for a, b in zip(grads, out):
                close(b, a.double() * f, (a.double() * f).abs() * 3e-6, "out")
                base = b._base
                assert bool(torch.isnan(base[:out_by]).all())
                assert bool(torch.isnan(base[out_by + b.numel():]).all())


def test_join_many_rows_of_one_cta_shape():
    """More rows than the persistent grid holds, rows left over in a CTA's
    groups, row gates read ahead."""
    for R, H in ((40_001, 64), (9_999, 200), (5_003, 512), (3_001, 511)):
        check_join(join_inputs(R, H, B16, B16, F32, "row", True, True, False, R), "rms")


# ---------------------------------------------------------------------------
# launches that start early, in graphs and back to back


def test_clip_in_a_graph_and_back_to_back():
    """Several launches a pass (over 1000 tensors), captured once and replayed
    on new values; then calls that follow one another without a wait."""
    rng = np.random.default_rng(3)
    sizes = [int(x) for x in rng.integers(1, 4000, 1300)]
    grads = grads_of(sizes, [(F32, B16)[k % 2] for k in range(len(sizes))], 3)
    out = [torch.empty(n, dtype=B16, device="cuda") for n in sizes]
    call = Z.ClipGradNorm(grads, 0.3, out=out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = call()
    for scale in (1.0, 7.0, 0.01):
        for g in grads:
            g.mul_(scale)
        ref = exact_norm(grads)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(float(norm) - ref) <= NORM_TOL * ref
        f = min(1.0, 0.3 / (ref + 1e-6))
        for k in (0, 1, 999, 1000, 1299):
            close(out[k], grads[k].double() * f, (grads[k].double() * f).abs() * 3e-6, f"tensor {k}")
    big = [torch.full((3_000_000,), 1.0, device="cuda")]
    halve = Z.ClipGradNorm(big, 1.0)
    refs = []
    for k in range(20):   # in place: each call's norm is the limit before it
        halve.max_norm = 1000.0 / 2 ** k
        refs.append(halve().clone())
    torch.cuda.synchronize()
    want = math.sqrt(3_000_000)
    for k, r in enumerate(refs):
        assert abs(float(r) - want) <= 1e-5 * want, k
        want *= min(1.0, 1000.0 / 2 ** k / (want + 1e-6))


def test_large_sort_and_join_in_a_graph():
    ids = choose(60_000, 2, 100, 9)
    v = join_inputs(700, 768, B16, B16, B16, "channel", True, True, False, 6)
    params = {k: t for k, t in v.items() if k not in ("x", "b")}

    def run():
        order = Z.zero_expert_sort(ids, 100)
        o, n, stats = Z.zero_block_join(v["x"], v["b"], want_stats=True, **params)
        g = Z.zero_block_join_backward(v["x"], v["b"], o, n, stats, **params)
        return [order.offsets, order.rows, order.pairs, o, n] + [t for t in g.values() if t is not None]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for seed in (1, 2):
        ids.copy_(choose(60_000, 2, 100, seed, 0.1))
        v["b"].mul_(0.9)
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_record_and_prepared_norm():
    g = [torch.full((100,), 3.0, device="cuda"), torch.full((7,), -4.0, dtype=H16, device="cuda")]
    call = Z.GradNorm(g)
    want = math.sqrt(100 * 9 + 7 * 16)
    assert abs(float(call()) - want) <= NORM_TOL * want
    r = call.read()
    assert abs(r.norm - want) <= NORM_TOL * want and r.coef == 1.0 and r.nonfinite == 0
    clip = Z.ClipGradNorm(g, 0.5)
    clip()
    r = clip.read()
    assert abs(r.norm - want) <= NORM_TOL * want
    assert abs(r.coef - 0.5 / want) <= 1e-6 * 0.5 / want
    mixed = Z.ClipGradNorm(g, 1e9, out=[g[0], torch.empty(7, device="cuda")])
    assert float(mixed()) > 0   # one in place, one elsewhere
    ws = torch.empty(Z.zero_grad_norm_workspace_bytes(g), dtype=torch.uint8, device="cuda")
    assert float(Z.GradNorm(g, workspace=ws)()) == float(Z.GradNorm(g)())
    with pytest.raises(ValueError):
        Z.GradNorm(g, workspace=ws[:16])


def test_calls_keep_nothing():
    """Neither memory nor references stay behind, after refusals either."""
    import gc
    import sys
    x, b, d = (torch.randn(6, 64, device="cuda") for _ in range(3))
    w = torch.ones(64, device="cuda")
    ids = torch.tensor([[0, 1], [1, 2], [2, 0], [0, 2], [1, 0], [2, 1]], dtype=torch.int32, device="cuda")
    weights = torch.rand(6, 2, device="cuda")

    def calls():
        _, _, stats = Z.zero_block_join(x, b, w_post=w, w_pre=w, want_stats=True)
        Z.zero_block_join_backward(x, b, d, d, stats, w_post=w, w_pre=w, want={"dx", "dw_pre"})
        assert Z.zero_block_join(x, w_pre=w)[0] is x
        order = Z.zero_expert_sort(ids, 3)
        ys = Z.zero_expert_dispatch(x, order)
        Z.zero_expert_combine(ys, weights, order)
        Z.zero_expert_combine_backward(d, ys, weights, order)
        Z.zero_expert_dispatch_backward(ys, order)
        for bad in (lambda: Z.zero_block_join(x, b, w_post=w, scale="x"),
                    lambda: Z.zero_block_join(x, b, w_post=w, eps=0.0),
                    lambda: Z.zero_expert_combine(ys, weights[:3], order)):
            with pytest.raises((TypeError, ValueError, Z.ZeroError)):
                bad()

    calls()
    torch.cuda.synchronize()
    gc.collect()
    held = [sys.getrefcount(t) for t in (x, b, d, w, ids, weights)] + [sys.getrefcount(None)]
    bytes_ = torch.cuda.memory_allocated()
    for _ in range(200):
        calls()
    torch.cuda.synchronize()
    gc.collect()
    now = [sys.getrefcount(t) for t in (x, b, d, w, ids, weights)] + [sys.getrefcount(None)]
    assert now[:-1] == held[:-1]
    assert abs(now[-1] - held[-1]) < 100    # None: immortal, or within the interpreter's own use
    assert torch.cuda.memory_allocated() == bytes_


@pytest.mark.parametrize("dtype", [H16, B16, F32])
@pytest.mark.parametrize("K", [1, 2, 3, 5])
@pytest.mark.parametrize("Hd", [1, 7, 8, 9, 16, 17, 31, 33, 60, 517, 2051])
def test_expert_rows_of_any_length_start_and_stride(Hd, K, dtype):
    """Inputs and outputs start at odd elements, the tokens' rows are `pad`
    apart, and what lies between and around them is NaN and stays so."""
    T, n_experts = 11, 4
    for by, pad in ((1, 0), (2, 3), (3, 1), (5, 8), (7, 5)):
        g = gen(by + Hd)
        order = Z.zero_expert_sort(choose(T, K, n_experts, by, 0.2), n_experts)
        M = int(order.offsets[-1])
        pairs = order.pairs[:M].long()
        token = pairs // K

        def rows(n, stride):
            store = torch.full((by + n * stride + 24,), float("nan"), dtype=dtype, device="cuda")
            view = store.as_strided((n, Hd), (stride, 1), by)
            view.copy_(torch.randn(n, Hd, device="cuda", generator=g))
            return view

        def outputs(n):
            store = torch.full((by + n * Hd + 24,), float("nan"), dtype=dtype, device="cuda")
            return store, store[by:by + n * Hd].view(n, Hd)

        def untouched(store, n):
            return bool(store[:by].isnan().all() and store[by + n * Hd:].isnan().all())

        x, dy = rows(T, Hd + pad), rows(T, Hd + pad)
        ys, dxs = rows(T * K, Hd), rows(T * K, Hd)
        ys[M:], dxs[M:] = float("nan"), float("nan")
        w = torch.rand(T, K, device="cuda", generator=g)
        wd = w.double().reshape(-1)[pairs][:, None]

        def back(t):
            return torch.zeros(T, Hd, dtype=torch.float64, device="cuda").index_add_(0, token, t)

        step = 10 * 2.0 ** -24    # K products and sums in binary32
        store, xs = outputs(T * K)
        Z.zero_expert_dispatch(x, order, out=xs)
        assert torch.equal(xs[:M], x[token]) and not xs[M:].any() and untouched(store, T * K)
        store, y = outputs(T)
        Z.zero_expert_combine(ys, w, order, out=y)
        terms = wd * ys[:M].double()
        close(y, back(terms), step * back(terms.abs()), "y")
        assert untouched(store, T)
        store, dx = outputs(T)
        Z.zero_expert_dispatch_backward(dxs, order, out=dx)
        close(dx, back(dxs[:M].double()), step * back(dxs[:M].double().abs()), "dx")
        assert untouched(store, T)
        dys, dw = Z.zero_expert_combine_backward(dy, ys, w, order)
        close(dys[:M], wd * dy[token].double(), step * (wd * dy[token].double()).abs(), "dys")
        assert not dys[M:].any()
        ref, size = (torch.zeros(T * K, dtype=torch.float64, device="cuda") for _ in range(2))
        prod = dy[token].double() * ys[:M].double()
        ref[pairs], size[pairs] = prod.sum(1), prod.abs().sum(1)
        close(dw.reshape(-1), ref, E * size, "dweights")
