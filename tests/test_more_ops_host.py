"""Host side of the embedding, the router and the cross entropy (no GPU needed):
the C calls refuse bad arguments with the documented status before they touch a
device, and so does the binding; what runs on a given stream is made there."""
import ctypes
import math
import types

import pytest
import torch

from zero_sharded_optimizer_flatten_gb300 import _build
from zero_sharded_optimizer_flatten_gb300 import train_ops as T
from zero_sharded_optimizer_flatten_gb300 import zero as Z

NAMES = ("ids", "table", "y", "dy", "dtable", "ws", "logits", "weights", "counts", "losses", "stats", "dw", "dl",
         "dz", "x", "w", "targets", "lse", "rows", "total", "d", "dx")
AT = {k: 0x10000000 + (i << 24) for i, k in enumerate(NAMES)}   # addresses that are never read


@pytest.fixture(scope="module")
def L():
    _build.build()
    return Z.lib()


@pytest.fixture(autouse=True)
def _launches_nothing(L):
    before = Z.zero_launch_count()
    yield
    assert Z.zero_launch_count() == before


def refused(status, want=Z.ZERO_ERR_INVALID, says=""):
    assert status == want and says in Z.zero_last_error() and Z.zero_last_error(), (status, Z.zero_last_error())


# ---------------------------------------------------------------------------
# embedding


def lookup(L, **c):
    a = dict(ids=AT["ids"], id_bytes=8, tokens=10, table=AT["table"], stride=64, type=1, vocab=100, hidden=64,
             scale=1.0, y=AT["y"], y_type=1) | c
    return L.zero_embedding(*a.values(), None)


def gradient(L, **c):
    a = dict(dy=AT["dy"], stride=64, dy_type=1, ids=AT["ids"], id_bytes=8, tokens=10, vocab=100, hidden=64,
             scale=1.0, accumulate=0, out=AT["dtable"], out_type=1, ws=AT["ws"], size=1 << 20) | c
    return L.zero_embedding_backward(*a.values(), None)


def test_embedding_refusals(L):
    for bad in (dict(ids=None), dict(id_bytes=2), dict(tokens=-1), dict(tokens=(1 << 28) + 1), dict(table=None),
                dict(stride=63), dict(type=3), dict(type=-1), dict(vocab=0), dict(vocab=(1 << 22) + 1),
                dict(hidden=0), dict(hidden=(1 << 20) + 1), dict(scale=math.nan), dict(scale=math.inf),
                dict(scale=1e300), dict(y=None), dict(y_type=0), dict(type=2, y_type=1)):
        refused(lookup(L, **bad))
    for bad in (dict(ids=AT["ids"] + 4), dict(table=AT["table"] + 1), dict(y=AT["y"] + 2, y_type=2)):
        refused(lookup(L, **bad), Z.ZERO_ERR_ALIGN)
    for at in (AT["ids"], AT["ids"] + 79, AT["table"], AT["table"] + 99 * 128 + 127):
        refused(lookup(L, y=at & ~1), says="y overlaps")
    assert lookup(L, tokens=0, ids=None, table=None, y=None) == 0


def test_embedding_gradient_refusals(L):
    need = ctypes.c_int64()
    assert L.zero_embedding_workspace_bytes(10, 100, 64, ctypes.byref(need)) == 0
    assert 0 < need.value <= 1 << 20
    for bad in (dict(dy=None), dict(stride=63), dict(dy_type=3), dict(ids=None), dict(id_bytes=3), dict(tokens=-1),
                dict(vocab=0), dict(vocab=(1 << 22) + 1), dict(hidden=0), dict(scale=math.nan), dict(out=None),
                dict(out_type=0), dict(out_type=5), dict(ws=None), dict(size=need.value - 1)):
        refused(gradient(L, **bad))
    for bad in (dict(dy=AT["dy"] + 1), dict(ids=AT["ids"] + 4), dict(out=AT["dtable"] + 1), dict(ws=AT["ws"] + 16)):
        refused(gradient(L, **bad), Z.ZERO_ERR_ALIGN)
    refused(gradient(L, out=AT["dy"]), says="dtable overlaps dy")
    refused(gradient(L, out=AT["dy"] - 100 * 128 + 2), says="dtable overlaps dy")
    refused(gradient(L, out=AT["ids"]), says="dtable overlaps ids")
    refused(gradient(L, ws=AT["dtable"] + 256), says="workspace overlaps dtable")
    refused(gradient(L, ws=AT["dy"]), says="workspace overlaps dy")
    for bad in ((-1, 100, 64), (10, 0, 64), (10, 100, 0)):
        refused(L.zero_embedding_workspace_bytes(*bad, ctypes.byref(need)))
    refused(L.zero_embedding_workspace_bytes(10, 100, 64, None))
    assert gradient(L, tokens=0, accumulate=1, dy=None, ids=None, ws=None) == 0
    last = 0
    for tokens in (1, 100, 10_000, 1 << 20):   # grows with the tokens
        assert L.zero_embedding_workspace_bytes(tokens, 32000, 4096, ctypes.byref(need)) == 0
        assert need.value > last
        last = need.value


# ---------------------------------------------------------------------------
# router


def route(L, **c):
    a = dict(z=AT["logits"], stride=16, type=2, tokens=10, experts=16, topk=2, normalize=1, ids=AT["ids"],
             weights=AT["weights"], counts=AT["counts"], losses=AT["losses"], stats=AT["stats"], ws=None, size=0) | c
    return L.zero_expert_route(*a.values(), None)


def route_back(L, **c):
    a = dict(z=AT["logits"], stride=16, type=2, tokens=10, experts=16, topk=2, normalize=1, ids=AT["ids"],
             weights=AT["weights"], counts=AT["counts"], stats=AT["stats"], dw=AT["dw"], dl=AT["dl"], dz=AT["dz"]) | c
    return L.zero_expert_route_backward(*a.values(), None)


def test_route_refusals(L):
    for bad in (dict(z=None), dict(stride=15), dict(type=3), dict(tokens=-1), dict(tokens=(1 << 24) + 1),
                dict(experts=0), dict(experts=1025, stride=2000), dict(topk=0), dict(topk=17),
                dict(experts=100, stride=100, topk=33), dict(ids=None), dict(weights=None), dict(counts=None),
                dict(losses=None), dict(stats=None), dict(tokens=1000), dict(tokens=1000, ws=AT["ws"], size=64)):
        refused(route(L, **bad))
    for bad in (dict(z=AT["logits"] + 2), dict(ids=AT["ids"] + 1), dict(stats=AT["stats"] + 2),
                dict(tokens=1000, ws=AT["ws"] + 1, size=1 << 20)):
        refused(route(L, **bad), Z.ZERO_ERR_ALIGN)
    refused(route(L, ids=AT["logits"]), says="ids overlaps logits")
    refused(route(L, weights=AT["ids"] + 4), says="weights overlaps ids")
    refused(route(L, stats=AT["counts"]), says="stats overlaps counts")
    refused(route(L, losses=AT["logits"] + 10 * 64 - 4), says="losses overlaps logits")
    need = ctypes.c_int64()
    assert L.zero_expert_route_workspace_bytes(10, 16, ctypes.byref(need)) == 0 and need.value == 0
    assert L.zero_expert_route_workspace_bytes(1000, 16, ctypes.byref(need)) == 0 and need.value > 0
    for bad in ((-1, 16), (10, 0), (10, 1025)):
        refused(L.zero_expert_route_workspace_bytes(*bad, ctypes.byref(need)))


def test_route_gradient_refusals(L):
    for bad in (dict(z=None), dict(stride=15), dict(type=-1), dict(tokens=-1), dict(topk=17), dict(ids=None),
                dict(weights=None), dict(counts=None), dict(stats=None), dict(dz=None)):
        refused(route_back(L, **bad))
    refused(route_back(L, dz=AT["dz"] + 2), Z.ZERO_ERR_ALIGN)
    for of in ("logits", "ids", "weights", "counts", "stats", "dw", "dl"):
        refused(route_back(L, dz=AT[of]), says="d_logits overlaps")
    assert route_back(L, tokens=0, z=None, ids=None, weights=None, counts=None, stats=None, dz=None) == 0


# ---------------------------------------------------------------------------
# cross entropy


class Desc(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in ("tokens", "hidden", "vocab", "x_stride", "w_stride")] + [
        ("dtype", ctypes.c_int32), ("dw_dtype", ctypes.c_int32), ("id_bytes", ctypes.c_int32),
        ("scale", ctypes.c_double)]


def desc(**c):
    return Desc(**(dict(tokens=10, hidden=64, vocab=100, x_stride=64, w_stride=64, dtype=1, dw_dtype=1, id_bytes=8,
                        scale=1.0) | c))


def loss(L, d=None, **c):
    a = dict(x=AT["x"], w=AT["w"], targets=AT["targets"], losses=AT["losses"], lse=AT["lse"], rows=AT["rows"],
             total=AT["total"], ws=AT["ws"], size=1 << 30) | c
    return L.zero_linear_cross_entropy(ctypes.byref(desc() if d is None else d), *a.values(), None)


def loss_back(L, desc_=None, **c):
    a = dict(x=AT["x"], w=AT["w"], targets=AT["targets"], lse=AT["lse"], rows=AT["rows"], d=AT["d"], reduction=2,
             dx=AT["dx"], dw=AT["dw"], ws=AT["ws"], size=1 << 40) | c
    return L.zero_linear_cross_entropy_backward(ctypes.byref(desc() if desc_ is None else desc_), *a.values(), None)


BAD = (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(hidden=0), dict(hidden=(1 << 20) + 1), dict(vocab=0),
       dict(vocab=(1 << 22) + 1), dict(x_stride=63), dict(w_stride=63), dict(dtype=2, dw_dtype=2), dict(dtype=3),
       dict(dw_dtype=0), dict(id_bytes=2), dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf),
       dict(scale=1e-9), dict(scale=-1e9))


def test_cross_entropy_refusals(L):
    need = ctypes.c_int64()
    for bad in BAD:
        refused(loss(L, desc(**bad)))
        refused(loss_back(L, desc(**bad)))
        refused(L.zero_linear_cross_entropy_workspace_bytes(ctypes.byref(desc(**bad)), None, 0, ctypes.byref(need)))
    refused(L.zero_linear_cross_entropy(None, *([AT["x"]] * 8), 1, None))
    for k in ("x", "w", "targets", "losses", "lse", "rows", "total", "ws"):
        refused(loss(L, **{k: None}))
    for k in ("x", "w", "targets", "lse", "rows", "d", "ws"):
        refused(loss_back(L, **{k: None}))
    for bad in (dict(x=AT["x"] + 1), dict(w=AT["w"] + 1), dict(targets=AT["targets"] + 4), dict(lse=AT["lse"] + 2),
                dict(ws=AT["ws"] + 128)):
        refused(loss(L, **bad), Z.ZERO_ERR_ALIGN)
        refused(loss_back(L, **bad), Z.ZERO_ERR_ALIGN)
    for bad in (-1, 3):
        refused(loss_back(L, reduction=bad))
    assert L.zero_linear_cross_entropy_workspace_bytes(ctypes.byref(desc()), AT["w"], 0, ctypes.byref(need)) == 0
    refused(loss(L, size=need.value - 1))
    forward = need.value
    assert L.zero_linear_cross_entropy_workspace_bytes(ctypes.byref(desc()), AT["w"], 1, ctypes.byref(need)) == 0
    refused(loss_back(L, size=need.value - 1))
    # a w whose rows bulk copies cannot take needs room for a copy, a binary32 dw for what rounding loses
    for d, w, more in ((desc(hidden=63), AT["w"], 0), (desc(w_stride=65), AT["w"], 0), (desc(), AT["w"] + 2, 0)):
        n = ctypes.c_int64()
        assert L.zero_linear_cross_entropy_workspace_bytes(ctypes.byref(d), w, 0, ctypes.byref(n)) == 0
        assert d.hidden == 63 or n.value > forward
    n = ctypes.c_int64()
    assert L.zero_linear_cross_entropy_workspace_bytes(ctypes.byref(desc(dw_dtype=2)), AT["w"], 1, ctypes.byref(n)) == 0
    assert n.value > need.value
    for out in ("losses", "lse", "rows", "total", "ws"):
        for of in ("x", "w", "targets"):
            refused(loss(L, **{out: AT[of]}), says=" overlaps ")
    refused(loss(L, losses=AT["x"] + 9 * 128 + 124), says="losses overlaps x")
    refused(loss(L, lse=AT["losses"] + 36), says="lse overlaps losses")
    for out in ("dx", "dw", "ws"):
        for of in ("x", "w", "targets", "lse", "rows", "d"):
            refused(loss_back(L, **{out: AT[of]}), says=" overlaps ")
    refused(loss_back(L, dx=AT["dw"] + 100 * 128 - 2), says="overlaps")
    assert loss_back(L, dx=None, dw=None) == 0   # nothing is wanted


def test_pieces_bound_the_workspace(L):
    """The logits' gradient takes half a GB at most, however many there are
    (or one tile's columns)."""
    need = ctypes.c_int64()
    for tokens, vocab in ((8192, 32000), (65536, 131072), (1 << 20, 1 << 20)):
        for dw in (1, 2):
            d = desc(tokens=tokens, vocab=vocab, dw_dtype=dw)
            assert L.zero_linear_cross_entropy_workspace_bytes(ctypes.byref(d), None, 1, ctypes.byref(need)) == 0
            rows = -(-tokens // 256) * 256
            others = rows * 64 * 2 + rows * 64 * 4 + 76 * 256 * 64 * 4 + rows * 12 + 4096
            assert need.value <= max(1 << 29, rows * 256 * 2 * dw) + others


# ---------------------------------------------------------------------------
# the binding


def test_host_tensors_and_wrong_arguments_are_refused(L):
    ids, t = torch.zeros(4, dtype=torch.int64), torch.zeros(5, 8)
    z = torch.zeros(4, 6)
    r = T.ExpertRoute(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(6, dtype=torch.int32),
                      torch.zeros(2), torch.zeros(5), True)
    h = torch.zeros(4, 8, dtype=torch.bfloat16)
    ce = T.CrossEntropy(torch.zeros(4), torch.zeros(4), torch.zeros(3), torch.zeros(5, dtype=torch.int32))
    for call in (lambda: T.zero_embedding(ids, t), lambda: T.zero_embedding_backward(t[:4], ids, 5),
                 lambda: T.zero_expert_route(z, 2), lambda: T.zero_expert_route_backward(z, r),
                 lambda: T.zero_linear_cross_entropy(h, h, ids),
                 lambda: T.zero_linear_cross_entropy_backward(h, h, ids, ce, torch.zeros(()))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: T.zero_embedding(None, t), lambda: T.zero_embedding(ids, 3),
                 lambda: T.zero_embedding(ids, t, dtype=torch.int32), lambda: T.zero_expert_route("z", 2),
                 lambda: T.zero_embedding_backward([1], ids, 5), lambda: T.zero_linear_cross_entropy(1, 2, 3),
                 lambda: T.zero_linear_cross_entropy_backward(h, h, ids, ce, h, dw_dtype=torch.int8)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        T.zero_linear_cross_entropy_backward(h, h, ids, ce, h, reduction="max")
    with pytest.raises(ValueError):
        T.zero_linear_cross_entropy_backward(h, h, ids, ce, h, want=("dz",))
    with pytest.raises(ValueError):
        T.linear_cross_entropy(h, h, ids, reduction="batchmean")


def test_public_names():
    import zero_sharded_optimizer_flatten_gb300 as P
    for name in ("embedding", "expert_route", "linear_cross_entropy", "zero_embedding", "zero_embedding_backward",
                 "zero_expert_route", "zero_expert_route_backward", "zero_linear_cross_entropy",
                 "zero_linear_cross_entropy_backward", "CrossEntropy", "ExpertRoute"):
        assert getattr(P, name) is getattr(T, name)


def test_calls_on_a_given_stream_make_their_buffers_there(monkeypatch):
    class Stream:
        pass

    class Made:
        def __init__(self):
            self.made_on, self.streams = current[-1], []

        def record_stream(self, stream):
            self.streams.append(stream)

    class Use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *error):
            current.pop()

    caller, side = Stream(), Stream()
    current = [caller]

    def make(n):
        return lambda *a: tuple(Made() for _ in range(n)) if n > 1 else Made()

    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(T, "_fast", types.SimpleNamespace(
        embedding=make(1), embedding_backward=make(1), expert_route=make(5), expert_route_backward=make(1),
        linear_cross_entropy=make(4), linear_cross_entropy_backward=make(2)))
    x = torch.ones(4, 8)

    def outputs(stream):
        r = T.zero_expert_route(x, 2, stream=stream)
        ce = T.zero_linear_cross_entropy(x, x, x, stream=stream)
        return [T.zero_embedding(x, x, stream=stream), T.zero_embedding_backward(x, x, 3, stream=stream), r.ids,
                r.weights, r.counts, r.losses, r.stats, T.zero_expert_route_backward(x, r, stream=stream), ce.losses,
                ce.lse, ce.total, ce.rows, *T.zero_linear_cross_entropy_backward(x, x, x, ce, x, stream=stream)]

    for t in outputs(side):
        assert t.made_on is side and caller in t.streams and side in t.streams
    for t in outputs(None):
        assert t.made_on is caller and t.streams == []
