"""The cross entropy's calls with the others' probability between them refuse
bad arguments with the documented status, without a GPU; its workspace."""
import ctypes

import pytest

from tests.test_more_ops_host import AT, L, desc, refused  # noqa: F401  (L: the library's fixture)
from zero_sharded_optimizer_flatten_gb300 import zero as Z

REST = 0x7000000000


def loss(L, d=None, **c):
    a = dict(x=AT["x"], w=AT["w"], targets=AT["targets"], losses=AT["losses"], lse=AT["lse"], rest=REST,
             rows=AT["rows"], total=AT["total"], ws=AT["ws"], size=1 << 30) | c
    return L.zero_linear_cross_entropy_rest(ctypes.byref(desc() if d is None else d), *a.values(), None)


def loss_back(L, d=None, **c):
    a = dict(x=AT["x"], w=AT["w"], targets=AT["targets"], lse=AT["lse"], rest=REST, rows=AT["rows"], d=AT["d"],
             reduction=2, dx=AT["dx"], dw=AT["dw"], ws=AT["ws"], size=1 << 40) | c
    return L.zero_linear_cross_entropy_rest_backward(ctypes.byref(desc() if d is None else d), *a.values(), None)


@pytest.fixture(autouse=True)
def _launches_nothing(L):  # noqa: F811
    before = Z.zero_launch_count()
    yield
    assert Z.zero_launch_count() == before


def test_refusals(L):  # noqa: F811
    for call in (loss, loss_back):
        refused(call(L, rest=None), says="rest is NULL")
        refused(call(L, rest=REST + 2), Z.ZERO_ERR_ALIGN)
        for bad in (dict(tokens=-1), dict(hidden=0), dict(scale=0.0)):
            refused(call(L, desc(**bad)))
        for k in ("x", "w", "targets", "lse", "rows", "ws"):
            refused(call(L, **{k: None}))
    for of in ("x", "w", "targets", "lse", "losses", "rows"):
        refused(loss(L, rest=AT[of]), says=" overlaps ")
    for out in ("dx", "dw", "ws"):
        refused(loss_back(L, **{out: REST & ~255}), says=f"{'workspace' if out == 'ws' else out} overlaps rest")
    assert loss_back(L, dx=None, dw=None) == 0   # nothing is wanted


def test_a_copy_of_w_is_in_the_workspace_where_rows_need_one(L):  # noqa: F811
    """w whose rows bulk copies cannot take needs room for a copy: rows off
    16-byte boundaries do, rows of 63 channels 64 apart do not."""
    n = ctypes.c_int64()

    def size(d, w):
        assert L.zero_linear_cross_entropy_workspace_bytes(ctypes.byref(d), w, 0, ctypes.byref(n)) == 0
        return n.value
    plain = size(desc(), AT["w"])
    assert size(desc(hidden=63, w_stride=64), AT["w"]) == plain
    for d, w in ((desc(hidden=63, w_stride=63), AT["w"]), (desc(w_stride=65), AT["w"]), (desc(), AT["w"] + 2)):
        assert size(d, w) >= plain + 100 * 64 * 2


def parts(pairs, tokens, hidden, columns):
    """Rows of dx's sums that the products write: k_loss_product's split of the sum over the vocabulary."""
    most = 0
    n_tiles, blocks = -(-hidden // 256), -(-columns // 256)
    for rows in range(1, -(-tokens // 256) + 1):
        tiles = rows * n_tiles
        splits = 1 if 2 * tiles > pairs else min(pairs // tiles, blocks)
        if splits > 1:
            most = max(most, splits * rows * 256)
    return most


def test_the_gradients_workspace_follows_what_is_summed_in_parts(L):  # noqa: F811
    """Eight tokens take tens of MB, not hundreds; what any number of pairs up to
    76 writes has its place."""
    n = ctypes.c_int64()

    def size(d):
        assert L.zero_linear_cross_entropy_workspace_bytes(ctypes.byref(d), AT["w"], 1, ctypes.byref(n)) == 0
        return n.value
    for hidden in (4096, 8192):
        d = desc(tokens=8, hidden=hidden, vocab=32000, x_stride=hidden, w_stride=hidden)
        assert size(d) <= 256 * 32000 * 2 + 256 * hidden * 2 + 76 * 256 * 256 * 4 + 65536
    big = desc(tokens=8192, hidden=4096, vocab=32000, x_stride=4096, w_stride=4096)
    assert size(big) <= (512 << 20) + 8192 * 4096 * 2 + 76 * 256 * 256 * 4 + (1 << 20)
    for tokens in (1, 200, 300, 1000, 5000, 40000):
        for hidden in (8, 256, 264, 1024, 4096, 9728, 9736, 20000):
            for vocab in (300, 5003, 32000):
                d = desc(tokens=tokens, hidden=hidden, vocab=vocab, x_stride=hidden, w_stride=hidden)
                rows = -(-tokens // 256) * 256
                columns = min(-(-vocab // 256) * 256, max(256, (256 << 20) // rows // 256 * 256))
                need = max(parts(pairs, tokens, hidden, columns) for pairs in (1, 2, 3, 37, 70, 75, 76))
                if columns < vocab:
                    need = max(need, rows)
                assert size(d) >= need * hidden * 4 + rows * columns * 2 + rows * hidden * 2
