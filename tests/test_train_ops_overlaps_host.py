"""Outputs of the block join and of the experts' calls that overlap an input or
another output are refused before a device is touched (no GPU needed)."""
import ctypes

import pytest

from zero_sharded_optimizer_flatten_gb300 import _build
from zero_sharded_optimizer_flatten_gb300 import train_ops as T
from zero_sharded_optimizer_flatten_gb300 import zero as Z

# addresses that are never read, 1 MB apart
AT = {k: 0x10000000 + (i << 20) for i, k in enumerate(
    ("x", "b", "gate", "w_post", "w_pre", "o", "n", "stats", "d_o", "d_n", "dx", "db", "dgate",
     "dw_post", "dw_pre", "ws", "ids", "offsets", "rows", "pairs", "xs", "weights", "dweights"))}
R, H = 4, 64
ROW = 2 * H   # bytes


@pytest.fixture(scope="module")
def L():
    _build.build()
    return Z.lib()


def overlap(status, out):
    assert status == Z.ZERO_ERR_INVALID and f": {out} overlaps " in Z.zero_last_error(), \
        (status, Z.zero_last_error())


def arguments(**changes):
    d = T.JoinDescC(rows=R, hidden=H, act_dtype=1, res_dtype=1, param_dtype=1, gate_dtype=1, kind=0,
                    gate_kind=3, eps=1e-6, scale=1.0, x_stride=H, b_stride=H, gate_stride=H,
                    do_stride=H, dn_stride=H)
    p = T.JoinInputsC(**{k: AT[k] for k in ("x", "b", "gate", "w_post", "w_pre")})
    for name, value in changes.items():
        setattr(d if name in dict(T.JoinDescC._fields_) else p, name, value)
    return ctypes.byref(d), ctypes.byref(p)


def test_join(L):
    def forward(out, at, **changes):
        places = {k: AT[k] for k in ("o", "n", "stats")} | {out: at}
        overlap(L.zero_block_join(*arguments(**changes), places["o"], places["n"], places["stats"],
                                  None), "stats" if (out, at) == ("n", AT["stats"]) else out)

    before = Z.zero_launch_count()
    for out in ("o", "n"):
        for of in ("w_post", "w_pre", "gate"):
            forward(out, AT[of])
        forward(out, AT["x"] + 2 * ROW)             # from the middle on
        forward(out, AT["b"] - 2 * ROW)             # up to the middle
        forward(out, AT["x"] + R * ROW - 2)         # the last element
        forward(out, AT["b"] - R * ROW + 2)         # the first element
    forward("o", AT["b"])
    forward("n", AT["x"])
    forward("o", AT["x"], x_stride=2 * H)           # in place, but the rows are apart
    forward("n", AT["b"], b_stride=H + 8)
    forward("o", AT["x"] + 2 * ROW, x_stride=2 * H)
    forward("o", AT["gate"] + 3 * 1000, gate_kind=2, gate_stride=1500)   # row gates, one number each
    forward("n", AT["o"])
    forward("n", AT["stats"])
    forward("stats", AT["o"] + R * ROW - 16)

    need = ctypes.c_int64()
    assert L.zero_block_join_workspace_bytes(arguments()[0], ctypes.byref(need)) == 0

    def backward(out, at, names=None, **changes):
        names = names or out
        places = {k: AT[k] for k in ("dx", "db", "dgate", "dw_post", "dw_pre", "ws")} | {out: at}
        g = T.JoinGradsC(**{k: v for k, v in places.items() if k != "ws"})
        overlap(L.zero_block_join_backward(*arguments(**changes), AT["d_o"], AT["d_n"], AT["stats"],
                                           ctypes.byref(g), places["ws"], need.value, None), names)

    for out in ("dx", "db", "dgate", "dw_post", "dw_pre"):
        for of in ("x", "b", "gate", "w_post", "w_pre", "d_o", "d_n", "stats"):
            if (out, of) not in (("dx", "d_o"), ("db", "d_n")):
                backward(out, AT[of])
    backward("dx", AT["d_o"], do_stride=H + 8)
    backward("db", AT["d_n"], dn_stride=2 * H)
    backward("db", AT["dx"])
    backward("dw_pre", AT["dw_post"] + ROW - 2)
    backward("ws", AT["d_o"], "workspace")
    backward("ws", AT["dw_pre"] - 16, "workspace")
    assert Z.zero_launch_count() == before


def test_experts(L):
    before = Z.zero_launch_count()
    tokens, topk, hidden, experts = 10, 2, 64, 4

    def at(out, place, *names):
        return [place if k == out else AT[k] for k in names]

    def sort(out, place, named=None):
        ids, offsets, rows, pairs = at(out, place, "ids", "offsets", "rows", "pairs")
        overlap(L.zero_expert_sort(ids, 4, tokens, topk, experts, offsets, rows, pairs, None, 0, None),
                named or out)

    for out in ("offsets", "rows", "pairs"):
        sort(out, AT["ids"])
        sort(out, AT["ids"] + 4 * (tokens * topk - 1))
    sort("rows", AT["offsets"] + 4 * experts)
    sort("pairs", AT["rows"] + 4)

    for place in (AT["x"], AT["x"] + 2 * (9 * 100 + 63), AT["rows"], AT["offsets"] + 4 * experts):
        overlap(L.zero_expert_dispatch(AT["x"], 100, 1, tokens, topk, hidden, AT["offsets"], experts,
                                       AT["rows"], place, None), "xs")
    for place in (AT["xs"], AT["rows"] + 4, AT["xs"] - 2 * tokens * hidden + 2):
        overlap(L.zero_expert_dispatch_backward(AT["xs"], 1, tokens, topk, hidden, AT["rows"], place,
                                                None), "dx")
    for place in (AT["xs"], AT["rows"], AT["weights"] + 4):
        overlap(L.zero_expert_combine(AT["xs"], 1, AT["weights"], 2, tokens, topk, hidden, AT["rows"],
                                      place, None), "y")

    def backward(dys, dweights, named):
        overlap(L.zero_expert_combine_backward(AT["d_o"], hidden, AT["xs"], 1, AT["weights"], 2, tokens,
                                               topk, hidden, AT["offsets"], experts, AT["rows"], dys,
                                               dweights, None), named)

    for place in (AT["d_o"], AT["xs"], AT["weights"], AT["rows"], AT["offsets"]):
        backward(place, AT["dweights"], "dys")
        backward(AT["dx"], place, "dweights")
    backward(AT["dx"], AT["dx"] + 4, "dweights")
    assert Z.zero_launch_count() == before
