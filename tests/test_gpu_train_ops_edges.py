"""Edges of the block join's and the experts' C calls: no rows, storage that
ends with the last row that is read, outputs in place of inputs, and rows that
the kernels for long rows take."""
import ctypes
import gc

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z
from zero_sharded_optimizer_flatten_gb300 import train_ops as T

from .test_gpu_train_ops import check_join, join_inputs

pytestmark = pytest.mark.gpu

H16, B16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _cuda_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_parameter_gradients_of_no_rows_are_zero_whatever_the_gate_holds(kind):
    layer = kind == "layer"
    for gate_value in (1.0, float("inf"), float("nan")):
        x = torch.empty(0, 64, device="cuda", dtype=B16)
        w, gate = torch.full((64,), float("nan"), device="cuda"), torch.full((64,), gate_value, device="cuda")
        bias = w if layer else None
        g = Z.zero_block_join_backward(x, x, x, x, None, w_post=w, bias_post=bias, w_pre=w,
                                       bias_pre=bias, gate=gate, kind=kind, scale=-2.0)
        for k in ("dgate", "dw_post", "dbias_post", "dw_pre", "dbias_pre"):
            if g[k] is not None:
                assert g[k].shape == (64,) and bool((g[k] == 0).all()), k


def test_no_rows_need_no_inputs():
    """The C call takes NULL for every input when there are no rows, a channel
    gate among them."""
    lib = Z.lib()
    d = T.JoinDescC(rows=0, hidden=64, act_dtype=1, res_dtype=1, param_dtype=2, gate_dtype=2, kind=1,
                    gate_kind=1, eps=1e-6, scale=0.5, x_stride=64, b_stride=64, gate_stride=64,
                    do_stride=64, dn_stride=64)
    out = torch.full((5, 64), 7.0, device="cuda")
    need = ctypes.c_int64()
    assert lib.zero_block_join_workspace_bytes(ctypes.byref(d), ctypes.byref(need)) == 0
    ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    g = T.JoinGradsC(dgate=out[0].data_ptr(), dw_post=out[1].data_ptr(), dbias_post=out[2].data_ptr(),
                     dw_pre=out[3].data_ptr(), dbias_pre=out[4].data_ptr())
    p = T.JoinInputsC()
    torch.cuda.synchronize()
    assert lib.zero_block_join_backward(ctypes.byref(d), ctypes.byref(p), None, None, None,
                                        ctypes.byref(g), ws.data_ptr(), need.value, None) == 0
    torch.cuda.synchronize()
    assert not out.any()


def join_case(R, H, act, res, par, gate, post, pre, layer, seed=1, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def t(*shape, dtype, scale, shift=0.0):
        wide = torch.randn(*shape[:-1], shape[-1] + (pad if len(shape) == 2 and shape[1] > 1 else 0),
                           device="cuda", generator=g)
        return (wide * scale + shift).to(dtype)[..., :shape[-1]]

    shape = {"none": None, "channel": (H,), "row": (R, 1), "full": (R, H)}[gate]
    params = dict(gate=None if shape is None else t(*shape, dtype=act, scale=0.3, shift=0.5))
    for k, there in (("w_post", post), ("w_pre", pre), ("bias_post", post and layer),
                     ("bias_pre", pre and layer)):
        params[k] = t(H, dtype=par, scale=0.1, shift=float(k[0] == "w")) if there else None
    return t(R, H, dtype=res, scale=2.0), t(R, H, dtype=act, scale=0.5, shift=0.1), params


def c_backward(x, b, d_o, d_n, stats, dx, db, kind, **params):
    """zero_block_join_backward with the caller's own dx and db."""
    code = {H16: 0, B16: 1, F32: 2}
    R, H = x.shape
    first = next((t for k, t in params.items() if k != "gate" and t is not None), None)
    gate = params["gate"]
    kinds = {None: 0, (H,): 1, (R, 1): 2, (R, H): 3}
    d = T.JoinDescC(rows=R, hidden=H, act_dtype=code[b.dtype], res_dtype=code[x.dtype],
                    param_dtype=code[b.dtype if first is None else first.dtype],
                    gate_dtype=code[b.dtype if gate is None else gate.dtype],
                    kind=int(kind == "layer"), gate_kind=kinds[None if gate is None else tuple(gate.shape)],
                    eps=1e-6, scale=0.7, x_stride=H, b_stride=H,
                    gate_stride=1 if gate is not None and gate.shape[-1] == 1 else H, do_stride=H,
                    dn_stride=H)
    p = T.JoinInputsC(x=x.data_ptr(), b=b.data_ptr(),
                      **{k: None if t is None else t.data_ptr() for k, t in params.items()})
    g = T.JoinGradsC(dx=dx.data_ptr(), db=db.data_ptr())
    return Z.lib().zero_block_join_backward(
        ctypes.byref(d), ctypes.byref(p), d_o.data_ptr(), d_n.data_ptr(), stats.data_ptr(),
        ctypes.byref(g), None, 0, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["channel", "row", "full"])
@pytest.mark.parametrize("act,res", [(B16, B16), (H16, F32), (F32, F32)], ids=lambda t: str(t)[6:])
def test_join_gradients_in_place(act, res, kind, gate):
    """dx over d_o and db over d_n, in every kernel: short rows, several warps,
    rows that start anywhere, rows above 8192."""
    for R, H in ((700, 96), (300, 1024), (200, 333), (40, 4096), (30, 8200), (9, 8203)):
        x, b, params = join_case(R, H, act, res, act, gate, True, True, kind == "layer")
        d_o, d_n = torch.randn_like(x), torch.randn_like(b)
        _, _, stats = Z.zero_block_join(x, b, want_stats=True, kind=kind, scale=0.7, **params)
        want = Z.zero_block_join_backward(x, b, d_o, d_n, stats, kind=kind, scale=0.7, want={"dx", "db"},
                                          **params)
        dx, db = d_o.clone(), d_n.clone()
        assert c_backward(x, b, dx, db, stats, dx, db, kind, **params) == 0, Z.zero_last_error()
        assert torch.equal(dx, want["dx"]) and torch.equal(db, want["db"]), (R, H)


def test_outputs_between_the_rows_of_an_input():
    """Memory between an input's rows is no part of it."""
    big = torch.randn(2, 40, 64, device="cuda").bfloat16()
    x, room = big[:, 0], big[0, 10:12]      # rows 0 and 40 of 64; o lies in rows 10 and 11
    b, w = torch.randn_like(room), torch.ones(64, device="cuda", dtype=B16)
    want, n, _ = Z.zero_block_join(x.contiguous(), b, w_pre=w)
    got = Z.zero_block_join(x, b, w_pre=w, o=room)
    assert torch.equal(got[0], want) and torch.equal(got[1], n) and torch.equal(room, want)
    ids = torch.tensor([[0], [1]], device="cuda", dtype=torch.int32)
    order = Z.zero_expert_sort(ids, 2)
    xs = Z.zero_expert_dispatch(x, order, out=big[0, 20:22])
    assert torch.equal(xs, x)
    with pytest.raises(Z.ZeroError, match="xs overlaps x"):
        Z.zero_expert_dispatch(x, order, out=big.view(-1, 64)[39:41])
    with pytest.raises(Z.ZeroError, match="o overlaps x"):
        Z.zero_block_join(x, b, w_pre=w, o=big.view(-1, 64)[40:42])


def test_errors_name_what_is_wrong():
    x = torch.ones(4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    with pytest.raises(ValueError, match=r"o: expected a contiguous Float tensor of shape \(4, 16, \), "
                                         r"got Half \(4, 16, \)"):
        Z.zero_block_join(x, x, w_pre=w, o=x.half())
    with pytest.raises(ValueError, match="stats: .*got Float .*not contiguous"):
        Z.zero_block_join_backward(x, x, x, None, torch.ones(4, 4, device="cuda").t())
    with pytest.raises(TypeError, match="w_pre: expected float16, bfloat16 or float32"):
        Z.zero_block_join(x, w_pre=w.double())
    with pytest.raises(TypeError, match="d_n: expected float16, bfloat16 or float32"):
        Z.zero_block_join_backward(x, None, None, x.double(), None, w_pre=w)
    with pytest.raises(RuntimeError, match="ambiguous"):   # torch's own, not a SystemError about it
        Z.zero_block_join(x, x, w_pre=w, want_o=torch.ones(2))
    with pytest.raises(RuntimeError, match="ambiguous"):
        Z.zero_block_join(x, x, w_pre=w, want_stats=torch.ones(2))


# Rows above 8192 channels, and those below of which no copy fits in shared
# memory, go element by element.  The sizes stay within 8200, up to which the
# tolerances of check_join are derived.

TYPES = [(H16, H16, H16), (B16, B16, F32), (B16, F32, B16), (H16, F32, F32), (F32, F32, F32)]


@pytest.mark.parametrize("act,res,par", TYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
def test_long_rows_of_every_kind(act, res, par, kind, gate):
    for post, pre in ((True, True), (True, False), (False, True), (False, False)):
        for R, H in ((5, 8200), (3, 8195)):
            check_join(join_inputs(R, H, act, res, par, gate, post, pre, kind == "layer", R * H + post),
                       kind, eps=1e-3)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_long_rows_with_one_gradient_strides_and_no_block(kind):
    layer = kind == "layer"
    for use_o, use_n in ((True, False), (False, True)):
        for gate in ("row", "full"):
            check_join(join_inputs(4, 8200, B16, B16, F32, gate, True, True, layer, 3), kind, eps=1e-3,
                       use_o=use_o, use_n=use_n)
    for pad in (1, 8):
        check_join(join_inputs(6, 8200, B16, F32, F32, "full", True, True, layer, pad, pad=pad), kind,
                   eps=1e-3)
        check_join(join_inputs(6, 8195, H16, H16, H16, "row", True, True, layer, pad, pad=pad), kind,
                   eps=1e-3)
    check_join(join_inputs(4, 8200, B16, B16, B16, "none", False, True, layer, 5, b=False), kind, eps=1e-3)


def test_long_rows_more_than_there_are_ctas():
    check_join(join_inputs(2500, 8200, B16, B16, B16, "row", True, True, True, 7), "layer", eps=1e-3)


def test_long_rows_in_place_and_on_zeros():
    for H in (8200, 8195):
        for gate in ("channel", "row", "full"):
            v = join_inputs(12, H, B16, B16, B16, gate, True, True, False, 8)
            params = {k: t for k, t in v.items() if k not in ("x", "b")}
            o, n, _ = Z.zero_block_join(v["x"], v["b"], **params)
            x, b = v["x"].clone(), v["b"].clone()
            Z.zero_block_join(x, b, o=x, n=b, **params)
            assert torch.equal(x, o) and torch.equal(b, n)
    x = torch.zeros(2, 8200, device="cuda")
    w = torch.ones(8200, device="cuda")
    for kind in ("rms", "layer"):
        o, n, _ = Z.zero_block_join(x, x, w_post=w, w_pre=w, kind=kind)
        assert not o.any() and not n.any()


@pytest.mark.parametrize("H", [6660, 6664, 7684, 7688, 8192])
def test_rows_that_leave_no_room_for_their_copies(H):
    """fp32 layer norms with a full gate: forward from 7688 channels, backward
    from 6664."""
    for gate in ("full", "none"):
        check_join(join_inputs(7, H, F32, F32, F32, gate, True, True, True, H), "layer", eps=1e-3)
    check_join(join_inputs(7, H, F32, F32, F32, "full", True, True, False, H), "rms", eps=1e-3)
    v = join_inputs(7, H, B16, F32, F32, "full", True, True, True, H)
    v["gate"] = v["gate"].float()
    check_join(v, "layer", eps=1e-3)
