"""Edges of the block join's and the experts' C calls: no rows, storage that
ends with the last row that is read, outputs in place of inputs, and rows that
the kernels for long rows take."""
import ctypes
import gc

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z
from zero_sharded_optimizer_flatten_gb300 import train_ops as T

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
