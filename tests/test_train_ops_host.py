"""Host side of the training-step operators (no GPU needed): the C calls
refuse bad arguments with the documented status before they touch a device,
and the binding's checks of tensor lists."""
import ctypes

import pytest
import torch

from zero_sharded_optimizer_flatten_gb300 import _build
from zero_sharded_optimizer_flatten_gb300 import train_ops as T
from zero_sharded_optimizer_flatten_gb300 import zero as Z

P = 0x10000   # an address that is never read


@pytest.fixture(scope="module")
def L():
    _build.build()
    return Z.lib()


def refused(status, want=Z.ZERO_ERR_INVALID):
    assert status == want, (status, Z.zero_last_error())
    assert Z.zero_last_error()


def tensors(**changes):
    t = (T.GradTensorC * 2)()
    for k in range(2):
        t[k].src, t[k].dst, t[k].numel = P + 4096 * k, P + 65536 + 4096 * k, 100
        t[k].src_dtype = t[k].dst_dtype = 2
    for name, value in changes.items():
        setattr(t[1], name, value)
    return t


def test_grad_norm_refusals(L):
    need = ctypes.c_int64()
    assert L.zero_grad_norm_workspace_bytes(tensors(), 2, ctypes.byref(need)) == 0
    n = need.value
    assert n > 0

    def clip(t, count=2, kind=0, max_norm=1.0, result=P, ws=P, size=n):
        return L.zero_clip_grad_norm(t, count, kind, max_norm, result, ws, size, None)

    before = Z.zero_launch_count()
    refused(clip(tensors(), count=-1))
    refused(clip(None))
    refused(clip(tensors(), kind=2))
    for bad in (-1.0, float("nan"), float("inf")):
        refused(clip(tensors(), max_norm=bad))
    refused(clip(tensors(numel=-1)))
    refused(clip(tensors(numel=(1 << 40) + 1)))
    refused(clip(tensors(src_dtype=3)))
    refused(clip(tensors(dst_dtype=-1)))
    refused(clip(tensors(src=None)))
    refused(clip(tensors(dst=None)))
    refused(clip(tensors(src=P + 1)), Z.ZERO_ERR_ALIGN)
    refused(clip(tensors(dst=P + 65536 + 4098)), Z.ZERO_ERR_ALIGN)
    refused(clip(tensors(dst=P + 4096, dst_dtype=1)))   # in place, another type
    refused(clip(tensors(), result=None))
    refused(clip(tensors(), ws=None))
    refused(clip(tensors(), ws=P + 8), Z.ZERO_ERR_ALIGN)
    refused(clip(tensors(), size=n - 1))
    refused(L.zero_grad_norm(tensors(src=None), 2, 0, P, P, n, None))
    refused(L.zero_grad_norm_workspace_bytes(tensors(), 2, None))
    assert Z.zero_launch_count() == before


def join(**changes):
    d = T.JoinDescC(rows=4, hidden=64, act_dtype=1, res_dtype=1, param_dtype=1, gate_dtype=1,
                    kind=0, gate_kind=0, eps=1e-6, scale=1.0, x_stride=64, b_stride=64,
                    gate_stride=64, do_stride=64, dn_stride=64)
    p = T.JoinInputsC(x=P, b=P, w_post=P, w_pre=P)
    for name, value in changes.items():
        setattr(d if name in dict(T.JoinDescC._fields_) else p, name, value)
    return d, p


def test_join_refusals(L):
    def forward(o=P, n=P, stats=P, **changes):
        d, p = join(**changes)
        return L.zero_block_join(ctypes.byref(d), ctypes.byref(p), o, n, stats, None)

    before = Z.zero_launch_count()
    for bad in (dict(rows=-1), dict(hidden=0), dict(hidden=1 << 31), dict(act_dtype=3),
                dict(res_dtype=0), dict(param_dtype=0), dict(kind=2), dict(gate_kind=4),
                dict(gate_kind=1), dict(gate_kind=1, gate=P, gate_dtype=0), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=1e-60), dict(eps=float("nan")), dict(scale=float("inf")),
                dict(x=None), dict(gate=P), dict(b=None), dict(bias_pre=P),
                dict(kind=1, bias_post=P, w_post=None), dict(x_stride=63), dict(b_stride=0),
                dict(gate_kind=3, gate=P, gate_stride=10), dict(o=None, n=None), dict(w_pre=None)):
        refused(forward(**bad))
    for bad in (dict(x=P + 1), dict(b=P + 1), dict(w_pre=P + 1), dict(o=P + 1), dict(n=P + 1),
                dict(stats=P + 8)):
        refused(forward(**bad), Z.ZERO_ERR_ALIGN)
    refused(L.zero_block_join(None, None, P, P, P, None))

    d, p = join()
    need = ctypes.c_int64()
    assert L.zero_block_join_workspace_bytes(ctypes.byref(d), ctypes.byref(need)) == 0

    def backward(do=P, dn=P, stats=P, ws=P, size=need.value, grads=None, **changes):
        d, p = join(**changes)
        g = T.JoinGradsC(dx=P, db=P, dw_post=P, dw_pre=P)
        for name, value in (grads or {}).items():
            setattr(g, name, value)
        return L.zero_block_join_backward(ctypes.byref(d), ctypes.byref(p), do, dn, stats,
                                          ctypes.byref(g), ws, size, None)

    for bad in (dict(do=None, dn=None), dict(stats=None), dict(w_pre=None), dict(ws=None),
                dict(size=need.value // 1000), dict(grads=dict(dgate=P)),
                dict(grads=dict(dbias_pre=P)), dict(w_post=None), dict(do_stride=1),
                dict(dn_stride=1), dict(dn=None),
                dict(b=None, w_post=None, grads=dict(dw_post=None))):
        refused(backward(**bad))
    refused(backward(grads=dict(dx=P + 1)), Z.ZERO_ERR_ALIGN)
    refused(backward(ws=P + 8), Z.ZERO_ERR_ALIGN)
    refused(L.zero_block_join_backward(ctypes.byref(d), ctypes.byref(p), P, P, P, None, P, 1 << 30,
                                       None))
    assert Z.zero_launch_count() == before


def test_expert_refusals(L):
    before = Z.zero_launch_count()

    def sort(ids=P, width=4, tokens=10, topk=2, n=4, offsets=P, rows=P, pairs=P, ws=None, size=0):
        return L.zero_expert_sort(ids, width, tokens, topk, n, offsets, rows, pairs, ws, size, None)

    for bad in (dict(ids=None), dict(width=2), dict(tokens=-1), dict(topk=0), dict(n=0),
                dict(n=4097), dict(offsets=None), dict(rows=None), dict(pairs=None),
                dict(tokens=1 << 30, topk=4), dict(tokens=100_000)):
        refused(sort(**bad))
    refused(sort(ids=P + 4, width=8), Z.ZERO_ERR_ALIGN)
    refused(sort(tokens=100_000, ws=P, size=16))
    need = ctypes.c_int64()
    assert L.zero_expert_sort_workspace_bytes(100, 2, 4, ctypes.byref(need)) == 0
    assert need.value == 0
    assert L.zero_expert_sort_workspace_bytes(100_000, 2, 4, ctypes.byref(need)) == 0
    assert need.value > 0
    refused(L.zero_expert_sort_workspace_bytes(100, 2, 0, ctypes.byref(need)))
    for bad in ((None, 64, 1, 10, 2, 64, P, 4, P, P), (P, 63, 1, 10, 2, 64, P, 4, P, P),
                (P, 64, 3, 10, 2, 64, P, 4, P, P), (P, 64, 1, -1, 2, 64, P, 4, P, P),
                (P, 64, 1, 10, 2, 0, P, 4, P, P), (P, 64, 1, 10, 2, 64, None, 4, P, P),
                (P, 64, 1, 10, 2, 64, P, 0, P, P), (P, 64, 1, 10, 2, 64, P, 4, None, P),
                (P, 64, 1, 10, 2, 64, P, 4, P, None)):
        refused(L.zero_expert_dispatch(*bad, None))
    refused(L.zero_expert_dispatch(P + 1, 64, 1, 10, 2, 64, P, 4, P, P, None), Z.ZERO_ERR_ALIGN)
    for bad in ((None, 1, 10, 2, 64, P, P), (P, 1, 10, 2, 64, None, P), (P, 1, 10, 2, 64, P, None),
                (P, 5, 10, 2, 64, P, P)):
        refused(L.zero_expert_dispatch_backward(*bad, None))
    for bad in ((None, 1, P, 2, 10, 2, 64, P, P), (P, 1, None, 2, 10, 2, 64, P, P),
                (P, 1, P, 0, 10, 2, 64, P, P), (P, 1, P, 2, 10, 2, 64, P, None)):
        refused(L.zero_expert_combine(*bad, None))
    for bad in ((P, 64, None, 1, P, 2, 10, 2, 64, P, 4, P, P, P),
                (P, 60, P, 1, P, 2, 10, 2, 64, P, 4, P, P, P),
                (P, 64, P, 1, P, 0, 10, 2, 64, P, 4, P, P, P),
                (P, 64, P, 1, P, 2, 10, 2, 64, P, 4, P, None, P)):
        refused(L.zero_expert_combine_backward(*bad, None))
    assert Z.zero_launch_count() == before


def test_nothing_to_do_launches_nothing(L):
    before = Z.zero_launch_count()
    d, p = join(rows=0)
    assert L.zero_block_join(ctypes.byref(d), ctypes.byref(p), P, P, P, None) == 0
    assert L.zero_expert_dispatch(None, 64, 1, 0, 2, 64, None, 4, None, None, None) == 0
    assert L.zero_expert_combine(None, 1, None, 2, 0, 2, 64, None, None, None) == 0
    assert Z.zero_launch_count() == before


def test_disjoint():
    T._check_disjoint([])
    T._check_disjoint([(0, 10, True), (10, 20, True), (20, 30, False), (25, 40, False)])
    for bad in ([(0, 10, True), (9, 20, True)], [(0, 10, True), (5, 6, False)],
                [(0, 100, False), (50, 60, True)], [(0, 10, True), (0, 10, True)],
                [(0, 100, False), (10, 20, False), (30, 40, True)]):
        with pytest.raises(ValueError):
            T._check_disjoint(bad)


def test_dense():
    t = torch.zeros(4, 6, 8)
    for ok in (t, t.permute(2, 0, 1), t[1], t[:, :1][:, 0].reshape(-1), torch.zeros(()),
               torch.zeros(5, 1)[:, 0], t.transpose(0, 1)):
        assert T._dense(ok)
    for bad in (t[:, 1:3], t[..., ::2], torch.zeros(3).expand(4, 3)):
        assert not T._dense(bad)


def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 8)
    for call in (lambda: T.zero_block_join(x, x), lambda: T.zero_grad_norm([x]),
                 lambda: T.zero_expert_sort(torch.zeros(4, 2, dtype=torch.int32), 3)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        T.zero_grad_norm([1.0])


def test_compiled_binding_refuses_before_it_launches():
    import torch
    x, w = torch.ones(2, 8), torch.ones(8)
    order = T.ExpertOrder(torch.zeros(3, dtype=torch.int32), torch.zeros(2, 1, dtype=torch.int32),
                          torch.zeros(2, dtype=torch.int32), 2, 2, 1)
    for call in (lambda: T.zero_block_join(x, w_pre=w), lambda: T.zero_expert_sort(order.rows, 2),
                 lambda: T.zero_block_join_backward(x, x, x, None, None),
                 lambda: T.zero_expert_dispatch(x, order),
                 lambda: T.zero_expert_combine(x, torch.ones(2, 1), order),
                 lambda: T.zero_expert_dispatch_backward(x, order),
                 lambda: T.zero_expert_combine_backward(x, x, torch.ones(2, 1), order)):
        with pytest.raises(ValueError):    # host tensors
            call()
    for call in (lambda: T.zero_block_join(None), lambda: T.zero_block_join([1.0], w_pre=w),
                 lambda: T.zero_expert_dispatch(3, order),
                 lambda: T.zero_expert_combine(None, None, order)):
        with pytest.raises(TypeError):
            call()
