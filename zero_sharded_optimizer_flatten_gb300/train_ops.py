"""Operators of a training step around the sharded optimizer: gradient norm
and clipping over many tensors, the block join, the expert permutation.

The ``zero_*`` functions bind the C calls of include/zero.h under their own
names (argument checks and marshalling only; the current CUDA stream unless
``stream`` is given; no fallback).  ``GradNorm`` and ``ClipGradNorm`` are the
prepared forms for gradients whose buffers stay in place from step to step.
``block_join``, ``expert_dispatch`` and ``expert_combine`` are the same calls
with autograd.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools

import torch

from . import zero as _zero
from .zero import _check

ZERO_FP32 = 2
_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: ZERO_FP32}
_NORMS = {"l2": 0, "inf": 1}
_KINDS = {"rms": 0, "layer": 1}
GATE_NONE, GATE_CHANNEL, GATE_ROW, GATE_FULL = range(4)


def _type(t, what: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: expected float16, bfloat16 or float32, got {t.dtype}")
    return code


def _choice(table, value, what: str) -> int:
    if value not in table:
        raise ValueError(f"{what} must be one of {sorted(table)}, got {value!r}")
    return table[value]


_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_lib = None


def _load():
    """The library, kept here after the first call (these calls are made many
    times a step: what they do on the host shows beside small kernels)."""
    global _lib
    _lib = _zero.lib()
    return _lib


def _stream(stream, device: int):
    """Handle of the given stream, or of the device's current one."""
    return _raw_stream(device) if stream is None else _zero._stream(stream)


def _on(t, what: str, device: int):
    """A CUDA tensor on device `device`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    if t.get_device() != device:
        raise ValueError(f"{what}: on {t.device}, expected cuda:{device}")
    return t


def _current(t, what: str) -> int:
    """Index of the tensor's device, which has to be the current one (launches
    go there)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{what}: tensor must be on a CUDA device")
    if device != _device():
        raise ValueError(f"{what}: on {t.device}, but the current device is cuda:{_device()}")
    return device


def _keep_for(stream, *tensors):
    """Tensors allocated here and used on another stream than the current one."""
    if stream is None:
        return
    s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
    for t in tensors:
        if t is not None:
            t.record_stream(s)


def _new(like):
    """A new contiguous tensor of `like`'s shape and type."""
    if like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(like.shape, dtype=like.dtype, device=like.device)


def _result(t, what: str, like, shape, dtype):
    """A caller's output tensor, checked, or a new one beside `like`."""
    if t is None:
        if like.shape == shape and like.dtype == dtype:
            return _new(like)
        return torch.empty(shape, dtype=dtype, device=like.device)
    _on(t, what, like.get_device())
    if t.dtype != dtype or t.shape != torch.Size(shape) or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor of shape {tuple(shape)}")
    return t


# ----------------------------------------------------------------------------
# gradient norm and clipping


class GradTensorC(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("src_dtype", ctypes.c_int32), ("dst_dtype", ctypes.c_int32)]


class NormResult(ctypes.Structure):
    """Host image of zero_norm_result (32 bytes)."""
    _fields_ = [("norm", ctypes.c_double), ("norm32", ctypes.c_float), ("coef", ctypes.c_float),
                ("nonfinite", ctypes.c_int32), ("pad_", ctypes.c_int32 * 3)]


NORM_RESULT_BYTES = ctypes.sizeof(NormResult)


def read_norm_result(result) -> NormResult:
    """The record on the host (this synchronises with the current stream)."""
    return NormResult.from_buffer_copy(bytes(result.cpu().numpy().tobytes()))


def _dense(t) -> bool:
    """Whether the tensor's elements fill one run of memory, in any order."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if stride != want:
            return False
        want *= size
    return True


def _grad_tensor(t, what: str):
    if not isinstance(t, torch.Tensor) or t.layout != torch.strided:
        raise TypeError(f"{what}: expected a dense torch.Tensor")
    if t.numel() and not t.is_cuda and not t.is_pinned():
        raise ValueError(f"{what}: tensor must be on a CUDA device or in pinned host memory")
    if not _dense(t):
        raise ValueError(f"{what}: the elements must fill one run of memory")
    return _type(t, what)


def _check_disjoint(entries):
    """No output overlaps another tensor (entries: lo, hi, written)."""
    end = {False: 0, True: 0}
    for lo, hi, written in sorted(entries):
        if lo < end[True] or (written and lo < end[False]):
            raise ValueError("out: a tensor to be written overlaps another one")
        end[written] = max(end[written], hi)


def zero_grad_norm_workspace_bytes(grads) -> int:
    """Device workspace of zero_grad_norm or zero_clip_grad_norm for this list."""
    kept = [g for g in grads if g is not None]
    tensors = (GradTensorC * max(1, len(kept)))()
    for k, g in enumerate(kept):
        tensors[k].src_dtype, tensors[k].numel = _grad_tensor(g, f"grads[{k}]"), g.numel()
        tensors[k].src = g.data_ptr() if g.numel() else None
    need = ctypes.c_int64()
    _check((_lib or _load()).zero_grad_norm_workspace_bytes(tensors, len(kept), ctypes.byref(need)))
    return need.value


def _workspace(t, need: int, device: int):
    """A caller's workspace, checked, or a new one."""
    if t is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _on(t, "workspace", device)
    if not t.is_contiguous() or t.numel() * t.element_size() < need:
        raise ValueError(f"workspace: needs {need} contiguous bytes")
    return t


class GradNorm:
    """A prepared zero_grad_norm over `grads` (None entries are left out):
    the list is checked and marshalled once, each call takes the norm of what
    the tensors hold then.  Returns the norm as a float32 tensor without
    dimensions, a view of `result`, which the next call overwrites.
    workspace: device scratch of zero_grad_norm_workspace_bytes (None: its
    own)."""

    def __init__(self, grads, kind: str = "l2", workspace=None):
        self._prepare([g for g in grads if g is not None], None, kind, workspace)

    def _prepare(self, grads, out, kind, workspace):
        self.kind = _choice(_NORMS, kind, "kind")
        self._keep = (grads, out)
        self._list = (GradTensorC * max(1, len(grads)))()
        self.n = len(grads)
        device = None
        spans = []
        for k, g in enumerate(grads):
            what = f"grads[{k}]"
            e = self._list[k]
            e.src_dtype, e.numel = _grad_tensor(g, what), g.numel()
            e.src = g.data_ptr() if g.numel() else None
            if g.is_cuda:
                if device is None:
                    device = _current(g, what)
                _on(g, what, device)
            if out is None:
                continue
            d = out[k]
            if d is not g:
                _grad_tensor(d, f"out[{k}]")
                if d.shape != g.shape or (d.stride() != g.stride() and not
                                          (d.is_contiguous() and g.is_contiguous())):
                    raise ValueError(f"out[{k}]: shape and order must be those of grads[{k}]")
                if d.is_cuda and device is not None:
                    _on(d, f"out[{k}]", device)
            e.dst_dtype = _type(d, f"out[{k}]")
            e.dst = d.data_ptr() if d.numel() else None
            if g.numel():
                spans.append((e.dst, e.dst + d.numel() * d.element_size(), True))
                if e.dst != e.src:
                    spans.append((e.src, e.src + g.numel() * g.element_size(), False))
        _check_disjoint(spans)
        if device is None:
            device = _device()
        need = ctypes.c_int64()
        _check((_lib or _load()).zero_grad_norm_workspace_bytes(self._list, self.n, ctypes.byref(need)))
        self.result = torch.empty(NORM_RESULT_BYTES, dtype=torch.uint8, device=device)
        self._workspace = _workspace(workspace, need.value, device)
        self._norm = self.result[8:12].view(torch.float32)[0]
        self._args = (self.result.data_ptr(), self._workspace.data_ptr(), need.value)
        self.device = device

    def __call__(self, stream=None):
        _check((_lib or _load()).zero_grad_norm(self._list, self.n, self.kind, *self._args,
                                    _stream(stream, self.device)))
        return self._norm

    def read(self) -> NormResult:
        return read_norm_result(self.result)


class ClipGradNorm(GradNorm):
    """A prepared zero_clip_grad_norm: the norm of `grads`, and each gradient
    times min(1, max_norm / (norm + 1e-6)) into `out` (None: in place).
    `out` may have other types, for instance the views of a 16-bit replica
    that fp32 gradients go to.  `max_norm` may be changed between calls."""

    def __init__(self, grads, max_norm: float, kind: str = "l2", out=None, workspace=None):
        grads = list(grads)
        self.max_norm = float(max_norm)
        if out is None:
            grads = out = [g for g in grads if g is not None]
        else:
            out = list(out)
            if len(out) != len(grads):
                raise ValueError(f"out: expected {len(grads)} entries, got {len(out)}")
            pairs = [(g, d) for g, d in zip(grads, out) if g is not None]
            grads, out = [g for g, _ in pairs], [d for _, d in pairs]
        self._prepare(grads, out, kind, workspace)

    def __call__(self, stream=None):
        _check((_lib or _load()).zero_clip_grad_norm(self._list, self.n, self.kind, self.max_norm,
                                         *self._args, _stream(stream, self.device)))
        return self._norm


def zero_grad_norm(grads, kind: str = "l2", stream=None):
    """Norm of all gradients as one vector (see zero.h); a float32 tensor."""
    call = GradNorm(grads, kind)
    if stream is not None:
        _keep_for(stream, call.result, call._workspace)
    return call(stream)


def zero_clip_grad_norm(grads, max_norm: float, kind: str = "l2", out=None, stream=None):
    """Norm and clipping (see zero.h); returns the norm before clipping."""
    call = ClipGradNorm(grads, max_norm, kind, out)
    if stream is not None:
        _keep_for(stream, call.result, call._workspace)
    return call(stream)


# ----------------------------------------------------------------------------
# block join


class JoinDescC(ctypes.Structure):
    _fields_ = ([("rows", ctypes.c_int64), ("hidden", ctypes.c_int64)]
                + [(k, ctypes.c_int32) for k in ("act_dtype", "res_dtype", "param_dtype",
                                                 "gate_dtype", "kind", "gate_kind")]
                + [("eps", ctypes.c_double), ("scale", ctypes.c_double)]
                + [(k, ctypes.c_int64) for k in ("x_stride", "b_stride", "gate_stride",
                                                 "do_stride", "dn_stride")])


class JoinInputsC(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("x", "b", "gate", "w_post", "bias_post", "w_pre",
                                               "bias_pre")]


class JoinGradsC(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("dx", "db", "dgate", "dw_post", "dbias_post",
                                               "dw_pre", "dbias_pre")]


def _row_stride(t, what: str, shape, device: int) -> int:
    """Elements between rows of a tensor [..., hidden] whose rows are
    contiguous and evenly spaced."""
    if t.get_device() != device:
        _on(t, what, device)
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return shape[-1]
    hidden = shape[-1]
    if t.stride(-1) == 1 or hidden == 1:
        if t.dim() == 2:
            return t.stride(0)
        try:
            return t.view(-1, hidden).stride(0)
        except RuntimeError:
            pass
    raise ValueError(f"{what}: rows must be contiguous and evenly spaced (use .contiguous())")


def _join_args(x, b, gate, w_post, bias_post, w_pre, bias_pre, kind, scale, eps, act,
               d_o=None, d_n=None):
    """(desc, inputs, device, act dtype, hidden) of a join's arguments."""
    device = _current(x, "x")
    shape = x.shape
    if not shape:
        raise ValueError("x: expected [..., hidden]")
    hidden = shape[-1]
    x_stride = _row_stride(x, "x", shape, device)
    b_stride = gate_stride = do_stride = dn_stride = 0
    p_b = p_gate = None
    if b is not None:
        act = b.dtype
        b_stride = _row_stride(b, "b", shape, device)
        p_b = b.data_ptr()
    elif act is None:
        act = w_pre.dtype if x.dtype == torch.float32 and w_pre is not None else x.dtype
    act_code = _TYPES.get(act)
    if act_code is None:
        raise TypeError(f"b: expected float16, bfloat16 or float32, got {act}")
    param = None
    for name, t in (("w_post", w_post), ("bias_post", bias_post), ("w_pre", w_pre),
                    ("bias_pre", bias_pre)):
        if t is None:
            continue
        if t.get_device() != device:
            _on(t, name, device)
        if t.dim() != 1 or t.shape[0] != hidden or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous vector of {hidden}")
        if param is None:
            param = t.dtype
        elif t.dtype != param:
            raise TypeError(f"{name}: {t.dtype}, but another parameter is {param}")
    param_code = act_code if param is None else _TYPES.get(param)
    if param_code is None:
        raise TypeError(f"parameters: expected float16, bfloat16 or float32, got {param}")
    gate_kind, gate_code = GATE_NONE, act_code
    if gate is not None:
        _on(gate, "gate", device)
        gate_code = _type(gate, "gate")
        if gate.dim() == 1 and gate.shape[0] == hidden and len(shape) != 1:
            if not gate.is_contiguous():
                raise ValueError("gate: expected a contiguous vector")
            gate_kind = GATE_CHANNEL
        elif gate.shape == shape:
            gate_kind = GATE_FULL
            gate_stride = _row_stride(gate, "gate", shape, device)
        elif gate.shape == shape[:-1] + (1,):
            gate_kind = GATE_ROW
            gate_stride = _row_stride(gate, "gate", gate.shape, device)
        else:
            raise ValueError(f"gate: shape {tuple(gate.shape)}, expected ({hidden},), "
                             f"{tuple(shape[:-1]) + (1,)} or {tuple(shape)}")
        p_gate = gate.data_ptr()
    if d_o is not None:
        if d_o.dtype != x.dtype:
            raise TypeError(f"d_o: expected {x.dtype}, got {d_o.dtype}")
        do_stride = _row_stride(d_o, "d_o", shape, device)
    if d_n is not None:
        if d_n.dtype != act:
            raise TypeError(f"d_n: expected {act}, got {d_n.dtype}")
        dn_stride = _row_stride(d_n, "d_n", shape, device)
    d = JoinDescC(x.numel() // hidden if hidden else 0, hidden, act_code, _type(x, "x"),
                  param_code, gate_code, _choice(_KINDS, kind, "kind"), gate_kind, eps, scale,
                  x_stride, b_stride, gate_stride, do_stride, dn_stride)
    p = JoinInputsC(x.data_ptr(), p_b, p_gate, None if w_post is None else w_post.data_ptr(),
                    None if bias_post is None else bias_post.data_ptr(),
                    None if w_pre is None else w_pre.data_ptr(),
                    None if bias_pre is None else bias_pre.data_ptr())
    return d, p, device, act, hidden


def zero_block_join(x, b=None, *, w_post=None, bias_post=None, w_pre=None, bias_pre=None,
                    gate=None, kind: str = "rms", scale: float = 1.0, eps: float = 1e-6, o=None,
                    n=None, want_o: bool = True, want_stats: bool = False, stream=None):
    """o = x + scale * gate * norm(b; w_post) and n = norm(o; w_pre) (see
    zero.h): (o, n, stats).  Without w_post there is no norm before the gate,
    without w_pre no n (None); b None takes the norm of x alone, and o is x.
    x, b, gate: [..., hidden]; the gate also [hidden] or [..., 1].  stats is
    what the backward call takes (None unless want_stats)."""
    d, p, device, act, hidden = _join_args(x, b, gate, w_post, bias_post, w_pre, bias_pre, kind,
                                           scale, eps, None if n is None else n.dtype)
    if n is not None and w_pre is None:
        raise ValueError("n: needs w_pre")
    if b is None and o is None:
        want_o = False
    given_o, given_n = o, n
    p_o = p_n = p_stats = stats = None
    if want_o:
        o = _result(o, "o", x, x.shape, x.dtype)
        p_o = o.data_ptr()
    if w_pre is not None:
        n = _result(n, "n", x, x.shape, act)
        p_n = n.data_ptr()
    if want_stats:
        stats = torch.empty((d.rows, 4), dtype=torch.float32, device=x.device)
        p_stats = stats.data_ptr()
    if stream is not None:
        _keep_for(stream, o if given_o is None and want_o else None,
                  n if given_n is None else None, stats)
    _check((_lib or _load()).zero_block_join(ctypes.byref(d), ctypes.byref(p), p_o, p_n, p_stats,
                                 _stream(stream, device)))
    if not want_o:
        o = x if b is None else None
    return o, n, stats


def zero_block_join_workspace_bytes(x, b=None, *, w_post=None, bias_post=None, w_pre=None,
                                    bias_pre=None, gate=None, kind: str = "rms",
                                    scale: float = 1.0, eps: float = 1e-6) -> int:
    """Device workspace of zero_block_join_backward for these arguments."""
    d = _join_args(x, b, gate, w_post, bias_post, w_pre, bias_pre, kind, scale, eps, None)[0]
    return _join_need(d)


def _join_need(d) -> int:
    need = ctypes.c_int64()
    _check((_lib or _load()).zero_block_join_workspace_bytes(ctypes.byref(d), ctypes.byref(need)))
    return need.value


def zero_block_join_backward(x, b, d_o, d_n, stats, *, w_post=None, bias_post=None, w_pre=None,
                             bias_pre=None, gate=None, kind: str = "rms", scale: float = 1.0,
                             eps: float = 1e-6, want=None, workspace=None, stream=None):
    """Gradients of zero_block_join's inputs from those of o and n (either
    may be None) and its stats: a dict with dx, db, dgate, dw_post,
    dbias_post, dw_pre and dbias_pre, None for what has no input or is not in
    `want` (a set of those names; None: all).  workspace: device scratch of
    zero_block_join_workspace_bytes (None: allocated here)."""
    d, p, device, act, hidden = _join_args(x, b, gate, w_post, bias_post, w_pre, bias_pre, kind,
                                           scale, eps, None if d_n is None else d_n.dtype, d_o,
                                           d_n)
    p_stats = None
    if stats is not None:
        p_stats = _result(stats, "stats", x, (d.rows, 4), torch.float32).data_ptr()
    out, at = {}, []
    unused = False
    for name, like in (("dx", x), ("db", b), ("dgate", gate), ("dw_post", w_post),
                       ("dbias_post", bias_post), ("dw_pre", w_pre), ("dbias_pre", bias_pre)):
        t = ptr = None
        if like is not None and (want is None or name in want):
            if d_n is None and name in ("dw_pre", "dbias_pre"):
                t = torch.zeros_like(like)  # n was not used
                unused = True
            else:
                t = (torch.empty_like(like) if like.is_contiguous() else
                     torch.empty(like.shape, dtype=like.dtype, device=like.device))
                ptr = t.data_ptr()
        out[name] = t
        at.append(ptr)
    sums = any(at[3:]) or (d.gate_kind == GATE_CHANNEL and at[2])
    p_ws, need, ws = None, 0, None
    if sums:
        need = _join_need(d)
        ws = _workspace(workspace, need, device)
        p_ws = ws.data_ptr()
    if stream is not None:
        _keep_for(stream, *out.values(), ws if workspace is None else None)
    if unused and not any(at):
        return out
    _check((_lib or _load()).zero_block_join_backward(
        ctypes.byref(d), ctypes.byref(p), None if d_o is None else d_o.data_ptr(),
        None if d_n is None else d_n.data_ptr(), p_stats, ctypes.byref(JoinGradsC(*at)), p_ws,
        need, _stream(stream, device)))
    return out


def _even_rows(t):
    """A gradient as the calls take it (autograd may hand out expanded ones)."""
    if t is None or t.is_contiguous() or (t.dim() == 2 and t.stride(1) == 1
                                          and t.stride(0) >= t.shape[1]):
        return t
    return t.contiguous()


class _BlockJoin(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, b, gate, w_post, bias_post, w_pre, bias_pre, kind, scale, eps):
        ctx.set_materialize_grads(False)
        ctx.how = dict(kind=kind, scale=scale, eps=eps)
        o, n, stats = zero_block_join(x, b, w_post=w_post, bias_post=bias_post, w_pre=w_pre,
                                      bias_pre=bias_pre, gate=gate, want_stats=True, **ctx.how)
        ctx.save_for_backward(x, b, gate, w_post, bias_post, w_pre, bias_pre, stats)
        if o is x:
            o = x.view_as(x)
        return o, n

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_o, d_n):
        x, b, gate, w_post, bias_post, w_pre, bias_pre, stats = ctx.saved_tensors
        names = ("dx", "db", "dgate", "dw_post", "dbias_post", "dw_pre", "dbias_pre")
        want = {k for k, needed in zip(names, ctx.needs_input_grad) if needed}
        if d_o is None and d_n is None:
            return (None,) * 10
        g = zero_block_join_backward(x, b, _even_rows(d_o), _even_rows(d_n), stats, w_post=w_post,
                                     bias_post=bias_post, w_pre=w_pre, bias_pre=bias_pre,
                                     gate=gate, want=want, **ctx.how)
        return tuple(g[k] for k in names) + (None, None, None)


def block_join(x, b=None, *, w_post=None, bias_post=None, w_pre=None, bias_pre=None, gate=None,
               kind: str = "rms", scale: float = 1.0, eps: float = 1e-6):
    """zero_block_join with autograd: (o, n), n None without w_pre."""
    return _BlockJoin.apply(x, b, gate, w_post, bias_post, w_pre, bias_pre, kind, scale, eps)


# ----------------------------------------------------------------------------
# expert permutation


@dataclasses.dataclass
class ExpertOrder:
    """What zero_expert_sort leaves on the device: offsets [n_experts + 1],
    rows [tokens, topk] (-1: dropped), pairs [tokens * topk] (-1: past the
    end), all int32."""
    offsets: torch.Tensor
    rows: torch.Tensor
    pairs: torch.Tensor
    n_experts: int
    tokens: int
    topk: int


def zero_expert_sort_workspace_bytes(tokens: int, topk: int, n_experts: int) -> int:
    """Device workspace of zero_expert_sort (0 up to some tens of thousands of choices)."""
    need = ctypes.c_int64()
    _check((_lib or _load()).zero_expert_sort_workspace_bytes(tokens, topk, n_experts, ctypes.byref(need)))
    return need.value


_sort_need = functools.lru_cache(maxsize=256)(zero_expert_sort_workspace_bytes)


def zero_expert_sort(ids, n_experts: int, workspace=None, stream=None) -> ExpertOrder:
    """Rows of every token's choices in expert order (see zero.h).  ids:
    [tokens, topk] int32 or int64; a choice outside [0, n_experts) is
    dropped.  workspace: device scratch of zero_expert_sort_workspace_bytes
    (None: allocated here)."""
    device = _current(ids, "ids")
    if ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids: expected a contiguous [tokens, topk] tensor")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids: expected int32 or int64, got {ids.dtype}")
    tokens, topk = ids.shape
    if topk < 1:
        raise ValueError("ids: topk must be at least 1")
    where = ids.device
    offsets = torch.empty(max(0, n_experts) + 1, dtype=torch.int32, device=where)
    rows = torch.empty(ids.shape, dtype=torch.int32, device=where)
    pairs = torch.empty(tokens * topk, dtype=torch.int32, device=where)
    need = _sort_need(tokens, topk, n_experts)
    ws = _workspace(workspace, need, device) if need else None
    if stream is not None:
        _keep_for(stream, offsets, rows, pairs, ws if workspace is None else None)
    _check((_lib or _load()).zero_expert_sort(ids.data_ptr() or None, ids.element_size(), tokens, topk,
                                  n_experts, offsets.data_ptr(), rows.data_ptr() or None,
                                  pairs.data_ptr() or None,
                                  None if ws is None else ws.data_ptr(), need,
                                  _stream(stream, device)))
    return ExpertOrder(offsets, rows, pairs, n_experts, tokens, topk)


def _sorted_rows(t, what: str, order: ExpertOrder):
    """(device, type, hidden) of a tensor [tokens * topk, hidden]."""
    device = _current(t, what)
    if order.rows.get_device() != device:
        _on(order.rows, "order", device)
    if t.dim() != 2 or t.shape[0] != order.tokens * order.topk or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous [{order.tokens * order.topk}, hidden] "
                         "tensor")
    return device, _type(t, what), t.shape[1]


def _token_rows(t, what: str, order: ExpertOrder):
    """(device, type, hidden, row stride) of a tensor [tokens, hidden]."""
    device = _current(t, what)
    if order.rows.get_device() != device:
        _on(order.rows, "order", device)
    if t.dim() != 2 or t.shape[0] != order.tokens:
        raise ValueError(f"{what}: expected [{order.tokens}, hidden], got {tuple(t.shape)}")
    return device, _type(t, what), t.shape[1], _row_stride(t, what, t.shape, device)


def _expert_weights(weights, order: ExpertOrder, device: int):
    if weights.get_device() != device:
        _on(weights, "weights", device)
    if weights.shape != order.rows.shape or not weights.is_contiguous():
        raise ValueError(f"weights: expected a contiguous [{order.tokens}, {order.topk}] tensor")
    return _type(weights, "weights")


def zero_expert_dispatch(x, order: ExpertOrder, out=None, stream=None):
    """Tokens copied to their rows in expert order, [tokens * topk, hidden];
    the rows past the last kept choice are zero."""
    device, code, hidden, stride = _token_rows(x, "x", order)
    xs = _result(out, "out", x, (order.tokens * order.topk, hidden), x.dtype)
    if stream is not None:
        _keep_for(stream, xs if out is None else None)
    _check((_lib or _load()).zero_expert_dispatch(x.data_ptr(), stride, code, order.tokens, order.topk, hidden,
                                      order.offsets.data_ptr(), order.n_experts,
                                      order.rows.data_ptr(), xs.data_ptr(),
                                      _stream(stream, device)))
    return xs


def zero_expert_dispatch_backward(dxs, order: ExpertOrder, out=None, stream=None):
    """Each token's gradient: the sum of its rows'."""
    device, code, hidden = _sorted_rows(dxs, "dxs", order)
    dx = _result(out, "out", dxs, (order.tokens, hidden), dxs.dtype)
    if stream is not None:
        _keep_for(stream, dx if out is None else None)
    _check((_lib or _load()).zero_expert_dispatch_backward(dxs.data_ptr(), code, order.tokens, order.topk,
                                               hidden, order.rows.data_ptr(), dx.data_ptr(),
                                               _stream(stream, device)))
    return dx


def zero_expert_combine(ys, weights, order: ExpertOrder, out=None, stream=None):
    """Each token's weighted sum of its rows; zero when all its choices were
    dropped."""
    device, code, hidden = _sorted_rows(ys, "ys", order)
    wcode = _expert_weights(weights, order, device)
    y = _result(out, "out", ys, (order.tokens, hidden), ys.dtype)
    if stream is not None:
        _keep_for(stream, y if out is None else None)
    _check((_lib or _load()).zero_expert_combine(ys.data_ptr(), code, weights.data_ptr(), wcode, order.tokens,
                                     order.topk, hidden, order.rows.data_ptr(), y.data_ptr(),
                                     _stream(stream, device)))
    return y


def zero_expert_combine_backward(dy, ys, weights, order: ExpertOrder, want_weights: bool = True,
                                 stream=None):
    """(dys, dweights) of zero_expert_combine; dweights None unless wanted."""
    device, code, hidden = _sorted_rows(ys, "ys", order)
    _, dcode, dhidden, stride = _token_rows(dy, "dy", order)
    if dcode != code or dhidden != hidden:
        raise TypeError(f"dy: expected {ys.dtype} rows of {hidden}, got {dy.dtype} of {dhidden}")
    wcode = _expert_weights(weights, order, device)
    dys = _new(ys)
    dweights = _new(weights) if want_weights else None
    if stream is not None:
        _keep_for(stream, dys, dweights)
    _check((_lib or _load()).zero_expert_combine_backward(
        dy.data_ptr(), stride, ys.data_ptr(), code, weights.data_ptr(), wcode, order.tokens,
        order.topk, hidden, order.offsets.data_ptr(), order.n_experts, order.rows.data_ptr(),
        dys.data_ptr(), None if dweights is None else dweights.data_ptr(),
        _stream(stream, device)))
    return dys, dweights


class _ExpertDispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order):
        ctx.order = order
        return zero_expert_dispatch(x, order)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dxs):
        return zero_expert_dispatch_backward(dxs.contiguous(), ctx.order), None


class _ExpertCombine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, order):
        ctx.order = order
        ctx.save_for_backward(ys, weights)
        return zero_expert_combine(ys, weights, order)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        ys, weights = ctx.saved_tensors
        dys, dw = zero_expert_combine_backward(_even_rows(dy), ys, weights, ctx.order,
                                               want_weights=ctx.needs_input_grad[1])
        return dys if ctx.needs_input_grad[0] else None, dw, None


def expert_dispatch(x, order: ExpertOrder):
    """zero_expert_dispatch with autograd."""
    return _ExpertDispatch.apply(x, order)


def expert_combine(ys, weights, order: ExpertOrder):
    """zero_expert_combine with autograd (of ys and of the weights)."""
    return _ExpertCombine.apply(ys, weights, order)
