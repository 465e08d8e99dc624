"""Operators of a training step around the sharded optimizer: gradient norm
and clipping over many tensors, the block join, the expert permutation and the
router before it, and a language model's two ends, the token embedding and the
cross entropy over the vocabulary.

The ``zero_*`` functions bind the C calls of include/zero.h under their own
names (argument checks and marshalling only, compiled but for the norm's,
csrc/train_ops_binding.cpp; the current CUDA stream unless
``stream`` is given, which then makes the call's buffers too; inputs are the
caller's to order; no fallback).  ``GradNorm`` and ``ClipGradNorm`` are the
prepared forms for gradients whose buffers stay in place from step to step.
``block_join``, ``expert_route``, ``expert_dispatch``, ``expert_combine``,
``embedding`` and ``linear_cross_entropy`` are the same calls with autograd.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _build
from . import zero as _zero
from .zero import _check

ZERO_FP32 = 2
_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: ZERO_FP32}
_NORMS = {"l2": 0, "inf": 1}


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


_fast = None


def _load_fast():
    """The compiled binding (built with the library, and linked against it)."""
    global _fast
    _load()
    problem = _build.binding_problem()
    if problem:
        raise RuntimeError(f"{problem}: run `python -c 'import __graft_entry__ as g; g.build()'`; "
                           "there is no fallback implementation")
    from . import _train_ops
    _train_ops.set_error(_zero.ZeroError)
    _fast = _train_ops
    return _fast


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


def _torch_stream(stream):
    """A stream object for a stream or a handle.  0 and 1 are the default
    stream's handles (ExternalStream(0) would be a new stream)."""
    if not isinstance(stream, int):
        return stream
    return torch.cuda.default_stream() if stream in (0, 1) else torch.cuda.ExternalStream(stream)


def _keep_for(stream, *tensors):
    """Tensors allocated here and used on another stream than the current one."""
    if stream is None:
        return
    s = _torch_stream(stream)
    for t in tensors:
        if t is not None:
            t.record_stream(s)


def _run_on(stream, call):
    """call() with `stream` as the current one (None: as it is).  What the call
    allocates then belongs to that stream, whose earlier work is done with the
    memory, and what it fills is filled there; the results, which the caller's
    stream goes on to use, are held for both."""
    if stream is None:
        return call()
    stream, caller = _torch_stream(stream), torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        got = call()
    made = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
    for s in (stream, caller):
        _keep_for(s, *made)
    return got


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
    """A prepared zero_grad_norm over `grads` (None entries are left out): the
    list is checked and marshalled here once, each call takes the norm of what
    the tensors hold then.  (The C call checks the list and fills its tables
    each time.)  Returns the norm as a float32 tensor without dimensions, a
    view of `result`, which the next call overwrites.  workspace: device
    scratch of zero_grad_norm_workspace_bytes (None: its own).

    Calls share the result and the workspace: those on different streams are
    the caller's to order, one after the other.  A graph that captured a call
    needs the object alive."""

    _ready = None

    def __init__(self, grads, kind: str = "l2", workspace=None):
        self._fill(grads, kind, workspace)
        self._mark()

    def _fill(self, grads, kind="l2", workspace=None):
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
        self._home = _raw_stream(device)  # the stream that the buffers were allocated on

    def _mark(self):
        """Notes the own stream's work so far, which may have used the buffers'
        memory before (nothing to wait for when they come from a capture)."""
        self._joined = set()
        if not torch.cuda.is_current_stream_capturing():
            self._ready = torch.cuda.Event()
            self._ready.record()

    def _on_stream(self, stream):
        """Handle of the stream that a call runs on; launches go to the current
        device.  Another stream than the buffers' own first waits for what used
        their memory before (not when it is captured: that begins with the
        device idle).  The object may be gone before the stream has done the
        call's work, so it is recorded on them."""
        if _device() != self.device:
            raise ValueError(f"prepared on cuda:{self.device}, but the current device is "
                             f"cuda:{_device()}")
        handle = _stream(stream, self.device)
        if handle != self._home:
            other = torch.cuda.current_stream() if stream is None else _torch_stream(stream)
            if self._ready is not None and handle not in self._joined:
                with torch.cuda.stream(other):
                    captured = torch.cuda.is_current_stream_capturing()
                if not captured:
                    other.wait_event(self._ready)
                    self._joined.add(handle)
            _keep_for(other, self.result, self._workspace)
        return handle

    def __call__(self, stream=None):
        _check((_lib or _load()).zero_grad_norm(self._list, self.n, self.kind, *self._args,
                                                self._on_stream(stream)))
        return self._norm

    def read(self) -> NormResult:
        return read_norm_result(self.result)


class ClipGradNorm(GradNorm):
    """A prepared zero_clip_grad_norm: the norm of `grads`, and each gradient
    times min(1, max_norm / (norm + 1e-6)) into `out` (None: in place).
    `out` may have other types, for instance the views of a 16-bit replica
    that fp32 gradients go to.  `max_norm` may be changed between calls."""

    def __init__(self, grads, max_norm: float, kind: str = "l2", out=None, workspace=None):
        self._fill(grads, max_norm, kind, out, workspace)
        self._mark()

    def _fill(self, grads, max_norm, kind="l2", out=None, workspace=None):
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
                                                     *self._args, self._on_stream(stream)))
        return self._norm


def _once(cls, *args):
    """A call of a list that is used once, on the stream that it is made on."""
    call = cls.__new__(cls)
    call._fill(*args)
    return call()


def zero_grad_norm(grads, kind: str = "l2", stream=None):
    """Norm of all gradients as one vector (see zero.h); a float32 tensor."""
    return _run_on(stream, lambda: _once(GradNorm, grads, kind))


def zero_clip_grad_norm(grads, max_norm: float, kind: str = "l2", out=None, stream=None):
    """Norm and clipping (see zero.h); returns the norm before clipping."""
    return _run_on(stream, lambda: _once(ClipGradNorm, grads, max_norm, kind, out))


# ----------------------------------------------------------------------------
# block join


class JoinDescC(ctypes.Structure):
    """Host image of zero_join_desc."""
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


def zero_block_join(x, b=None, *, w_post=None, bias_post=None, w_pre=None, bias_pre=None,
                    gate=None, kind: str = "rms", scale: float = 1.0, eps: float = 1e-6, o=None,
                    n=None, want_o: bool = True, want_stats: bool = False, stream=None):
    """o = x + scale * gate * norm(b; w_post) and n = norm(o; w_pre) (see
    zero.h): (o, n, stats).  Without w_post there is no norm before the gate,
    without w_pre no n (None); b None takes the norm of x alone, and o is x.
    x, b, gate: [..., hidden]; the gate also [hidden] or [..., 1].  stats is
    what the backward call takes (None unless want_stats)."""
    if stream is not None:
        return _run_on(stream, lambda: zero_block_join(
            x, b, w_post=w_post, bias_post=bias_post, w_pre=w_pre, bias_pre=bias_pre, gate=gate,
            kind=kind, scale=scale, eps=eps, o=o, n=n, want_o=want_o, want_stats=want_stats))
    return (_fast or _load_fast()).block_join(x, b, w_post, bias_post, w_pre, bias_pre, gate, kind,
                                              scale, eps, o, n, want_o, want_stats)


def zero_block_join_workspace_bytes(x, b=None, *, w_post=None, bias_post=None, w_pre=None,
                                    bias_pre=None, gate=None, kind: str = "rms",
                                    scale: float = 1.0, eps: float = 1e-6) -> int:
    """Device workspace of zero_block_join_backward for these arguments."""
    return (_fast or _load_fast()).block_join_workspace_bytes(x, b, w_post, bias_post, w_pre,
                                                              bias_pre, gate, kind, scale, eps)


def zero_block_join_backward(x, b, d_o, d_n, stats, *, w_post=None, bias_post=None, w_pre=None,
                             bias_pre=None, gate=None, kind: str = "rms", scale: float = 1.0,
                             eps: float = 1e-6, want=None, workspace=None, stream=None):
    """Gradients of zero_block_join's inputs from those of o and n (either
    may be None) and its stats: a dict with dx, db, dgate, dw_post,
    dbias_post, dw_pre and dbias_pre, None for what has no input or is not in
    `want` (a set of those names; None: all).  workspace: device scratch of
    zero_block_join_workspace_bytes (None: allocated here)."""
    return _run_on(stream, lambda: (_fast or _load_fast()).block_join_backward(
        x, b, w_post, bias_post, w_pre, bias_pre, gate, kind, scale, eps, d_o, d_n, stats, want,
        workspace))


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


def zero_expert_sort(ids, n_experts: int, workspace=None, stream=None) -> ExpertOrder:
    """Rows of every token's choices in expert order (see zero.h).  ids:
    [tokens, topk] int32 or int64; a choice outside [0, n_experts) is
    dropped.  workspace: device scratch of zero_expert_sort_workspace_bytes
    (None: allocated here)."""
    got = _run_on(stream, lambda: (_fast or _load_fast()).expert_sort(ids, n_experts, workspace))
    return ExpertOrder(*got, n_experts, ids.shape[0], ids.shape[1])


def zero_expert_dispatch(x, order: ExpertOrder, out=None, stream=None):
    """Tokens copied to their rows in expert order, [tokens * topk, hidden];
    the rows past the last kept choice are zero."""
    return _run_on(stream, lambda: (_fast or _load_fast()).expert_dispatch(
        x, order.offsets, order.rows, order.n_experts, order.tokens, order.topk, out))


def zero_expert_dispatch_backward(dxs, order: ExpertOrder, out=None, stream=None):
    """Each token's gradient: the sum of its rows'."""
    return _run_on(stream, lambda: (_fast or _load_fast()).expert_dispatch_backward(
        dxs, order.offsets, order.rows, order.n_experts, order.tokens, order.topk, out))


def zero_expert_combine(ys, weights, order: ExpertOrder, out=None, stream=None):
    """Each token's weighted sum of its rows; zero when all its choices were
    dropped."""
    return _run_on(stream, lambda: (_fast or _load_fast()).expert_combine(
        ys, weights, order.offsets, order.rows, order.n_experts, order.tokens, order.topk, out))


def zero_expert_combine_backward(dy, ys, weights, order: ExpertOrder, want_weights: bool = True,
                                 stream=None):
    """(dys, dweights) of zero_expert_combine; dweights None unless wanted."""
    return _run_on(stream, lambda: (_fast or _load_fast()).expert_combine_backward(
        dy, ys, weights, order.offsets, order.rows, order.n_experts, order.tokens, order.topk,
        want_weights))


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


# ----------------------------------------------------------------------------
# router


@dataclasses.dataclass
class ExpertRoute:
    """What zero_expert_route leaves on the device: ids [tokens, topk] and
    counts [n_experts] int32, weights [tokens, topk] and losses [2] (balance
    and z loss) float32; stats, which the backward call takes."""
    ids: torch.Tensor
    weights: torch.Tensor
    counts: torch.Tensor
    losses: torch.Tensor
    stats: torch.Tensor
    normalize: bool


def zero_expert_route_workspace_bytes(tokens: int, n_experts: int) -> int:
    """Device workspace of zero_expert_route."""
    need = ctypes.c_int64()
    _check((_lib or _load()).zero_expert_route_workspace_bytes(tokens, n_experts, ctypes.byref(need)))
    return need.value


def zero_expert_route(logits, topk: int, *, normalize: bool = True, workspace=None,
                      stream=None) -> ExpertRoute:
    """Every token's experts with their weights, the experts' counts, and the
    losses that keep them in balance (see zero.h).  logits: [tokens,
    n_experts]; -inf bars an expert, a row of nothing else leaves its token
    out (ids -1, weights 0).  workspace: device scratch of
    zero_expert_route_workspace_bytes (None: allocated here)."""
    got = _run_on(stream, lambda: (_fast or _load_fast()).expert_route(logits, topk, normalize,
                                                                       workspace))
    return ExpertRoute(*got, bool(normalize))


def zero_expert_route_backward(logits, route: ExpertRoute, d_weights=None, d_losses=None, *,
                               out=None, stream=None):
    """The logits' gradient from those of the weights and of the two losses
    (float32 [2]), either None: no gradient comes that way."""
    return _run_on(stream, lambda: (_fast or _load_fast()).expert_route_backward(
        logits, route.normalize, route.ids, route.weights, route.counts, route.stats, d_weights,
        d_losses, out))


class _ExpertRoute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk, normalize):
        ctx.set_materialize_grads(False)
        r = zero_expert_route(logits, topk, normalize=normalize)
        ctx.normalize = r.normalize
        ctx.save_for_backward(logits, r.ids, r.weights, r.counts, r.stats)
        ctx.mark_non_differentiable(r.ids, r.counts)
        return r.ids, r.weights, r.counts, r.losses

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _ids, d_weights, _counts, d_losses):
        if d_weights is None and d_losses is None:
            return None, None, None
        logits, ids, weights, counts, stats = ctx.saved_tensors
        route = ExpertRoute(ids, weights, counts, None, stats, ctx.normalize)
        return zero_expert_route_backward(
            logits, route, None if d_weights is None else d_weights.contiguous(),
            None if d_losses is None else d_losses.contiguous()), None, None


def expert_route(logits, topk: int, *, normalize: bool = True):
    """zero_expert_route with autograd (of the weights and the losses): (ids,
    weights, counts, losses)."""
    return _ExpertRoute.apply(logits, topk, normalize)


# ----------------------------------------------------------------------------
# token embedding


def _code(dtype, what: str) -> int:
    """A type's number, -1 for None."""
    if dtype is None:
        return -1
    if dtype not in _TYPES:
        raise TypeError(f"{what}: expected float16, bfloat16 or float32, got {dtype}")
    return _TYPES[dtype]


def zero_embedding(ids, table, *, scale: float = 1.0, dtype=None, out=None, stream=None):
    """scale * table[ids], zero rows for ids outside the table (see zero.h).
    ids: [...], int32 or int64; table: [vocab, hidden].  dtype: the table's
    (None) or float32."""
    code = _code(dtype, "dtype")
    return _run_on(stream, lambda: (_fast or _load_fast()).embedding(ids, table, scale, code, out))


def zero_embedding_workspace_bytes(tokens: int, vocab: int, hidden: int) -> int:
    """Device workspace of zero_embedding_backward."""
    need = ctypes.c_int64()
    _check((_lib or _load()).zero_embedding_workspace_bytes(tokens, vocab, hidden, ctypes.byref(need)))
    return need.value


def zero_embedding_backward(dy, ids, vocab: int, *, scale: float = 1.0, dtype=None, out=None,
                            accumulate: bool = False, workspace=None, stream=None):
    """The table's gradient [vocab, hidden]: scale times the sum of every id's
    rows of dy (see zero.h).  dtype: dy's (None) or another; a 16-bit one and
    float32 mix.  accumulate: added to `out`, whose other rows are left
    alone.  workspace: 256-byte aligned device scratch of
    zero_embedding_workspace_bytes (None: allocated here)."""
    code = _code(dtype, "dtype")
    return _run_on(stream, lambda: (_fast or _load_fast()).embedding_backward(
        dy, ids, vocab, scale, code, out, accumulate, workspace))


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale, dtype):
        ctx.save_for_backward(ids)
        ctx.scale, ctx.vocab, ctx.dtype = scale, table.shape[0], table.dtype
        return zero_embedding(ids, table, scale=scale, dtype=dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        ids, = ctx.saved_tensors
        return None, zero_embedding_backward(_even_rows(dy), ids, ctx.vocab, scale=ctx.scale,
                                             dtype=ctx.dtype), None, None


def embedding(ids, table, *, scale: float = 1.0, dtype=None):
    """zero_embedding with autograd (of the table)."""
    return _Embedding.apply(ids, table, scale, dtype)


# ----------------------------------------------------------------------------
# linear softmax cross entropy

_REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}


@dataclasses.dataclass
class CrossEntropy:
    """What zero_linear_cross_entropy leaves on the device: losses and lse of
    the targets' shape (0 where a token is left out), total [3] (mean, sum and
    number of the losses), all float32; rows and rest (1 - p of the targets),
    which the backward call takes.  Without rest it forms 1 - p from lse, of
    which little is left where p is near 1."""
    losses: torch.Tensor
    lse: torch.Tensor
    total: torch.Tensor
    rows: torch.Tensor
    rest: torch.Tensor | None = None


def zero_linear_cross_entropy_workspace_bytes(x, w, targets, *, scale: float = 1.0,
                                              backward: bool = False, dw_dtype=None) -> int:
    """Device workspace of zero_linear_cross_entropy, or of its backward call."""
    return (_fast or _load_fast()).linear_cross_entropy_workspace_bytes(
        x, w, targets, scale, backward, _code(dw_dtype, "dw_dtype"))


def zero_linear_cross_entropy(x, w, targets, *, scale: float = 1.0, workspace=None,
                              stream=None) -> CrossEntropy:
    """Cross entropy of the logits scale * x w^T with the targets (see zero.h),
    the logits never in memory.  x: [..., hidden], w: [vocab, hidden], both
    float16 or bfloat16; targets: [...], int32 or int64, a token whose target
    lies outside [0, vocab) is left out.  workspace: 256-byte aligned device
    scratch of zero_linear_cross_entropy_workspace_bytes (None: allocated
    here)."""
    return CrossEntropy(*_run_on(stream, lambda: (_fast or _load_fast()).linear_cross_entropy(
        x, w, targets, scale, workspace)))


def zero_linear_cross_entropy_backward(x, w, targets, ce: CrossEntropy, d_loss, *,
                                       reduction: str = "mean", scale: float = 1.0,
                                       want=("dx", "dw"), dx=None, dw=None, dw_dtype=None,
                                       workspace=None, stream=None):
    """(dx, dw) of zero_linear_cross_entropy from the gradient of its mean
    (ce.total[0]), its sum (ce.total[1]), each one float32 number on the
    device, or of the losses (reduction "none").  None for what is not in
    `want`.  dw_dtype: the type of w (None) or float32, for which the logits'
    gradient is held in two 16-bit numbers: a quarter more operations."""
    kind = _choice(_REDUCTIONS, reduction, "reduction")
    if not set(want) <= {"dx", "dw"}:
        raise ValueError(f"want must name dx or dw, got {want!r}")
    code = _code(dw_dtype, "dw_dtype")
    return _run_on(stream, lambda: (_fast or _load_fast()).linear_cross_entropy_backward(
        x, w, targets, scale, ce.lse, ce.rows, d_loss, kind, "dx" in want, "dw" in want, dx, dw,
        code, workspace, ce.rest))


# These make and take `rest`.
zero_linear_cross_entropy_rest = zero_linear_cross_entropy
zero_linear_cross_entropy_rest_backward = zero_linear_cross_entropy_backward


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, targets, scale, reduction):
        ce = zero_linear_cross_entropy(x, w, targets, scale=scale)
        ctx.how = dict(scale=scale, reduction=reduction)
        ctx.save_for_backward(x, w, targets, ce.lse, ce.rows, ce.rest)
        if reduction == "none":
            return ce.losses
        return ce.total[1 if reduction == "sum" else 0]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d):
        x, w, targets, lse, rows, rest = ctx.saved_tensors
        want = [k for k, needed in zip(("dx", "dw"), ctx.needs_input_grad) if needed]
        dx, dw = zero_linear_cross_entropy_backward(x, w, targets, CrossEntropy(None, lse, None, rows, rest),
                                                    d.contiguous(), want=want, **ctx.how)
        return dx, dw, None, None, None


def linear_cross_entropy(x, w, targets, *, scale: float = 1.0, reduction: str = "mean"):
    """zero_linear_cross_entropy with autograd: its mean or sum over the tokens
    that are not left out (0 when all are), or ("none") every token's loss."""
    _choice(_REDUCTIONS, reduction, "reduction")
    return _LinearCrossEntropy.apply(x, w, targets, scale, reduction)
