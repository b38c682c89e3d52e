"""Network operators around the coder: group norm with an activation, rotary
positions and attention, forward and backward (``include/lic_layers.h``).

A learned image codec's transforms and its entropy model run right before the
coder; these are the parts of them that convolutions and matrix products leave
over, as hand-written HIP kernels in ``liblic_layers.so``.  Sums are taken in an
order that a call's sizes, windows and key lengths alone decide, wherever its values
lie, so an encoder and a decoder that make the same call predict the same scales, bit
for bit.  A call of another size (a single token instead of a whole latent) may differ
in the last bits: an encoder has to step where its decoder does.

:func:`group_norm`, :func:`rotary` and :func:`attention` work with autograd (what they cannot
differentiate they refuse: forward mode, second derivatives but rotary's).  The
``*_forward`` and ``*_backward`` functions are the calls beneath them, for programs that
keep their own gradients.  As in :mod:`.binding`, torch only supplies device memory and
the current stream, nothing is synchronised, and there is no CPU path.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import torch
from torch.autograd import forward_ad

from .binding import NAME_TO_CODE, _check_rc

PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(PKG, "liblic_layers.so")

# every symbol the public header declares
EXPORTS = (
    "lic_group_norm_workspace_bytes",
    "lic_group_norm_forward",
    "lic_group_norm_backward",
    "lic_rotary_table",
    "lic_rotary",
    "lic_attention_workspace_bytes",
    "lic_attention_forward",
    "lic_attention_backward",
    "lic_layers_target",
)

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
MAX_HEAD_DIM = 128

_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load the compiled library; raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIBRARY
        if not os.path.exists(p):
            raise RuntimeError(
                f"{p} is missing: build it with `python -m learned_image_compression_amd.build` "
                "(hipcc, gfx950); there is no CPU fallback")
        lib = ctypes.CDLL(p)
        vp, u64, i64, i32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int64, ctypes.c_int32
        f32, f64, st = ctypes.c_float, ctypes.c_double, ctypes.c_char_p
        lib.lic_group_norm_workspace_bytes.argtypes = [i32, i64, i32, i32]
        lib.lic_group_norm_workspace_bytes.restype = u64
        lib.lic_group_norm_forward.argtypes = [vp, i64, i64, i32, i64, i32, i32, i32, vp, vp, i32,
                                               f32, i32, vp, i64, i64, vp, vp, vp, u64, vp]
        lib.lic_group_norm_forward.restype = ctypes.c_int
        lib.lic_group_norm_backward.argtypes = [vp, i64, i64, vp, i64, i64, i32, i64, i32, i32,
                                                i32, vp, vp, i32, i32, vp, vp, vp, i64, i64, vp,
                                                vp, vp, u64, vp]
        lib.lic_group_norm_backward.restype = ctypes.c_int
        lib.lic_rotary_table.argtypes = [vp, i64, i32, i32, f64, f64, f64, f64, f64, f64, vp, vp,
                                         vp]
        lib.lic_rotary_table.restype = ctypes.c_int
        lib.lic_rotary.argtypes = [st, vp]
        lib.lic_rotary.restype = ctypes.c_int
        lib.lic_attention_workspace_bytes.argtypes = [st, i32]
        lib.lic_attention_workspace_bytes.restype = u64
        for name in ("lic_attention_forward", "lic_attention_backward"):
            getattr(lib, name).argtypes = [st, vp, u64, vp]
            getattr(lib, name).restype = ctypes.c_int
        lib.lic_layers_target.argtypes = []
        lib.lic_layers_target.restype = ctypes.c_char_p
        if path is None:
            _lib = lib
        return lib


# ---- device, stream, workspace --------------------------------------------


def _device_of(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, which is not the current device")
    return t.device


def _stream(device) -> int:
    """The current stream's handle (without an object around it, which takes 2 us)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _dense_like(t: torch.Tensor) -> torch.Tensor:
    if t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _like(t, dtype, device, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is dtype and t.device == device:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _out_like(out, t, dtype, device, name):
    """Checks of an output that the caller gives; two of its entries must not be one."""
    _like(out, dtype, device, name)
    if out.shape != t.shape:
        raise ValueError(f"{name} differs in shape")
    if any(stride == 0 and size > 1 for stride, size in zip(out.stride(), out.shape)):
        raise ValueError(f"{name} overlaps itself")


_NO_WORKSPACE = (None, 0, None)  # address, bytes, owner
_E_WORKSPACE = NAME_TO_CODE["RANS_E_WORKSPACE"]


class _Workspace:
    """A stream's scratch memory, and the lock under which a call enqueues its launches."""

    __slots__ = ("lock", "held")

    def __init__(self):
        # the allocator may run finalizers, which may call operators: the same thread enters again
        self.lock = threading.RLock()
        self.held = _NO_WORKSPACE


_workspaces: dict = {}


def _with_workspace(device, stream: int, call, size, where: str):
    """``call(address, bytes)`` with this stream's scratch memory, grown when it is refused.

    Kept per device and stream.  A call is several launches that pass sums to each other
    through that memory, so all of them are enqueued under the stream's lock: those of two
    threads would otherwise mix (the interpreter's own lock is let go of within a call).  A
    buffer that is replaced goes back to the allocator of the stream that still uses it.
    Under stream capture the memory is the graph's own.
    """
    workspace = _workspaces.get((device.index, stream))
    if workspace is None:
        workspace = _workspaces.setdefault((device.index, stream), _Workspace())
    with workspace.lock:
        capturing = torch.cuda.is_current_stream_capturing()
        held = _NO_WORKSPACE if capturing else workspace.held
        rc = call(held[0], held[1])
        if rc == _E_WORKSPACE:
            nbytes = max(size(), 1 << 20)
            buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
            held = (buf.data_ptr(), nbytes, buf)
            if not capturing:
                workspace.held = held
            rc = call(held[0], held[1])
    if rc:
        _check_rc(rc, where)


def release_workspaces() -> None:
    """Give the scratch memory of all streams back to the allocator.

    It is as large as a stream's largest call needed and otherwise kept for the next.  Work that
    is still queued may go on using it, as any freed tensor of its stream.
    """
    for workspace in list(_workspaces.values()):
        with workspace.lock:
            workspace.held = _NO_WORKSPACE


# ---- derivatives -----------------------------------------------------------


def _wants_gradient(*tensors) -> bool:
    """Whether autograd has to know of a call.  Forward mode does not know the operators: their
    results would have no tangents, so tensors that have one are refused."""
    if forward_ad._current_level >= 0:
        for t in tensors:
            if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError("forward-mode derivatives are not supported")
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


class _Once(torch.autograd.Function):
    """Gradients as functions of what they were formed from, so that whoever differentiates them
    again is refused instead of missing a term."""

    @staticmethod
    def forward(ctx, form, *inputs):
        return form()

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("second derivatives are not supported")


def _once(form, *inputs):
    """``form()``, a tuple of gradients; with a graph (``create_graph``) that refuses."""
    return _Once.apply(form, *inputs) if torch.is_grad_enabled() else form()


# ---- group norm --------------------------------------------------------------


def _rows(t: torch.Tensor, name: str):
    """(sample stride, row stride, positions) of a channels-last [N, C, ...] tensor."""
    shape, strides = t.shape, t.stride()
    if len(shape) < 2:
        raise ValueError(f"{name} must be [N, C, ...]")
    if len(shape) == 4 and strides[1] == 1 and strides[2] == strides[3] * shape[3] and shape[3] > 1:
        return strides[0], strides[3], shape[2] * shape[3]
    if shape[1] > 1 and strides[1] != 1:
        raise ValueError(f"{name} must be channels last (its channels next to each other)")
    positions, row = 1, None
    for size, stride in zip(reversed(shape[2:]), reversed(strides[2:])):
        if size != 1 and positions > 0:
            if row is None:
                row = stride
            elif stride != row * positions and size > 0:
                raise ValueError(f"{name}: positions must be evenly spaced in memory")
        positions *= size
    return strides[0], shape[1] if row is None else row, positions


def _channels_last_empty(x: torch.Tensor) -> torch.Tensor:
    if x.dim() == 4 and x.is_contiguous(memory_format=torch.channels_last) and \
            (x.shape[1] == 1 or x.stride(1) == 1):
        return torch.empty_like(x)
    n, c, *rest = x.shape
    return torch.empty((n, *rest, c), dtype=x.dtype, device=x.device).movedim(-1, 1)


def _norm_params(x, num_groups, weight, bias, activation):
    device = _device_of(x, "x")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}")
    if x.dim() < 2 or num_groups < 1 or x.shape[1] % num_groups or x.shape[1] == 0:
        raise ValueError("num_groups must divide x's channels")
    kind = torch.float32
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            kind = t.dtype
            if kind not in DTYPES:
                raise TypeError(f"{name} must be float32, float16 or bfloat16, got {kind}")
            if t.device != device:
                raise ValueError(f"{name} must be on {device}, got {t.device}")
            if t.numel() != x.shape[1] or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous, one value a channel")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias differ in type")
    return device, kind


def group_norm_forward(x: torch.Tensor, num_groups: int, weight=None, bias=None, *,
                       eps: float = 1e-5, activation: str = "none", out=None):
    """Enqueue ``act(group_norm(x))``; returns (y, mean, rstd).

    ``x`` is [N, C, ...] with its channels last in memory (for example
    ``x.to(memory_format=torch.channels_last)``, or tokens [N, S, C] as
    ``x.transpose(1, 2)``); ``y`` is laid out the same.  ``mean`` and ``rstd`` are
    float32 [N, num_groups].
    """
    device, kind = _norm_params(x, num_groups, weight, bias, activation)
    xs, xr, positions = _rows(x, "x")
    if out is None:
        out = _channels_last_empty(x)
    else:
        _out_like(out, x, x.dtype, device, "out")
    ys, yr, _ = _rows(out, "out")
    n, c = x.shape[0], x.shape[1]
    stats = torch.empty((2, n, num_groups), dtype=torch.float32, device=device)
    mean, rstd = stats[0], stats[1]
    if positions == 0 or n == 0:
        return out, mean.fill_(math.nan), rstd.fill_(math.nan)
    lib = load()
    stream = _stream(device)
    args = (x.data_ptr(), xs, xr, n, positions, c, num_groups, DTYPES[x.dtype],
            weight.data_ptr() if weight is not None else None,
            bias.data_ptr() if bias is not None else None, DTYPES[kind], eps,
            ACTIVATIONS[activation], out.data_ptr(), ys, yr, mean.data_ptr(), rstd.data_ptr())
    _with_workspace(device, stream, lambda p, size: lib.lic_group_norm_forward(*args, p, size, stream),
                    lambda: lib.lic_group_norm_workspace_bytes(n, positions, c, num_groups),
                    "lic_group_norm_forward")
    return out, mean, rstd


def group_norm_backward(dy: torch.Tensor, x: torch.Tensor, num_groups: int, weight, bias,
                        mean: torch.Tensor, rstd: torch.Tensor, *, activation: str = "none"):
    """Enqueue the gradients; returns (dx, dweight, dbias), the last two of the
    parameters' type (float32 without parameters)."""
    device, kind = _norm_params(x, num_groups, weight, bias, activation)
    _like(dy, x.dtype, device, "dy")
    if dy.shape != x.shape:
        raise ValueError("dy and x differ in shape")
    n, c = x.shape[0], x.shape[1]
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _like(t, torch.float32, device, name)
        if t.numel() != n * num_groups or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous [N, num_groups]")
    xs, xr, positions = _rows(x, "x")
    gs, gr, _ = _rows(dy, "dy")
    dx = _channels_last_empty(x)
    ds, dr, _ = _rows(dx, "dx")
    grads = torch.empty((2, c), dtype=kind, device=device)
    dweight, dbias = grads[0], grads[1]
    if positions == 0 or n == 0:
        return dx, dweight.zero_(), dbias.zero_()
    lib = load()
    stream = _stream(device)
    args = (dy.data_ptr(), gs, gr, x.data_ptr(), xs, xr, n, positions, c, num_groups,
            DTYPES[x.dtype], weight.data_ptr() if weight is not None else None,
            bias.data_ptr() if bias is not None else None, DTYPES[kind], ACTIVATIONS[activation],
            mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), ds, dr, dweight.data_ptr(),
            dbias.data_ptr())
    _with_workspace(device, stream, lambda p, size: lib.lic_group_norm_backward(*args, p, size, stream),
                    lambda: lib.lic_group_norm_workspace_bytes(n, positions, c, num_groups),
                    "lic_group_norm_backward")
    return dx, dweight, dbias


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, num_groups, weight, bias, eps, activation):
        y, mean, rstd = group_norm_forward(x, num_groups, weight, bias, eps=eps,
                                           activation=activation)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        ctx.num_groups, ctx.activation = num_groups, activation
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        try:
            _rows(dy, "dy")
        except ValueError:  # a gradient of another layout
            dy = _channels_last_empty(dy).copy_(dy)
        dx, dw, db = _once(lambda: group_norm_backward(dy, x, ctx.num_groups, weight, bias, mean, rstd,
                                                       activation=ctx.activation),
                           dy, x, weight, bias)
        need = ctx.needs_input_grad
        return (dx if need[0] else None, None, dw.view_as(weight) if need[2] else None,
                db.view_as(bias) if need[3] else None, None, None)


def group_norm(x: torch.Tensor, num_groups: int, weight=None, bias=None, eps: float = 1e-5,
               activation: str = "none") -> torch.Tensor:
    """Group norm of a channels-last [N, C, ...] tensor and an activation ("none",
    "relu", "silu", "gelu"), differentiable (once, in reverse) in x, weight and bias."""
    if _wants_gradient(x, weight, bias):
        return _GroupNorm.apply(x, num_groups, weight, bias, eps, activation)
    return group_norm_forward(x, num_groups, weight, bias, eps=eps, activation=activation)[0]


# ---- rotary positions ----------------------------------------------------------


def rotary_table(coords: torch.Tensor, rotary_dim: int, *, base: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, low: float = 1.0, high: float = 32.0,
                 original: int = 0, amplitude: float | None = None):
    """Cosines and sines for :func:`rotary`; returns (cos, sin), float32 [rows, rotary_dim / 2].

    ``coords`` (float64, on the GPU) is [rows], a row's position, or [rows, axes],
    for example an image position's row and column: the pairs are split evenly
    over the axes.  For contexts longer than a model was trained on (``original``
    positions), ``scaling`` is

    * "linear": every angle divided by ``factor``;
    * "base": the base raised to ``base * factor ** (n / (n - 1))``, n the pairs of an
      axis, so the slowest pair is divided by ``factor`` and the fastest kept;
    * "ramp": pairs that turn fewer than ``low`` times within ``original`` positions are
      divided by ``factor``, those that turn more than ``high`` times are kept, with a
      straight ramp between; ``amplitude`` defaults to 0.1 ln(factor) + 1.
    """
    if not isinstance(coords, torch.Tensor) or coords.dtype != torch.float64:
        raise TypeError("coords must be a float64 tensor")
    if not coords.is_cuda or coords.device.index != torch.cuda.current_device():
        raise ValueError(f"coords must be on the current device, got {coords.device}")
    if coords.dim() not in (1, 2) or not coords.is_contiguous():
        raise ValueError("coords must be contiguous [rows] or [rows, axes]")
    axes = 1 if coords.dim() == 1 else coords.shape[1]
    if rotary_dim < 2 or rotary_dim % 2 or axes < 1 or (rotary_dim // 2) % axes:
        raise ValueError("rotary_dim must be even, its pairs a multiple of the axes")
    if scaling not in ("none", "linear", "base", "ramp"):
        raise ValueError("scaling must be none, linear, base or ramp")
    if not factor > 0 or not base > 0:
        raise ValueError("base and factor must be positive")
    gain = 1.0 if amplitude is None else amplitude
    if scaling == "none":
        factor = 1.0
    elif scaling == "linear":
        low = high = 0.0
    elif scaling == "base":
        n = rotary_dim // 2 // axes
        if n > 1:
            base = base * factor ** (n / (n - 1))
        factor = 1.0
    else:
        if original <= 0 or not high > low:
            raise ValueError("ramp scaling needs original > 0 and high > low")
        if amplitude is None:
            gain = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    rows = coords.shape[0]
    cos = torch.empty((rows, rotary_dim // 2), dtype=torch.float32, device=coords.device)
    sin = torch.empty_like(cos)
    stream = _stream(coords.device)
    rc = load().lic_rotary_table(coords.data_ptr(), rows, axes, rotary_dim, base, factor, low, high,
                                 float(original), gain, cos.data_ptr(), sin.data_ptr(), stream)
    if rc:
        _check_rc(rc, "lic_rotary_table")
    return cos, sin


_ROTARY = struct.Struct("=8Qq12q7q3q")


def _heads(t: torch.Tensor, name: str):
    """Strides (batch, row, head) of a [B, S, heads, dim] tensor."""
    s = t.stride()
    if len(s) != 4:
        raise ValueError(f"{name} must be [batch, rows, heads, dim]")
    if s[3] != 1 and t.shape[3] > 1:
        raise ValueError(f"{name}: a head's values must be next to each other")
    return s[:3]


def _rotary(q, k, cos, sin, positions, interleaved, inverse, status, out):
    device = _device_of(q, "q")
    qs = _heads(q, "q")
    b, s, h, d = q.shape
    if h < 1:
        raise ValueError("q has no heads")
    kh, ks, kos = 0, (0, 0, 0), (0, 0, 0)
    if k is not None:
        _like(k, q.dtype, device, "k")
        ks = _heads(k, "k")
        kh = k.shape[2]
        if k.shape[0] != b or k.shape[1] != s or k.shape[3] != d:
            raise ValueError("q and k differ in batch, rows or dim")
    _like(cos, torch.float32, device, "cos")
    _like(sin, torch.float32, device, "sin")
    if cos.shape != sin.shape or cos.dim() != 2 or not (cos.is_contiguous() and sin.is_contiguous()):
        raise ValueError("cos and sin must be contiguous [rows, rotary_dim / 2]")
    rows, pairs = cos.shape
    if pairs < 1 or 2 * pairs > d:
        raise ValueError("the tables have more pairs than a head")
    batch_step = 0
    if positions is not None:
        _like(positions, torch.int32, device, "positions")
        if not positions.is_contiguous() or tuple(positions.shape) not in ((s,), (b, s)):
            raise ValueError("positions must be contiguous [rows] or [batch, rows]")
        batch_step = s if positions.dim() == 2 else 0
    elif rows < s:
        raise ValueError("the tables have fewer rows than there are positions")
    if status is not None:
        _like(status, torch.int32, device, "status")
    if out is None:
        qo = _dense_like(q)
        ko = _dense_like(k) if kh else None
    else:
        qo, ko = out
        for o, t, name in ((qo, q, "q"), (ko, k, "k")):
            if t is not None:
                _out_like(o, t, q.dtype, device, f"out of {name}")
    qos = _heads(qo, "out of q")
    if kh:
        kos = _heads(ko, "out of k")
    if q.numel() == 0:
        return qo, ko if kh else (k if k is None else torch.empty_like(k))
    args = _ROTARY.pack(q.data_ptr(), k.data_ptr() if kh else 0, qo.data_ptr(),
                        ko.data_ptr() if kh else 0, cos.data_ptr(), sin.data_ptr(),
                        positions.data_ptr() if positions is not None else 0,
                        status.data_ptr() if status is not None else 0, batch_step, *qs, *ks, *qos,
                        *kos, b, s, h, kh, d, 2 * pairs, rows, DTYPES[q.dtype],
                        1 if interleaved else 0, 1 if inverse else 0)
    rc = load().lic_rotary(args, _stream(device))
    if rc:
        _check_rc(rc, "lic_rotary")
    return qo, ko


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, cos, sin, positions, interleaved, inverse, status):
        ctx.save_for_backward(cos, sin, positions)
        ctx.options = interleaved, inverse
        qo, ko = _rotary(q, k, cos, sin, positions, interleaved, inverse, status, None)
        return (qo, ko) if k is not None else qo

    @staticmethod
    def backward(ctx, dq, dk=None):
        cos, sin, positions = ctx.saved_tensors
        interleaved, inverse = ctx.options
        dq = dq if dq.stride(-1) == 1 else dq.contiguous()
        if dk is not None and dk.stride(-1) != 1:
            dk = dk.contiguous()
        # the turn is linear: its gradient is the inverse, which autograd knows in its turn
        gq, gk = rotary(dq, dk, cos, sin, positions=positions, interleaved=interleaved,
                        inverse=not inverse)
        return gq, gk, None, None, None, None, None, None


def rotary(q: torch.Tensor, k: torch.Tensor | None, cos: torch.Tensor, sin: torch.Tensor, *,
           positions: torch.Tensor | None = None, interleaved: bool = False,
           inverse: bool = False, status: torch.Tensor | None = None, out=None):
    """Turn the first ``2 * cos.shape[1]`` values of each head; returns (q, k).

    ``q`` is [B, S, heads, dim], ``k`` [B, S, kv_heads, dim] or None.  Pairs are
    (j, j + half) or, interleaved, (2 j, 2 j + 1).  ``positions`` (int32, [S] or
    [B, S]) are rows of the tables, by default 0 .. S - 1; one outside them gives
    a token of NaN and, where ``status`` (int32[1], zeroed by the caller) is given,
    RANS_E_INDEX in it.  ``inverse`` turns back, which is also the gradient with
    respect to the inputs.  ``out`` is a pair of outputs, possibly (q, k) themselves;
    it is for calls outside autograd.  Gradients are those of q and k, of any order; the tables
    have none.
    """
    if _wants_gradient(cos, sin):
        raise NotImplementedError("cos and sin have no gradients")
    if _wants_gradient(q, k):
        if out is not None:
            raise ValueError("out is for calls outside autograd")
        r = _Rotary.apply(q, k, cos, sin, positions, interleaved, inverse, status)
        return r if k is not None else (r, None)
    return _rotary(q, k, cos, sin, positions, interleaved, inverse, status, out)


# ---- attention -------------------------------------------------------------------


_ATTENTION = struct.Struct("=11Q24q4q9qd")
_NO_STRIDES = (0, 0, 0)


def _attention_common(q, k, v, causal, window, mask, key_lengths, scale):
    device = _device_of(q, "q")
    _like(k, q.dtype, device, "k")
    _like(v, q.dtype, device, "v")
    qs, ks, vs = _heads(q, "q"), _heads(k, "k"), _heads(v, "v")
    b, n, h, d = q.shape
    if k.shape != v.shape or k.shape[0] != b or k.shape[3] != d:
        raise ValueError("q, k and v differ in batch or dim, or k and v in shape")
    m, kv = k.shape[1], k.shape[2]
    if kv < 1 or h % kv or h < 1:
        raise ValueError("heads must be a multiple of kv heads")
    if not 1 <= d <= MAX_HEAD_DIM:
        raise ValueError(f"dim must be 1 .. {MAX_HEAD_DIM}")
    left, right = -1, -1
    if window is not None:
        left, right = (-1 if w is None else int(w) for w in window)
        if left < -1 or right < -1:
            raise ValueError("window must be (left, right), each at least 0 or None")
    if causal:
        right = 0
    mask_ptr, ms = 0, (0, 0, 0, 0)
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError("mask must be a bool or uint8 tensor")
        if mask.device != device:
            raise ValueError(f"mask must be on {device}, got {mask.device}")
        try:
            ms = mask.expand(b, h, n, m).stride()
        except RuntimeError:
            raise ValueError("mask must be broadcast to [batch, heads, queries, keys]") from None
        mask_ptr = mask.data_ptr()
    length_ptr = 0
    if key_lengths is not None:
        _like(key_lengths, torch.int32, device, "key_lengths")
        if key_lengths.shape != (b,) or not key_lengths.is_contiguous():
            raise ValueError("key_lengths must be contiguous [batch]")
        length_ptr = key_lengths.data_ptr()
    if scale is None:
        scale = d ** -0.5
    elif not (scale > 0 and math.isfinite(scale)):
        raise ValueError("scale must be positive and finite")
    sizes = (b, n, m, h, kv, d, DTYPES[q.dtype], left, right, scale)
    return device, (qs, ks, vs), (mask_ptr, length_ptr), ms, sizes


def attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = False,
                      window=None, mask=None, key_lengths=None, scale: float | None = None,
                      out=None):
    """Enqueue softmax(scale q k^T) v over the visible keys; returns (out, lse).

    ``q`` is [B, Q, heads, dim], ``k`` and ``v`` [B, S, kv_heads, dim] (any strides
    but the last; kv_heads divides heads), ``out`` like q and ``lse`` float32
    [B, heads, Q].  ``key_lengths`` (int32 [B]) are the keys in use, for example of a
    cache; queries are a batch's last positions.  ``causal`` and ``window``
    = (left, right) limit a query to keys around its position, ``mask`` (bool or
    uint8, broadcast to [B, heads, Q, S]) to those where it is true.  A query that
    sees nothing gives 0 and an lse of -inf.
    """
    device, (qs, ks, vs), ptrs, ms, sizes = _attention_common(q, k, v, causal, window, mask,
                                                              key_lengths, scale)
    b, n, h, d = q.shape
    if out is None:
        out = _dense_like(q)
    else:
        _out_like(out, q, q.dtype, device, "out")
    lse = torch.empty((b, h, n), dtype=torch.float32, device=device)
    args = _ATTENTION.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           lse.data_ptr(), 0, 0, 0, 0, *ptrs, *qs, *ks, *vs, *_heads(out, "out"),
                           *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES, *ms, *sizes)
    lib = load()
    stream = _stream(device)
    _with_workspace(device, stream, lambda p, size: lib.lic_attention_forward(args, p, size, stream),
                    lambda: lib.lic_attention_workspace_bytes(args, 0), "lic_attention_forward")
    return out, lse


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       out: torch.Tensor, lse: torch.Tensor, *, causal: bool = False, window=None,
                       mask=None, key_lengths=None, scale: float | None = None):
    """Enqueue the gradients of :func:`attention_forward`; returns (dq, dk, dv).

    Takes the forward call's inputs, options and outputs.  The probabilities are
    formed again from q, k and lse.  dk and dv of heads that share a kv head are
    their sums; rows past ``key_lengths`` are 0.
    """
    device, (qs, ks, vs), ptrs, ms, sizes = _attention_common(q, k, v, causal, window, mask,
                                                              key_lengths, scale)
    for t, name in ((dout, "dout"), (out, "out")):
        _like(t, q.dtype, device, name)
        if t.shape != q.shape:
            raise ValueError(f"{name} and q differ in shape")
    _like(lse, torch.float32, device, "lse")
    b, n, h, d = q.shape
    if lse.shape != (b, h, n) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous [batch, heads, queries]")
    dq, dk, dv = _dense_like(q), _dense_like(k), _dense_like(v)
    s = dk.stride()[:3]
    args = _ATTENTION.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                           dv.data_ptr(), *ptrs, *qs, *ks, *vs, *_heads(out, "out"),
                           *_heads(dout, "dout"), *dq.stride()[:3], *s, *s, *ms, *sizes)
    lib = load()
    stream = _stream(device)
    _with_workspace(device, stream, lambda p, size: lib.lic_attention_backward(args, p, size, stream),
                    lambda: lib.lic_attention_workspace_bytes(args, 1), "lic_attention_backward")
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, mask, key_lengths, causal, window, scale):
        options = {"causal": causal, "window": window, "scale": scale}
        out, lse = attention_forward(q, k, v, mask=mask, key_lengths=key_lengths, **options)
        ctx.save_for_backward(q, k, v, out, lse, mask, key_lengths)
        ctx.options = options
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    def backward(ctx, dout, _):
        q, k, v, out, lse, mask, key_lengths = ctx.saved_tensors
        if dout.stride(-1) != 1:
            dout = dout.contiguous()
        grads = _once(lambda: attention_backward(dout, q, k, v, out, lse, mask=mask,
                                                 key_lengths=key_lengths, **ctx.options),
                      dout, q, k, v)
        return (*grads, None, None, None, None, None)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = False,
              window=None, mask=None, key_lengths=None, scale: float | None = None) -> torch.Tensor:
    """Attention as :func:`attention_forward`, differentiable (once, in reverse) in q, k and v;
    returns out."""
    if _wants_gradient(q, k, v):
        return _Attention.apply(q, k, v, mask, key_lengths, causal, window, scale)[0]
    return attention_forward(q, k, v, causal=causal, window=window, mask=mask,
                             key_lengths=key_lengths, scale=scale)[0]
