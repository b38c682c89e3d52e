"""Network operators around the coder: group norm with an activation, RMS norm with the
residual's addition, rotary positions, attention and linear attention, forward and backward,
and clipping of gradients (``include/lic_layers.h``).

A learned image codec's transforms and its entropy model run right before the
coder; these are the parts of them that convolutions and matrix products leave
over, as hand-written HIP kernels in ``liblic_layers.so``.  Sums are taken in an
order that a call's sizes, windows and key lengths alone decide, wherever its values
lie, so an encoder and a decoder that make the same call predict the same scales, bit
for bit.  A call of another size (a single token instead of a whole latent) may differ
in the last bits: an encoder has to step where its decoder does.

:func:`group_norm`, :func:`rms_norm`, :func:`rotary`, :func:`attention` and
:func:`linear_attention` work with autograd (what they cannot differentiate they refuse: forward
mode, second derivatives but rotary's).  The
``*_forward`` and ``*_backward`` functions are the calls beneath them, for programs that
keep their own gradients.  As in :mod:`.binding`, torch only supplies device memory and
the current stream, nothing is synchronised, and there is no CPU path.
"""
from __future__ import annotations

import array
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
    "lic_rms_norm_workspace_bytes",
    "lic_rms_norm_forward",
    "lic_rms_norm_backward",
    "lic_rotary_table",
    "lic_rotary",
    "lic_attention_workspace_bytes",
    "lic_attention_forward",
    "lic_attention_backward",
    "lic_linear_attention_workspace_bytes",
    "lic_linear_attention_forward",
    "lic_linear_attention_backward",
    "lic_clip_gradients_workspace_bytes",
    "lic_gradient_norm",
    "lic_clip_gradients",
    "lic_layers_target",
)

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
FORMATS = {"e4m3": (1, torch.float8_e4m3fn), "int8": (2, torch.int8)}
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
        lib.lic_rms_norm_workspace_bytes.argtypes = [i64, i64, i64]
        lib.lic_rms_norm_workspace_bytes.restype = u64
        lib.lic_rms_norm_forward.argtypes = [st, vp]
        lib.lic_rms_norm_forward.restype = ctypes.c_int
        lib.lic_rms_norm_backward.argtypes = [st, vp, u64, vp]
        lib.lic_rms_norm_backward.restype = ctypes.c_int
        lib.lic_linear_attention_workspace_bytes.argtypes = [st, i32]
        lib.lic_linear_attention_workspace_bytes.restype = u64
        for name in ("lic_linear_attention_forward", "lic_linear_attention_backward"):
            getattr(lib, name).argtypes = [st, vp, u64, vp]
            getattr(lib, name).restype = ctypes.c_int
        lib.lic_clip_gradients_workspace_bytes.argtypes = [st, i64]
        lib.lic_clip_gradients_workspace_bytes.restype = u64
        lib.lic_gradient_norm.argtypes = [st, i64, vp, vp, u64, vp]
        lib.lic_gradient_norm.restype = ctypes.c_int
        lib.lic_clip_gradients.argtypes = [st, i64, f64, vp, vp, u64, vp]
        lib.lic_clip_gradients.restype = ctypes.c_int
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
    device = t.device
    if device.index != torch._C._cuda_getDevice():  # a tensor there has initialised the GPU
        raise ValueError(f"{name} is on {device}, which is not the current device")
    return device


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
    _out_of(out, t.shape, dtype, device, name)


def _out_of(out, shape, dtype, device, name):
    _like(out, dtype, device, name)
    if out.shape != shape:
        raise ValueError(f"{name} differs in shape")
    if out.is_contiguous():
        return
    end = 1  # of what the narrower strides reach
    for stride, size in sorted((st, n) for st, n in zip(out.stride(), out.shape) if n > 1):
        if stride < end:
            raise ValueError(f"{name} overlaps itself")
        end += stride * (size - 1)


def _written(tensors):
    """Tells autograd of tensors of the caller's that a call writes, so that a graph that still needs
    their old values says so."""
    torch.autograd.graph.increment_version([t for t in tensors if t is not None and not t.is_inference()])


def _runs(t):
    """Where a tensor's values lie: the bytes of its runs without gaps, and the (stride, count) of their
    repetitions, widest first, in bytes."""
    run, dims = t.element_size(), []
    for stride, n in sorted((st * t.element_size(), n) for st, n in zip(t.stride(), t.shape) if n > 1 and st > 0):
        if dims and stride == dims[0][0] * dims[0][1]:
            dims[0] = (dims[0][0], dims[0][1] * n)
        elif not dims and stride == run:
            run *= n
        else:
            dims.insert(0, (stride, n))
    return run, dims


_MANY = 64


def _meet(apart, run, dims, other_run, other_dims) -> bool:
    """Whether runs and others that begin ``apart`` bytes behind them have a byte in common.  Where that would
    take more than some comparisons (strides that are no multiples of each other), they count as if they had."""
    end = run + sum(stride * (n - 1) for stride, n in dims)
    other_end = other_run + sum(stride * (n - 1) for stride, n in other_dims)
    if apart >= end or apart + other_end <= 0:
        return False
    if not dims and not other_dims:
        return True
    stride, n = dims[0] if dims else (0, 1)
    other, m = other_dims[0] if other_dims else (0, 1)
    # the repetitions of the wider stride, of both where it is the same: only their difference counts
    wide, first, last = max(stride, other), 0, 0
    if stride == wide:
        dims, last, end = dims[1:], n - 1, end - stride * (n - 1)
    if other == wide:
        other_dims, first, other_end = other_dims[1:], 1 - m, other_end - other * (m - 1)
    first, last = max(first, (apart - end) // wide + 1), min(last, -((-apart - other_end) // wide) - 1)
    return last - first >= _MANY or any(_meet(apart - i * wide, run, dims, other_run, other_dims)
                                        for i in range(first, last + 1))


def _overlapping(out, tensors):
    """Those that have memory in common with ``out``."""
    at, found = out.data_ptr(), []
    end = at + out.untyped_storage().nbytes()
    for t in tensors:
        if t is not None:
            begin = t.data_ptr()
            # a look at the storages first, which is quick
            if begin < end and at < begin + t.untyped_storage().nbytes() and t.numel() and out.numel() and \
                    _meet(begin - at, *_runs(out), *_runs(t)):
                found.append(t)
    return found


def _in_place(out, name, inputs, others=()):
    """An output may be one of ``inputs`` entry by entry: not overlap one that is shifted or lies otherwise, and
    none of ``others``."""
    if out is None:
        return
    for t in _overlapping(out, [t for t in inputs if t is not out]):
        if t.data_ptr() != out.data_ptr() or t.dtype is not out.dtype or \
                any(n > 1 and a != b for n, a, b in zip(out.shape, out.stride(), t.stride())):
            raise ValueError(f"{name} overlaps an input and is laid out differently, or shifted")
    if _overlapping(out, others):
        raise ValueError(f"{name} overlaps what it must not be")


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


# ---- RMS norm ------------------------------------------------------------------


_RMS_NORM = struct.Struct("=11Q14q6qd")
_NO_ROWS = (0, 0)


def _token_rows(t: torch.Tensor, name: str):
    """(sample stride, row stride) of a [N, ..., C] tensor whose rows are evenly spaced within a sample."""
    shape, strides = t.shape, t.stride()
    if shape[-1] > 1 and strides[-1] != 1:
        raise ValueError(f"{name}: a row's values must be next to each other")
    if len(shape) == 1:
        return 0, shape[0]
    if len(shape) == 2:
        return 0, strides[0]
    positions, row = 1, None
    for size, stride in zip(reversed(shape[1:-1]), reversed(strides[1:-1])):
        if size != 1 and positions > 0:
            if row is None:
                row = stride
            elif stride != row * positions and size > 0:
                raise ValueError(f"{name}: rows must be evenly spaced in memory")
        positions *= size
    return strides[0], shape[-1] if row is None else row


def _sample_rows(shape):
    """(samples, positions): all but the first axis count as positions, a matrix is one sample."""
    if len(shape) < 3:
        return 1, shape[0] if len(shape) == 2 else 1
    return shape[0], math.prod(shape[1:-1])


def _rms_params(x, name, weight, eps):
    device = _device_of(x, name)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{name} must be [..., C]")
    if not 0 <= eps < 1e30:
        raise ValueError("eps must be at least 0")
    if weight is None:
        return device, torch.float32
    if not isinstance(weight, torch.Tensor) or weight.dtype not in DTYPES:
        raise TypeError("weight must be a float32, float16 or bfloat16 tensor")
    if weight.device != device:
        raise ValueError(f"weight must be on {device}, got {weight.device}")
    if weight.numel() != x.shape[-1] or not weight.is_contiguous():
        raise ValueError("weight must be contiguous, one value a channel")
    return device, weight.dtype


def _same(t, x, device, name):
    _like(t, x.dtype, device, name)
    if t.shape != x.shape:
        raise ValueError(f"{name} and x differ in shape")


def _rms_forward(x, weight, residual, eps, code, y, stat, rstd, sum_out, device, kind):
    """The call beneath the forward functions; returns h.  ``stat`` holds the scales of 8 bits."""
    h, rs, hs = x, _NO_ROWS, _NO_ROWS
    if residual is not None:
        _same(residual, x, device, "residual")
        if sum_out is None:
            h = _dense_like(x)
        else:
            _out_like(sum_out, x, x.dtype, device, "sum_out")
            h = sum_out
        if sum_out is not None and _overlapping(h, (y,)):
            raise ValueError("out and sum_out must not be one place")
    elif sum_out is not None:
        raise ValueError("sum_out is for calls with a residual")
    c = x.shape[-1]
    if x.is_contiguous() and y.is_contiguous() and \
            (residual is None or (residual.is_contiguous() and h.is_contiguous())):
        samples, positions = 1, x.numel() // c  # the usual layout: all rows one after another
        xs = rs = ys = hs = (0, c)
    else:
        samples, positions = _sample_rows(x.shape)
        xs, ys = _token_rows(x, "x"), _token_rows(y, "out")
        if residual is not None:
            rs, hs = _token_rows(residual, "residual"), _token_rows(h, "sum_out")
    if samples and positions:
        args = _RMS_NORM.pack(x.data_ptr(), residual.data_ptr() if residual is not None else 0,
                              weight.data_ptr() if weight is not None else 0, y.data_ptr(),
                              h.data_ptr() if residual is not None else 0,
                              rstd.data_ptr() if rstd is not None else 0,
                              stat.data_ptr() if stat is not None else 0, 0, 0, 0, 0, *xs, *rs, *ys,
                              *hs, 0, 0, 0, 0, 0, 0, samples, positions, c, DTYPES[x.dtype],
                              DTYPES[kind], code, eps)
        rc = load().lic_rms_norm_forward(args, _stream(device))
        if rc:
            _check_rc(rc, "lic_rms_norm_forward")
    return h


def rms_norm_forward(x: torch.Tensor, weight=None, *, residual=None, eps: float = 1e-6, out=None,
                     sum_out=None):
    """Enqueue the norm of ``h = x + residual`` over the last axis; returns (y, h, rstd).

    ``x`` is [..., C] with a row's values next to each other and the rows of a sample (all axes but
    the first) evenly spaced, for example tokens [N, S, C] cut out of a wider tensor; ``residual`` is
    like it.  ``h`` is rounded to x's type before the norm (without a residual it is ``x``
    itself), ``y = weight * h * rstd`` and ``rstd = 1 / sqrt(mean(h^2) + eps)``, float32 [...].
    ``out`` and ``sum_out`` are places for y and h, and each may be x or residual, but not overlap
    them otherwise.
    """
    device, kind = _rms_params(x, "x", weight, eps)
    given = (out, sum_out)
    if out is None:
        out = _dense_like(x)
    else:
        _out_like(out, x, x.dtype, device, "out")
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
    if given[0] is not None or given[1] is not None:
        _in_place(given[0], "out", (x, residual), (weight,))
        _in_place(given[1], "sum_out", (x, residual), (weight,))
        _written(given)
    h = _rms_forward(x, weight, residual, eps, 0, out, None, rstd, sum_out, device, kind)
    return out, h, rstd


def rms_norm_8bit(x: torch.Tensor, weight=None, *, residual=None, eps: float = 1e-6,
                  format: str = "e4m3", out=None, sum_out=None):
    """The norm of ``h = x + residual`` in 8 bits, for a product that takes them; returns
    (y, scales, h).

    ``y`` is float8_e4m3fn ("e4m3") or int8 ("int8") and stands for ``y * scales[..., None]``: a
    row's scale (float32) is its largest size over 448 or 127, so nothing is cut off.  A row that is
    not all finite stands for NaN.  The rest is as in :func:`rms_norm_forward`.  There is no gradient.
    """
    if _wants_gradient(x, weight, residual):
        raise NotImplementedError("the norm in 8 bits has no gradients")
    device, kind = _rms_params(x, "x", weight, eps)
    if format not in FORMATS:
        raise ValueError(f"format must be one of {', '.join(FORMATS)}")
    code, dtype = FORMATS[format]
    given = (out, sum_out)
    if out is None:
        out = torch.empty(x.shape, dtype=dtype, device=device)
    else:
        _out_like(out, x, dtype, device, "out")
    scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
    if given[0] is not None or given[1] is not None:
        _in_place(given[0], "out", (x, residual), (weight,))
        _in_place(given[1], "sum_out", (x, residual), (weight,))
        _written(given)
    h = _rms_forward(x, weight, residual, eps, code, out, scales, None, sum_out, device, kind)
    return out, scales, h


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight, rstd: torch.Tensor, *, dsum=None,
                      out=None):
    """Enqueue the gradients; returns (dx, dweight).

    Takes the forward call's h and rstd.  ``dx`` is the gradient of x and of the residual alike;
    ``dsum`` is what comes to h from elsewhere (the residual stream behind it), and is in it.
    ``dweight`` is of the weight's type (float32 without one).  ``out`` is a place for dx, and may
    be dy or dsum.
    """
    device, kind = _rms_params(h, "h", weight, 0.0)
    _same(dy, h, device, "dy")
    if dsum is not None:
        _same(dsum, h, device, "dsum")
    _like(rstd, torch.float32, device, "rstd")
    if rstd.shape != h.shape[:-1] or not rstd.is_contiguous():
        raise ValueError("rstd must be contiguous, one value a row")
    if out is None:
        out = _dense_like(h)
    else:
        _out_like(out, h, h.dtype, device, "out")
        _in_place(out, "out", (dy, dsum, h), (weight, rstd))
        _written((out,))
    c = h.shape[-1]
    dweight = torch.empty(c, dtype=kind, device=device)
    if h.is_contiguous() and dy.is_contiguous() and out.is_contiguous() and \
            (dsum is None or dsum.is_contiguous()):
        samples, positions = 1, h.numel() // c
        hs = gs = ss = outs = (0, c)
    else:
        samples, positions = _sample_rows(h.shape)
        hs, gs, outs = _token_rows(h, "h"), _token_rows(dy, "dy"), _token_rows(out, "out")
        ss = _token_rows(dsum, "dsum") if dsum is not None else _NO_ROWS
    args = _RMS_NORM.pack(h.data_ptr(), 0, weight.data_ptr() if weight is not None else 0, 0, 0,
                          rstd.data_ptr(), 0, dy.data_ptr(),
                          dsum.data_ptr() if dsum is not None else 0, out.data_ptr(),
                          dweight.data_ptr(), *hs, 0, 0, 0, 0, 0, 0, *gs, *ss, *outs, samples, positions,
                          c, DTYPES[h.dtype], DTYPES[kind], 0, 0.0)
    if samples == 0 or positions == 0:
        return out, dweight.zero_()
    lib = load()
    stream = _stream(device)
    _with_workspace(device, stream, lambda p, size: lib.lic_rms_norm_backward(args, p, size, stream),
                    lambda: lib.lic_rms_norm_workspace_bytes(samples, positions, c),
                    "lic_rms_norm_backward")
    return out, dweight


def _rows_or_dense(t, name):
    """A gradient as it is if its layout is taken, else a copy."""
    if t is None:
        return None
    try:
        _token_rows(t, name)
    except ValueError:
        return t.contiguous()
    return t


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, rstd = rms_norm_forward(x, weight, residual=residual, eps=eps)
        ctx.save_for_backward(h, weight, rstd)
        ctx.set_materialize_grads(False)
        return y, (h if residual is not None else None)

    @staticmethod
    def backward(ctx, dy, dsum):
        h, weight, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dy is None:  # the norm itself was not used
            return dsum, None, dsum if need[2] else None, None
        dy, dsum = _rows_or_dense(dy, "dy"), _rows_or_dense(dsum, "dsum")
        inputs = [t for t in (dy, dsum, h, weight) if t is not None]
        dx, dw = _once(lambda: rms_norm_backward(dy, h, weight, rstd, dsum=dsum), *inputs)
        return (dx if need[0] else None, dw.view_as(weight) if need[1] else None,
                dx if need[2] else None, None)


def rms_norm(x: torch.Tensor, weight=None, residual=None, eps: float = 1e-6):
    """RMS norm over the last axis, differentiable (once, in reverse) in x, weight and residual.

    Returns y; with a ``residual`` it returns (y, x + residual), so the sum is formed where it is
    read.
    """
    if _wants_gradient(x, weight, residual):
        y, h = _RMSNorm.apply(x, weight, residual, eps)
    else:
        y, h, _ = rms_norm_forward(x, weight, residual=residual, eps=eps)
    return (y, h) if residual is not None else y


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


# ---- linear attention ---------------------------------------------------------------


_LINEAR = struct.Struct("=15Q36q7qd")


def _state(t, shape, device, name):
    """Address and strides (batch, head, row) of a state, or of none."""
    if t is None:
        return 0, _NO_STRIDES
    _like(t, torch.float32, device, name)
    if t.shape != shape:
        raise ValueError(f"{name} must be [batch, heads, dim, value dim]")
    s = t.stride()
    if s[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name}: a row's values must be next to each other")
    return t.data_ptr(), s[:3]


def _linear_common(q, k, v, log_decay, state, lengths, scale):
    device = _device_of(q, "q")
    _like(k, q.dtype, device, "k")
    _like(v, q.dtype, device, "v")
    strides = _heads(q, "q"), _heads(k, "k"), _heads(v, "v")
    b, s, h, d = q.shape
    vb, vs, kv, e = v.shape
    if k.shape != (b, s, kv, d) or vb != b or vs != s:
        raise ValueError("q, k and v differ in batch, rows or dim, or k and v in heads")
    if kv < 1 or h % kv or h < 1:
        raise ValueError("heads must be a multiple of kv heads")
    if not (1 <= d <= MAX_HEAD_DIM and 1 <= e <= MAX_HEAD_DIM):
        raise ValueError(f"dim and value dim must be 1 .. {MAX_HEAD_DIM}")
    _like(log_decay, torch.float32, device, "log_decay")
    if log_decay.shape != (h,) or not log_decay.is_contiguous():
        raise ValueError("log_decay must be contiguous [heads]")
    length_ptr = 0
    if lengths is not None:
        _like(lengths, torch.int32, device, "lengths")
        if lengths.shape != (b,) or not lengths.is_contiguous():
            raise ValueError("lengths must be contiguous [batch]")
        length_ptr = lengths.data_ptr()
    if scale is None:
        scale = d ** -0.5
    elif not (scale > 0 and math.isfinite(scale)):
        raise ValueError("scale must be positive and finite")
    shape = (b, h, d, e)
    return device, strides, _state(state, shape, device, "state"), length_ptr, shape, \
        (b, s, h, kv, d, e, DTYPES[q.dtype], scale)


def linear_attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             log_decay: torch.Tensor, *, state=None, lengths=None,
                             scale: float | None = None, out=None, state_out=None):
    """Enqueue linear attention with a decay for each head; returns (out, state_out).

    A head's state S, float32 [dim, value dim], goes from token to token:
    ``S = exp(log_decay[head]) * S + outer(k, v)``, ``out = scale * q @ S``.  ``q`` is [B, S, heads,
    dim], ``k`` [B, S, kv_heads, dim], ``v`` [B, S, kv_heads, value_dim] (any strides but the last;
    kv_heads divides heads), ``log_decay`` float32 [heads], ``out`` [B, S, heads, value_dim].
    ``state`` and ``state_out``, [B, heads, dim, value_dim], are S before the first token (None:
    zeros) and behind the last; a decoder that steps passes one tensor as both.  ``out`` must not
    overlap an input or ``state_out``, nor that one any input but ``state`` as a whole.  ``lengths``
    (int32 [B]) are the tokens in use: rows behind them are not read, their out is 0, and the
    state is that behind the last one in use.
    """
    device, strides, (state_ptr, ss), length_ptr, shape, sizes = \
        _linear_common(q, k, v, log_decay, state, lengths, scale)
    out_shape, given = (*q.shape[:3], shape[3]), out
    if out is None:
        out = torch.empty(out_shape, dtype=q.dtype, device=device)
    else:
        _out_of(out, out_shape, q.dtype, device, "out")
        if _overlapping(out, (q, k, v, log_decay, state, lengths)):
            raise ValueError("out must not be an input")
        _written((out,))
    if state_out is None:
        state_out = torch.empty(shape, dtype=torch.float32, device=device)
    else:
        _out_of(state_out, shape, torch.float32, device, "state_out")
        _in_place(state_out, "state_out", (state,), (q, k, v, log_decay, lengths, given))
        _written((state_out,))
    last_ptr, ls = _state(state_out, shape, device, "state_out")
    args = _LINEAR.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), state_ptr, length_ptr,
                        out.data_ptr(), last_ptr, 0, 0, 0, 0, 0, 0, 0, *strides[0], *strides[1], *strides[2],
                        *_heads(out, "out"), *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES, *ss, *ls,
                        *_NO_STRIDES, *_NO_STRIDES, *sizes)
    lib = load()
    stream = _stream(device)
    if q.shape[1] == 1:  # a single token takes no scratch memory
        rc = lib.lic_linear_attention_forward(args, None, 0, stream)
        if rc:
            _check_rc(rc, "lic_linear_attention_forward")
        return out, state_out
    _with_workspace(device, stream, lambda p, size: lib.lic_linear_attention_forward(args, p, size, stream),
                    lambda: lib.lic_linear_attention_workspace_bytes(args, 0),
                    "lic_linear_attention_forward")
    return out, state_out


def linear_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                              log_decay: torch.Tensor, *, dstate=None, state=None, lengths=None,
                              scale: float | None = None, decay: bool = True):
    """Enqueue the gradients of :func:`linear_attention_forward`; returns (dq, dk, dv, dlog_decay,
    dstate_in).

    Takes the forward call's inputs, ``dout``, and ``dstate``, the gradient that comes to
    ``state_out`` (None: 0).  ``dlog_decay`` is float32 [heads], or None with ``decay=False``;
    ``dstate_in`` is the gradient of ``state``, or None without one.  dk and dv of heads that share a
    kv head are their sums; rows behind ``lengths`` are 0.
    """
    device, strides, (state_ptr, ss), length_ptr, shape, sizes = \
        _linear_common(q, k, v, log_decay, state, lengths, scale)
    _like(dout, q.dtype, device, "dout")
    if dout.shape != (*q.shape[:3], shape[3]):
        raise ValueError("dout must be [batch, rows, heads, value dim]")
    dstate_ptr, ds = _state(dstate, shape, device, "dstate")
    dq, dk, dv = _dense_like(q), _dense_like(k), _dense_like(v)
    dlog = torch.empty(shape[1], dtype=torch.float32, device=device) if decay else None
    first = torch.empty(shape, dtype=torch.float32, device=device) if state is not None else None
    first_ptr, fs = _state(first, shape, device, "dstate_in")
    args = _LINEAR.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), state_ptr, length_ptr, 0, 0,
                        dout.data_ptr(), dstate_ptr, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                        dlog.data_ptr() if decay else 0, first_ptr, *strides[0], *strides[1], *strides[2],
                        *_NO_STRIDES, *_heads(dout, "dout"), *dq.stride()[:3], *dk.stride()[:3], *dv.stride()[:3],
                        *ss, *_NO_STRIDES, *ds, *fs, *sizes)
    lib = load()
    stream = _stream(device)
    _with_workspace(device, stream, lambda p, size: lib.lic_linear_attention_backward(args, p, size, stream),
                    lambda: lib.lic_linear_attention_workspace_bytes(args, 1),
                    "lic_linear_attention_backward")
    return dq, dk, dv, dlog, first


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, state, lengths, scale):
        out, last = linear_attention_forward(q, k, v, log_decay, state=state, lengths=lengths, scale=scale)
        ctx.save_for_backward(q, k, v, log_decay, state, lengths)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return out, last

    @staticmethod
    def backward(ctx, dout, dstate):
        q, k, v, log_decay, state, lengths = ctx.saved_tensors
        if dout is None:
            dout = q.new_zeros((*q.shape[:3], v.shape[3]))
        elif dout.stride(-1) != 1 and dout.shape[-1] > 1:
            dout = dout.contiguous()
        if dstate is not None and dstate.stride(-1) != 1 and dstate.shape[-1] > 1:
            dstate = dstate.contiguous()
        need = ctx.needs_input_grad
        inputs = [t for t in (dout, dstate, q, k, v, log_decay, state) if t is not None]

        def form():
            grads = linear_attention_backward(dout, q, k, v, log_decay, dstate=dstate, state=state,
                                              lengths=lengths, scale=ctx.scale, decay=need[3])
            return tuple(g for g in grads if g is not None)

        grads = list(_once(form, *inputs))
        if not need[3]:
            grads.insert(3, None)
        return (*grads, *[None] * (7 - len(grads)))


def linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *,
                     state=None, lengths=None, scale: float | None = None):
    """Linear attention as :func:`linear_attention_forward`, differentiable (once, in reverse) in q, k,
    v, log_decay and state; returns (out, state_out)."""
    if _wants_gradient(q, k, v, log_decay, state):
        return _LinearAttention.apply(q, k, v, log_decay, state, lengths, scale)
    return linear_attention_forward(q, k, v, log_decay, state=state, lengths=lengths, scale=scale)


# ---- clipping of gradients -----------------------------------------------------------


def _dense(t) -> bool:
    """Whether a tensor's values fill a piece of memory, in whatever order of its axes."""
    if t.is_contiguous():
        return True
    step = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if stride != step:
            return False
        step *= size
    return True


def _gradients(tensors, out):
    """The packed list, its length and the tensors' device (None without tensors)."""
    if isinstance(tensors, torch.Tensor):
        tensors = [tensors]
    tensors = [t for t in tensors if t is not None]
    if out is not None:
        out = [out] if isinstance(out, torch.Tensor) else [o for o in out if o is not None]
        if len(out) != len(tensors):
            raise ValueError("out has to have a place for each tensor")
    if _wants_gradient(*tensors):
        raise NotImplementedError("clipping has no gradients")
    flat, device = [], None
    places = tensors if out is None else out
    for i, (t, to) in enumerate(zip(tensors, places)):
        if device is None or not isinstance(t, torch.Tensor) or t.dtype not in DTYPES or \
                t.get_device() != device.index:
            device = _device_of(t, f"tensor {i}")
        whole = t.is_contiguous()
        if not (whole or _dense(t)):
            raise ValueError(f"tensor {i} has gaps between its values")
        if to is not t and not (whole and isinstance(to, torch.Tensor) and to.dtype is t.dtype and
                                to.shape == t.shape and to.get_device() == device.index and
                                to.is_contiguous()):
            _out_like(to, t, t.dtype, device, f"out {i}")
            if to.stride() != t.stride():
                raise ValueError(f"out {i} differs in layout")
        flat += (t.data_ptr(), to.data_ptr(), t.numel(), DTYPES[t.dtype])
    return array.array("q", flat).tobytes(), places, device


def _clip(tensors, max_norm, out, where):
    packed, places, device = _gradients(tensors, out)
    n = len(places)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    norm = torch.empty((), dtype=torch.float32, device=device)
    lib = load()
    stream = _stream(device)
    if max_norm is None:
        def call(p, size):
            return lib.lic_gradient_norm(packed, n, norm.data_ptr(), p, size, stream)
    else:
        _written(places)

        def call(p, size):
            return lib.lic_clip_gradients(packed, n, max_norm, norm.data_ptr(), p, size, stream)
    _with_workspace(device, stream, call, lambda: lib.lic_clip_gradients_workspace_bytes(packed, n), where)
    return norm


def gradient_norm(tensors) -> torch.Tensor:
    """Enqueue the norm of all values of all tensors together; returns it, float32 [].

    ``tensors`` is a list of tensors without gaps, of any types and shapes (None is passed over), or
    one tensor.  Squares are summed in 64 bits.
    """
    return _clip(tensors, None, None, "lic_gradient_norm")


def clip_gradients(tensors, max_norm: float, *, out=None) -> torch.Tensor:
    """Enqueue the scaling of all tensors by min(1, max_norm / (norm + 1e-6)); returns the norm, float32 [].

    As in :func:`gradient_norm`; in place, or into ``out``, a list of tensors laid out the same.
    No tensor may overlap another that is written.  A NaN anywhere makes everything NaN; with an
    infinity the factor is 0.
    """
    max_norm = float(max_norm)
    if not (max_norm >= 0 and math.isfinite(max_norm)):
        raise ValueError("max_norm must be finite and at least 0")
    return _clip(tensors, max_norm, out, "lic_clip_gradients")
