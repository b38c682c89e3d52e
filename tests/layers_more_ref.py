"""Plain 64-bit forms of RMS norm, linear attention with a decay for each head, and clipping, and
the error bounds their tests use (units and the 32-bit share as in `layers_ref`).

Linear attention is a sum of products of inputs with weights that are not negative, so the same
form of the inputs' absolute values is the sum of the absolute terms.  These bounds are wide: a result
may be off by its last rounding (u times itself), by u times the absolute sum (16-bit types) and by what
32-bit sums and two-part operands lose (2e-5 of the absolute sum; a value in two bfloat16 parts is off by
2^-17 of itself at most, which is 0.8e-5).  `test_gpu_linear_exact` holds results to what the arithmetic
allows, without the second of these.
"""
from __future__ import annotations

import torch

from layers_ref import F32, STEP, UNIT


def rms_norm(x, weight, residual, eps, dy=None, dsum=None):
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    t = h.double()
    c = x.shape[-1]
    w = torch.ones(c, dtype=t.dtype, device=t.device) if weight is None else weight.double()
    rstd = 1 / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)
    xh = t * rstd
    r = {"h": h, "rstd": rstd[..., 0], "y": w * xh}
    if dy is not None:
        g = dy.double()
        a = w * g
        r["dx"] = rstd * (a - xh * (a * xh).mean(-1, keepdim=True))
        r["dx_abs"] = rstd * (a.abs() + xh.abs() * (a * xh).abs().mean(-1, keepdim=True))
        if dsum is not None:
            r["dx"] = r["dx"] + dsum.double()
            r["dx_abs"] = r["dx_abs"] + dsum.double().abs()
        lead = tuple(range(x.dim() - 1))
        r["dw"], r["dw_abs"] = (g * xh).sum(lead), (g * xh).abs().sum(lead)
    return r


def linear(q, k, v, log_decay, state=None, lengths=None, scale=None, dout=None, dstate=None):
    """64-bit results, [B, S, heads, dim] and [B, heads, dim, value dim]; rows behind the lengths count as
    zeros, whatever they hold."""
    b, s, h, d = q.shape
    kv, e = v.shape[2:]
    m = h // kv
    scale = d ** -0.5 if scale is None else scale
    dev = q.device
    n = torch.full((b,), s, device=dev) if lengths is None else lengths.long().clamp(0, s)
    at = torch.arange(s, device=dev)
    live = at < n[:, None]

    def rows(t, share=1):
        t = torch.where(live[:, :, None, None], t.double(), 0.0).permute(0, 2, 1, 3)
        return t.repeat_interleave(share, dim=1).contiguous()

    def back(t):
        return t.permute(0, 2, 1, 3)

    def shared(t):
        return back(t.reshape(b, kv, m, s, -1).sum(2))

    def tr(t):
        return t.transpose(2, 3).contiguous()

    g = log_decay.double()

    def power(steps, where):  # g^steps by head, [.., heads, ..]; g^0 is 1 also of g = 0
        p = torch.exp(g.view(1, h, 1, 1) * steps.clamp(min=1))
        return torch.where(where, torch.where(steps == 0, 1.0, p), 0.0)

    q_, k_, v_ = rows(q), rows(k, m), rows(v, m)
    first = torch.zeros(b, h, d, e, dtype=torch.float64, device=dev) if state is None else state.double()
    lag = (at[:, None] - at[None, :]).view(1, 1, s, s)
    w = power(lag, lag >= 0) * scale
    there = live[:, None, :, None]
    come = power((at + 1).view(1, 1, s, 1), there) * scale
    steps = n.view(b, 1, 1, 1) - 1 - at.view(1, 1, s, 1)
    go = power(steps, there)
    stay = power(n.view(b, 1, 1, 1), torch.ones(1, 1, 1, 1, dtype=torch.bool, device=dev))
    a = (q_ @ tr(k_)) * w
    r = {"out": back(a @ v_ + (q_ @ first) * come), "last": stay * first + tr(k_ * go) @ v_}
    if dout is None:
        return r
    do = rows(dout)
    da = (do @ tr(v_)) * w
    last = torch.zeros_like(first) if dstate is None else dstate.double()
    r["dq"] = back(da @ k_ + (do @ tr(first)) * come)
    r["dk"] = shared(tr(da) @ q_ + (v_ @ tr(last)) * go)
    r["dv"] = shared(tr(a) @ do + (k_ @ last) * go)
    r["dstate"] = stay * last + tr(q_ * come) @ do
    pairs = (a * (do @ tr(v_)) * lag.clamp(min=0)).sum((0, 2, 3))
    pairs = pairs + ((at + 1).view(1, 1, s, 1) * come * q_ * (do @ tr(first))).sum((0, 2, 3))
    pairs = pairs + (steps.clamp(min=0) * go * k_ * (v_ @ tr(last))).sum((0, 2, 3))
    r["dlog"] = pairs + (n.view(b, 1, 1, 1) * stay * first * last).sum((0, 2, 3))
    return r


def linear_abs(q, k, v, log_decay, **more):
    """The absolute sums of the same results."""
    def size(t):
        return t.abs() if isinstance(t, torch.Tensor) and t.is_floating_point() else t
    return linear(size(q), size(k), size(v), log_decay, **{n: size(t) for n, t in more.items()})


def linear_bound(want, size, dtype):
    """For results of the inputs' type."""
    u = UNIT[dtype]
    return u * want.abs() + (F32 + (0 if dtype == torch.float32 else u)) * size + STEP[dtype]
