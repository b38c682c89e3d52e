"""Plain 64-bit forms of the network operators (group norm with an activation,
rotary positions, attention) and the error bounds their tests use.

Bounds.  u is half a unit in the last place of a type's 1: 2^-24, 2^-11 and 2^-8
for float32, float16 and bfloat16.  A result rounded once from 32 bits is off by
u times itself; an operand rounded to the inputs' type before a sum is off by
u times the sum of absolute values (float16 ends at 2^-24, so either is off by 2^-25
at least); what the 32-bit arithmetic itself loses
(sums of up to some thousand terms in short chains, hardware exponential and
reciprocal of about 2^-22) is given 2e-5 of the same absolute sums.
"""
from __future__ import annotations

import math

import torch

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
STEP = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
F32 = 2e-5


def act(u, kind):
    """Value and slope."""
    if kind == "none":
        return u, torch.ones_like(u)
    if kind == "relu":
        return torch.where(u > 0, u, 0 * u), (u > 0).to(u.dtype)
    if kind == "silu":
        s = 1 / (1 + torch.exp(-u))
        return u * s, s * (1 + u * (1 - s))
    phi = 0.5 * torch.erfc(-u / math.sqrt(2))
    return u * phi, phi + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)


def group_norm(x, groups, weight, bias, eps, kind, dy=None):
    """x [N, C, ...]; returns a dict of 64-bit results."""
    x = x.double()
    n, c = x.shape[:2]
    flat = x.reshape(n, groups, -1)
    mean = flat.mean(2, keepdim=True)
    var = ((flat - mean) ** 2).mean(2, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xh = ((flat - mean) * rstd).view_as(x)
    wide = (1, c) + (1,) * (x.dim() - 2)
    w = torch.ones(wide, dtype=x.dtype, device=x.device) if weight is None else weight.double().view(wide)
    b = torch.zeros(wide, dtype=x.dtype, device=x.device) if bias is None else bias.double().view(wide)
    u = xh * w + b
    y, slope = act(u, kind)
    r = {"y": y, "mean": mean[..., 0], "rstd": rstd[..., 0], "u": u, "xh": xh}
    if dy is not None:
        du = dy.double() * slope
        dims = [0] + list(range(2, x.dim()))
        r["db"], r["dw"] = du.sum(dims), (du * xh).sum(dims)
        r["db_abs"], r["dw_abs"] = dy.double().abs().sum(dims) * 1.2, (dy.double() * xh).abs().sum(dims) * 1.2
        v = (du * w).reshape(n, groups, -1)
        xg = xh.reshape(n, groups, -1)
        a, s = v.mean(2, keepdim=True), (v * xg).mean(2, keepdim=True)
        r["dx"] = (rstd * (v - a - xg * s)).view_as(x)
        m = dy.double().abs().max() * 1.2
        r["dx_abs"] = (rstd.expand_as(v) * (w.abs() * m).expand_as(x).reshape(n, groups, -1)).view_as(x) * \
            (1 + xh.abs())
    return r


def turn(x, cos, sin, positions, interleaved, inverse=False):
    """x [B, S, heads, dim]."""
    x = x.double()
    b, s = x.shape[:2]
    if positions is None:
        positions = torch.arange(s, device=x.device)
    at = positions.long().expand(b, s)
    c, n = cos.double()[at][:, :, None], sin.double()[at][:, :, None]
    if inverse:
        n = -n
    half = cos.shape[1]
    y = x.clone()
    i = torch.arange(half, device=x.device)
    i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, e = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - e * n, a * n + e * c
    return y


def seen(b, h, q, s, device, causal=False, window=None, mask=None, key_lengths=None):
    """[B, H, Q, S]: which keys a query sees."""
    n = torch.full((b,), s, device=device) if key_lengths is None else key_lengths.long().clamp(0, s)
    n = n.view(b, 1, 1, 1)
    at = torch.arange(q, device=device).view(1, 1, q, 1) + n - q
    key = torch.arange(s, device=device).view(1, 1, 1, s)
    ok = (key < n).expand(b, h, q, s).clone()
    left, right = window if window is not None else (None, None)
    if causal:
        right = 0
    if left is not None:
        ok &= key >= at - left
    if right is not None:
        ok &= key <= at + right
    if mask is not None:
        ok &= mask.bool().expand(b, h, q, s)
    return ok


def attention(q, k, v, dout=None, scale=None, **options):
    """64-bit results [B, rows, heads, dim], their absolute sums (`*_abs`, for the
    bounds) and which keys are seen; values in unseen places count for nothing."""
    b, n, h, d = q.shape
    s, kv = k.shape[1], k.shape[2]
    g = h // kv
    scale = d ** -0.5 if scale is None else scale
    ok = seen(b, h, n, s, q.device, **options)

    def split(x):
        return x.double().permute(0, 2, 1, 3)

    def share(x):
        return split(x).repeat_interleave(g, dim=1)

    def t(x):
        return x.transpose(2, 3).contiguous()

    def back(x):
        return x.permute(0, 2, 1, 3)

    def gather(x):
        return back(x.reshape(b, kv, g, s, d).sum(2))

    q_, k_, v_ = split(q), share(k), share(v)
    a = (q_ @ t(k_)) * scale
    a = torch.where(ok, a, -math.inf)
    m = a.amax(3, keepdim=True)
    e = torch.where(ok, torch.exp(a - torch.where(m == -math.inf, 0.0, m)), 0.0)
    total = e.sum(3, keepdim=True)
    p = e / torch.where(total == 0, 1.0, total)
    r = {"lse": (m + torch.log(total))[..., 0], "out": back(p @ v_), "out_abs": back(p @ v_.abs()), "seen": ok}
    # what scores of 32-bit sums may be off by, which the exponential passes on
    slack = 4 * d ** 0.5 * 2.0 ** -24 * scale * (q_.abs() @ t(k_.abs())).amax().item()
    r["slack"] = slack
    if dout is not None:
        do, o = split(dout), split(r["out"])
        delta = (do * o).sum(3, keepdim=True)
        ds = torch.where(ok, p * (do @ t(v_) - delta), 0.0)
        big = torch.where(ok, p * (do.abs() @ t(v_.abs()) + (do.abs() * o.abs()).sum(3, keepdim=True)), 0.0)
        # sums that a least operand error of 1 would make
        r["dq_ones"], r["dk_ones"] = back(ok.double() @ k_.abs()) * scale, gather(t(ok.double()) @ q_.abs()) * scale
        r["dq"], r["dq_abs"] = back(ds @ k_) * scale, back(big @ k_.abs()) * scale
        r["dk"], r["dk_abs"] = gather(t(ds) @ q_) * scale, gather(t(big) @ q_.abs()) * scale
        r["dv"], r["dv_abs"] = gather(t(p) @ do), gather(t(p) @ do.abs())
    return r


def worst(got, want, bound):
    """Largest error over its bound (at most 1 passes); infinities and NaN must agree."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), "infinities or NaN in other places"
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    other = ~fine & ~torch.isnan(want)
    assert torch.equal(got[other], want[other])
    if not bool(fine.any()):
        return 0.0
    bound = bound.expand_as(want) if isinstance(bound, torch.Tensor) else torch.full_like(want, bound)
    return float(((got - want).abs()[fine] / bound[fine].clamp(min=1e-30)).max())
