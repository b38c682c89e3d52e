"""The network operators around the coder as cases to be measured: group norm with an
activation (channels last), rotary positions and attention, forward and backward.

`run` computes a case in plain form (elementary torch operations in 32 bits, rounded
once at the end) or, where `own` is true, with the package's kernels.  Sizes: the
latents of `workloads` (z 192 x 17 x 30, y of 1080p 192 x 68 x 120 = 8160 positions, y
of 4K 136 x 240 = 32640 positions), the transforms' activations at those images'
resolutions, and training crops of 256 x 256 pixels.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # the z latent's hyper-decoder: six channels a group, odd sides, one small launch
        {"name": "norm_z", "op": "norm", "type": "f32", "N": 1, "C": 192, "H": 17, "W": 30, "G": 32, "act": "silu", "train": False},
        # the synthesis transform's last hidden stage of a 1080p image, half its sides
        {"name": "norm_1080p_half", "op": "norm", "type": "bf16", "N": 1, "C": 192, "H": 544, "W": 960, "G": 32, "act": "silu", "train": False},
        # training crops after two strided convolutions
        {"name": "norm_crops_train", "op": "norm", "type": "bf16", "N": 16, "C": 192, "H": 64, "W": 64, "G": 32, "act": "silu", "train": True},
        # a wider transform at a crop's half resolution, ten channels a group
        {"name": "norm_wide_train", "op": "norm", "type": "f16", "N": 8, "C": 320, "H": 128, "W": 128, "G": 32, "act": "gelu", "train": True},
        # one token of each of 16 latents decoded side by side, keys shared by heads: the smallest call
        {"name": "rotary_step", "op": "rotary", "type": "bf16", "B": 16, "S": 1, "H": 16, "K": 4, "D": 64, "R": 64, "inter": False, "train": False},
        # all positions of eight 4K latents, 192 channels as six heads
        {"name": "rotary_4k", "op": "rotary", "type": "bf16", "B": 8, "S": 32640, "H": 6, "K": 6, "D": 32, "R": 32, "inter": False, "train": False},
        # a training pass over half of each head, neighbours paired
        {"name": "rotary_train", "op": "rotary", "type": "f16", "B": 4, "S": 4095, "H": 16, "K": 4, "D": 128, "R": 64, "inter": True, "train": True},
        # one token a latent over a ragged cache of a 1080p latent's positions
        {"name": "attention_step", "op": "attention", "type": "bf16", "B": 16, "Q": 1, "S": 8160, "H": 16, "K": 4, "D": 64, "mask": "ragged", "train": False},
        # the z latent's positions, trained in 32 bits
        {"name": "attention_z_train", "op": "attention", "type": "f32", "B": 4, "Q": 510, "S": 510, "H": 6, "K": 6, "D": 32, "mask": "none", "train": True},
        # crops' latents (16 x 16), each position seeing the slices coded before its own: the first slice sees nothing
        {"name": "attention_crops_train", "op": "attention", "type": "f16", "B": 32, "Q": 256, "S": 256, "H": 6, "K": 6, "D": 32, "mask": "slices", "train": True},
        # every position of a 1080p latent with every other, 192 channels as three heads of 64
        {"name": "attention_1080p", "op": "attention", "type": "bf16", "B": 2, "Q": 8160, "S": 8160, "H": 3, "K": 3, "D": 64, "mask": "none", "train": False},
        # an autoregressive model trained over a 1080p latent's positions: the largest
        {"name": "attention_long_train", "op": "attention", "type": "bf16", "B": 1, "Q": 8160, "S": 8160, "H": 16, "K": 4, "D": 128, "mask": "causal", "train": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    kind = rng.choice(["norm", "norm", "rotary", "rotary", "step", "attention", "attention"])
    typ = rng.choice(["bf16", "bf16", "f16", "f32"])
    train = rng.random() < 0.5
    if kind == "norm":
        G = rng.choice([1, 2, 4, 8, 16, 32, 32, 32])
        # a rectified unit's slope jumps at zero, where any rounding decides: it is drawn without gradients
        return {"op": "norm", "type": typ, "N": _log(rng, 1, 32), "C": G * _log(rng, 1, 1024 // G),
                "H": _log(rng, 1, 544), "W": _log(rng, 1, 960), "G": G,
                "act": rng.choice(["none", "silu", "silu", "gelu"] if train else ["relu", "silu", "silu", "gelu"]), "train": train}
    K = rng.choice([1, 2, 3, 4, 6, 8])
    H = K * rng.choice([1, 1, 2, 4, 8])
    D = rng.choice([16, 24, 32, 40, 64, 64, 72, 96, 128, 128])
    if kind == "rotary":
        return {"op": "rotary", "type": typ, "B": _log(rng, 1, 32), "S": _log(rng, 1, 32640), "H": H, "K": K, "D": D,
                "R": rng.choice([D, D, 2 * (D // 4)]), "inter": rng.random() < 0.5, "train": train}
    if kind == "step":
        return {"op": "attention", "type": typ, "B": _log(rng, 1, 64), "Q": 1, "S": _log(rng, 1, 131072), "H": H, "K": K, "D": D,
                "mask": rng.choice(["none", "ragged"]), "train": False}
    S = _log(rng, 16, 8160)
    return {"op": "attention", "type": typ, "B": _log(rng, 1, 32), "Q": S if rng.random() < 0.7 else _log(rng, 2, 4096), "S": S,
            "H": H, "K": K, "D": D, "mask": rng.choice(["none", "causal", "ragged", "slices", "window"]), "train": train}


def draw(rng):
    # no more than the largest listed cases have: products, bytes and, where 32 bits are
    # multiplied, a sixteenth of the products
    while True:
        case = _drawn(rng)
        w = work(case)
        if case["op"] == "attention":
            pairs = case["B"] * case["H"] * case["Q"] * case["S"]
            if pairs <= 16 * 8160 ** 2 and w["flops"] <= (5.9e10 if case["type"] == "f32" else 9.4e11) and w["bytes"] <= 4e8:
                return case
        elif w["bytes"] <= 4e8 and (case["op"] != "norm" or case["H"] * case["W"] * case["C"] >= 64 * case["G"]):
            return case  # of a group of two or three values next to nothing is left after its mean and slope


def _lengths(case):
    """Keys of each latent in use: from all of them down to about a half, odd numbers among them."""
    S = case["S"]
    return [S - (b * 37) % (S // 2 + 1) for b in range(case["B"])]


def _pairs(case):
    """Visible pairs of one head, over the whole batch."""
    B, Q, S = case["B"], case["Q"], case["S"]
    if case["mask"] == "none":
        return B * Q * S
    if case["mask"] == "ragged":
        return Q * sum(_lengths(case))
    if case["mask"] == "slices":
        q, k = [len(range(g, Q, 4)) for g in range(4)], [len(range(g, S, 4)) for g in range(4)]
        return B * sum(q[g] * sum(k[:g]) for g in range(4))
    reach = S if case["mask"] == "causal" else _window(case)
    return B * sum(max(0, i + S - Q + 1 - max(0, i + S - Q - reach)) for i in range(Q))


def _window(case):
    return max(1, case["S"] // 8)


def work(case):
    b = BYTES[case["type"]]
    if case["op"] == "norm":
        n = case["N"] * case["C"] * case["H"] * case["W"]
        return {"bytes": n * b * (4 if case["train"] else 2) + 2 * 4 * case["C"], "flops": n * (30 if case["train"] else 10)}
    if case["op"] == "rotary":
        n = case["B"] * case["S"] * (case["H"] + case["K"]) * case["D"]
        tables = case["S"] * case["R"] * 4
        return {"bytes": n * b * (4 if case["train"] else 2) + tables, "flops": 3 * n * (2 if case["train"] else 1)}
    rows, keys = case["B"] * case["Q"] * case["H"] * case["D"], case["B"] * case["S"] * case["K"] * case["D"]
    if case["mask"] == "ragged":
        keys = sum(_lengths(case)) * case["K"] * case["D"]
    more = case["Q"] * case["S"] if case["mask"] == "slices" else 0
    flops = 4 * _pairs(case) * case["H"] * case["D"]
    if case["train"]:  # q, k, v, dout in; out, dq, dk, dv out; the probabilities again and four products more
        return {"bytes": (4 * rows + 4 * keys) * b + more, "flops": flops * 7 // 2}
    return {"bytes": (2 * rows + 2 * keys) * b + more, "flops": flops}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    typ = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "norm":
        shape = (case["N"], case["H"], case["W"], case["C"])
        # features differ in size and have means of their own
        size, mean = torch.exp(0.5 * normal(case["C"])), normal(case["C"])
        s = {"case": case, "x": (normal(*shape) * size + mean).to(typ).permute(0, 3, 1, 2),
             "weight": 1 + 0.2 * normal(case["C"]), "bias": 0.2 * normal(case["C"])}
        if case["train"]:
            s["dy"] = normal(*shape).to(typ).permute(0, 3, 1, 2)
        return s
    B, S, H, K, D = (case[k] for k in "BSHKD")
    if case["op"] == "rotary":
        R = case["R"]
        # a cache's rows are further along than the call's own tokens are
        rows = S + 1024
        turn = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * \
            10000.0 ** (-2.0 * torch.arange(R // 2, dtype=torch.float64, device="cuda") / R)
        first = torch.randint(0, 1024, (B, 1), generator=g, device="cuda")
        s = {"case": case, "cos": turn.cos().float(), "sin": turn.sin().float(),
             "positions": (first + torch.arange(S, device="cuda")).to(torch.int32),
             "q": normal(B, S, H, D).to(typ), "k": normal(B, S, K, D).to(typ)}
        if case["train"]:
            s["dq"], s["dk"] = normal(B, S, H, D).to(typ), normal(B, S, K, D).to(typ)
        return s
    s = {"case": case, "q": normal(B, case["Q"], H, D).to(typ), "k": normal(B, S, K, D).to(typ), "v": normal(B, S, K, D).to(typ),
         "options": {}}
    if case["train"]:
        s["dout"] = normal(B, case["Q"], H, D).to(typ)
    if case["mask"] == "ragged":
        s["options"]["key_lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    elif case["mask"] == "slices":
        s["options"]["mask"] = torch.arange(S, device="cuda")[None, :] % 4 < torch.arange(case["Q"], device="cuda")[:, None] % 4
    elif case["mask"] == "causal":
        s["options"]["causal"] = True
    elif case["mask"] == "window":
        s["options"]["window"] = (_window(case), 0)
    return s


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "rotary": _plain_rotary, "attention": _plain_attention}[state["case"]["op"]](state)


def _own(s):
    from learned_image_compression_amd import layers as L

    case = s["case"]
    if case["op"] == "norm":
        y, mean, rstd = L.group_norm_forward(s["x"], case["G"], s["weight"], s["bias"], activation=case["act"])
        if not case["train"]:
            return y
        return (y, *L.group_norm_backward(s["dy"], s["x"], case["G"], s["weight"], s["bias"], mean, rstd, activation=case["act"]))
    if case["op"] == "rotary":
        out = L.rotary(s["q"], s["k"], s["cos"], s["sin"], positions=s["positions"], interleaved=case["inter"])
        if not case["train"]:
            return out
        return (*out, *L.rotary(s["dq"], s["dk"], s["cos"], s["sin"], positions=s["positions"], interleaved=case["inter"], inverse=True))
    out, lse = L.attention_forward(s["q"], s["k"], s["v"], **s["options"])
    if not case["train"]:
        return out, lse
    return (out, lse, *L.attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, **s["options"]))


def _plain_norm(s):
    case, x = s["case"], s["x"]
    N, C, H, W = x.shape
    G = case["G"]
    w, b = s["weight"], s["bias"]
    t = x.float().permute(0, 2, 3, 1).reshape(N, H * W, G, C // G)
    t = t - t.mean(dim=(1, 3), keepdim=True)
    r = torch.rsqrt((t * t).mean(dim=(1, 3), keepdim=True) + 1e-5)
    xh = (t * r).reshape(N, H * W, C)
    u = xh * w + b
    if case["act"] == "none":
        y = u
    elif case["act"] == "relu":
        y = u * (u > 0)
    elif case["act"] == "silu":
        y = u / (1 + torch.exp(-u))
    else:
        y = u * 0.5 * (1 + torch.erf(u * math.sqrt(0.5)))
    y = y.to(x.dtype).view(N, H, W, C).permute(0, 3, 1, 2)
    if not case["train"]:
        return y
    dy = s["dy"].float().permute(0, 2, 3, 1).reshape(N, H * W, C)
    if case["act"] == "none":
        du = dy
    elif case["act"] == "relu":
        du = dy * (u > 0)
    elif case["act"] == "silu":
        e = 1 / (1 + torch.exp(-u))
        du = dy * e * (1 + u * (1 - e))
    else:
        du = dy * (0.5 * (1 + torch.erf(u * math.sqrt(0.5))) + u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi))
    dw, db = (du * xh).sum(dim=(0, 1)), du.sum(dim=(0, 1))
    v = (du * w).view(N, H * W, G, C // G)
    xg = xh.view(N, H * W, G, C // G)
    dx = r * (v - v.mean(dim=(1, 3), keepdim=True) - xg * (v * xg).mean(dim=(1, 3), keepdim=True))
    return y, dx.to(x.dtype).view(N, H, W, C).permute(0, 3, 1, 2), dw, db


def _turned(x, c, s, inter):
    """x [B, S, heads, D] with its first R values of each head turned by the angles of c and s [B, S, 1, R/2]."""
    n = c.shape[-1]
    t, rest = x[..., :2 * n].float(), x[..., 2 * n:]
    a, b = (t[..., 0::2], t[..., 1::2]) if inter else (t[..., :n], t[..., n:])
    a, b = a * c - b * s, a * s + b * c
    t = torch.stack((a, b), dim=-1).flatten(-2) if inter else torch.cat((a, b), dim=-1)
    return torch.cat((t.to(x.dtype), rest), dim=-1)


def _plain_rotary(s):
    case = s["case"]
    at = s["positions"].long()
    c, n = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    out = [_turned(s["q"], c, n, case["inter"]), _turned(s["k"], c, n, case["inter"])]
    if case["train"]:
        out += [_turned(s["dq"], c, -n, case["inter"]), _turned(s["dk"], c, -n, case["inter"])]
    return tuple(out)


def _visible(case, options, device):
    """Which keys a query sees: [B or 1, 1, Q, S], or None for all of them."""
    Q, S = case["Q"], case["S"]
    if case["mask"] == "ragged":
        return torch.arange(S, device=device) < options["key_lengths"][:, None, None, None]
    if case["mask"] == "slices":
        return options["mask"][None, None]
    at = torch.arange(Q, device=device)[:, None] + (S - Q)
    keys = torch.arange(S, device=device)[None, :]
    if case["mask"] == "causal":
        return (keys <= at)[None, None]
    if case["mask"] == "window":
        return ((keys <= at) & (keys >= at - options["window"][0]))[None, None]
    return None


def _plain_attention(s):
    case = s["case"]
    B, Q, S, H, K, D = (case[k] for k in "BQSHKD")
    scale = D ** -0.5
    q = s["q"].float().permute(0, 2, 1, 3).reshape(B, K, H // K * Q, D)  # the heads that share keys, side by side
    k = s["k"].float().permute(0, 2, 1, 3).contiguous()
    v = s["v"].float().permute(0, 2, 1, 3).contiguous()
    p = torch.matmul(q * scale, k.transpose(2, 3).contiguous()).view(B, H, Q, S)
    seen = _visible(case, s["options"], q.device)
    if seen is not None:
        p = p.masked_fill_(~seen, -math.inf)
    m = p.amax(dim=-1, keepdim=True)
    p = torch.exp(p - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(dim=-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    p = (p / torch.where(total == 0, 1.0, total)).view(B, K, H // K * Q, S)

    def back(t, heads, n):
        return t.reshape(B, heads, n, D).permute(0, 2, 1, 3).to(s["q"].dtype)

    o = torch.matmul(p, v)
    out = back(o, H, Q)
    if not case["train"]:
        return out, lse
    do = s["dout"].float().permute(0, 2, 1, 3).reshape(B, K, H // K * Q, D)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
    ds = torch.matmul(do, v.transpose(2, 3).contiguous())
    ds = p * (ds - (do * o).sum(dim=-1, keepdim=True))
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q) * scale
    return out, lse, back(dq, H, Q), back(dk, K, S), back(dv, K, S)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotary": _exact_rotary, "attention": _exact_attention}[case["op"]](case, s)


def _exact_norm(case, s):
    G = case["G"]
    x = s["x"].double()  # [N, C, H, W]
    N, C, H, W = x.shape
    wide = (1, C, 1, 1)
    w, b = s["weight"].double().view(wide), s["bias"].double().view(wide)
    per = x.reshape(N, G, -1)
    var, mean = torch.var_mean(per, dim=2, unbiased=False)
    sd = torch.sqrt(var + 1e-5)

    def spread(t):
        return t.repeat_interleave(C // G, dim=1).view(N, C, 1, 1)

    z = (x - spread(mean)) / spread(sd)
    u = z * w + b
    if case["act"] == "none":
        y, slope = u, torch.ones_like(u)
    elif case["act"] == "relu":
        y, slope = u.clamp(min=0), (u > 0).double()
    elif case["act"] == "silu":
        g = torch.sigmoid(u)
        y, slope = u * g, g + u * g * (1 - g)
    else:
        g = torch.special.ndtr(u)
        y, slope = u * g, g + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    if not case["train"]:
        return y
    du = s["dy"].double() * slope
    dz = du * w
    low = dz.reshape(N, G, -1).mean(dim=2)
    tilt = (dz * z).reshape(N, G, -1).mean(dim=2)
    dx = (dz - spread(low) - z * spread(tilt)) / spread(sd)
    return y, dx, (du * z).sum(dim=(0, 2, 3)), du.sum(dim=(0, 2, 3))


def _exact_rotary(case, s):
    R = case["R"]
    at = s["positions"].long()
    turn = torch.complex(s["cos"].double(), s["sin"].double())[at].unsqueeze(2)

    def through(x, turn):
        y = x.double().clone()
        first, second = (slice(0, R, 2), slice(1, R, 2)) if case["inter"] else (slice(0, R // 2), slice(R // 2, R))
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = [through(s["q"], turn), through(s["k"], turn)]
    if case["train"]:
        out += [through(s["dq"], turn.conj()), through(s["dk"], turn.conj())]
    return tuple(out)


def _exact_attention(case, s):
    B, Q, S, H, K, D = (case[k] for k in "BQSHKD")
    seen = _visible(case, s["options"], "cuda")
    out = torch.zeros(B, Q, H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, H, Q, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(out), *(torch.zeros(B, S, K, D, dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(B):
        for h in range(H):
            j = h // (H // K)
            q, k, v = s["q"][b, :, h].double(), s["k"][b, :, j].double(), s["v"][b, :, j].double()
            a = (q @ k.t()) / math.sqrt(D)
            if seen is not None:
                a = a.masked_fill(~seen[b % seen.shape[0], 0], -math.inf)
            lse[b, h] = torch.logsumexp(a, dim=1)
            p = torch.nan_to_num(torch.softmax(a, dim=1), nan=0.0)  # a row that sees nothing gives nothing
            out[b, :, h] = p @ v
            if case["train"]:
                do = s["dout"][b, :, h].double()
                dv[b, :, j] += p.t() @ do
                dp = do @ v.t()
                ds = p * (dp - (p * dp).sum(dim=1, keepdim=True)) / math.sqrt(D)
                dq[b, :, h] = ds @ k
                dk[b, :, j] += ds.t() @ q
    return (out, lse, dq, dk, dv) if case["train"] else (out, lse)
