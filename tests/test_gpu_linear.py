"""Linear attention with a decay for each head on the GPU against plain 64-bit forms (`layers_more_ref`,
where the bounds are derived), at the sizes, lengths, strides and values where it can go wrong."""
from __future__ import annotations

import math
import threading

import pytest
import torch

import layers_more_ref as M
import layers_ref as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ALL = (F32, F16, BF16)


@pytest.fixture(scope="module")
def L():
    from learned_image_compression_amd import layers
    layers.load()
    return layers


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def passes(got, want, bound, what):
    if got.dtype == F16:
        # a result beyond float16's last number (65504; half a step more rounds to infinity) is infinite, and
        # within the bound of that it may be either
        size, end = want.abs(), 65520.0
        want = torch.where(size - bound > end, math.inf * want, want)
        want = torch.where((size - end).abs() <= bound, got.double(), want)
    w = R.worst(got, want, bound)
    print(f"{what}: {w:.3f} of the bound", flush=True)
    assert w <= 1.0, (what, w)


def decays(h, g):
    """Memories of 2 to 1000 positions, none at all, and no decay."""
    reach = torch.exp2(1 + 9 * torch.rand(h, generator=g, device="cuda"))
    log = torch.log1p(-1 / reach)
    if h > 2:
        log[0], log[1] = 0.0, -40.0
    return log


def inputs(b, s, h, kv, d, e, dtype, state, ragged, seed=0, size=1.0):
    g = gen(seed + 7 * s + d)
    x = {"q": normal(g, b, s, h, d, dtype=dtype), "k": normal(g, b, s, kv, d, dtype=dtype),
         "v": (size * normal(g, b, s, kv, e)).to(dtype), "log_decay": decays(h, g)}
    more = {"state": normal(g, b, h, d, e) if state else None, "lengths": None}
    if ragged:
        more["lengths"] = torch.tensor([max(0, s - 29 * i) if i < 3 else s + 5 for i in range(b)], dtype=torch.int32, device="cuda")
    grads = {"dout": (size * normal(g, b, s, h, e)).to(dtype), "dstate": normal(g, b, h, d, e) if state else None}
    return x, more, grads


def check(L, x, more, grads, backward=True, scale=None):
    dtype = x["q"].dtype
    r = M.linear(**x, **more, scale=scale, **(grads if backward else {}))
    size = M.linear_abs(**x, **more, scale=scale, **(grads if backward else {}))
    out, last = L.linear_attention_forward(**x, **more, scale=scale)
    assert out.dtype == dtype and last.dtype == F32
    passes(out, r["out"], M.linear_bound(r["out"], size["out"], dtype), "out")
    passes(last, r["last"], R.F32 * size["last"], "state")
    if not backward:
        return
    dq, dk, dv, dlog, first = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more, scale=scale)
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert got.dtype == dtype
        passes(got, r[name], M.linear_bound(r[name], size[name], dtype), name)
    passes(dlog, r["dlog"], R.F32 * size["dlog"], "dlog_decay")
    assert (first is None) == (more["state"] is None)
    if first is not None:
        passes(first, r["dstate"], R.F32 * size["dstate"], "dstate")


CASES = [
    # B, S, heads, kv heads, dim, value dim, state, ragged
    (1, 1, 1, 1, 1, 1, False, False),
    (2, 1, 4, 2, 64, 64, True, False),
    (3, 1, 3, 1, 33, 20, True, False),
    (2, 2, 2, 2, 32, 32, False, False),
    (1, 31, 3, 3, 32, 32, True, False),
    (2, 32, 4, 1, 64, 64, True, False),
    (1, 33, 3, 3, 40, 40, False, False),
    (4, 64, 6, 3, 32, 32, True, True),
    (4, 65, 3, 3, 96, 64, True, True),
    (1, 63, 4, 4, 128, 128, False, False),
    (4, 127, 8, 2, 64, 64, True, True),
    (2, 130, 3, 1, 72, 33, True, False),
    (3, 200, 4, 2, 128, 128, True, True),
    (1, 257, 5, 5, 16, 16, False, False),
    (5, 100, 6, 6, 20, 5, True, True),
    (1, 300, 2, 1, 5, 128, False, False),
    (2, 129, 2, 2, 128, 8, True, False),
    (1, 700, 4, 4, 32, 32, True, False),
    (4, 510, 6, 6, 32, 32, False, False),
    (2, 1100, 3, 3, 64, 64, True, True),
]


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("b,s,h,kv,d,e,state,ragged", CASES)
def test_linear_attention(L, b, s, h, kv, d, e, state, ragged, dtype):
    check(L, *inputs(b, s, h, kv, d, e, dtype, state, ragged))


@pytest.mark.parametrize("dtype", ALL)
def test_step_by_step(L, dtype):
    """Tokens one at a time, the state in place, against the whole call."""
    b, s, h, kv, d, e = 3, 70, 4, 2, 64, 48
    x, more, _ = inputs(b, s, h, kv, d, e, dtype, True, False)
    r, size = M.linear(**x, **more), M.linear_abs(**x, **more)
    state = more["state"].clone()
    outs = []
    for i in range(s):
        out, last = L.linear_attention_forward(*(x[n][:, i:i + 1] for n in "qkv"), x["log_decay"], state=state, state_out=state)
        assert last is state
        outs.append(out)
    # a step rounds its state to 32 bits each time: 2^-24 of what is left of each of 70 steps
    passes(torch.cat(outs, 1), r["out"], M.linear_bound(r["out"], size["out"], dtype), "out")
    passes(state, r["last"], R.F32 * size["last"], "state")


@pytest.mark.parametrize("dtype", ALL)
def test_calls_carry_the_state(L, dtype):
    """A long call and the same in pieces of odd lengths, the state given on (in place)."""
    x, more, _ = inputs(2, 333, 3, 3, 40, 72, dtype, True, False)
    r, size = M.linear(**x, **more), M.linear_abs(**x, **more)
    state, outs, at = more["state"].clone(), [], 0
    for n in (1, 2, 64, 65, 100, 101):
        out, _ = L.linear_attention_forward(*(x[m][:, at:at + n] for m in "qkv"), x["log_decay"], state=state, state_out=state)
        outs.append(out)
        at += n
    assert at == 333
    passes(torch.cat(outs, 1), r["out"], M.linear_bound(r["out"], size["out"], dtype), "out")
    passes(state, r["last"], R.F32 * size["last"], "state")


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("d,e", [(64, 32), (36, 28), (128, 128)])
def test_bits_do_not_depend_on_layout(L, d, e, dtype):
    b, s, h, kv = 2, 131, 4, 2
    x, more, grads = inputs(b, s, h, kv, d, e, dtype, True, False)
    want = (*L.linear_attention_forward(**x, **more),
            *L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more))

    def laid(t, how):
        n, rows, heads, dim = t.shape
        if how == "heads first":
            return t.transpose(1, 2).contiguous().transpose(1, 2)
        if how == "cut out":
            return torch.full((n, rows + 1, heads + 1, dim + 3), math.nan, dtype=t.dtype, device="cuda")[:, 1:, :-1, 3:].copy_(t)
        return torch.full((t.numel() + 1,), math.nan, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)

    for how in ("heads first", "cut out", "odd"):
        y = {n: laid(t, how) if n in "qkv" else t for n, t in x.items()}
        m = {**more, "state": laid(more["state"], how)}
        out = laid(want[0], how).fill_(5.0)
        state_out = laid(more["state"], how).fill_(5.0)
        got = (*L.linear_attention_forward(**y, **m, out=out, state_out=state_out),
               *L.linear_attention_backward(laid(grads["dout"], how), *y.values(), dstate=laid(grads["dstate"], how), **m))
        assert got[0] is out and got[1] is state_out
        assert all(torch.equal(a, b) for a, b in zip(got, want)), how
        if how == "cut out":
            assert bool(torch.isnan(out._base[:, 0]).all()) and bool(torch.isnan(out._base[..., :3]).all())
            assert bool(torch.isnan(state_out._base[:, :, -1]).all())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("s", [1, 40, 150])
def test_rows_behind_the_lengths(L, s, dtype):
    """They are not read, their results are 0; a length of 0 gives the state on."""
    b, h, kv, d, e = 4, 4, 2, 64, 40
    x, more, grads = inputs(b, s, h, kv, d, e, dtype, True, False)
    more["lengths"] = torch.tensor([0, s, s // 2, -3], dtype=torch.int32, device="cuda")
    check(L, x, more, grads)
    want = (*L.linear_attention_forward(**x, **more), *L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more))
    for i, n in enumerate((0, s, s // 2, 0)):
        for t in (x["q"], x["k"], x["v"], grads["dout"]):
            t[i, n:] = math.nan
        assert n == s or bool((want[0][i, n:] == 0).all()) and all(bool((g[i, n:] == 0).all()) for g in want[2:5])
    assert torch.equal(want[1][0], more["state"][0]) and torch.equal(want[1][3], more["state"][3])
    got = (*L.linear_attention_forward(**x, **more), *L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("at", [0, 5, 40, 70, 149])
@pytest.mark.parametrize("s", [150, 1500])
def test_nothing_shows_before_its_token(L, s, at, value, dtype):
    b, h, d, e = 1, 2, 64, 64
    x, more, grads = inputs(b, s, h, h, d, e, dtype, True, False)
    clean = L.linear_attention_forward(**x, **more)
    back = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more)
    for name in "qkv":
        y = dict(x)
        y[name] = x[name].clone()
        y[name][0, at, 0, 3] = value
        out, last = L.linear_attention_forward(**y, **more)
        assert torch.equal(out[:, :at], clean[0][:, :at]) and torch.equal(out[:, :, 1], clean[0][:, :, 1])
        assert torch.equal(last[:, 1], clean[1][:, 1])
        if name == "q":  # its own row only
            assert not bool(torch.isfinite(out[0, at, 0]).any())
            assert torch.equal(out[0, at + 1:, 0], clean[0][0, at + 1:, 0]) and torch.equal(last, clean[1])
        elif name == "v":  # its column, from there on
            assert not bool(torch.isfinite(out[0, at, 0, 3]))
            keep = torch.arange(e, device="cuda") != 3
            assert torch.equal(out[..., keep], clean[0][..., keep]) and torch.equal(last[..., keep], clean[1][..., keep])
        else:
            assert not bool(torch.isfinite(out[0, at, 0]).any())
            keep = torch.arange(d, device="cuda") != 3
            assert torch.equal(last[:, :, keep], clean[1][:, :, keep])
        dq, dk, dv, dlog, first = L.linear_attention_backward(grads["dout"], *y.values(), dstate=grads["dstate"], **more)
        assert bool(torch.isfinite(dlog[1])) and torch.equal(dlog[1], back[3][1])
        if name == "q":
            assert torch.equal(dk[:, at + 1:], back[1][:, at + 1:]) and torch.equal(dv[:, at + 1:], back[2][:, at + 1:])
        else:
            assert torch.equal(dq[:, :at], back[0][:, :at])
    dout = grads["dout"].clone()
    dout[0, at, 0, 3] = value
    dq, dk, dv, _, first = L.linear_attention_backward(dout, *x.values(), dstate=grads["dstate"], **more)
    assert not bool(torch.isfinite(dq[0, at, 0]).any()) and not bool(torch.isfinite(dv[0, at, 0, 3]))
    rows = torch.arange(s, device="cuda") != at
    assert torch.equal(dq[:, rows], back[0][:, rows])
    assert torch.equal(dk[:, at + 1:], back[1][:, at + 1:]) and torch.equal(dv[:, at + 1:], back[2][:, at + 1:])
    keep = torch.arange(e, device="cuda") != 3
    assert torch.equal(dv[..., keep], back[2][..., keep]) and torch.equal(first[..., keep], back[4][..., keep])


@pytest.mark.parametrize("size", [1e-5, 1e-3, 3e3])
def test_half_results_of_any_size(L, size):
    """In float16 what is rounded for a product keeps its bits whatever the size of v and dout."""
    for b, s, h, kv, d, e in ((2, 150, 4, 2, 64, 64), (1, 600, 2, 2, 32, 128)):
        x, more, grads = inputs(b, s, h, kv, d, e, F16, False, False, size=size)
        x["k"] = (x["k"].float() * (1e-2 if size > 1 else 1.0)).half()
        check(L, x, more, grads)


@pytest.mark.parametrize("dtype", ALL)
def test_decays(L, dtype):
    """None, almost none, all of it at once, growth, and one that ends 32-bit powers."""
    x, more, grads = inputs(1, 200, 6, 6, 32, 32, dtype, True, False)
    x["log_decay"] = torch.tensor([0.0, -1e-6, -math.inf, 0.01, -1.5, -100.0], device="cuda")
    r = M.linear(**x, **more)
    size = M.linear_abs(**x, **more)
    out, last = L.linear_attention_forward(**x, **more)
    passes(out, r["out"], M.linear_bound(r["out"], size["out"], dtype), "out")
    passes(last, r["last"], R.F32 * size["last"] + 1e-37, "state")
    x["log_decay"] = torch.tensor([0.0, -1e-6, -20.0, 0.01, -1.5, -100.0], device="cuda")
    check(L, x, more, grads)


@pytest.mark.parametrize("dtype", ALL)
def test_memory_without_an_end(L, dtype):
    """Ten thousand positions without decay: the state is a plain sum, and dlog_decay counts every step."""
    s, d = 10_000, 16
    g = gen(3)
    q, k, v = (normal(g, 1, s, 1, d, dtype=dtype) for _ in range(3))
    for log in (0.0, -2.0 ** -20):
        decay = torch.full((1,), log, device="cuda")
        out, last = L.linear_attention_forward(q, k, v, decay)
        w = torch.exp(decay.double() * torch.arange(s - 1, -1, -1, device="cuda", dtype=torch.float64))[:, None]
        kd, vd = k[0, :, 0].double(), v[0, :, 0].double()
        passes(last[0, 0], (kd * w).t() @ vd, R.F32 * ((kd * w).abs().t() @ vd.abs()), "state")
        # g^(i-j) = g^(s-1-j) / g^(s-1-i)
        steps = torch.cumsum(kd[:, :, None] * vd[:, None, :] * w[:, :, None], 0) / w[:, :, None]
        want = (q[0, :, 0].double()[:, None, :] @ steps)[:, 0] * d ** -0.5
        most = torch.cumsum(kd.abs()[:, :, None] * vd.abs()[:, None, :], 0)
        size = (q[0, :, 0].double().abs()[:, None, :] @ most)[:, 0] * d ** -0.5
        passes(out[0, :, 0], want, M.linear_bound(want, size, dtype), "out")


def test_scale_and_options(L):
    x, more, grads = inputs(2, 90, 4, 2, 64, 32, F32, True, False)
    check(L, x, more, grads, scale=0.7)
    full = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more)
    part = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more, decay=False)
    assert part[3] is None and all(torch.equal(a, b) for i, (a, b) in enumerate(zip(full, part)) if i != 3)
    # dstate alone, and neither
    for dstate in (grads["dstate"], None):
        r = M.linear(**x, dout=torch.zeros_like(grads["dout"]), dstate=dstate)
        size = M.linear_abs(**x, dout=torch.zeros_like(grads["dout"]), dstate=dstate)
        got = L.linear_attention_backward(torch.zeros_like(grads["dout"]), *x.values(), dstate=dstate)
        for a, n in zip(got, ("dq", "dk", "dv", "dlog")):
            passes(a, r[n], R.F32 * size[n] + 2.0 ** -24 * r[n].abs(), n)


def test_autograd_and_differences(L):
    g = gen(8)
    b, s, h, kv, d, e = 2, 37, 4, 2, 8, 12
    leaves = [normal(g, b, s, h, d), normal(g, b, s, kv, d), normal(g, b, s, kv, e), decays(h, g), normal(g, b, h, d, e)]
    leaves[3][1] = -0.7
    for t in leaves:
        t.requires_grad_()
    dout, dlast = normal(g, e, s, h, b).permute(3, 1, 2, 0), normal(g, b, h, e, d).transpose(2, 3)
    out, last = L.linear_attention(*leaves[:4], state=leaves[4])
    got = torch.autograd.grad((out, last), leaves, (dout, dlast))
    args = [t.detach() for t in leaves]
    r = M.linear(*args[:4], state=args[4], dout=dout, dstate=dlast)
    size = M.linear_abs(*args[:4], state=args[4], dout=dout, dstate=dlast)
    for a, n in zip(got, ("dq", "dk", "dv", "dlog", "dstate")):
        passes(a, r[n], R.F32 * (size[n] + r[n].abs()), n)
    step = 2.0 ** -7  # central differences: off by step^2 of third derivatives and 2^-24 / step of the sums
    for i, t in enumerate(leaves):
        way = normal(g, *t.shape) * (0.05 if i == 3 else 1.0)
        ends = []
        for sign in (step, -step):
            moved = list(args)
            moved[i] = args[i] + sign * way
            o, z = L.linear_attention(*moved[:4], state=moved[4])
            ends.append((o.double() * dout).sum() + (z.double() * dlast).sum())
        have, most = float((got[i].double() * way).sum()), float((got[i].double() * way).abs().sum())
        assert abs(float(ends[0] - ends[1]) / (2 * step) - have) <= 16 * step * step * (most + 1)
    # parts of the inputs and of the results
    out, last = L.linear_attention(*args[:3], leaves[3])
    assert torch.autograd.grad(last, leaves[3], dlast)[0].shape == (h,)
    out, last = L.linear_attention(leaves[0], *args[1:4])
    assert torch.equal(torch.autograd.grad(out, leaves[0], dout)[0], L.linear_attention_backward(dout.contiguous(), *args[:4])[0])
    first, = torch.autograd.grad(L.linear_attention(leaves[0], *args[1:4])[0].sum(), leaves[0], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(first.sum(), leaves[0])


def test_empty_calls(L):
    dev = "cuda"
    q, log = torch.zeros(2, 0, 4, 8, device=dev), torch.zeros(4, device=dev)
    state = torch.randn(2, 4, 8, 8, device=dev)
    out, last = L.linear_attention_forward(q, q, q, log, state=state)
    assert out.shape == q.shape and torch.equal(last, state)
    dq, dk, dv, dlog, first = L.linear_attention_backward(q, q, q, q, log, state=state, dstate=state)
    assert torch.equal(first, state) and bool((dlog == 0).all())
    q = torch.zeros(0, 5, 4, 8, device=dev)
    out, last = L.linear_attention_forward(q, q, q, log)
    assert out.shape == q.shape and last.shape == (0, 4, 8, 8)
    assert bool((L.linear_attention_backward(q, q, q, q, log)[3] == 0).all())


def test_refusals(L):
    q = torch.zeros(2, 6, 4, 8, device="cuda")
    k, v, log = q[:, :, :2], torch.zeros(2, 6, 2, 5, device="cuda"), torch.zeros(4, device="cuda")
    state = torch.zeros(2, 4, 8, 5, device="cuda")
    f = L.linear_attention
    for call, error, match in (
            (lambda: f(q.cpu(), k, v, log), ValueError, "on the GPU"),
            (lambda: f(q, k.half(), v, log), TypeError, "k must be"),
            (lambda: f(q, k, v.half(), log), TypeError, "v must be"),
            (lambda: f(q, q[:, :, :3], torch.zeros(2, 6, 3, 5, device="cuda"), log), ValueError, "multiple of kv heads"),
            (lambda: f(q, k[:, :5], v, log), ValueError, "differ"),
            (lambda: f(q, k[..., :4], v, log), ValueError, "differ"),
            (lambda: f(q, k, v[:, :, :1], log), ValueError, "differ"),
            (lambda: f(q, k, v, log[:3]), ValueError, "log_decay"),
            (lambda: f(q, k, v, log.double()), TypeError, "log_decay"),
            (lambda: f(q, k, v, log.cpu()), ValueError, "log_decay"),
            (lambda: f(q, k, v, log, state=state.half()), TypeError, "state"),
            (lambda: f(q, k, v, log, state=state[:1]), ValueError, "state"),
            (lambda: f(q, k, v, log, state=torch.zeros(2, 4, 5, 8, device="cuda").transpose(2, 3)), ValueError, "next to each other"),
            (lambda: f(q, k, v, log, lengths=torch.zeros(2, device="cuda")), TypeError, "lengths"),
            (lambda: f(q, k, v, log, lengths=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError, "lengths"),
            (lambda: f(q, k, v, log, scale=0.0), ValueError, "scale"),
            (lambda: f(q, k, v, log, scale=math.nan), ValueError, "scale"),
            (lambda: f(q.transpose(1, 3), k, v, log), ValueError, "next to each other"),
            (lambda: f(torch.zeros(1, 2, 1, 129, device="cuda"), torch.zeros(1, 2, 1, 129, device="cuda"), torch.zeros(1, 2, 1, 8, device="cuda"), log[:1]), ValueError, "128"),
            (lambda: L.linear_attention_forward(q, k, v, log, out=q), ValueError, "out"),
            (lambda: L.linear_attention_forward(q, k, v, log, state_out=state[:1].expand(2, 4, 8, 5)), ValueError, "overlap"),
            (lambda: L.linear_attention_backward(q, q, k, v, log), ValueError, "dout"),
            (lambda: L.linear_attention_backward(torch.zeros(2, 6, 4, 5, device="cuda"), q, k, v, log, dstate=state[:1]), ValueError, "dstate"),
    ):
        with pytest.raises(error, match=match):
            call()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(q, torch.ones_like(q))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            f(dual, k, v, log)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_captured(L, dtype):
    """Two graphs of one stream's calls, replayed in turn with eager calls between."""
    x, more, grads = inputs(2, 140, 4, 2, 64, 64, dtype, True, False)
    step, more1, _ = inputs(2, 1, 4, 2, 64, 64, dtype, True, False)

    def whole():
        return (*L.linear_attention_forward(**x, **more),
                *L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more))

    def one():
        return L.linear_attention_forward(**step, **more1)

    whole(), one()
    graphs, outs = [], []
    for f in (whole, one):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(f())
        graphs.append(graph)
    g = gen(1)
    for turn in range(3):
        for t in (x["q"], x["v"], grads["dout"], step["k"], more["state"], more1["state"]):
            t.copy_(normal(g, *t.shape))
        want = [[t.clone() for t in f()] for f in (whole, one)]
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert all(torch.equal(s, t) for s, t in zip(a, b)), turn


def test_places(L):
    """out is no input; state_out is the state's own layout or apart from it."""
    g = gen(13)
    q, k, v = (normal(g, 3, 70, 3, 8, dtype=F16) for _ in range(3))
    log = torch.tensor([-0.1, -0.2, -0.3], device="cuda")
    state = normal(g, 3, 3, 8, 8)
    for t in (q, k, v):
        with pytest.raises(ValueError, match="must not be an input"):
            L.linear_attention_forward(q, k, v, log, out=t)
    was = state.clone()
    for s in (1, 70):
        with pytest.raises(ValueError, match="laid out differently"):
            L.linear_attention_forward(q[:, :s], k[:, :s], v[:, :s], log, state=state, state_out=state.transpose(0, 1))
    assert torch.equal(state, was)
    for s in (1, 70):
        a = q[:, :s], k[:, :s], v[:, :s], log
        want = L.linear_attention_forward(*a, state=state)
        out, last = L.linear_attention_forward(*a, state=state, state_out=state)
        assert last is state and torch.equal(out, want[0]) and torch.equal(state, want[1])


def test_threads_that_share_a_stream(L):
    """Each thread's results are the bits that it gets alone."""
    jobs = [inputs(2, 400 + 100 * i, 4, 2, 32 * (i + 1), 48, dtype, True, False) for i, dtype in enumerate(ALL)]

    def work(i):
        x, more, grads = jobs[i]
        y, h, rstd = L.rms_norm_forward(x["q"])
        both = [x["k"].clone(), x["v"].clone()]
        return (*L.linear_attention_forward(**x, **more),
                *L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more),
                y, *L.rms_norm_backward(h, h, None, rstd), L.clip_gradients(both, 1.0), *both)

    want = [work(i) for i in range(3)]
    wrong, start = [], threading.Barrier(3)

    def repeat(i):
        start.wait(60)
        for _ in range(20):
            if not all(torch.equal(a, b) for a, b in zip(work(i), want[i])):
                wrong.append(i)

    threads = [threading.Thread(target=repeat, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not any(t.is_alive() for t in threads) and wrong == []


def test_another_stream(L):
    """The same bits on a stream of the caller's, with scratch memory of its own."""
    x, more, grads = inputs(2, 700, 4, 2, 64, 64, BF16, True, True)

    def work():
        y, h, rstd = L.rms_norm_forward(x["q"])
        return (*L.linear_attention_forward(**x, **more),
                *L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more),
                y, *L.rms_norm_backward(h, h, None, rstd), L.gradient_norm([x["k"], x["v"]]))

    want = work()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = [work() for _ in range(3)]
    here = work()  # meanwhile
    torch.cuda.synchronize()
    for r in (*got, here):
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_results_do_not_depend_on_timing(L):
    x, more, grads = inputs(3, 700, 4, 2, 64, 64, BF16, True, True)
    runs = [(*L.linear_attention_forward(**x, **more), *L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more))
            for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_rows_far_apart(L):
    """Offsets past 32 bits: a batch, a row and a state far from the first."""
    d = 32
    big = torch.zeros(3, (1 << 30) + 4096, dtype=F16, device="cuda")
    rows = big[:, :1 << 30].view(3, 64, 1, 1 << 24)[:, :, :, :d]  # rows 2^24 values apart
    g = gen(2)
    q, v = normal(g, 3, 64, 1, d, dtype=F16), normal(g, 3, 64, 1, d, dtype=F16)
    rows.copy_(normal(g, 3, 64, 1, d, dtype=F16))
    log = torch.full((1,), -0.1, device="cuda")
    assert torch.equal(L.linear_attention_forward(q, rows, v, log)[0], L.linear_attention_forward(q, rows.contiguous(), v, log)[0])
    dout = normal(g, 3, 64, 1, d, dtype=F16)
    for a, b in zip(L.linear_attention_backward(dout, q, rows, v, log)[:4], L.linear_attention_backward(dout, q, rows.contiguous(), v, log)[:4]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("s", [600, 4000])
def test_overflow_costs_little(L, s, dtype):
    """A training pass whose values are NaN everywhere takes little longer than one of numbers."""
    x, more, grads = inputs(2, s, 8, 8, 64, 64, dtype, False, False)
    bad = {**x, "v": torch.full_like(x["v"], math.nan)}

    def took(y):
        best = math.inf
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(5):
                L.linear_attention_forward(**y, **more)
                L.linear_attention_backward(grads["dout"], *y.values(), **more)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    plain, odd = took(x), took(bad)
    print(f"{odd / plain:.2f} times as long", flush=True)
    assert odd < 6 * plain
    out, last = L.linear_attention_forward(**bad, **more)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(last).all())


def test_what_is_written_is_known_to_autograd(L):
    """A state that a graph keeps, and that a step then overwrites, is an error and no wrong gradient."""
    x, more, _ = inputs(1, 40, 2, 2, 16, 16, F32, True, False)
    q = x["q"].clone().requires_grad_()
    out, _ = L.linear_attention(q, x["k"], x["v"], x["log_decay"], state=more["state"])
    L.linear_attention_forward(*(x[n][:, :1] for n in "qkv"), x["log_decay"], state=more["state"], state_out=more["state"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    w = torch.randn(3, 8, device="cuda", requires_grad=True)
    loss = (w * w).sum()
    L.clip_gradients(w.detach(), 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        state = torch.zeros(1, 2, 16, 16, device="cuda")
        L.linear_attention_forward(*(x[n][:, :1] for n in "qkv"), x["log_decay"], state=state, state_out=state)
        assert bool((state != 0).any())
