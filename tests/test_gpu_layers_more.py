"""The network operators on the GPU where their first tests did not look: gradients of small
size, layouts of the same values, infinities, launches past 2^32 threads, threads that share a stream."""
from __future__ import annotations

import math
import threading

import pytest
import torch

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
    w = R.worst(got, want, bound)
    print(f"{what}: {w:.3f} of the bound", flush=True)
    assert w <= 1.0, (what, w)


# ---- threads that share a stream ---------------------------------------------------


def test_threads_that_share_a_stream(L):
    """Each thread's results are the bits that it gets alone: calls of several launches do not mix."""
    def job(i):
        g = gen(i)
        x = normal(g, 2, 3000 + 100 * i, 64).transpose(1, 2)                  # sums, join, outputs
        q = normal(g, 2, 1, 8, 64, dtype=BF16)                                # split keys, join
        k, v = (normal(g, 2, 2000 + 300 * i, 2, 64, dtype=BF16) for _ in range(2))
        t = [normal(g, 1, 300 + 10 * i, 4, 32, dtype=F16) for _ in range(4)]  # row statistics, both gradients

        def call():
            y, mean, rstd = L.group_norm_forward(x, 8, activation="silu")
            out, lse = L.attention_forward(*t[:3], causal=True)
            return (y, *L.group_norm_backward(y, x, 8, None, None, mean, rstd, activation="silu"),
                    *L.attention_forward(q, k, v), *L.attention_backward(t[3], *t[:3], out, lse, causal=True))
        return call

    calls = [job(i) for i in range(4)]
    alone = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(4)

    def work(i):
        start.wait(30)
        for turn in range(50):
            for n, (a, b) in enumerate(zip(calls[i](), alone[i])):
                if not torch.equal(a, b):
                    wrong.append((i, turn, n))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not any(t.is_alive() for t in threads) and wrong == []


# ---- half precision -------------------------------------------------------------


@pytest.mark.parametrize("q,s,h,kv,d,options", [
    (64, 8160, 2, 2, 64, {}),
    (300, 1000, 4, 2, 128, {"causal": True}),
    (130, 4000, 2, 1, 40, {"mask": True}),
    (40, 700, 2, 2, 33, {"causal": True}),
])
@pytest.mark.parametrize("size,v_size", [(2.0 ** -7, 1.0), (2.0 ** -10, 1.0), (2.0 ** -13, 4.0), (1.0, 2.0 ** -10),
                                         (2.0 ** 9, 2.0 ** 7)])
def test_half_gradients_of_any_size(L, q, s, h, kv, d, options, size, v_size):
    """The products' operands keep their relative precision whatever the size of dout or v: the
    bound has no term for float16's least step but the results' own."""
    g = gen(q + s)
    options = dict(options)
    if "mask" in options:
        options["mask"] = torch.rand(q, s, generator=g, device="cuda") < 0.5
    qt, k = normal(g, 1, q, h, d, dtype=F16), normal(g, 1, s, kv, d, dtype=F16)
    v, dout = (v_size * normal(g, 1, s, kv, d)).half(), (size * normal(g, 1, q, h, d)).half()
    out, lse = L.attention_forward(qt, k, v, **options)
    r = R.attention(qt, k, v, dout, **options)
    u, e = R.UNIT[F16], R.F32 + r["slack"]
    # out, as the forward call rounded it, is an operand of D: off by u (and half a least step)
    low = R.STEP[F16] * dout.double().abs().sum(3).amax().item() * max(qt.abs().max().item(), k.abs().max().item())
    for x, name, n in zip(L.attention_backward(dout, qt, k, v, out, lse, **options), ("dq", "dk", "dv"), (3, 3, 2)):
        passes(x, r[name], (n * u + 2 * e) * r[name + "_abs"] + R.STEP[F16] + low * d ** -0.5, name)


@pytest.mark.parametrize("b,n,h", [(600, 1, 2), (20, 70, 8), (1, 16384, 2)])
def test_half_probabilities_of_a_long_row(L, b, n, h):
    """One key far above 40000 equal others, which together still count: their probabilities lie
    among float16's last numbers, where rounding them would move the sum by per cents."""
    s, d, high = 40000, 32, 14.4921875  # exp(-high) = 8.53 of float16's least steps
    q, k, v = (torch.zeros(m, r, h, d, device="cuda", dtype=F16) for m, r in ((b, n), (1, s), (1, s)))
    q[..., 0], k[:, 7, :, 0] = 1.0, high  # in the first tile, so all others are taken with its maximum
    v.fill_(1.0)
    v[:, 7] = 0.0
    out, lse = L.attention_forward(q, k.expand(b, s, h, d), v.expand(b, s, h, d), scale=1.0)
    share = (s - 1) * math.exp(-high) / (1 + (s - 1) * math.exp(-high))
    passes(out, torch.full_like(out, share, dtype=torch.float64), (2 * R.UNIT[F16] + R.F32) * share, "out")
    want = high + math.log1p((s - 1) * math.exp(-high))
    passes(lse, torch.full_like(lse, want, dtype=torch.float64), R.F32 * (1 + want), "lse")


# ---- the same bits from the same values --------------------------------------------


def laid_out(x, how):
    """The same values [N, S, C] in other places: at an odd address, with rows further apart, ..."""
    n, s, c = x.shape
    if how == "odd address":
        y = torch.empty(n * s * c + 1, dtype=x.dtype, device="cuda")[1:].view(n, s, c)
    elif how == "odd rows":
        y = torch.empty(n, s, c + 3, dtype=x.dtype, device="cuda")[..., 1:c + 1]
    elif how == "pairs":
        y = torch.empty(n, s, c + 2, dtype=x.dtype, device="cuda")[..., 2:]
    else:  # samples apart by an odd number
        y = torch.empty(n, s * c + 1, dtype=x.dtype, device="cuda")[:, 1:].unflatten(1, (s, c))
    y.copy_(x)
    return y


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("how", ["odd address", "odd rows", "pairs", "odd samples"])
@pytest.mark.parametrize("n,s,c,groups", [(1, 510, 192, 32), (2, 1600, 192, 32), (3, 4000, 64, 4), (2, 77, 30, 5),
                                          (40, 700, 24, 3), (1, 9000, 320, 32)])
def test_group_norm_bits_do_not_depend_on_layout(L, n, s, c, groups, how, dtype):
    g = gen(s)
    x, dy = (normal(g, n, s, c, dtype=dtype) for _ in range(2))
    w, b = normal(g, c), normal(g, c)

    def call(x, dy):
        x, dy = x.transpose(1, 2), dy.transpose(1, 2)
        out = L.group_norm_forward(x, groups, w, b, activation="silu")
        return (*out, *L.group_norm_backward(dy, x, groups, w, b, *out[1:], activation="silu"))

    first = call(x, dy)
    for a, b_ in ((laid_out(x, how), dy), (x, laid_out(dy, how)), (laid_out(x, how), laid_out(dy, how))):
        for got, want, name in zip(call(a, b_), first, ("y", "mean", "rstd", "dx", "dw", "db")):
            assert torch.equal(got, want), name


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("how", ["odd address", "odd rows", "odd samples"])
@pytest.mark.parametrize("b,q,s,h,kv,d,options", [
    (1, 1, 20000, 2, 1, 32, {}),                      # many splits
    (2, 1, 9000, 3, 1, 64, {}),
    (1, 20, 7000, 2, 2, 96, {"causal": True}),
    (32, 140, 200, 4, 2, 32, {"causal": True}),
    (32, 140, 200, 4, 2, 64, {"window": (30, 40)}),
    (3, 300, 300, 2, 2, 40, {"lengths": True}),
    (1, 1030, 1030, 2, 1, 96, {"mask": True}),
    (1, 1030, 1030, 4, 2, 128, {"causal": True}),
])
def test_attention_bits_do_not_depend_on_layout(L, b, q, s, h, kv, d, options, how, dtype):
    g = gen(s)
    options = dict(options)
    if "lengths" in options:
        options = {"key_lengths": torch.tensor([s, s // 2, 1], dtype=torch.int32, device="cuda")}
    if "mask" in options:
        options["mask"] = torch.rand(q, s, generator=g, device="cuda") < 0.7
    t = [normal(g, b, q, h, d, dtype=dtype), normal(g, b, s, kv, d, dtype=dtype), normal(g, b, s, kv, d, dtype=dtype),
         normal(g, b, q, h, d, dtype=dtype)]

    def call(q, k, v, dout):
        out, lse = L.attention_forward(q, k, v, **options)
        return (out, lse, *L.attention_backward(dout, q, k, v, out, lse, **options))

    first = call(*t)
    moved = [laid_out(x.flatten(2), how).unflatten(2, x.shape[2:]) for x in t]
    for args in (moved, [moved[0], *t[1:]], [*t[:2], moved[2], t[3]]):
        for got, want, name in zip(call(*args), first, ("out", "lse", "dq", "dk", "dv")):
            assert torch.equal(got, want), name


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,r", [(64, 64), (40, 20), (96, 48), (24, 24)])
def test_rotary_bits_do_not_depend_on_layout(L, d, r, interleaved, dtype):
    g = gen(d)
    a = torch.rand(60, r // 2, generator=g, device="cuda", dtype=torch.float64) * 7
    cos, sin = a.cos().float(), a.sin().float()
    q = normal(g, 3, 60, 4, d, dtype=dtype)
    want, _ = L.rotary(q, None, cos, sin, interleaved=interleaved)
    for how in ("odd address", "odd rows", "pairs", "odd samples"):
        moved = laid_out(q.flatten(2), how).unflatten(2, (4, d))
        for out in (None, (torch.empty_like(q), None)):
            assert torch.equal(L.rotary(moved, None, cos, sin, interleaved=interleaved, out=out)[0], want), how
    odd = torch.empty(2, 60 * (r // 2) + 1, device="cuda")[:, 1:].unflatten(1, (60, r // 2))
    odd[0], odd[1] = cos, sin
    assert torch.equal(L.rotary(q, None, odd[0], odd[1], interleaved=interleaved)[0], want)


# ---- derivatives ---------------------------------------------------------------------


def operators(L, g):
    """(name, function of one tensor, the tensor) of each operator that autograd knows."""
    cos, sin = normal(g, 6, 4), normal(g, 6, 4)
    k = normal(g, 1, 6, 2, 8)
    return [("group_norm", lambda x: L.group_norm(x, 2, activation="silu"), normal(g, 1, 5, 8).transpose(1, 2)),
            ("rotary", lambda x: L.rotary(x, k, cos, sin)[0], normal(g, 1, 6, 2, 8)),
            ("attention", lambda x: L.attention(x, k, k), normal(g, 1, 6, 2, 8))]


@pytest.mark.parametrize("which", [0, 2])
def test_second_derivatives_are_refused(L, which):
    """Also where the first gradient is but a part of what is differentiated, which is how it would
    go missing; a graph that nobody walks costs nothing."""
    _, f, x = operators(L, gen(1))[which]
    x = x.detach().requires_grad_()
    plain, = torch.autograd.grad(f(x).square().sum(), x)
    for penalty in (lambda first: first.square().sum(), lambda first: first.square().sum() + x.square().sum()):
        for again in (lambda y: torch.autograd.grad(y, x), lambda y: y.backward()):
            first, = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
            assert torch.equal(first, plain)
            with pytest.raises(RuntimeError, match="second derivatives"):
                again(penalty(first))


def test_rotary_second_derivatives(L):
    """The rotation is linear: its gradient's gradient is the rotation again."""
    g = gen(2)
    cos, sin = normal(g, 6, 4), normal(g, 6, 4)
    x, k = normal(g, 1, 6, 2, 8).requires_grad_(), normal(g, 1, 6, 1, 8).requires_grad_()
    a, b = L.rotary(x, k, cos, sin)
    first = torch.autograd.grad((a.pow(3).sum() + b.pow(3).sum()) / 3, (x, k), create_graph=True)
    w = normal(g, 1, 6, 2, 8), normal(g, 1, 6, 1, 8)
    second = torch.autograd.grad(first, (x, k), w)
    for t, v, got in ((x, w[0], second[0]), (k, w[1], second[1])):
        turned, along = (R.turn(y.detach(), cos, sin, None, False) for y in (t, v))
        want = R.turn(2 * turned * along, cos, sin, None, False, inverse=True)
        passes(got, want, 1e-5 * (1 + want.abs().max()), "second")


@pytest.mark.parametrize("which", [0, 1, 2])
def test_forward_mode_is_refused(L, which):
    from torch.autograd import forward_ad
    _, f, x = operators(L, gen(3))[which]
    for grad in (False, True):
        with forward_ad.dual_level():
            dual = forward_ad.make_dual(x.detach().requires_grad_(grad), torch.ones_like(x))
            with pytest.raises(NotImplementedError, match="forward"):
                f(dual)
    f(x)


def test_rotary_tables_that_want_gradients_are_refused(L):
    g = gen(4)
    cos, sin, q = normal(g, 6, 4), normal(g, 6, 4), normal(g, 1, 6, 2, 8)
    for tables in ((cos.clone().requires_grad_(), sin), (cos, sin.clone().requires_grad_())):
        for x in (q, q.clone().requires_grad_()):
            with pytest.raises(NotImplementedError, match="cos and sin"):
                L.rotary(x, None, *tables)
        with torch.no_grad():
            L.rotary(q, None, *tables)


# ---- infinities ----------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("s", [100, 30000])  # one launch, three
@pytest.mark.parametrize("at", [0, 57])
def test_group_norm_statistics_of_infinities(L, s, value, at, dtype):
    x = normal(gen(s), 2, s, 64, dtype=dtype)
    x[1, at, 19] = value
    y, mean, rstd = L.group_norm_forward(x.transpose(1, 2), 8)
    assert bool(torch.isnan(rstd[1, 2])) and not bool(torch.isfinite(mean[1, 2]))
    assert bool(torch.isnan(y[1, 16:24]).all())
    clean = torch.ones(2, 64, dtype=torch.bool, device="cuda")
    clean[1, 16:24] = False
    assert bool(torch.isfinite(y[clean]).all())
    clean = clean[:, ::8]
    assert bool(torch.isfinite(mean[clean]).all()) and bool(torch.isfinite(rstd[clean]).all())


@pytest.mark.parametrize("s", [100, 30000])
def test_relu_of_minus_infinity_is_zero(L, s):
    x = normal(gen(s), 1, s, 64).transpose(1, 2)
    bias = torch.zeros(64, device="cuda")
    bias[5], bias[6], bias[7] = -math.inf, math.inf, math.nan
    y = L.group_norm_forward(x, 8, None, bias, activation="relu")[0]
    assert bool((y[:, 5] == 0).all()) and bool((y[:, 6] == math.inf).all()) and bool(torch.isnan(y[:, 7]).all())
    assert bool(torch.isfinite(y[:, :5]).all())
    assert not bool(torch.signbit(y[:, :5]).any())  # and no zeros with a sign


# ---- rotary ----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("d,r", [(16, 8), (64, 32), (24, 10)])
def test_rotary_positions_outside_the_tables_take_the_whole_token(L, d, r, in_place, dtype):
    g = gen(d)
    cos, sin = normal(g, 10, r // 2), normal(g, 10, r // 2)
    q, k = normal(g, 1, 4, 3, d, dtype=dtype), normal(g, 1, 4, 1, d, dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, -1, 9, 10], dtype=torch.int32, device="cuda")
    got = L.rotary(q, k, cos, sin, positions=at, status=status, out=(q, k) if in_place else None)
    assert int(status) == -3
    for y in got:
        assert bool(torch.isnan(y[:, [1, 3]]).all()) and bool(torch.isfinite(y[:, [0, 2]]).all())


def test_rotary_without_query_heads_is_refused(L):
    """It used to return keys that no kernel had written."""
    c, k = torch.zeros(4, 4, device="cuda"), torch.ones(1, 4, 2, 8, device="cuda")
    with pytest.raises(ValueError, match="heads"):
        L.rotary(torch.empty(1, 4, 0, 8, device="cuda"), k, c, c)
    q, k = L.rotary(torch.empty(1, 0, 2, 8, device="cuda"), k[:, :0], c, c)
    assert q.shape == (1, 0, 2, 8) and k.shape == (1, 0, 2, 8)


def test_outputs_that_overlap_are_refused(L):
    g = gen(5)
    q = normal(g, 2, 4, 2, 8)
    c = normal(g, 4, 4)
    with pytest.raises(ValueError, match="overlap"):
        L.attention_forward(q, q, q, out=torch.empty(1, 4, 2, 8, device="cuda").expand(2, 4, 2, 8))
    with pytest.raises(ValueError, match="overlap"):
        L.rotary(q, None, c, c, out=(torch.empty(2, 4, 1, 8, device="cuda").expand(2, 4, 2, 8), None))
    x = normal(g, 2, 4, 8).transpose(1, 2)
    with pytest.raises(ValueError, match="overlap"):
        L.group_norm_forward(x, 2, out=torch.empty(2, 1, 8, device="cuda").expand(2, 4, 8).transpose(1, 2))


# ---- launches past 2^32 threads ---------------------------------------------------------


def test_rotary_of_more_threads_than_a_launch_has(L):
    """2^32 threads and more of two values each (heads of 6): several launches."""
    g = gen(1)
    s, h = 1 << 20, 1366
    cos, sin = normal(g, s, 3), normal(g, s, 3)
    some = normal(g, 1, 1, h, 6, dtype=BF16)
    q = torch.empty(1, s, h, 6, dtype=BF16, device="cuda")
    q.copy_(some.expand(1, s, h, 6))
    got, _ = L.rotary(q, None, cos, sin, out=(q, None))
    at = torch.cat((torch.arange(3, device="cuda"), torch.randint(0, s, (200,), generator=g, device="cuda"),
                    torch.arange(s - 3, s, device="cuda")))
    want = R.turn(some.expand(1, len(at), h, 6), cos[at], sin[at], None, False)
    passes(got[:, at], want, R.UNIT[BF16] * want.abs() + 4 * 2.0 ** -24 * some.double().abs().max() * 4, "turned")


def test_attention_of_more_threads_than_a_launch_has(L):
    """More than 2^24 blocks of 256 threads: one query on one key, whose value is the result."""
    b, h, d = 1 << 20, 17, 8
    g = gen(2)
    q, k, v, dout = (normal(g, b, 1, h, d, dtype=BF16) for _ in range(4))
    out, lse = L.attention_forward(q, k, v)
    assert torch.equal(out, v)
    want = (q.float() * k.float()).sum(3).transpose(1, 2) * d ** -0.5
    assert float((lse - want).abs().max()) <= R.F32 * (1 + float(want.abs().max()))
    dq, dk, dv = L.attention_backward(dout, q, k, v, out, lse)
    # the probability is 1, off by what exp and lse leave of it
    assert float(((dv.float() - dout.float()).abs() - (2.0 ** -8 + 1e-4) * dout.float().abs()).max()) <= 0
    assert float(dq.abs().max()) < 0.01 and float(dk.abs().max()) < 0.01


# ---- scratch memory ----------------------------------------------------------------------


def test_scratch_memory_can_be_given_back_while_it_is_used(L):
    g = gen(6)
    q, k, v = normal(g, 8, 1, 8, 64, dtype=BF16), *(normal(g, 8, 6000, 2, 64, dtype=BF16) for _ in range(2))
    want, _ = L.attention_forward(q, k, v)
    before = torch.cuda.memory_allocated()
    out = [L.attention_forward(q, k, v)[0]]
    L.release_workspaces()
    assert torch.cuda.memory_allocated() < before
    torch.full((1 << 22,), math.nan, device="cuda")  # takes the memory, behind the call
    out.append(L.attention_forward(q, k, v)[0])
    assert all(torch.equal(o, want) for o in out)


# ---- what a NaN costs --------------------------------------------------------------------


def microseconds(f):
    f()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for _ in range(3):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) * 1000 / 3


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("options", [{}, {"causal": True}, {"window": (100, 50)}, {"mask": True}])
@pytest.mark.parametrize("where,value", [("q", math.nan), ("q", math.inf), ("v", math.nan), ("dout", math.nan)])
def test_overflow_costs_little(L, options, where, value, dtype):
    """A training step that has overflowed takes about as long as any other (it took 14 to 216 times as
    long): what is NaN because of what a row sees is not formed again."""
    g = gen(3)
    b, n, h, d = 2, 1500, 4, 64
    options = dict(options)
    if "mask" in options:
        options["mask"] = torch.rand(n, n, generator=g, device="cuda") < 0.5
    t = {name: normal(g, b, n, h, d, dtype=dtype) for name in ("q", "k", "v", "dout")}

    def call():
        out, lse = L.attention_forward(t["q"], t["k"], t["v"], **options)
        L.attention_backward(t["dout"], t["q"], t["k"], t["v"], out, lse, **options)

    usual = microseconds(call)
    t[where].fill_(value)
    strange = microseconds(call)
    print(f"{usual:.0f} us, with {value} in {where} {strange:.0f} us", flush=True)
    assert strange < 10 * usual


def seen_sum(weights, values, ok):
    """[.., rows, dim] sums of weights x values over the last axis of `ok` [.., rows, others], over what it
    shows alone: 0 times an infinity is not formed."""
    return torch.where(ok[..., None], weights[..., None] * values[..., None, :, :], 0.0).sum(-2)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("b,q,s,h,kv,d,options", [
    (1, 1, 300, 4, 2, 32, {}),
    (2, 20, 200, 2, 1, 64, {"causal": True}),
    (3, 150, 150, 2, 2, 32, {"causal": True}),
    (12, 70, 130, 8, 4, 24, {"window": (20, 9)}),
    (2, 140, 140, 2, 1, 128, {"mask": 0.5}),
    (3, 130, 190, 2, 2, 40, {"lengths": [190, 77, 0]}),
    (1, 140, 600, 1, 1, 96, {"mask": 0.9}),
    (2, 129, 129, 2, 2, 33, {"causal": True}),
])
@pytest.mark.parametrize("where", ["k", "v", "q", "dout", "k v q dout"])
def test_attention_of_scattered_infinities(L, b, q, s, h, kv, d, options, where, dtype):
    """What is not finite is so in the very places, and of the very kind, that the formula gives when
    it is summed over what is seen alone."""
    g = gen(q + s)
    options = dict(options)
    if "mask" in options:
        options["mask"] = torch.rand(b, 1, q, s, generator=g, device="cuda") < options["mask"]
    if "lengths" in options:
        options = {"key_lengths": torch.tensor(options["lengths"], dtype=torch.int32, device="cuda")}
    t = {"q": normal(g, b, q, h, d), "k": normal(g, b, s, kv, d), "v": normal(g, b, s, kv, d),
         "dout": normal(g, b, q, h, d)}
    for name in where.split():
        x = t[name]
        rows = torch.rand(x.shape[:3], generator=g, device="cuda")[..., None]
        part = torch.rand(x.shape, generator=g, device="cuda")
        x[(rows < 0.03) & (part < 0.1)] = math.inf       # here and there in a row
        x[(rows > 0.97) & (part < 0.1)] = -math.inf
        x[(rows > 0.48) & (rows < 0.5) & (part < 0.2)] = math.nan
        x[((rows > 0.5) & (rows < 0.51)).expand_as(x)] = math.nan  # all of a row
    t = {k: x.to(dtype) for k, x in t.items()}
    out, lse = L.attention_forward(t["q"], t["k"], t["v"], **options)
    dq, dk, dv = L.attention_backward(t["dout"], t["q"], t["k"], t["v"], out, lse, **options)

    ok = R.seen(b, h, q, s, "cuda", **options)
    qd, dod = (t[n].double().permute(0, 2, 1, 3) for n in ("q", "dout"))
    kd, vd = (t[n].double().permute(0, 2, 1, 3).repeat_interleave(h // kv, 1) for n in ("k", "v"))
    scale = d ** -0.5
    a = torch.where(ok, (qd @ kd.transpose(2, 3).contiguous()) * scale, -math.inf)
    m = torch.nan_to_num(a, nan=-math.inf, posinf=math.inf).amax(3, keepdim=True)
    e = torch.where(ok, torch.exp(a - torch.where(m == -math.inf, 0.0, m)), 0.0)
    total = e.sum(3, keepdim=True)
    p = e / torch.where(total == 0, 1.0, total)
    o = seen_sum(p, vd, ok)
    od = out.double().permute(0, 2, 1, 3)  # D is formed from what the forward call gave
    ds = p * (dod @ vd.transpose(2, 3).contiguous() - (dod * od).sum(3, keepdim=True))
    turned = ok.transpose(2, 3)

    def back(x):
        return x.permute(0, 2, 1, 3)

    def gather(x):
        return back(x.reshape(b, kv, h // kv, s, d).sum(2))

    want = {"out": back(o), "dq": back(seen_sum(ds, kd, ok)) * scale,
            "dk": gather(seen_sum(ds.transpose(2, 3), qd, turned)) * scale,
            "dv": gather(seen_sum(p.transpose(2, 3), dod, turned))}
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        w = want[name]
        kinds = [torch.nan_to_num(x.double(), nan=3.0, posinf=2.0, neginf=-2.0).where(~torch.isfinite(x), 0.0)
                 for x in (got, w)]
        assert torch.equal(*kinds), name
        fine = torch.isfinite(w)
        if bool(fine.any()):
            assert float((got.double() - w)[fine].abs().max()) <= 0.05 * max(1.0, float(w[fine].abs().max())), name


# ---- group norm at other sizes -----------------------------------------------------------


def norm_passes(L, n, s, c, groups, dtype, kind, backward=True):
    g = gen(s + c)
    x = (1.5 * normal(g, n, s, c) + normal(g, c)).to(dtype).transpose(1, 2)
    w, b = 1 + 0.3 * normal(g, c), 0.3 * normal(g, c)
    dy = normal(g, n, s, c, dtype=dtype).transpose(1, 2) if backward else None
    y, mean, rstd = L.group_norm_forward(x, groups, w, b, activation=kind)
    r = R.group_norm(x, groups, w, b, 1e-5, kind, dy)
    u = R.UNIT[dtype]
    passes(y, r["y"], u * r["y"].abs() + R.F32 * (1 + r["u"].abs()), "y")
    passes(mean, r["mean"], R.F32 * (1 + r["mean"].abs()), "mean")
    passes(rstd, r["rstd"], R.F32 * r["rstd"], "rstd")
    if backward:
        dx, dw, db = L.group_norm_backward(dy, x, groups, w, b, mean, rstd, activation=kind)
        passes(dx, r["dx"], u * r["dx"].abs() + R.F32 * r["dx_abs"], "dx")
        passes(dw, r["dw"], R.UNIT[F32] * r["dw"].abs() + R.F32 * (r["dw_abs"] + r["db_abs"]), "dw")
        passes(db, r["db"], R.UNIT[F32] * r["db"].abs() + R.F32 * r["db_abs"], "db")


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("n,s,c,groups", [(1, 8160, 192, 32), (2, 32640, 96, 8), (3, 5001, 30, 5), (1, 130560, 64, 1)])
def test_group_norm_of_many_positions(L, n, s, c, groups, dtype):
    norm_passes(L, n, s, c, groups, dtype, "silu")


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("s", [1360, 1530, 1531, 1701])  # one launch up to about here, three from here on
def test_group_norm_where_one_launch_becomes_three(L, s, dtype):
    norm_passes(L, 16, s, 192, 32, dtype, "gelu")


@pytest.mark.parametrize("dtype,c", [(BF16, 128), (F32, 64), (F16, 96)])
def test_group_norm_past_the_caches(L, c, dtype):
    """Inputs and outputs of more than 256 MB: the outputs' stores pass the caches."""
    norm_passes(L, 1, 1100 * 1000, c, 8, dtype, "silu", backward=False)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("b,q,s,h,kv,d", [(24, 140, 197, 4, 4, 32), (24, 140, 197, 4, 2, 64), (8, 300, 300, 4, 4, 96),
                                          (4, 130, 400, 2, 1, 128), (2, 9, 700, 4, 2, 64)])
def test_attention_bits_do_not_depend_on_the_masks_layout(L, b, q, s, h, kv, d, dtype):
    g = gen(s + d)
    t = [normal(g, b, n, m, d, dtype=dtype) for n, m in ((q, h), (s, kv), (s, kv), (q, h))]
    mask = torch.rand(b, 1, q, s, generator=g, device="cuda") < 0.6
    spread = torch.zeros(b, 1, q, 2 * s + 1, dtype=torch.bool, device="cuda")[..., 1::2]
    spread.copy_(mask)
    layouts = [mask, mask.transpose(2, 3).contiguous().transpose(2, 3), mask.expand(b, h, q, s).contiguous(),
               spread, torch.nn.functional.pad(mask, (3, 2))[..., 3:3 + s]]

    def call(mask):
        out, lse = L.attention_forward(*t[:3], mask=mask)
        return (out, lse, *L.attention_backward(t[3], *t[:3], out, lse, mask=mask))

    first = call(mask)
    for other in layouts[1:]:
        for got, want, name in zip(call(other), first, ("out", "lse", "dq", "dk", "dv")):
            assert torch.equal(got, want), name
