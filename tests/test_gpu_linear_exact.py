"""Linear attention held to what its arithmetic allows: outputs and gradients to their last rounding, states and
the decay's gradient to 32-bit sums, near and far sizes of values side by side, many segments."""
from __future__ import annotations

import pytest
import torch

import layers_more_ref as M
import layers_ref as R
from test_gpu_linear import ALL, BF16, F16, F32, L, decays, gen, inputs, normal, passes  # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu

# What 32-bit arithmetic loses of a sum of absolute terms: powers of g and the scale (4 roundings of 2^-24), the
# state's step from run to run (2^-21 at most, 8 of them), and sums in short chains, whose roundings have no
# common sign (4, for chains of up to some hundred).
SUMS = 16 * 2.0 ** -24
# What an operand of a product that forms an output loses in its two parts: x = part + rest, |rest| < u of x, so rest
# is rounded by u / 2 of u at most; float32 is its own operand.
PARTS = {F32: 0.0, F16: 2.0 ** -23, BF16: 2.0 ** -17}


def once(want, size, dtype):
    """Rounded once from sums of operands in parts."""
    return R.UNIT[dtype] * want.abs() + (SUMS + PARTS[dtype]) * size + R.STEP[dtype]


def both(x, more, grads):
    return M.linear(**x, **more, **grads), M.linear_abs(**x, **more, **grads)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("b,s,h,kv,d,e,state,ragged", [
    (2, 1, 4, 2, 64, 64, True, False), (2, 2, 3, 3, 32, 32, True, False), (1, 31, 3, 1, 40, 33, True, False),
    (4, 65, 6, 3, 32, 32, True, True), (2, 130, 4, 1, 96, 72, True, False), (3, 200, 4, 2, 128, 128, True, True),
    (1, 700, 4, 4, 64, 64, False, False), (4, 510, 6, 6, 32, 32, False, False), (2, 1100, 3, 3, 20, 5, True, True),
])
def test_outputs_are_rounded_once(L, b, s, h, kv, d, e, state, ragged, dtype):  # noqa: F811
    """Scores and states keep their bits on the way into the products that form out, dq, dk and dv."""
    x, more, grads = inputs(b, s, h, kv, d, e, dtype, state, ragged, seed=1)
    r, size = both(x, more, grads)
    out, _ = L.linear_attention_forward(**x, **more)
    dq, dk, dv, _, _ = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more)
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        passes(got, r[name], once(r[name], size[name], dtype), name)


def alone(b, s, h, d, e, at, size, dtype=F16):
    """Tokens of `size` in one component."""
    t = torch.zeros(b, s, h, e if e else d, device="cuda")
    t[..., at] = size
    return t.to(dtype)


@pytest.mark.parametrize("s", [2, 40, 700])
@pytest.mark.parametrize("state,scale", [(2.0 ** 100, None), (2.0 ** 120, None), (2.0 ** 80, 2.0 ** -30), (2.0 ** 60, 2.0 ** -60)])
def test_half_beside_a_very_large_state(L, s, state, scale):  # noqa: F811
    """A state's large entry that no token sees leaves what they do see as it is, forward and backward."""
    d = 32
    q, v = (normal(gen(i), 1, s, 2, d, dtype=F16) * 2.0 ** -6 for i in (1, 2))
    k = normal(gen(3), 1, s, 2, d, dtype=F16) * 2.0 ** -6
    for t in (q, k):
        t[..., 0] = 0
    first = torch.zeros(1, 2, d, d, device="cuda")
    first[:, :, 0, 0] = state
    log = torch.tensor([-0.01, 0.0], device="cuda")
    x = {"q": q, "k": k, "v": v, "log_decay": log}
    more = {"state": first, "lengths": None, "scale": scale}
    grads = {"dout": normal(gen(4), 1, s, 2, d, dtype=F16) * 2.0 ** -6, "dstate": torch.zeros_like(first)}
    grads["dout"][..., 0] = 0
    grads["dstate"][:, :, 0, 0] = state
    v[..., 0] = 0
    r, size = both(x, more, grads)
    out, last = L.linear_attention_forward(**x, **more)
    passes(out, r["out"], once(r["out"], size["out"], F16), "out")
    # the large entry stays beside what the tokens add
    passes(last, r["last"], R.F32 * size["last"], "state")
    dq, dk, dv, _, _ = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more)
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        passes(got, r[name], once(r[name], size[name], F16), name)


def test_half_tokens_of_one_component_beside_a_very_large_state(L):  # noqa: F811
    x = {"q": alone(1, 2, 1, 32, 0, 1, 2.0 ** -14), "k": alone(1, 2, 1, 32, 0, 1, 2.0 ** -14),
         "v": torch.ones(1, 2, 1, 32, dtype=F16, device="cuda"), "log_decay": torch.zeros(1, device="cuda")}
    state = torch.zeros(1, 1, 32, 32, device="cuda")
    state[0, 0, 0, 0] = 2.0 ** 100
    out, last = L.linear_attention_forward(**x, state=state)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(last).all()) and float(last[0, 0, 0, 0]) == 2.0 ** 100


@pytest.mark.parametrize("s", [40, 700])
def test_half_columns_far_apart_in_size(L, s):  # noqa: F811
    """One column of v (dout, q, k) twenty-eight powers of two above its neighbours takes none of their bits."""
    def columns(t):
        t = t.float() * 2.0 ** -14
        t[..., 5] *= 2.0 ** 28
        return t.half()

    x, more, grads = inputs(2, s, 4, 2, 64, 64, F16, False, False, seed=2)
    x["q"], x["k"] = 4 * x["q"], 4 * x["k"]
    x["v"], grads["dout"] = columns(x["v"]), columns(grads["dout"])
    r, size = both(x, more, grads)
    out, _ = L.linear_attention_forward(**x, **more)
    passes(out, r["out"], once(r["out"], size["out"], F16), "out")
    dv = L.linear_attention_backward(grads["dout"], *x.values(), **more)[2]
    passes(dv, r["dv"], once(r["dv"], size["dv"], F16), "dv")


def plain_state(k, v, log_decay, lengths=None):
    """sum over tokens of g^(n - 1 - j) k_j v_j' in 64 bits, of one kv head a head, and of absolute values."""
    b, s, h, _ = k.shape
    n = torch.full((b,), s, device="cuda") if lengths is None else lengths.long()
    steps = n[:, None] - 1 - torch.arange(s, device="cuda")  # [B, S]
    w = torch.exp(steps.clamp(min=0)[:, None].double() * log_decay.double()[None, :, None]) * (steps >= 0)[:, None]
    kd, vd = (t.double().permute(0, 2, 1, 3) for t in (k, v))
    return ((kd * w[..., None]).transpose(2, 3).contiguous() @ vd.contiguous(),
            (kd.abs() * w[..., None]).transpose(2, 3).contiguous() @ vd.abs().contiguous())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("s,lengths", [(32640, None), (16400, (16400, 9001)), (5000, (4999, 37)), (2500, None)])
def test_long_memories_do_not_drift(L, s, lengths, dtype):  # noqa: F811
    """States of values of one sign, with memories of a thousand to a million positions, over up to 255 segments: the
    powers that carry a state on are off by no common part."""
    h, d, b = 4, 16, 1 if lengths is None else 2
    g = gen(s)
    q, k, v, dout = (normal(g, b, s, h, d).abs().to(dtype) for _ in range(4))
    log = torch.log1p(-torch.tensor([1e-3, 1e-4, 1.3e-5, 1e-6], device="cuda"))
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    state, dstate = (normal(g, b, h, d, d).abs() * 100 for _ in range(2))
    stay = torch.exp((torch.full((b,), s, device="cuda") if n is None else n)[:, None].double() * log.double())[:, :, None, None]
    _, last = L.linear_attention_forward(q, k, v, log, state=state, lengths=n)
    want, size = plain_state(k, v, log, n)
    passes(last, want + stay * state.double(), SUMS * (size + stay * state.double()), "state")
    first = L.linear_attention_backward(dout, q, k, v, log, state=state, dstate=dstate, lengths=n)[4]
    # the gradient of the first state: sum over tokens of g^(i + 1) scale q_i dout_i', the same read from behind
    i = torch.arange(s, device="cuda")
    w = torch.exp((i + 1)[None, None].double() * log.double()[None, :, None]) * d ** -0.5
    if n is not None:
        w = w * (i < n[:, None].long())[:, None]
    qd, gd = (t.double().permute(0, 2, 1, 3).contiguous() for t in (q, dout))
    want = (qd * w[..., None]).transpose(2, 3).contiguous() @ gd + stay * dstate.double()
    passes(first, want, SUMS * want, "dstate")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_steps_do_not_drift(L, dtype):  # noqa: F811
    """A state that a decoder carries through thousands of single tokens, values of one sign."""
    s, h, d = 3000, 16, 8
    g = gen(5)
    q, k, v = (normal(g, 1, s, h, d).abs().to(dtype) for _ in range(3))
    log = torch.log1p(-torch.logspace(-5, -2, h, device="cuda"))
    state = torch.zeros(1, h, d, d, device="cuda")
    outs = [L.linear_attention_forward(q[:, i:i + 1], k[:, i:i + 1], v[:, i:i + 1], log, state=state, state_out=state)[0]
            for i in range(s)]
    want, size = plain_state(k, v, log)
    # two roundings a step, of no common sign: four times the root of their number
    bound = SUMS + 4 * (2 * s) ** 0.5 * 2.0 ** -24
    passes(state, want, bound * size, "state")
    out = (q[:, -1].double()[:, :, None] @ want)[:, :, 0] * d ** -0.5
    passes(outs[-1][:, 0], out, (R.UNIT[dtype] + bound) * out, "out")


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("signs", ["both", "one"])
@pytest.mark.parametrize("s,d,e", [(2, 1, 1), (3, 2, 1), (5, 1, 2), (33, 1, 1), (40, 8, 8), (70, 3, 40), (300, 64, 64), (130, 128, 96)])
def test_states_and_the_decays_gradient_keep_32_bits(L, s, d, e, signs, dtype):  # noqa: F811
    """What leaves a call in 32 bits, where few terms make it up (so errors of the terms do not average out), many heads
    of them, and values of one sign.  Operands in two parts of bfloat16 are off by up to 2^-17 of a term, eight bounds."""
    h = 64 if d < 64 else 4
    x, more, grads = inputs(1, s, h, h, d, e, dtype, True, False, seed=3)
    if signs == "one":
        x, more, grads = ({n: t.abs() if isinstance(t, torch.Tensor) and n != "log_decay" else t for n, t in part.items()}
                          for part in (x, more, grads))
    for given in (True, False):
        if not given:  # from nothing: the tokens' terms alone
            more, grads = {**more, "state": None}, {**grads, "dstate": None}
        r, size = both(x, more, grads)
        _, last = L.linear_attention_forward(**x, **more)
        _, _, _, dlog, first = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more)
        passes(last, r["last"], SUMS * size["last"], "state")
        passes(dlog, r["dlog"], SUMS * size["dlog"], "dlog_decay")
        if given:
            passes(first, r["dstate"], SUMS * size["dstate"], "dstate")


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("b,s,h,kv,lengths", [(1, 8301, 2, 1, None), (2, 4500, 1, 1, (4133, 4500)), (2, 16390, 1, 1, (5000, 11))])
def test_gradients_over_many_segments(L, b, s, h, kv, lengths, dtype):  # noqa: F811
    """More than 64 segments (of 64 and 96 tokens), lengths that end inside one in the middle, state and dstate."""
    d, e = 24, 16
    x, more, grads = inputs(b, s, h, kv, d, e, dtype, True, False, seed=4)
    x["log_decay"] = torch.log1p(-torch.tensor([2e-4, 0.03], device="cuda"))[:h]
    if lengths is not None:
        more["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    r, size = both(x, more, grads)
    out, last = L.linear_attention_forward(**x, **more)
    dq, dk, dv, dlog, first = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more)
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        passes(got, r[name], once(r[name], size[name], dtype), name)
    for name, got in (("last", last), ("dlog", dlog), ("dstate", first)):
        passes(got, r[name], SUMS * size[name], name)


@pytest.mark.parametrize("dtype", ALL)
def test_decays_gradient_counts_every_step(L, dtype):  # noqa: F811
    """Ten thousand positions with no decay at all: each pair counts as often as there are positions between."""
    s, d = 10_000, 16
    g = gen(3)
    q, k, v, dout = (normal(g, 1, s, 1, d, dtype=dtype) for _ in range(4))
    log = torch.zeros(1, device="cuda")
    r, size = both({"q": q, "k": k, "v": v, "log_decay": log}, {"state": None, "lengths": None}, {"dout": dout, "dstate": None})
    got = L.linear_attention_backward(dout, q, k, v, log)[3]
    passes(got, r["dlog"], SUMS * size["dlog"], "dlog_decay")


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("s", [20, 32])
def test_powers_of_strong_decays(L, s, dtype):  # noqa: F811
    """One token far back is all there is: its power of g has 32 bits however small it is."""
    h, d = 64, 8
    x, more, grads = inputs(1, s, h, h, d, d, dtype, False, False, seed=6)
    x["log_decay"] = -torch.linspace(0.1, 2.6, h, device="cuda")
    x["k"][:, 1:], grads["dout"][:, :-1] = 0, 0
    r, size = both(x, more, grads)
    _, last = L.linear_attention_forward(**x, **more)
    _, _, _, dlog, _ = L.linear_attention_backward(grads["dout"], *x.values(), **more)
    bound = SUMS * size["last"] + 2.0 ** -126
    if dtype == F16:
        # What a state takes in is lifted by a power of two for each column of a run, so that the largest v g^(n-1-j) of
        # the column's tokens is at least 2^13; its two parts end at float16's last step, 2^-24, so each value
        # is off by 2^-25 of at least 2^13 of the largest: 2^-38 of it, times k.
        steps = torch.arange(s - 1, -1, -1, device="cuda")[:, None, None]
        largest = (x["v"][0].double().abs() * torch.exp(steps * x["log_decay"].double()[:, None])).amax(0)  # [heads, columns]
        bound = bound + 2.0 ** -38 * x["k"][0, 0].double().abs()[:, :, None] * largest[:, None, :]
    passes(last, r["last"], bound, "state")
    passes(dlog, r["dlog"], SUMS * size["dlog"] + 2.0 ** -126, "dlog_decay")


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("s", [1, 2, 40, 700])
def test_an_infinity_of_the_state_stays_one(L, s, dtype):  # noqa: F811
    """Nothing of it is NaN (a number less itself), and other columns keep their bits."""
    x, more, grads = inputs(1, s, 2, 2, 32, 32, dtype, True, False, seed=7)
    x["log_decay"] = torch.tensor([-0.01, -0.02], device="cuda")
    for n in "qk":
        x[n][..., 1] = x[n][..., 1].abs() + 0.125
    clean = L.linear_attention_forward(**x, **more)
    back = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more)
    for t in (more["state"], grads["dstate"]):
        t[0, 0, 1, 3] = float("inf")
    out, last = L.linear_attention_forward(**x, **more)
    _, _, dv, _, first = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more)
    for got, want in ((out, clean[0]), (dv, back[2])):
        assert bool((got[0, :, 0, 3] == float("inf")).all())
        rest = torch.arange(32, device="cuda") != 3
        assert torch.equal(got[..., rest], want[..., rest]) and torch.equal(got[:, :, 1], want[:, :, 1])
    for got, want in ((last, clean[1]), (first, back[4])):
        assert float(got[0, 0, 1, 3]) == float("inf")
        got[0, 0, 1, 3] = want[0, 0, 1, 3]
        assert torch.equal(got, want)
