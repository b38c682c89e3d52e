"""RMS norm with the residual's addition and its 8-bit output on the GPU against plain 64-bit forms."""
from __future__ import annotations

import math

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
    w = R.worst(got, want, bound)
    print(f"{what}: {w:.3f} of the bound", flush=True)
    assert w <= 1.0, (what, w)


def check(L, x, residual, weight, eps, dy, dsum):
    dtype = x.dtype
    u = R.UNIT[dtype]
    r = M.rms_norm(x, weight, residual, eps, dy, dsum)
    y, h, rstd = L.rms_norm_forward(x, weight, residual=residual, eps=eps)
    assert torch.equal(h, r["h"]) and (residual is not None or h is x)
    assert y.dtype == dtype and rstd.dtype == F32 and rstd.shape == x.shape[:-1]
    passes(rstd, r["rstd"], R.F32 * r["rstd"], "rstd")
    passes(y, r["y"], u * r["y"].abs() + R.F32 * r["y"].abs() + R.STEP[dtype], "y")
    dx, dw = L.rms_norm_backward(dy, h, weight, rstd, dsum=dsum)
    kind = F32 if weight is None else weight.dtype
    assert dx.dtype == dtype and dw.dtype == kind
    passes(dx, r["dx"], u * r["dx"].abs() + R.F32 * r["dx_abs"] + R.STEP[dtype], "dx")
    passes(dw, r["dw"], R.UNIT[kind] * r["dw"].abs() + R.F32 * r["dw_abs"] + R.STEP[kind], "dw")


SHAPES = [
    (1, 1), (1, 2), (3, 3), (5, 7), (1, 8), (16, 33), (7, 64), (2, 100, 119), (4, 5, 6, 192), (65, 192), (16, 1, 1024),
    (300, 257), (33, 1000), (9, 2048), (5, 2049), (6, 4096), (3, 4099), (2, 8192), (3, 8200), (2, 20001), (1, 65536),
    (5000, 40), (257, 320),
]


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("shape", SHAPES)
def test_rms_norm(L, shape, dtype):
    g = gen(sum(shape))
    x, residual, dy, dsum = (normal(g, *shape, dtype=dtype) for _ in range(4))
    weight = (1 + 0.3 * normal(g, shape[-1])).to((F32, dtype)[sum(shape) % 2])
    check(L, x, residual, weight, 1e-6, dy, dsum)
    check(L, x, None, None, 1e-5, dy, None)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("c", [96, 119, 8196])
def test_rms_norm_strides(L, c, dtype):
    """Rows cut out of wider ones, samples apart, odd addresses: the same bits; neighbours stay as they are."""
    g = gen(c)
    n, s = 3, 5
    base = [normal(g, n, s, c, dtype=dtype) for _ in range(4)]
    weight = 1 + 0.3 * normal(g, c)
    want = L.rms_norm_forward(base[0], weight, residual=base[1])
    grads = L.rms_norm_backward(base[2], want[1], weight, want[2], dsum=base[3])

    def laid(t, how):
        if how == "rows":
            w = torch.full((n, s, c + 7), 9.0, dtype=dtype, device="cuda")[..., 3:3 + c]
        elif how == "samples":
            w = torch.full((n, s + 2, c), 9.0, dtype=dtype, device="cuda")[:, 1:-1]
        else:
            w = torch.full((n * s * c + 1,), 9.0, dtype=dtype, device="cuda")[1:].view(n, s, c)
        return w.copy_(t)

    for how in ("rows", "samples", "odd"):
        x, r, dy, ds = (laid(t, how) for t in base)
        out, total, dx = (laid(t, how) for t in base[:3])
        y, h, rstd = L.rms_norm_forward(x, weight, residual=r, out=out, sum_out=total)
        assert y is out and h is total
        assert all(torch.equal(a, b) for a, b in zip((y, h, rstd), want)), how
        got = L.rms_norm_backward(dy, h, weight, rstd, dsum=ds, out=dx)
        assert got[0] is dx and all(torch.equal(a, b) for a, b in zip(got, grads)), how
        if how == "rows":
            for t in (out, total, dx):
                around = t._base
                assert bool((around[..., :3] == 9).all()) and bool((around[..., 3 + c:] == 9).all())
        elif how == "samples":
            assert bool((out._base[:, 0] == 9).all()) and bool((out._base[:, -1] == 9).all())
        # in place: the sum where the residual was, the norm where x was, dx where dsum was
        y, h, _ = L.rms_norm_forward(x, weight, residual=r, out=x, sum_out=r)
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])
        assert torch.equal(L.rms_norm_backward(dy, h, weight, rstd, dsum=ds, out=ds)[0], grads[0])
    with pytest.raises(ValueError, match="evenly spaced"):
        L.rms_norm_forward(normal(g, n, s, 4, c, dtype=dtype)[:, :, 1:3])
    with pytest.raises(ValueError, match="next to each other"):
        L.rms_norm_forward(base[0].transpose(1, 2))


@pytest.mark.parametrize("format", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("shape", [(1, 1), (3, 5), (16, 1, 1024), (100, 192), (7, 333), (2, 9, 4100), (2, 9001), (1, 65536)])
def test_rms_norm_8bit(L, shape, dtype, format):
    g = gen(sum(shape) + 1)
    x, residual = normal(g, *shape, dtype=dtype), normal(g, *shape, dtype=dtype)
    weight = 1 + 0.3 * normal(g, shape[-1])
    x.view(-1, shape[-1])[0] = 0
    residual.view(-1, shape[-1])[0] = 0  # a row of zeros
    most = 448.0 if format == "e4m3" else 127.0
    y, scales, h = L.rms_norm_8bit(x, weight, residual=residual, format=format)
    r = M.rms_norm(x, weight, residual, 1e-6)
    assert torch.equal(h, r["h"]) and y.dtype == (torch.float8_e4m3fn if format == "e4m3" else torch.int8)
    top = r["y"].abs().amax(-1).clamp(min=1e-30)
    passes(scales, top / most, R.F32 * top / most, "scales")
    assert bool((y.float().abs() <= most).all())
    assert bool((y.float().view(-1, shape[-1])[0] == 0).all())
    # half a step of what the value is between: e4m3 steps are 2^-3 of a power of two, 2^-9 below 2^-6
    exact = r["y"] * (most / top)[..., None]
    step = torch.ones_like(exact) if format == "int8" else \
        torch.exp2(torch.floor(torch.log2((exact.abs() * (1 + R.F32)).clamp(min=2.0 ** -6))) - 3)
    passes(y.double(), exact, step / 2 + 2 * R.F32 * exact.abs(), "y")


def test_rms_norm_8bit_of_what_is_not_finite(L):
    for format in ("e4m3", "int8"):
        for c in (40, 9000):
            x = normal(gen(2), 6, c)
            x[1, 3], x[2, 0], x[4, c - 1] = math.nan, math.inf, -math.inf
            y, scales, _ = L.rms_norm_8bit(x, format=format)
            value = y.float() * scales[:, None]
            assert bool(torch.isfinite(value[[0, 3, 5]]).all()) and bool(torch.isnan(value[[1, 2, 4]]).all())


def test_rms_norm_of_what_is_not_finite(L):
    for dtype in ALL:
        x, dy = normal(gen(3), 6, 70, dtype=dtype), normal(gen(4), 6, 70, dtype=dtype)
        x[1, 3], x[4, 69] = math.nan, math.inf
        y, h, rstd = L.rms_norm_forward(x)
        rows = torch.tensor([0, 2, 3, 5], device="cuda")
        want = L.rms_norm_forward(x[rows])
        assert torch.equal(y[rows], want[0]) and bool(torch.isnan(y[1]).all())
        # an infinity: rstd is 0, the others 0, itself NaN
        assert float(rstd[4]) == 0 and bool((y[4, :69] == 0).all()) and math.isnan(float(y[4, 69]))
        dx, _ = L.rms_norm_backward(dy, h, None, rstd)
        assert torch.equal(dx[rows], L.rms_norm_backward(dy[rows], x[rows], None, rstd[rows])[0])


def test_rms_norm_large_and_small_values(L):
    """Squares beyond float16's range are sums of 32 bits; rows below eps."""
    g = gen(6)
    for dtype, size in ((F16, 6e4), (F16, 1e-7), (BF16, 1e15), (BF16, 1e-30), (F32, 1e15), (F32, 1e-25)):
        x = (normal(g, 9, 200).clamp(-1, 1) * size).to(dtype)
        r = M.rms_norm(x, None, None, 1e-6)
        y, _, _ = L.rms_norm_forward(x, eps=1e-6)
        passes(y, r["y"], (R.UNIT[dtype] + R.F32) * r["y"].abs() + R.STEP[dtype], f"{dtype} {size}")


def test_rms_norm_autograd_and_differences(L):
    g = gen(5)
    n, s, c = 2, 5, 24
    x, r = normal(g, n, s, c).requires_grad_(), normal(g, n, s, c).requires_grad_()
    w = (1 + 0.2 * normal(g, c)).requires_grad_()
    dy, dh = normal(g, n, s, c), normal(g, c, s, n).permute(2, 1, 0)  # one of another layout
    got = torch.autograd.grad(L.rms_norm(x, w, r), (x, w, r), (dy, dh))
    want = M.rms_norm(x.detach(), w.detach(), r.detach(), 1e-6, dy, dh)
    assert torch.equal(got[0], got[2])
    passes(got[0], want["dx"], R.F32 * (want["dx_abs"] + want["dx"].abs()), "dx")
    passes(got[1], want["dw"], R.F32 * (want["dw_abs"] + want["dw"].abs()), "dw")
    step = 2.0 ** -6  # central differences: off by step^2 and by 2^-24 / step
    for i, t in enumerate((x, w, r)):
        d = normal(g, *t.shape)
        ends = []
        for sign in (step, -step):
            args = [p.detach() for p in (x, w, r)]
            args[i] = args[i] + sign * d
            y, h = L.rms_norm(*args)
            ends.append((y.double() * dy).sum() + (h.double() * dh).sum())
        have = float((got[i].double() * d).sum())
        size = float((got[i].double() * d).abs().sum())
        assert abs(float(ends[0] - ends[1]) / (2 * step) - have) <= 8 * step * step * size
    # one of the two results only
    y, h = L.rms_norm(x, w, r)
    a = torch.autograd.grad(y, (x, w), dy)
    assert torch.equal(a[1], got[1])
    y, h = L.rms_norm(x, w, r)
    assert torch.equal(torch.autograd.grad(h, r, dh)[0], dh)
    assert isinstance(L.rms_norm(x, w), torch.Tensor)
    assert torch.autograd.grad(L.rms_norm(x), x, dy)[0].shape == x.shape


def test_rms_norm_refusals(L):
    x = torch.zeros(2, 3, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    for call, error, match in (
            (lambda: L.rms_norm(x.cpu()), ValueError, "on the GPU"),
            (lambda: L.rms_norm(x.int()), TypeError, "float32"),
            (lambda: L.rms_norm(x, w[:4]), ValueError, "one value a channel"),
            (lambda: L.rms_norm(x, w.double()), TypeError, "weight"),
            (lambda: L.rms_norm(x, w, x.half()), TypeError, "residual"),
            (lambda: L.rms_norm(x, w, x[:1]), ValueError, "residual"),
            (lambda: L.rms_norm(x, w, eps=-1.0), ValueError, "eps"),
            (lambda: L.rms_norm(x, w, eps=math.nan), ValueError, "eps"),
            (lambda: L.rms_norm(torch.zeros((), device="cuda")), ValueError, "C"),
            (lambda: L.rms_norm_8bit(x, w, format="int4"), ValueError, "format"),
            (lambda: L.rms_norm_8bit(x.clone().requires_grad_(), w), NotImplementedError, "gradients"),
            (lambda: L.rms_norm_8bit(x, w, out=x), TypeError, "out"),
            (lambda: L.rms_norm_forward(x, w, sum_out=x), ValueError, "sum_out"),
            (lambda: L.rms_norm_forward(x, w, out=torch.zeros(2, 1, 8, device="cuda").expand(2, 3, 8)), ValueError, "overlap"),
            (lambda: L.rms_norm_backward(x[:1], x, w, torch.ones(2, 3, device="cuda")), ValueError, "dy"),
            (lambda: L.rms_norm_backward(x, x, w, torch.ones(3, device="cuda")), ValueError, "rstd"),
    ):
        with pytest.raises(error, match=match):
            call()
    leaf = x.clone().requires_grad_()
    y = L.rms_norm(leaf, w)
    first, = torch.autograd.grad(y.sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(first.sum(), leaf)


def test_rms_norm_places(L):
    """An output may be an input of the same layout; another layout at its address, and one place for both
    outputs, are refused before anything is written."""
    g = gen(12)
    x, r = normal(g, 6, 6, 16, dtype=BF16), normal(g, 6, 6, 16, dtype=BF16)
    was = x.clone()
    turned = x.transpose(0, 1)
    for call in (
            lambda: L.rms_norm_forward(x, residual=r, out=turned),
            lambda: L.rms_norm_forward(x, residual=r, sum_out=turned),
            lambda: L.rms_norm_forward(r, residual=turned, out=x),
            lambda: L.rms_norm_8bit(x, out=x.view(torch.float8_e4m3fn)[..., :16]),
            lambda: L.rms_norm_backward(x, r, None, torch.ones(6, 6, device="cuda"), out=turned),
            lambda: L.rms_norm_backward(r, r, None, torch.ones(6, 6, device="cuda"), dsum=x, out=turned),
    ):
        with pytest.raises(ValueError, match="laid out differently"):
            call()
    with pytest.raises(ValueError, match="one place"):
        L.rms_norm_forward(r, residual=r, out=x, sum_out=x)
    assert torch.equal(x, was)
    want = L.rms_norm_forward(x, residual=r)
    y, h, _ = L.rms_norm_forward(x, residual=r, out=x, sum_out=r)
    assert y is x and h is r and torch.equal(x, want[0]) and torch.equal(r, want[1])


def test_rms_norm_empty(L):
    for shape in ((0, 8), (2, 0, 8), (0, 3, 8)):
        x = torch.zeros(shape, device="cuda")
        y, h, rstd = L.rms_norm_forward(x, residual=x)
        dx, dw = L.rms_norm_backward(x, h, None, rstd)
        assert y.shape == dx.shape == x.shape and rstd.shape == x.shape[:-1] and bool((dw == 0).all())
        assert L.rms_norm_8bit(x)[0].shape == x.shape


def test_rms_norm_captured(L):
    g = gen(9)
    x, r, dy = (normal(g, 40, 192, dtype=BF16) for _ in range(3))
    w = 1 + 0.1 * normal(g, 192)

    def step():
        y, h, rstd = L.rms_norm_forward(x, w, residual=r)
        return (y, h, *L.rms_norm_backward(dy, h, w, rstd), *L.rms_norm_8bit(x, w)[:2])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for turn in range(3):
        x.copy_(normal(g, 40, 192, dtype=BF16))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want)), turn
