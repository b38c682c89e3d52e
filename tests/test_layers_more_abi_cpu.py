"""RMS norm, linear attention and clipping without a GPU: what the library refuses on the host, the
scratch memory it asks for, and (with a stand-in of the runtime, `host_runtime.cpp`) its launches."""
from __future__ import annotations

import array
import ctypes
import re
import struct

import pytest
import torch

from test_layers_abi_cpu import HEADER, layers  # noqa: F401 - a fixture
from test_layers_launches_cpu import stand_in  # noqa: F401 - a fixture

RMS_POINTERS = ("x", "residual", "weight", "y", "sum", "rstd", "scales", "dy", "dsum", "dx", "dweight")
RMS_STRIDES = ("xs", "rs", "ys", "hs", "gs", "ss", "ds")
RMS_SIZES = ("n", "s", "c", "dtype", "pdtype", "format", "eps")
RMS = {**{p: 256 for p in RMS_POINTERS}, **{s: (64, 8) for s in RMS_STRIDES}, "n": 2, "s": 8, "c": 8, "dtype": 2, "pdtype": 0,
       "format": 0, "eps": 1e-6}


def rms_args(layers, **kw):  # noqa: F811
    a = {**RMS, **kw}
    return layers._RMS_NORM.pack(*(a[p] for p in RMS_POINTERS), *(v for s in RMS_STRIDES for v in a[s]),
                                 *(a[s] for s in RMS_SIZES))


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), -1), (dict(y=0), -1), (dict(residual=0), -1), (dict(sum=0), -1), (dict(n=-1), -1), (dict(s=-1), -1),
    (dict(c=0), -1), (dict(c=65537), -1), (dict(dtype=3), -1), (dict(pdtype=-1), -1), (dict(format=3), -1),
    (dict(format=-1), -1), (dict(format=1, scales=0), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(xs=(-1, 8)), -1), (dict(rs=(64, -8)), -1), (dict(ys=(64, -8)), -1),
    (dict(hs=(-64, 8)), -1), (dict(n=1 << 31, s=1 << 31), -1), (dict(n=0, x=0), 0), (dict(s=0, x=0), 0),
])
def test_rms_norm_forward_host_checks(layers, kw, code):  # noqa: F811
    assert layers.load().lic_rms_norm_forward(rms_args(layers, **kw), 0) == code
    assert layers.load().lic_rms_norm_forward(None, 0) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), -1), (dict(rstd=0), -1), (dict(dy=0), -1), (dict(dx=0), -1), (dict(format=1), -1), (dict(gs=(-1, 8)), -1),
    (dict(ds=(64, -1)), -1), (dict(ss=(64, -1)), -1), (dict(c=0), -1), (dict(n=0, x=0), 0), (dict(s=0, dy=0), 0),
])
def test_rms_norm_backward_host_checks(layers, kw, code):  # noqa: F811
    assert layers.load().lic_rms_norm_backward(rms_args(layers, **kw), 256, 1 << 30, 0) == code


def test_rms_norm_workspace(layers):  # noqa: F811
    lib = layers.load()
    for bad in ((0, 8, 8), (2, 0, 8), (2, 8, 0), (2, 8, 65537)):
        assert lib.lic_rms_norm_workspace_bytes(*bad) == 0
    need = lib.lic_rms_norm_workspace_bytes(2, 8, 8)
    assert need >= 64 * 8 * 4
    args = rms_args(layers)
    for at, size in ((None, need), (257, need), (256, need - 1)):
        assert lib.lic_rms_norm_backward(args, at, size, 0) == -7


LINEAR_POINTERS = ("q", "k", "v", "log_decay", "state", "lengths", "out", "state_out", "dout", "dstate", "dq", "dk", "dv", "dlog",
                   "dstate_in")
LINEAR_SIZES = ("b", "s", "h", "kv", "d", "e", "dtype", "scale")
LINEAR = {**{p: 256 for p in LINEAR_POINTERS}, "strides": (4096, 64, 16) * 8, "states": (4096, 1024, 16) * 4, "b": 2, "s": 64,
          "h": 4, "kv": 2, "d": 16, "e": 16, "dtype": 2, "scale": 0.25}


def linear_args(layers, **kw):  # noqa: F811
    a = {**LINEAR, **kw}
    return layers._LINEAR.pack(*(a[p] for p in LINEAR_POINTERS), *a["strides"], *a["states"], *(a[s] for s in LINEAR_SIZES))


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(log_decay=0), -1), (dict(b=-1), -1), (dict(s=-1), -1),
    (dict(s=(1 << 28) + 1), -1), (dict(h=3), -1), (dict(kv=0), -1), (dict(h=0), -1), (dict(d=0), -1), (dict(d=129), -1),
    (dict(e=0), -1), (dict(e=129), -1), (dict(dtype=3), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(strides=(-1, 64, 16) * 8), -1), (dict(states=(4096, -1, 16) * 4), -1),
    (dict(b=1 << 20, h=512, kv=512), -1), (dict(b=1 << 20, s=1 << 28), -1),
])
def test_linear_attention_host_checks(layers, kw, code):  # noqa: F811
    lib = layers.load()
    args = linear_args(layers, **kw)
    assert lib.lic_linear_attention_forward(args, 256, 1 << 60, 0) == code
    assert lib.lic_linear_attention_backward(args, 256, 1 << 60, 0) == code


def test_linear_attention_more_host_checks(layers):  # noqa: F811
    lib = layers.load()
    assert lib.lic_linear_attention_forward(None, 256, 1 << 30, 0) == -1
    assert lib.lic_linear_attention_forward(linear_args(layers, b=0, q=0), None, 0, 0) == 0
    assert lib.lic_linear_attention_backward(linear_args(layers, b=0, q=0, dlog=0), None, 0, 0) == 0
    assert lib.lic_linear_attention_forward(linear_args(layers, out=0), 256, 1 << 30, 0) == -1
    for kw in (dict(dout=0), dict(dq=0), dict(dk=0), dict(dv=0)):
        assert lib.lic_linear_attention_backward(linear_args(layers, **kw), 256, 1 << 30, 0) == -1


def test_linear_attention_workspace(layers):  # noqa: F811
    lib = layers.load()
    size = lib.lic_linear_attention_workspace_bytes
    assert size(linear_args(layers, h=3), 1) == 0 and size(linear_args(layers, d=200), 0) == 0
    assert size(linear_args(layers, s=1), 0) == 0 and size(linear_args(layers, b=512, h=4), 0) == 0
    for backward, call in ((0, lib.lic_linear_attention_forward), (1, lib.lic_linear_attention_backward)):
        args = linear_args(layers, s=8000, strides=(1 << 20, 64, 16) * 8)
        need = size(args, backward)
        assert need > 0
        for at, n in ((None, need), (257, need), (256, need - 1)):
            assert call(args, at, n, 0) == -7
    # parts of heads that share keys, of each gradient
    assert size(linear_args(layers), 1) >= 2 * 4 * 64 * (16 + 16) * 4


def test_the_header_names_what_sizes_the_linear_workspace(layers):  # noqa: F811
    said = re.search(r"/\* Bytes for lic_linear_attention_forward.*?\*/", open(HEADER).read(), flags=re.S).group(0)
    names = dict(zip(LINEAR_SIZES, ("batch", "tokens", "heads", "kv_heads", "dim", "value_dim", "dtype", "scale")))
    base = {**LINEAR, "s": 3000}
    other = dict(b=3, s=700, h=8, kv=1, d=96, e=128, dtype=0, scale=0.5)
    for backward in (0, 1):
        for field, name in names.items():
            a = layers.load().lic_linear_attention_workspace_bytes(linear_args(layers, **base), backward)
            b = layers.load().lic_linear_attention_workspace_bytes(linear_args(layers, **{**base, field: other[field]}), backward)
            assert a == b or re.search(r"\b%s\b" % name, said), name


def gradients(*entries):
    return array.array("q", [v for e in entries for v in e]).tobytes()


A, B = (4096, 4096, 100, 0), (8192, 8192, 50, 2)


@pytest.mark.parametrize("entries,norm,max_norm,code", [
    ((A, B), 0, 1.0, -1), ((A, B), 256, -1.0, -1), ((A, B), 256, float("nan"), -1), ((A, B), 256, float("inf"), -1),
    (((0, 4096, 100, 0),), 256, 1.0, -1), (((4096, 0, 100, 0),), 256, 1.0, -1), (((4096, 4096, -1, 0),), 256, 1.0, -1),
    (((4096, 4096, 100, 3),), 256, 1.0, -1), ((A, A), 256, 1.0, -1), ((A, (4096 + 396, 4096 + 396, 10, 0)), 256, 1.0, -1),
    ((A, (8192, 4096, 10, 0)), 256, 1.0, -1), (((4096, 4100, 100, 0),), 256, 1.0, -1),
    (((4096, 8192, 100, 0), (8192, 4096, 100, 0)), 256, 1.0, -1),
    # what does not overlap, ends where another begins, or has no values
    ((A, (4096 + 400, 4096 + 400, 10, 0)), 256, 1.0, -7), ((A, (4096, 4096, 0, 0)), 256, 1.0, -7),
    (((4096, 8192, 100, 0), (4096, 12288, 100, 0)), 256, 1.0, -7),
])
def test_clip_host_checks(layers, entries, norm, max_norm, code):  # noqa: F811
    lib = layers.load()
    assert lib.lic_clip_gradients(gradients(*entries), len(entries), max_norm, norm or None, None, 0, 0) == code


def test_clip_workspace(layers):  # noqa: F811
    lib = layers.load()
    size = lib.lic_clip_gradients_workspace_bytes
    assert size(gradients(A), -1) == 0 and size(None, 1) == 0 and size(gradients((0, 0, 5, 0)), 1) == 0 and size(b"", 0) == 0
    assert size(gradients(A, B), 2) == 2 * 8 and size(gradients((4096, 4096, 1 << 30, 0)), 1) == 1024 * 8
    assert lib.lic_gradient_norm(None, 1, 256, 256, 1 << 20, 0) == -1
    assert lib.lic_gradient_norm(gradients(A), 1, 256, 256, 7, 0) == -7
    assert lib.lic_gradient_norm(gradients(A), 1, 256, 300, 1 << 20, 0) == -7


def test_host_tensors_are_refused(layers):  # noqa: F811
    x, q = torch.zeros(4, 8), torch.zeros(1, 4, 2, 8)
    for call in (lambda: layers.rms_norm(x), lambda: layers.rms_norm_8bit(x), lambda: layers.linear_attention(q, q, q, torch.zeros(2)),
                 lambda: layers.clip_gradients([x], 1.0), lambda: layers.gradient_norm(x)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()


def test_more_argument_blocks_match_the_header(layers):  # noqa: F811
    """The packed blocks are as long as the C structs (all members of 8 bytes)."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name, size in (("lic_rms_norm_args", layers._RMS_NORM.size), ("lic_linear_attention_args", layers._LINEAR.size),
                       ("lic_gradient", struct.calcsize("=2Q2q"))):
        body = re.search(r"typedef struct %s \{(.*?)\}" % name, text, flags=re.S).group(1)
        total = 0
        for field in re.split(r"[;,]", body):
            if field.strip():
                many = re.search(r"\[(\d+)\]", field)
                total += int(many.group(1)) if many else 1
        assert size == 8 * total, name
    assert ctypes.sizeof(ctypes.c_void_p) == 8


# ---- launches --------------------------------------------------------------------------


def rms(layers, backward=0, device=0, **kw):  # noqa: F811
    args = rms_args(layers, **kw).hex()
    if backward:
        return [device, 0, "lic_rms_norm_backward", "bpQp", [args, 256, 1 << 46, 0]]
    return [device, 0, "lic_rms_norm_forward", "bp", [args, 0]]


def linear(layers, backward=0, device=0, refuses=0, **kw):  # noqa: F811
    name = "lic_linear_attention_backward" if backward else "lic_linear_attention_forward"
    return [device, refuses, name, "bpQp", [linear_args(layers, **kw).hex(), 256, 1 << 60, 0]]


def clip(*entries):
    return [0, 0, "lic_clip_gradients", "bqdppQp", [gradients(*entries).hex(), len(entries), 1.0, 256, 256, 1 << 30, 0]]


def every_linear_kernel(layers, device):  # noqa: F811
    return [linear(layers, backward, device, dtype=dtype, d=d, e=e, s=s, state_out=256 if last else 0, state=256 if last else 0,
                   dstate_in=256 if last else 0, strides=strides)
            for backward in (0, 1) for dtype in (0, 1, 2) for d, e in ((32, 8), (64, 64), (16, 96), (128, 128))
            for s in (1, 40, 3000) for last in (0, 1) for strides in ((1 << 20, 512, 128) * 8, (1 << 20, 513, 129) * 8)]


def test_each_device_is_told_of_large_linear_kernels(layers, stand_in):  # noqa: F811
    there = [every_linear_kernel(layers, device) for device in (0, 1, 0)]
    n = len(there[0])
    rows = stand_in(*(job for jobs in there for job in jobs))
    assert all(r["rc"] == 0 and r["launches"] >= 1 for r in rows)
    assert sum(r["too_much_lds"] + r["too_many_threads"] for r in rows) == 0
    told = [sum(r["attributes"] for r in rows[i:i + n]) for i in range(0, 3 * n, n)]
    assert told[0] == told[1] > 0 and told[2] == 0


def test_a_device_without_the_lds_is_an_error_of_linear_attention(layers, stand_in):  # noqa: F811
    jobs = [linear(layers, backward, 0, refuses, dtype=0, d=128, e=128, s=40) for refuses in (1, 0) for backward in (0, 1)]
    rows = stand_in(*jobs)
    assert [r["rc"] for r in rows] == [-8, -8, 0, 0] and rows[0]["launches"] == 0


def test_no_launch_of_these_has_more_threads_than_it_can(layers, stand_in):  # noqa: F811
    wide = (1 << 50, 1 << 20, 1 << 10) * 8
    jobs = [linear(layers, 0, b=1 << 20, h=256, kv=256, s=1, d=8, e=8, strides=wide),
            linear(layers, 0, b=1 << 20, h=255, kv=255, s=20, d=128, e=128, strides=wide),
            linear(layers, 1, b=1 << 20, h=255, kv=51, s=20, d=128, e=128, strides=wide),
            rms(layers, 0, n=1 << 20, s=1 << 20, c=8, xs=(1 << 23, 8)), rms(layers, 1, n=1 << 20, s=1 << 20, c=65536),
            clip((1 << 40, 1 << 40, 1 << 37, 2)), clip(*[((i + 1) << 20, (i + 1) << 20, 1 << 18, 0) for i in range(1000)])]
    rows = stand_in(*jobs)
    assert all(r["rc"] == 0 and r["launches"] >= 1 and r["too_many_threads"] == 0 for r in rows)
    assert rows[0]["blocks"] >= 1 << 28 and rows[1]["blocks"] >= 255 << 20 and rows[2]["blocks"] >= 4 * 255 << 20
    # a list of a thousand tensors: nine lists of 120 and their sums
    assert rows[-1]["launches"] == 18


def test_an_empty_batch_still_has_a_sum(layers, stand_in):  # noqa: F811
    row, = stand_in(linear(layers, 1, b=0))
    assert row["rc"] == 0 and row["launches"] == 1
