"""The network operators' C ABI without a GPU: the library exports what its header declares,
sizes its workspaces and rejects bad arguments on the host before any launch."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lic_layers.h")


@pytest.fixture(scope="module")
def layers():
    from learned_image_compression_amd import build as hip_build
    from learned_image_compression_amd import layers as L
    if not os.path.exists(L.LIBRARY):
        hip_build.build()
    L.load()
    return L


def test_every_declared_function_is_exported(layers):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lic_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(layers.EXPORTS)
    for name in names:
        assert hasattr(layers.load(), name), name
    assert layers.load().lic_layers_target() == b"gfx950"


def test_refuses_to_run_without_library(layers, tmp_path):
    with pytest.raises(RuntimeError, match="no CPU fallback"):
        layers.load(str(tmp_path / "missing.so"))


def test_host_tensors_are_refused(layers):
    x = torch.zeros(1, 8, 4, 4).to(memory_format=torch.channels_last)
    with pytest.raises(ValueError, match="on the GPU"):
        layers.group_norm(x, 2)
    q = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError, match="on the GPU"):
        layers.attention(q, q, q)
    with pytest.raises(ValueError, match="on the GPU"):
        layers.rotary(q, q, torch.zeros(4, 4), torch.zeros(4, 4))
    with pytest.raises(ValueError, match="current device"):
        layers.rotary_table(torch.zeros(4, dtype=torch.float64), 8)


NORM = dict(x=256, xs=64, xr=8, n=2, s=8, c=8, g=2, dtype=0, w=0, b=0, pdtype=0, eps=1e-5, act=0, y=512, ys=64,
            yr=8, mean=1024, rstd=2048, ws=4096, bytes=1 << 30)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), -1), (dict(y=0), -1), (dict(mean=0), -1), (dict(rstd=0), -1), (dict(n=-1), -1), (dict(n=65536), -1),
    (dict(s=-1), -1), (dict(c=0), -1), (dict(c=65537), -1), (dict(g=0), -1), (dict(g=3), -1), (dict(dtype=3), -1),
    (dict(pdtype=-1), -1), (dict(act=4), -1), (dict(act=-1), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(xr=-8), -1), (dict(ys=-1), -1), (dict(ws=0), -7), (dict(ws=4100), -7), (dict(bytes=16), -7),
    (dict(n=0, x=0, y=0), 0), (dict(s=0, x=0, y=0), 0),
])
def test_group_norm_forward_host_checks(layers, kw, code):
    a = {**NORM, **kw}
    assert layers.load().lic_group_norm_forward(
        a["x"], a["xs"], a["xr"], a["n"], a["s"], a["c"], a["g"], a["dtype"], a["w"], a["b"], a["pdtype"], a["eps"],
        a["act"], a["y"], a["ys"], a["yr"], a["mean"], a["rstd"], a["ws"], a["bytes"], 0) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=0), -1), (dict(x=0), -1), (dict(dx=0), -1), (dict(mean=0), -1), (dict(rstd=0), -1), (dict(n=0), -1),
    (dict(s=0), -1), (dict(c=9), -1), (dict(dtype=9), -1), (dict(act=7), -1), (dict(dxs=-1), -1), (dict(ws=0), -7),
    (dict(bytes=16), -7),
])
def test_group_norm_backward_host_checks(layers, kw, code):
    a = {**NORM, "dy": 256, "dx": 512, "dxs": 64, **kw}
    assert layers.load().lic_group_norm_backward(
        a["dy"], 64, 8, a["x"], a["xs"], a["xr"], a["n"], a["s"], a["c"], a["g"], a["dtype"], a["w"], a["b"],
        a["pdtype"], a["act"], a["mean"], a["rstd"], a["dx"], a["dxs"], 8, 0, 0, a["ws"], a["bytes"], 0) == code


def test_group_norm_workspace(layers):
    size = layers.load().lic_group_norm_workspace_bytes
    assert size(0, 10, 8, 2) == 0 and size(1, 10, 8, 3) == 0
    # every chunk's sums of every channel: up to 1024 / n + 1 chunks
    for n, c in ((1, 192), (16, 192), (5000, 64)):
        assert size(n, 1 << 20, c, 1) >= 8 * n * c * (1024 // n + 1 + 2)


ROTARY = dict(q=256, k=512, qo=256, ko=512, cos=1024, sin=2048, pos=0, status=0, step=0, strides=(64, 16, 8) * 4, b=1,
              s=4, h=2, kh=2, d=8, r=8, rows=4, dtype=0, inter=0, inv=0)


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(k=0), dict(qo=0), dict(ko=0), dict(cos=0), dict(sin=0), dict(b=-1), dict(s=-1), dict(h=0),
    dict(kh=-1), dict(d=1), dict(r=0), dict(r=7), dict(r=10), dict(rows=3), dict(dtype=3), dict(step=-1),
    dict(strides=(64, -16, 8) * 4),
])
def test_rotary_host_checks(layers, kw):
    a = {**ROTARY, **kw}
    args = layers._ROTARY.pack(*(a[k] for k in ("q", "k", "qo", "ko", "cos", "sin", "pos", "status", "step")),
                               *a["strides"], *(a[k] for k in ("b", "s", "h", "kh", "d", "r", "rows", "dtype",
                                                               "inter", "inv")))
    assert layers.load().lic_rotary(args, 0) == -1


def test_rotary_empty_calls(layers):
    for kw in (dict(b=0), dict(s=0)):
        a = {**ROTARY, **kw, "q": 0, "cos": 0}
        args = layers._ROTARY.pack(*(a[k] for k in ("q", "k", "qo", "ko", "cos", "sin", "pos", "status", "step")),
                                   *a["strides"], *(a[k] for k in ("b", "s", "h", "kh", "d", "r", "rows", "dtype",
                                                                   "inter", "inv")))
        assert layers.load().lic_rotary(args, 0) == 0
    assert layers.load().lic_rotary(None, 0) == -1


@pytest.mark.parametrize("kw", [
    dict(coords=0), dict(cos=0), dict(sin=0), dict(rows=-1), dict(axes=0), dict(axes=3), dict(r=7), dict(r=0),
    dict(base=0.0), dict(base=float("inf")), dict(factor=0.0), dict(factor=float("nan")), dict(original=-1.0),
    dict(amplitude=float("inf")),
])
def test_rotary_table_host_checks(layers, kw):
    a = {**dict(coords=256, rows=4, axes=1, r=8, base=1e4, factor=1.0, low=1.0, high=2.0, original=0.0, amplitude=1.0,
                cos=512, sin=1024), **kw}
    assert layers.load().lic_rotary_table(a["coords"], a["rows"], a["axes"], a["r"], a["base"], a["factor"], a["low"],
                                          a["high"], a["original"], a["amplitude"], a["cos"], a["sin"], 0) == -1


POINTERS = ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "mask", "lengths")
SIZES = ("b", "n", "m", "h", "kv", "d", "dtype", "left", "right", "scale")
ATTENTION = {**{p: 256 for p in POINTERS}, "mask": 0, "lengths": 0, "strides": (4096, 64, 16) * 8,
             "mask_strides": (0, 0, 64, 1), "b": 2, "n": 64, "m": 64, "h": 4, "kv": 2, "d": 16, "dtype": 2, "left": -1,
             "right": -1, "scale": 0.25}


def attention_args(layers, **kw):
    a = {**ATTENTION, **kw}
    return layers._ATTENTION.pack(*(a[k] for k in POINTERS), *a["strides"], *a["mask_strides"],
                                  *(a[k] for k in SIZES))


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(out=0), -1), (dict(lse=0), -1), (dict(b=-1), -1),
    (dict(n=-1), -1), (dict(m=(1 << 28) + 1), -1), (dict(h=3), -1), (dict(kv=0), -1), (dict(h=0), -1), (dict(d=0), -1),
    (dict(d=129), -1), (dict(dtype=4), -1), (dict(left=-2), -1), (dict(right=-2), -1), (dict(scale=0.0), -1),
    (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(strides=(-1, 64, 16) * 8), -1), (dict(mask=256, mask_strides=(0, 0, -1, 1)), -1),
    (dict(b=0, q=0), 0), (dict(n=0, m=0, q=0, k=0), 0),
])
def test_attention_host_checks(layers, kw, code):
    lib = layers.load()
    args = attention_args(layers, **kw)
    big = 1 << 40
    assert lib.lic_attention_forward(args, 256, big, 0) == code
    assert lib.lic_attention_backward(args, 256, big, 0) == code


@pytest.mark.parametrize("kw", [dict(dout=0), dict(dq=0), dict(dk=0), dict(dv=0)])
def test_attention_backward_host_checks(layers, kw):
    assert layers.load().lic_attention_backward(attention_args(layers, **kw), 256, 1 << 40, 0) == -1


def test_attention_workspace_checks(layers):
    lib = layers.load()
    one = attention_args(layers, n=1, m=5000, b=1)
    need = lib.lic_attention_workspace_bytes(one, 0)
    assert need > 0
    assert lib.lic_attention_forward(one, None, need, 0) == -7
    assert lib.lic_attention_forward(one, 257, need, 0) == -7
    assert lib.lic_attention_forward(one, 256, need - 1, 0) == -7
    back = attention_args(layers)
    # dout . out of every row at least
    assert lib.lic_attention_workspace_bytes(back, 1) >= 2 * 4 * 64 * 4
    assert lib.lic_attention_backward(back, None, 0, 0) == -7
    assert lib.lic_attention_workspace_bytes(attention_args(layers, h=3), 1) == 0
    assert lib.lic_attention_forward(None, 256, 1 << 30, 0) == -1


def test_argument_blocks_match_the_header(layers):
    """The packed blocks are as long as the C structs (all members of 8 bytes)."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)

    def members(name):
        body = re.search(r"typedef struct %s \{(.*?)\}" % name, text, flags=re.S).group(1)
        total = 0
        for line in body.split(";"):
            for field in line.split(","):
                if field.strip():
                    size = re.search(r"\[(\d+)\]", field)
                    total += int(size.group(1)) if size else 1
        return total

    assert layers._ROTARY.size == 8 * members("lic_rotary_args")
    assert layers._ATTENTION.size == 8 * members("lic_attention_args")
    assert ctypes.sizeof(ctypes.c_void_p) == 8
