"""What the network operators' host side decides from a call's sizes, without a GPU."""
from __future__ import annotations

import re

import pytest

from test_layers_abi_cpu import HEADER, SIZES, attention_args, layers  # noqa: F401 - a fixture


def size_of(layers, backward, **kw):  # noqa: F811
    return layers.load().lic_attention_workspace_bytes(attention_args(layers, **kw), backward)


LONG = dict(b=8, n=2080, m=2080, h=2, kv=2, d=64)
WINDOWS = [(-1, -1), (0, 0), (-1, 0), (300, -1), (300, 0), (100, 900)]


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("left,right", WINDOWS)
def test_a_call_takes_the_workspace_of_its_sizes_and_windows(layers, left, right, backward):  # noqa: F811
    lib = layers.load()
    for sizes in (LONG, dict(b=1, n=510, m=510, h=2, kv=1, d=32), dict(b=2, n=1, m=9000, h=4, kv=1, d=96)):
        need = size_of(layers, backward, left=left, right=right, **sizes)
        call = lib.lic_attention_backward if backward else lib.lic_attention_forward
        if need:  # one byte less is refused on the host
            args = attention_args(layers, left=left, right=right, **sizes)
            assert call(args, 256, need - 1, 0) == -7


def test_the_header_names_what_sizes_the_workspace(layers):  # noqa: F811
    """Each field that the size depends on is named where the header says what is read."""
    said = re.search(r"/\* Bytes for lic_attention_forward.*?\*/", open(HEADER).read(), flags=re.S).group(0)
    names = dict(zip(SIZES, ("batch", "queries", "keys", "heads", "kv_heads", "dim", "dtype", "window_left",
                             "window_right", "scale")))
    base = {**LONG, "left": -1, "right": -1, "dtype": 2, "scale": 0.25}
    other = dict(b=3, n=700, m=500, h=4, kv=1, d=96, dtype=0, left=64, right=0, scale=0.5)
    for backward in (0, 1):
        for start in (base, {**base, "left": 64, "right": 64}):
            for field, name in names.items():
                if size_of(layers, backward, **start) != size_of(layers, backward, **{**start, field: other[field]}):
                    assert re.search(r"\b%s\b" % name, said), name
    # and the windows do count
    assert size_of(layers, 0, **base) != size_of(layers, 0, **{**base, "right": 0})


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("kw", [dict(left=-2), dict(right=-2), dict(left=(1 << 40) + 1), dict(right=1 << 62),
                                dict(left=(1 << 63) - 1, right=(1 << 63) - 1)])
def test_windows_out_of_range_have_no_size(layers, kw, backward):  # noqa: F811
    assert size_of(layers, backward, **{**LONG, **kw}) == 0
    args = attention_args(layers, **{**LONG, **kw})
    assert layers.load().lic_attention_forward(args, 256, 1 << 40, 0) == -1
    assert layers.load().lic_attention_backward(args, 256, 1 << 40, 0) == -1
