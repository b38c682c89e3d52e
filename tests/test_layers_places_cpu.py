"""Which places a caller may give for outputs, without a GPU: the overlap of two layouts against the sets of their
bytes, and the calls of RMS norm and linear attention with a stand-in for the library."""
from __future__ import annotations

import random

import pytest
import torch

from learned_image_compression_amd import layers


def views(rng, base):
    """A view of `base` with any strides, and the bytes of its values."""
    dtype = rng.choice([torch.uint8, torch.float16, torch.float32])
    size = torch.empty(0, dtype=dtype).element_size()
    shape = [rng.randint(0 if rng.random() < 0.05 else 1, 5) for _ in range(rng.randint(1, 4))]
    strides = [rng.choice([0, 1, 1, 2, 3, 4, 5, 8, 12, 16, 20, 24, 40]) for _ in shape]
    start = rng.randint(0, 200) * 4 // size
    values = torch.as_strided(torch.arange(base.numel() // size), shape, strides, start).flatten().tolist()
    return torch.as_strided(base.view(dtype), shape, strides, start), {i * size + k for i in values for k in range(size)}


@pytest.mark.parametrize("seed", range(4))
def test_overlap_is_that_of_the_bytes(seed):
    rng, base = random.Random(seed), torch.zeros(4000, dtype=torch.uint8)
    seen = set()
    for _ in range(5000):
        (a, its), (b, others) = views(rng, base), views(rng, base)
        want = bool(its & others)
        seen.add(want)
        assert bool(layers._overlapping(a, (None, b))) == want, (a.shape, a.stride(), a.storage_offset(), b.shape, b.stride(), b.storage_offset())
    assert seen == {True, False}


def test_overlap_of_large_layouts():
    """As many rows as a picture has, decided without going over them."""
    wide = torch.empty(4, 32640, 512, dtype=torch.float16)
    a, b, c = wide[..., :192], wide[..., 192:384], wide[..., 191:383]
    assert not layers._overlapping(a, (b,)) and layers._overlapping(a, (c,)) and layers._overlapping(b, (c,))
    assert not layers._overlapping(wide[:, ::2], (wide[:, 1::2],)) and layers._overlapping(wide[:, 1:], (wide[:, :-1],))
    assert not layers._overlapping(wide[:2], (wide[2:],)) and layers._overlapping(wide[:2], (wide[1:2, :5],))


class Library:
    """Counts the calls and says that they went well."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(layers, "load", lambda: lib)
    monkeypatch.setattr(layers, "_device_of", lambda t, name: t.device)
    monkeypatch.setattr(layers, "_stream", lambda device: 0)
    monkeypatch.setattr(layers, "_with_workspace", lambda device, stream, call, size, where: call(None, 0))
    return lib


def test_rms_norm_places(library):
    buf, other = torch.zeros(9, 16), torch.zeros(8, 16)
    rstd = torch.ones(8)
    wide = torch.zeros(8, 48)
    for call in (
            lambda: layers.rms_norm_forward(buf[:-1], out=buf[1:]),
            lambda: layers.rms_norm_forward(buf[1:], out=buf[:-1]),
            lambda: layers.rms_norm_forward(other, residual=buf[:-1], out=buf[1:]),
            lambda: layers.rms_norm_forward(other, residual=buf[:-1], sum_out=buf[1:]),
            lambda: layers.rms_norm_forward(other, residual=other, out=buf[1:], sum_out=buf[:-1]),
            lambda: layers.rms_norm_forward(wide[:, :16], out=wide[:, 8:24]),
            lambda: layers.rms_norm_forward(other, buf[3], out=buf[1:]),
            lambda: layers.rms_norm_8bit(other, out=other.view(torch.float8_e4m3fn).view(-1)[64:192].view(8, 16)),
            lambda: layers.rms_norm_backward(buf[:-1], other, None, rstd, out=buf[1:]),
            lambda: layers.rms_norm_backward(other, other, None, rstd, dsum=buf[:-1], out=buf[1:]),
            lambda: layers.rms_norm_backward(other, other, None, buf.view(-1)[16:24], out=buf[1:]),
    ):
        with pytest.raises(ValueError, match="overlaps|one place"):
            call()
    assert library.calls == 0
    # entry by entry, side by side, or one behind the other
    for call in (
            lambda: layers.rms_norm_forward(other, residual=buf[1:], out=other, sum_out=buf[1:]),
            lambda: layers.rms_norm_forward(wide[:, :16], residual=wide[:, 16:32], out=wide[:, 32:], sum_out=wide[:, :16]),
            lambda: layers.rms_norm_forward(buf[:4], residual=buf[4:8], out=other[:4], sum_out=other[4:]),
            lambda: layers.rms_norm_backward(other, buf[:-1], None, rstd, dsum=other, out=other),
    ):
        call()
    assert library.calls == 4


@pytest.mark.parametrize("s", [1, 70])
def test_linear_attention_places(library, s):
    wide = torch.zeros(2, s, 3, 32)
    q, k, v = wide[..., :8], wide[..., 8:16], wide[..., 16:24]
    log = torch.zeros(3)
    ring = torch.zeros(3, 3, 8, 8)  # two batches' states from each place on
    flat = torch.zeros(2 * s * 24 + 2 * 192)

    def call(**more):
        return layers.linear_attention_forward(q, k, v, log, **more)

    for more in (
            dict(out=wide[..., 4:12]), dict(out=k), dict(state=ring[1:], state_out=ring[:-1]),
            dict(state=ring[:-1], state_out=ring[1:]),
            dict(out=flat[:48 * s].view(2, s, 3, 8), state_out=flat[48 * s - 1:48 * s + 383].view(2, 3, 8, 8)),
    ):
        with pytest.raises(ValueError, match="must not|laid out differently"):
            call(**more)
    assert library.calls == 0
    state = torch.zeros(2, 3, 8, 8)
    call(out=wide[..., 24:], state=state, state_out=state)
    call(state=ring[:2], state_out=torch.zeros(2, 3, 8, 8))
    call(out=flat[:48 * s].view(2, s, 3, 8), state_out=flat[48 * s:].view(2, 3, 8, 8))
    assert library.calls == 3


def test_outputs_that_overlap_themselves(library):
    """A sliding window's entries are written by several rows, in no order; any other strides are taken."""
    flat, x = torch.zeros(4096), torch.zeros(6, 16)
    for out in (flat.as_strided((6, 16), (8, 1)), flat.as_strided((6, 16), (15, 1)), flat.as_strided((6, 16), (0, 1)), flat.unfold(0, 16, 4)[:6]):
        with pytest.raises(ValueError, match="overlaps itself"):
            layers.rms_norm_forward(x, out=out)
    q, state = torch.zeros(2, 1, 3, 8), torch.zeros(2, 3, 8, 8)
    with pytest.raises(ValueError, match="overlaps itself"):
        layers.linear_attention_forward(q, q, q, torch.zeros(3), state_out=flat.as_strided((2, 3, 8, 8), (192, 60, 8, 1)))
    assert library.calls == 0
    layers.rms_norm_forward(x, out=flat.as_strided((6, 16), (16, 1)))
    layers.rms_norm_forward(x, out=flat.as_strided((6, 16), (100, 1)))
    layers.rms_norm_forward(torch.zeros(4, 6, 16), out=flat.as_strided((4, 6, 16), (16, 64, 1)))
    layers.linear_attention_forward(q, q, q, torch.zeros(3), out=flat.as_strided((2, 1, 3, 8), (8, 4000, 16, 1)),
                                    state_out=state.transpose(0, 1).contiguous().transpose(0, 1))
    assert library.calls == 4
