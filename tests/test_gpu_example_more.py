"""The example's recurrent model: RMS norms with the residual, rotary positions, linear attention and clipping
together, trained and used to code; its gradients against the same model of plain 64-bit operators."""
from __future__ import annotations

import math

import pytest
import torch

import layers_more_ref as M
import layers_ref as R
from test_gpu_example import load

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,columns,channels,heads", [(32, 48, 64, 2), (20, 28, 96, 4)])
def test_recurrent_model_trains_and_codes(rows, columns, channels, heads):
    r = load().run(rows, columns, channels, heads, steps=8, model="recurrent", clip=1.0, say=lambda s: print(s, flush=True))
    assert r["same"] and all(math.isfinite(v) for v in r["history"])


class Plain:
    """The operators of the model in 64 bits, with torch's own gradients."""

    @staticmethod
    def rms_norm(x, weight, residual, eps=1e-6):
        h = x + residual
        return weight * h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps), h

    @staticmethod
    def rotary(q, k, cos, sin):
        return R.turn(q, cos, sin, None, False), R.turn(k, cos, sin, None, False)

    @staticmethod
    def linear_attention(q, k, v, log_decay):
        r = M.linear(q, k, v, log_decay)
        return r["out"], r["last"]


@pytest.mark.parametrize("rows,columns,channels,heads", [(8, 12, 64, 2), (16, 20, 48, 3)])
def test_recurrent_models_gradients(rows, columns, channels, heads, monkeypatch):
    example = load()
    torch.manual_seed(1)
    z, y = example.synthetic(rows, columns, channels, 1)
    model = example.LatentRecurrent(channels, heads).cuda()
    table = example.positions(rows, columns, channels // heads)
    loss = example.bits(y, *model(z, table))
    got = torch.autograd.grad(loss, list(model.parameters()))
    exact = example.LatentRecurrent(channels, heads).cuda().double()
    exact.load_state_dict({n: p.double() for n, p in model.state_dict().items()})
    for block in exact.blocks:  # the example takes decays in 32 bits
        block.rate.data = block.rate.data.float()
    for name in ("rms_norm", "rotary", "linear_attention"):
        monkeypatch.setattr(example.L, name, getattr(Plain, name))
    want_loss = example.bits(y, *exact(z.double(), table))
    want = torch.autograd.grad(want_loss, list(exact.parameters()))
    # 32-bit sums of some hundred to some thousand terms through a dozen layers: 1e-3 of a gradient's norm, where
    # one wrong term would be of the gradient's size
    assert abs(float(loss.detach()) - float(want_loss.detach())) <= 1e-4 * float(want_loss.detach())
    for (name, _), a, b in zip(model.named_parameters(), got, want):
        off = float((a.double() - b.double()).norm() / b.double().norm().clamp(min=1e-12))
        print(f"{name}: {off:.2e}", flush=True)
        assert off <= 1e-3, name


def test_clipped_gradients_of_a_step():
    """Clipping a model's gradients in place, in the middle of a step, against torch's sums in 64 bits."""
    example = load()
    torch.manual_seed(2)
    z, y = example.synthetic(16, 16, 64, 2)
    model = example.LatentRecurrent(64, 2).cuda().to(torch.bfloat16)
    example.bits(y, *model(z.to(torch.bfloat16), example.positions(16, 16, 32))).backward()
    grads = [p.grad for p in model.parameters()]
    held = [g.double() for g in grads]
    norm = math.sqrt(sum(float(g.square().sum()) for g in held))
    got = example.L.clip_gradients(grads, norm / 4)
    assert float(got) == pytest.approx(norm, rel=1e-6)
    c = (norm / 4) / (norm + 1e-6)
    for g, h in zip(grads, held):
        assert R.worst(g, h * c, (2.0 ** -8 + 2.0 ** -22) * (h * c).abs() + 2.0 ** -133) <= 1.0
