"""A transformer that predicts a latent's means and scales, trained and then used to code it.

    python examples/latent_transformer.py [--rows 68 --columns 120 --channels 192 --steps 40]

From a hyper latent z (a quarter of y's sides) the model predicts mean and scale of every value
of y.  Its blocks are group norm (channels last), attention with rotary positions (rows turn one
half of a head's pairs, columns the other) and group norm with SiLU, all from
``learned_image_compression_amd.layers``; what multiplies features by weights is torch's.  It is
trained on the number of bits that the coder will need, then y is coded with its predictions: the
encoder's front end and coder run fused, the decoder predicts again from z, which gives the same
bits, looks up the same tables and gets the same symbols.  z and y are synthetic.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch
from torch import nn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from learned_image_compression_amd import binding as B  # noqa: E402
from learned_image_compression_amd import layers as L  # noqa: E402


class Norm(nn.Module):
    """Group norm of [N, H, W, C] and an activation."""

    def __init__(self, channels, groups=8, activation="none"):
        super().__init__()
        self.weight, self.bias = nn.Parameter(torch.ones(channels)), nn.Parameter(torch.zeros(channels))
        self.groups, self.activation = groups, activation

    def forward(self, x):
        y = L.group_norm(x.permute(0, 3, 1, 2), self.groups, self.weight, self.bias, activation=self.activation)
        return y.permute(0, 2, 3, 1)


class Block(nn.Module):
    def __init__(self, channels, heads):
        super().__init__()
        self.heads = heads
        self.before, self.between = Norm(channels), Norm(channels, activation="silu")
        self.qkv, self.out = nn.Linear(channels, 3 * channels), nn.Linear(channels, channels)
        self.mix = nn.Linear(channels, channels)

    def forward(self, x, table):
        n, h, w, c = x.shape
        q, k, v = self.qkv(self.before(x)).view(n, h * w, 3, self.heads, c // self.heads).unbind(2)
        q, k = L.rotary(q, k, *table)
        x = x + self.out(L.attention(q, k, v).reshape(n, h, w, c))
        return x + self.mix(self.between(x))


class LatentTransformer(nn.Module):
    """z [N, H / 4, W / 4, channels] -> means and scales of y [N, H, W, channels]."""

    def __init__(self, channels, heads, blocks=2):
        super().__init__()
        self.up = nn.Linear(channels, 16 * channels)
        self.blocks = nn.ModuleList(Block(channels, heads) for _ in range(blocks))
        self.head = nn.Linear(channels, 2 * channels)

    def forward(self, z, table):
        n, h, w, c = z.shape
        x = self.up(z).view(n, h, w, 4, 4, c).permute(0, 1, 3, 2, 4, 5).reshape(n, 4 * h, 4 * w, c)
        for block in self.blocks:
            x = block(x, table)
        means, logs = self.head(x).float().chunk(2, dim=-1)
        return means, torch.exp(logs.clamp(-2.0, 5.0)) + 0.11


def positions(rows, columns, dim):
    """Tables of an image's positions, its rows and columns as two axes."""
    at = torch.cartesian_prod(torch.arange(rows, dtype=torch.float64), torch.arange(columns, dtype=torch.float64))
    return L.rotary_table(at.cuda().contiguous(), dim)


def bits(y, means, scales):
    """Bits a value of y takes under the discretised Gaussian, on average."""
    up, low = (torch.special.ndtr((y - means + s) / scales) for s in (0.5, -0.5))
    return -torch.log2((up - low).clamp(min=1e-9)).mean()


def synthetic(rows, columns, channels, seed):
    """z, and a y whose means and spreads follow z's neighbourhood."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(1, rows // 4, columns // 4, channels, generator=g, device="cuda")
    wide = z.repeat_interleave(4, dim=1).repeat_interleave(4, dim=2)
    spread = torch.exp(0.7 * wide.roll(1, dims=-1))
    return z, 3.0 * wide + spread * torch.randn(wide.shape, generator=g, device="cuda")


def run(rows=32, columns=48, channels=64, heads=2, steps=40, seed=0, say=print):
    torch.manual_seed(seed)
    z, y = synthetic(rows, columns, channels, seed)
    model = LatentTransformer(channels, heads).cuda().to(torch.bfloat16)
    table = positions(rows, columns, channels // heads)
    z16 = z.to(torch.bfloat16)
    optimizer = torch.optim.Adam(model.parameters(), lr=2e-3)
    history = []
    for step in range(steps):
        loss = bits(y, *model(z16, table))
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        history.append(float(loss.detach()))
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step}: {history[-1]:.3f} bits a value")

    # one table row for each of 64 scales, as the coder takes them
    scale_table = torch.exp(torch.linspace(math.log(0.11), math.log(256.0), 64, dtype=torch.float64, device="cuda"))
    tables, row_status = B.gaussian_tables(scale_table, 6.1094, 3133)
    B.check_rows(row_status, "tables")
    streams = max(1, y.numel() // 32768)
    with torch.no_grad():
        means, scales = (t.reshape(-1).contiguous() for t in model(z16, table))
        stream, words, status = B.encode_interleaved_latent(y.reshape(-1), means, scales, scale_table.float(), tables,
                                                            streams)
        B.check(status, "encode")
        # the decoder: nothing but z and the stream
        means2, scales2 = (t.reshape(-1).contiguous() for t in model(z16, table))
        _, indexes = B.latent_symbols(torch.zeros_like(means2), means2, scales2, scale_table.float())
        symbols, status = B.decode_interleaved(stream, indexes, tables, streams)
        B.check(status, "decode")
        y_hat = B.dequantize(symbols, means2)
        want = torch.round(y.reshape(-1) - means) + means
    coded = 32 * int(words) / y.numel()
    same = torch.equal(means, means2) and torch.equal(scales, scales2) and torch.equal(y_hat, want)
    say(f"coded at {coded:.3f} bits a value; the decoder's latent {'equals' if same else 'DIFFERS FROM'} the encoder's")
    return {"history": history, "coded": coded, "same": same}


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--rows", type=int, default=68)
    parser.add_argument("--columns", type=int, default=120)
    parser.add_argument("--channels", type=int, default=192)
    parser.add_argument("--heads", type=int, default=6)
    parser.add_argument("--steps", type=int, default=40)
    a = parser.parse_args()
    sys.exit(0 if run(a.rows, a.columns, a.channels, a.heads, a.steps)["same"] else 1)
