"""The example that trains an entropy model from the network operators and codes with it."""
from __future__ import annotations

import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def load():
    spec = importlib.util.spec_from_file_location("latent_transformer",
                                                  os.path.join(ROOT, "examples", "latent_transformer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("rows,columns,channels,heads", [(32, 48, 64, 2), (20, 28, 96, 4)])
def test_trains_and_codes(rows, columns, channels, heads):
    r = load().run(rows, columns, channels, heads, steps=30, say=lambda s: print(s, flush=True))
    assert r["same"]
    assert r["history"][-1] < r["history"][0] - 0.5
    # the stream holds what the loss promised, and its own headers and table rounding
    assert r["coded"] < r["history"][-1] + 1.0
