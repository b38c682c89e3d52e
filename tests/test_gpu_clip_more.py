"""Clipping where its factor is below the numbers of 32 bits."""
from __future__ import annotations

import math

import pytest
import torch

import layers_ref as R
from test_gpu_clip import BF16, F16, F32, L, made  # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size,n,max_norm", [(3e38, 1, 1e-6), (1e38, 5000, 1.0), (1e38, 70000, 1e-2), (1e38, 9, 1e-30), (1e20, 4096, 1e-5)])
def test_clip_of_very_large_values(L, size, n, max_norm, dtype):  # noqa: F811
    """The result is of max_norm's size, so it has all of its bits, whatever the factor's are."""
    grads = [t.clamp(-2, 2).mul_(size / 2).to(dtype) for t in made([n, 37], (F32,), seed=n)]
    held = [t.double() for t in grads]
    norm = math.sqrt(sum(float(t.square().sum()) for t in held))
    c = max_norm / (norm + 1e-6)
    for out in ([torch.empty_like(t) for t in grads], None):
        L.clip_gradients(grads, max_norm, out=out)
        for t, h in zip(grads if out is None else out, held):
            # the factor is rounded to 32 bits, the product to the type; results below 2^-126 in steps of 2^-149 (2^-133)
            want = h * c
            bound = (R.UNIT[dtype] + 2.0 ** -23) * want.abs() + (2.0 ** -149 if dtype == F32 else 2.0 ** -133)
            assert R.worst(t, want, bound) <= 1.0
    assert math.sqrt(sum(float(t.double().square().sum()) for t in grads)) == pytest.approx(max_norm, rel=4e-3)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("place", ["in place", "out"])
def test_clip_past_the_caches(L, place, dtype):  # noqa: F811
    """More bytes than the last-level cache holds, which the stores then pass; odd lengths and addresses."""
    sizes = [90_000_001 if dtype != F32 else 45_000_001, 1, 12_345_677]
    grads = [t[1:] if i == 2 else t for i, t in enumerate(made(sizes, (dtype,), seed=4))]
    assert 2 * sum(t.numel() * t.element_size() for t in grads) > 256 << 20
    held = [t.clone() for t in grads]
    out = [torch.empty_like(t) for t in grads] if place == "out" else None
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in held))
    got = L.clip_gradients(grads, 0.25 * norm, out=out)
    assert float(got) == pytest.approx(norm, rel=2.0 ** -23)
    c = 0.25 * norm / (norm + 1e-6)
    for t, h in zip(grads if out is None else out, held):
        want = h.double() * c
        assert R.worst(t, want, (R.UNIT[dtype] + 2.0 ** -23) * want.abs() + R.STEP[dtype] + 2.0 ** -126) <= 1.0
