"""RMS norm where its arrays are larger than the last-level cache, which its stores then pass."""
from __future__ import annotations

import pytest
import torch

from test_gpu_rms import ALL, L, check, gen, normal  # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,c", [(400_000, 192), (700_001, 119), (9000, 8196), (4100, 20001)])
def test_rms_norm_past_the_caches(L, rows, c, dtype):  # noqa: F811
    g = gen(c)
    x, residual, dy, dsum = (normal(g, rows, c, dtype=dtype) for _ in range(4))
    assert 3 * x.numel() * x.element_size() > 256 << 20
    check(L, x, residual, 1 + 0.3 * normal(g, c), 1e-6, dy, dsum)
