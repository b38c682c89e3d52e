"""Linear attention held to what its arithmetic allows: outputs and gradients to their last rounding, states and
the decay's gradient to 32-bit sums, near and far sizes of values side by side, many segments."""
from __future__ import annotations

import pytest
import torch

import layers_more_ref as M
import layers_ref as R
from test_gpu_linear import ALL, BF16, F16, F32, L, decays, gen, inputs, normal, passes  # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu

# What 32-bit arithmetic loses of a sum of absolute terms: powers of g and the scale (4 roundings of 2^-24), the
# state's step from run to run (2^-21 at most, 8 of them), and sums in short chains, whose roundings have no
# common sign (4, for chains of up to some hundred).
SUMS = 16 * 2.0 ** -24
# What an operand of a product that forms an output loses in its two parts: x = part + rest, |rest| < u of x, so rest
# is rounded by u / 2 of u at most; float32 is its own operand.
PARTS = {F32: 0.0, F16: 2.0 ** -23, BF16: 2.0 ** -17}


def once(want, size, dtype):
    """Rounded once from sums of operands in parts."""
    return R.UNIT[dtype] * want.abs() + (SUMS + PARTS[dtype]) * size + R.STEP[dtype]


def both(x, more, grads):
    return M.linear(**x, **more, **grads), M.linear_abs(**x, **more, **grads)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("b,s,h,kv,d,e,state,ragged", [
    (2, 1, 4, 2, 64, 64, True, False), (2, 2, 3, 3, 32, 32, True, False), (1, 31, 3, 1, 40, 33, True, False),
    (4, 65, 6, 3, 32, 32, True, True), (2, 130, 4, 1, 96, 72, True, False), (3, 200, 4, 2, 128, 128, True, True),
    (1, 700, 4, 4, 64, 64, False, False), (4, 510, 6, 6, 32, 32, False, False), (2, 1100, 3, 3, 20, 5, True, True),
])
def test_outputs_are_rounded_once(L, b, s, h, kv, d, e, state, ragged, dtype):  # noqa: F811
    """Scores and states keep their bits on the way into the products that form out, dq, dk and dv."""
    x, more, grads = inputs(b, s, h, kv, d, e, dtype, state, ragged, seed=1)
    r, size = both(x, more, grads)
    out, _ = L.linear_attention_forward(**x, **more)
    dq, dk, dv, _, _ = L.linear_attention_backward(grads["dout"], *x.values(), dstate=grads["dstate"], **more)
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        passes(got, r[name], once(r[name], size[name], dtype), name)
