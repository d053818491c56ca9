"""The losses over an FP8 head on the GPU where their arithmetic has an edge: teachers whose scaled
logits do not fit fp32.  Tolerances as in test_loss_ops.py."""

import numpy as np
import pytest

import block_quant_gb300 as bq
from test_loss_ops import Head, empty

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_quant_gb300 import build

    build.build()
    return bq.load()


def both_grads(c, g):
    """(dx, dw) of a head whose forward pass has run."""
    import torch

    dx, dw = empty(c.n, c.cols, c.dev, torch.bfloat16)[0], empty(c.rows, c.cols, c.dev, torch.bfloat16)[0]
    c.grad(torch.as_tensor(g).to(c.dev), dx, dw)
    return dx, dw


@pytest.mark.parametrize("n", [5, 70])
@pytest.mark.parametrize("teacher", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [2.0, -2.0, 1.0, -1.0, 1e-38, 0.0])
def test_teachers_of_the_types_limits(cuda, n, teacher, scale):
    """Rows of the type's lowest value alone, whose scaled logits overflow and whose weights are equal all the
    same; one such logit, and the largest, beside others."""
    import torch

    def edit(c):
        t = torch.finfo(c.z.dtype)
        c.ids[:5] = np.arange(c.k) * 3
        c.ids[4, 1::2] = -1
        c.z[0] = t.min
        c.z[1, 2] = t.min
        c.z[2, 1], c.z[2, 3] = t.min, t.max
        c.z[3] = t.max
        c.z[4] = t.min
        c.z[4, 2] = -np.inf

    c = Head(cuda, n, 600, 128, scale=scale, k=11, teacher=teacher, seed=40, edit=edit)
    assert np.all(np.isfinite(c.pairs[1])) and np.all(c.pairs[1][0] == c.pairs[1][0, 0])
    c.forward().check_forward()
    if scale == 1e-38:
        return  # (gradients below bf16's smallest normal value)
    g = c.rng.standard_normal(n).astype(np.float32)
    c.check_grads(g, *both_grads(c, g))
