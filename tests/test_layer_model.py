"""The layer operators as a user runs them together: the example model's gradients
against the same model in fp64 on the same FP8 weights, and its training."""

import math
import os
import sys

import numpy as np
import pytest

import block_quant_gb300 as bq
from oracle import layer as L

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_quant_gb300 import build

    build.build()
    return bq.load()


def test_gradients_match_the_model_in_fp64(cuda):
    """Relative distance of each parameter's gradient from autograd in fp64 through the
    same FP8 weights.  The model rounds activations to E4M3 (2^-4 of a value, at random:
    a product of k such values is off by about 2^-5 of its own size) at up to nine places
    between a loss and a weight, so 9 * 2^-5 = 0.28 bounds what is expected."""
    import torch

    from fp8_lm import EPS, Model

    torch.manual_seed(0)
    m = Model(300, 256, 384, 2, 200, cuda, seed=3)
    ids = torch.randint(0, 300, (200,), device=cuda)
    ids[3] = -1  # padding
    logits, saved = m.forward(ids)
    dlogits = (torch.randn(200, 300, device=cuda) / 200).bfloat16()
    m.backward(ids, dlogits, saved)
    m.check()

    w = {}
    for name, (r, c) in m.shapes.items():
        if r == 1:
            t = m.vector(name).double().cpu()
        else:
            codes, scales = m.weight(name)
            t = torch.as_tensor(L.decode_tiles(codes.cpu().numpy(), scales.cpu().numpy()))
        w[name] = t.clone().requires_grad_(True)
    cpu = ids.cpu()
    x = w["embed"][cpu.clamp(min=0)] * (cpu >= 0)[:, None]
    norm = lambda h, g: h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * g  # noqa: E731
    h = x
    for i in range(2):
        u = norm(h, w[f"norm{i}"]) @ w[f"up{i}"].t()
        h = h + torch.relu(u).square() @ w[f"down{i}"].t()
    out = norm(h, w["norm"]) @ w["head"].t()
    far = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert far(logits, out.detach()) < 0.28
    out.backward(dlogits.double().cpu())
    for name in m.names:
        got = m.grads[name]
        assert far(got.view_as(w[name]), w[name].grad) < 0.28, name


def test_training_lowers_the_loss(cuda):
    from fp8_lm import train

    losses = train(40, vocab=500, width=256, hidden=512, layers=2, tokens=1000)
    assert np.all(np.isfinite(losses))
    assert abs(losses[0] - math.log(500)) < 1.5  # as good as guessing
    assert losses[-1] < 0.5 * losses[0]


def test_same_seed_same_losses(cuda):
    """No operator sums in an order of its own choosing."""
    from fp8_lm import train

    a = train(5, vocab=300, width=256, hidden=256, layers=1, tokens=700)
    b = train(5, vocab=300, width=256, hidden=256, layers=1, tokens=700)
    assert a == b
