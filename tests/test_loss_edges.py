"""The losses over an FP8 head on the GPU where their arithmetic has an edge: teachers whose scaled
logits do not fit fp32, or that give next to nothing to a word, and logits that do not fit
it.  Tolerances as in test_loss_ops.py."""

import numpy as np
import pytest

import block_quant_gb300 as bq
from test_loss_ops import Head, empty, f64

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


@pytest.mark.parametrize("n", [5, 70, 300])
@pytest.mark.parametrize("teacher", ["fp32", "bf16"])
def test_small_weights_of_a_teacher(cuda, n, teacher):
    """Words to which teacher and student give little, down to 2^-30: what u = p - q holds of them."""
    def edit(c):
        c.ids[:] = np.argsort(c.rng.random(c.ids.shape), axis=1) + 16 * c.rng.integers(0, 30, (n, 1))
        c.z[:] = -torch_like(c, np.arange(c.k) * (0.02 + 0.02 * c.rng.random((n, 1))))

    c = Head(cuda, n, 600, 128, scale=64.0, k=16, teacher=teacher, seed=41, edit=edit)
    q = c.pairs[1]
    assert np.sum(q > 0.5) and np.sum((q < 2.0 ** -14) & (q > 2.0 ** -28)) > n
    c.forward().check_forward()
    g = c.rng.standard_normal(n).astype(np.float32)
    c.check_grads(g, *both_grads(c, g))


def torch_like(c, v):
    import torch

    return torch.as_tensor(v).to(c.z.dtype)


@pytest.mark.parametrize("n", [6, 200])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.filterwarnings("ignore:invalid value")
def test_a_teacher_without_weights_stays_in_its_row(cuda, n, bad):
    """Logits that have no softmax, alone and beside others, whatever the student makes of their words."""
    def edit(c):
        c.ids[::2] = -1
        c.ids[::2, 0] = np.arange(c.ids[::2].shape[0])
        c.z[2, 0] = bad
        c.ids[3] = np.arange(c.k) + 5
        c.z[3, 1] = bad

    c = Head(cuda, n, 400, 128, scale=8.0, k=5, teacher="fp32", seed=42, edit=edit)
    c.x[2], c.xs[:, 2] = c.w[1], 4 * c.ws_[0, 0]  # (sure of its word)
    c.forward()
    wrong = np.isin(np.arange(n), [2, 3])
    assert float(c.logp[2, 0]) > -0.5
    assert np.array_equal(np.isnan(f64(c.loss)), wrong)
    dx, dw = both_grads(c, np.ones(n, np.float32))
    assert np.array_equal(np.isnan(f64(dx)).all(axis=1), wrong) and np.array_equal(np.isnan(f64(dx)).any(axis=1), wrong)
    assert np.isnan(f64(dw)[1]).all() and np.isnan(f64(dw)[6]).all()


@pytest.mark.parametrize("n", [8, 300])
@pytest.mark.parametrize("k", [None, 2])
def test_infinite_logits_are_not_hidden(cuda, n, k):
    """Logits past fp32 are infinities: a largest one has no log-probability (inf - inf), and the losses and
    gradients of its row are not finite, whichever the target; a row without a target gives nothing."""
    import torch

    rows, cols, scale = 200, 16, 1e36
    up, down = 0x7E, 0xFE  # 448 and -448: 448 * 16 * scale is past fp32's largest
    x, xs = torch.full((n, cols), 0x38, dtype=torch.uint8, device=cuda), torch.ones(1, n, device=cuda)  # 1.0
    ws_ = torch.ones(2, 1, device=cuda)
    words = torch.tensor([3, 5, 0, -1], device=cuda).repeat(n // 4)
    none = (words < 0).cpu().numpy()
    for case, lse in (("largest", np.inf), ("all", -np.inf)):
        w = torch.full((rows, cols), down if case == "all" else 0, dtype=torch.uint8, device=cuda)
        if case == "largest":
            w[3], w[5] = up, down
        c = Head.__new__(Head)
        c.n, c.rows, c.cols, c.k, c.scale, c.dev, c.head = n, rows, cols, k, scale, cuda, (x, xs, w, ws_)
        if k is None:
            c.t = words
        else:
            c.t, c.z = torch.stack([words, torch.where(words < 0, words, 7)], 1).contiguous(), torch.zeros(n, k, device=cuda)
        c.forward()
        loss = f64(c.loss)
        assert np.all(f64(c.lse) == lse)
        # the largest and, where all are -inf, every word: inf - inf; the others: inf
        undefined = (f64(words) == 3) | (case == "all")
        assert np.all(loss[none] == 0)
        assert np.all(np.isnan(loss[undefined & ~none])) and np.all(loss[~undefined & ~none] == np.inf)
        if k:
            assert np.all(f64(c.logp)[none] == 0) and not np.any(np.isfinite(f64(c.logp)[~none]))
        dx, dw = both_grads(c, np.ones(n, np.float32))
        assert np.all(np.isnan(f64(dx)[~none])) and np.all(f64(dx)[none] == 0)
        assert np.all(np.isnan(f64(dw)[3]))
