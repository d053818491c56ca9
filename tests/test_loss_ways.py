"""The ways that the losses over an FP8 head choose by size, each at sizes that take it, which the
tests see from the workspaces: dx of few tokens by three E4M3 terms of u, a teacher's words taken from
the product's tiles, the product on pairs of CTAs and on single ones.  Tolerances as in test_loss_ops.py."""

import numpy as np
import pytest

import block_quant_gb300 as bq
from oracle import loss as O
from test_loss_ops import E, Head, empty, f64, near, outside_kept, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_quant_gb300 import build

    build.build()
    return bq.load()


def up(x, to=256):
    return -(-x // to) * to


# ----------------------------------------------------------------------------- few tokens' dx
# 42 tokens fill a tile of the transposed product: one tile's rows and the next ones', all of them and a single one.
# The heads of at most 2^24 codes make dw beside dx, the others in turn.


FEW = [(4, 1298, 608), (13, 2500, 512), (42, 5000, 1040), (43, 9000, 1040), (85, 5000, 608), (126, 9000, 1040), (43, 17000, 1040)]


def takes_terms(n, rows, cols):
    """Without W in fp16 the workspace is smaller than that."""
    return bq.loss_fp8_grad_workspace(n, rows, cols) < 2 * rows * cols


def few_head(dev, n, rows, cols, **kw):
    assert takes_terms(n, rows, cols)
    return Head(dev, n, rows, cols, **kw)


@pytest.mark.parametrize("n,rows,cols", FEW)
@pytest.mark.parametrize("k,teacher", [(None, None), (9, "bf16")])
def test_gradients_of_few_tokens(cuda, n, rows, cols, k, teacher):
    """Both outputs, dx alone, and dw added to what is there; outputs at odd addresses inside wider matrices."""
    import torch

    c = few_head(cuda, n, rows, cols, scale=0.8, k=k, teacher=teacher, seed=50, pitch=16, spare=3).forward()
    g = c.rng.standard_normal(n).astype(np.float32) / n
    dloss = torch.as_tensor(g).to(cuda)
    dx, fx = empty(n, cols, cuda, torch.bfloat16, 5, 1)
    dw, fw = empty(rows, cols, cuda, torch.bfloat16, 24)
    c.grad(dloss, dx, dw)
    c.check_grads(g, dx, dw)
    assert outside_kept(dx, fx, 1) and outside_kept(dw, fw, 0)
    alone, again = empty(n, cols, cuda, torch.bfloat16)[0], empty(rows, cols, cuda, torch.bfloat16, 3)[0]
    c.grad(dloss, alone, None)
    assert torch.equal(alone, dx)
    old = torch.randn(rows, cols, device=cuda).bfloat16() / n
    again.copy_(old)
    c.grad(dloss, alone, again, accumulate=True)
    assert torch.equal(alone, dx)
    c.check_grads(g, None, again, old=f64(old))


@pytest.mark.parametrize("n,rows,cols", FEW[:4])
@pytest.mark.parametrize("k", [None, 4])
def test_few_rows_without_a_target_hold_anything(cuda, n, rows, cols, k):
    """NaN codes, scales, logits and gradients of those rows, and W's, stay out of them and of the others."""
    import torch

    def none(c):
        if k is None:
            c.targets[1::3] = -1
        else:
            c.ids[1::3] = -1
            c.z[1::3] = float("nan")
            c.z[0, 1] = -np.inf

    c = few_head(cuda, n, rows, cols, k=k, seed=51, edit=none)
    some = c.pairs[2].any(axis=1)
    g = c.rng.standard_normal(n).astype(np.float32)
    out = []
    for broken in (False, True):
        if broken:
            c.x[1::3] = 0x7F
            c.xs[:, 1::3] = float("nan")
            g[~some] = np.where(np.arange((~some).sum()) % 2, np.nan, np.inf)
        c.forward()
        dx, dw = empty(n, cols, cuda, torch.bfloat16)[0], empty(rows, cols, cuda, torch.bfloat16)[0]
        c.grad(torch.as_tensor(g).to(cuda), dx, dw)
        assert np.all(f64(c.loss)[~some] == 0) and np.all(f64(dx)[~some] == 0)
        out.append([f64(t) for t in (c.loss, dx, dw)])
    assert all(np.array_equal(a, b) for a, b in zip(*out))
    c.check_grads(np.where(some, g, 0), dx, dw)
    c.w[rows // 2, 7] = 0xFF
    c.forward()
    c.grad(torch.as_tensor(g).to(cuda), dx, dw)
    assert np.array_equal(np.isnan(f64(dx)).any(axis=1), some) and np.all(f64(dx)[~some] == 0)


# ----------------------------------------------------------------------------- what the forward pass took


def forward_way(c):
    """(whether the product ran on pairs, whether the teacher's words were taken from its tiles) of a forward
    pass, by what it wrote into a workspace of ones: the pairs copy X's scales where their pitch is odd, and the
    words are listed behind the parts' statistics."""
    assert c.xs.stride(0) % 4
    ws = workspace(bq.loss_fp8_workspace(c.n, c.rows, c.cols), c.dev)
    c.forward(ws)
    parts, groups = -(-c.rows // 64), -(-c.cols // 128)
    lists = 256 + up(groups * up(c.n, 4) * 4) + up(parts * c.n * 8) + up(parts * c.n)
    wrote = [bool((ws[at:at + 4 * c.n] != 0xFF).any()) for at in (256, lists)]
    return tuple(wrote)


@pytest.mark.parametrize("n,rows,cols,k,pairs", [(2001, 900, 1024, 130, False), (2001, 3001, 4096, 130, True), (1999, 2950, 2064, 300, True)])
@pytest.mark.parametrize("scale", [1.0, -0.5])
def test_a_teachers_words_from_the_tiles(cuda, n, rows, cols, k, pairs, scale):
    """Single CTAs, and more tiles than pairs of them, so that a pair's second tile finds its words where the first
    has been: several words of a row in one part, all of them, and none; the last block of columns ragged."""
    def edit(c):
        c.ids[::3] = 64 + c.rng.integers(0, 64, c.ids[::3].shape)
        c.ids[2::5] = rows - 1 - c.rng.integers(0, 70, c.ids[2::5].shape)
        c.ids[1] = -1

    c = Head(cuda, n, rows, cols, scale=scale, k=k, teacher="bf16", bits=32, spare=0, edit=edit)
    assert forward_way(c) == (pairs, True)
    c.check_forward()


# ----------------------------------------------------------------------------- every word and token counts


def whole_head(dev, n, rows, cols, k=None, seed=60):
    """Logits that fp32 holds as they are, in [-1/2, 1/2]: codes of -1, 0 and 1, scales and the factor powers of two."""
    import torch

    rng = np.random.default_rng([seed, n, rows, cols])
    c = Head.__new__(Head)
    c.n, c.rows, c.cols, c.k, c.dev, c.rng = n, rows, cols, k, dev, rng
    x, w = rng.integers(-1, 2, (n, cols)), rng.integers(-1, 2, (rows, cols))
    groups = -(-cols // 128)
    xs = rng.choice([0.5, 1.0], (groups, n))
    ws = rng.choice([1.0, 2.0], (-(-rows // 128), groups))
    c.x64 = x * np.repeat(xs.T, 128, axis=1)[:, :cols]
    c.w64 = w * np.repeat(np.repeat(ws, 128, axis=0), 128, axis=1)[:rows, :cols]
    z = (c.x64.astype(np.float32) @ c.w64.astype(np.float32).T).astype(np.float64)  # (exact: halves below 2^18)
    c.scale = float(2.0 ** -np.ceil(np.log2(2 * np.abs(z).max())))
    c.logits = c.scale * z
    code = lambda v: torch.as_tensor(np.array([0xB8, 0, 0x38], np.uint8)[v + 1]).to(dev)  # noqa: E731
    c.x, c.xs = code(x), torch.as_tensor(xs.astype(np.float32)).to(dev)
    c.head = c.x, c.xs, code(w), torch.as_tensor(ws.astype(np.float32)).to(dev)
    if k is None:
        c.targets = np.where(rng.random(n) < 0.1, -1, rng.integers(0, rows, n))
        c.t, c.pairs = torch.as_tensor(c.targets).to(dev), O.class_pairs(c.targets, rows)
    else:
        ids, t = rng.integers(0, rows, (n, k)), rng.standard_normal((n, k)).astype(np.float32)
        c.t, c.z, c.pairs = torch.as_tensor(ids).to(dev), torch.as_tensor(t).to(dev), O.teacher_pairs(ids, t, c.scale, rows)
    return c


def sum_error(n, rows):
    """Relative, of a row's sum of exponentials of such logits.  A term: exp2 and its argument, at most 1.45, 2^-21;
    up to 66 additions in its part; each of the joins that it passes scales it (2^-21, and two additions): one for each 16
    parts or more, and nine by shuffles."""
    joins = -(-rows // 64) / 16 + 10
    return 2.0 ** -21 + 66 * E + joins * (2.0 ** -21 + 2 * E)


# single CTAs, whole tiles and tiles split; pairs with less and more than one tile each; rows and words ragged
@pytest.mark.parametrize("n,rows,cols,pairs", [(1, 1000, 512, False), (85, 8999, 144, False), (301, 4100, 1040, False), (333, 9000, 2880, True),
                                               (521, 1500, 2064, False), (801, 9001, 1040, True), (2001, 3001, 4096, True), (3001, 8193, 528, True)])
@pytest.mark.parametrize("k", [None, 130])
def test_every_word_counts(cuda, n, rows, cols, pairs, k):
    """A sum of exponentials is off by less than any word's share of it."""
    c = whole_head(cuda, n, rows, cols, k)
    assert forward_way(c)[0] == pairs
    by = sum_error(n, rows)
    loss, lse, logp = O.loss(c.logits, c.pairs)
    assert by < 0.5 * np.exp(c.logits - lse[:, None]).min()
    near(f64(c.lse), lse, by + 3 * E * np.abs(lse))
    ids, q, kept = c.pairs
    if k is None:
        near(f64(c.loss), loss, by + 4 * E * np.abs(loss))
    else:
        near(f64(c.logp), logp, by + 4 * E * np.abs(logp))
        # (each term by 2^-20: q and log q)
        near(f64(c.loss), loss, by + 2.0 ** -20 * (1 + np.abs(q * logp).sum(axis=1) + np.abs(q * np.log(q)).sum(axis=1)) + k * E)


@pytest.mark.parametrize("n,rows,cols", [(43, 9000, 1040), (126, 9000, 1040), (130, 129, 144), (700, 690, 272), (1300, 1290, 512)])
def test_every_target_reaches_the_gradients(cuda, n, rows, cols):
    """Each of the last words a target, and each token with one: there u is near -1, far above what a sum may
    be off by."""
    import torch

    c = Head(cuda, n, rows, cols, seed=61, edit=lambda c: c.targets.__setitem__(slice(None), rows - 1 - np.arange(n) % rows))
    c.forward().check_forward()
    g = (1 + c.rng.random(n)).astype(np.float32)
    dx, dw = empty(n, cols, cuda, torch.bfloat16)[0], empty(rows, cols, cuda, torch.bfloat16)[0]
    c.grad(torch.as_tensor(g).to(cuda), dx, dw)
    c.check_grads(g, dx, dw)
