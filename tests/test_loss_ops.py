"""The losses over an FP8 head on the GPU against their formulas in fp64: cross entropy,
distillation from a teacher's top logits, and their gradients.

Tolerances: half a step relative to the result, that is half of the type's epsilon: e = 2^-24 for a rounding
to fp32 (epsilon 2^-23), h = 2^-11 to fp16 (2^-10), u = 2^-8 to bf16 (2^-7).

A logit is a sum over 128 products at a time in the tensor cores (each addition may truncate: 2^-23), then of
the groups in fp32: off by at most (cols + 4) 2^-23 A, A the sum of the magnitudes of its terms.  The
log-sum of logits that are off by d is off by d at most, plus the roundings of exp (2^-22 relative, and e
times the magnitude of its argument, which the sum weighs with the probabilities: at most 2^-24 max|z|), of the sum (rows e
at most) and of the result.  A loss adds the target's logit, d again.  The gradients' u = p - q is off by
p (2 d + 2^-21) from its logits, and by h |u| + 2^-25 2^-14 from its rounding; their operands X and W by h each, their sums
by 2^-23 a term, their result by 2^-8 of itself."""

import numpy as np
import pytest

import block_quant_gb300 as bq
from oracle import layer as L
from oracle import loss as O
from oracle.codecs import e4m3_encode

pytestmark = pytest.mark.gpu

E, H, U = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_quant_gb300 import build

    build.build()
    return bq.load()


# ----------------------------------------------------------------------------- helpers


def fp8_weight(rng, rows, cols, dev, size=0.5, pitch=0):
    import torch

    codes = e4m3_encode((rng.standard_normal((rows, cols)) * 60).astype(np.float32))
    scale = (np.exp(0.3 * rng.standard_normal((-(-rows // 128), -(-cols // 128)))) * size / 60).astype(np.float32)
    c = torch.full((rows, cols + pitch), 0x7F, dtype=torch.uint8, device=dev)  # NaN codes beside the rows
    c[:, :cols] = torch.as_tensor(codes).to(dev)
    return c[:, :cols], torch.as_tensor(scale).to(dev), L.decode_tiles(codes, scale)


def fp8_rows(rng, n, cols, dev, pitch=0, spare=0, towards=None):
    """FP8 rows; towards: rows that they lean to."""
    import torch

    x = rng.standard_normal((n, cols)) * np.exp(0.5 * rng.standard_normal((n, 1)))
    if towards is not None:
        x = x + 4 * rng.random((n, 1)) * towards / np.sqrt(np.mean(towards ** 2, axis=1, keepdims=True) + 1e-30)
    x = x / np.sqrt(cols)
    scale = np.maximum(L.row_scales(x), 1e-30).astype(np.float32)
    codes = e4m3_encode((x / L.spread_rows(scale, cols)).astype(np.float32))
    c = torch.full((n, cols + pitch), 0x7F, dtype=torch.uint8, device=dev)
    c[:, :cols] = torch.as_tensor(codes).to(dev)
    s = torch.full((scale.shape[0], n + spare), float("nan"), dtype=torch.float32, device=dev)
    s[:, :n] = torch.as_tensor(scale).to(dev)
    return c[:, :cols], s[:, :n], L.decode_rows(codes, scale)


def f64(t):
    return t.double().cpu().numpy()


def empty(n, c, dev, dtype, pitch=0, shift=0, fill=7.0):
    import torch

    flat = torch.full((n * (c + pitch) + shift,), fill, dtype=dtype, device=dev)
    return flat[shift:].view(n, c + pitch)[:, :c], flat


def outside_kept(m, flat, shift, fill=7.0):
    n, c = m.shape
    rest = flat[shift:].double().cpu().numpy().reshape(n, m.stride(0))[:, c:]
    return np.all(rest == fill) and np.all(flat[:shift].double().cpu().numpy() == fill)


def near(got, want, by):
    """|got - want| <= by everywhere; a NaN on either side is far."""
    off = np.abs(np.asarray(got) - want)
    bad = ~(off <= by)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, off / np.maximum(by, 1e-300), 0)), bad.shape)
        raise AssertionError(f"{bad.sum()} of {bad.size} too far; at {i}: {np.asarray(got)[i]!r}, want {want[i]!r} "
                             f"within {np.broadcast_to(by, bad.shape)[i]!r}")


def vectors(n, dev, count):
    import torch

    return [torch.full((n,), 5.0, dtype=torch.float32, device=dev) for _ in range(count)]


def workspace(size, dev, fill=0xFF):
    """A workspace that holds anything but for its first 256 bytes."""
    import torch

    ws = torch.full((size,), fill, dtype=torch.uint8, device=dev)
    ws[:256] = 0
    return ws


class Head:
    """Rows, weight, targets and their fp64 forms."""

    def __init__(self, dev, n, rows, cols, scale=1.0, k=None, teacher="fp32", bits=64, seed=0, pitch=0, spare=0, edit=None):
        import torch

        rng = np.random.default_rng([seed, n, rows, cols, k or 0])
        self.dev, self.n, self.rows, self.cols, self.scale, self.k, self.rng = dev, n, rows, cols, scale, k, rng
        self.w, self.ws_, self.w64 = fp8_weight(rng, rows, cols, dev, pitch=pitch)
        words = rng.integers(0, rows, n)
        self.x, self.xs, self.x64 = fp8_rows(rng, n, cols, dev, pitch, spare, self.w64[words])
        kind = torch.int64 if bits == 64 else torch.int32
        if k is None:
            self.targets = words.copy()
            gone = rng.random(n) < 0.15
            self.targets[gone] = rng.choice([-1, -100, rows, rows + 5, 2 ** 31 - 1], gone.sum())
            if edit:
                edit(self)
            self.pairs = O.class_pairs(self.targets, rows)
            self.t = torch.as_tensor(self.targets).to(kind).to(dev)
        else:
            self.ids = rng.integers(0, rows, (n, k))
            self.ids[:, 0] = words
            self.ids[rng.random((n, k)) < 0.1] = -1
            self.ids[rng.random((n, k)) < 0.05] = rows
            self.ids[rng.random(n) < 0.1] = -7
            z = rng.standard_normal((n, k)) * 3
            z[rng.random((n, k)) < 0.05] = -np.inf
            z[rng.random((n, k)) < 0.05] = -3.4028234e38 if teacher == "fp32" else -3.38e38
            self.z = torch.as_tensor(z.astype(np.float32)).to(torch.float32 if teacher == "fp32" else torch.bfloat16)
            if edit:
                edit(self)
            self.pairs = O.teacher_pairs(self.ids, self.z.double().numpy(), scale, rows)
            wide = torch.full((n, k + spare), 3, dtype=kind)
            wide[:, :k] = torch.as_tensor(self.ids)
            self.t = wide.to(dev)[:, :k]
            self.z = self.z.to(dev)
        self.logits, self.size = O.logits(self.x64, self.w64, scale)
        self.off = (cols + 4) * 2.0 ** -23 * self.size.max(axis=1)  # of a row's logits
        self.head = self.x, self.xs, self.w, self.ws_

    def forward(self, ws=None, stream=None):
        ws = workspace(bq.loss_fp8_workspace(self.n, self.rows, self.cols), self.dev) if ws is None else ws
        self.loss, self.lse = vectors(self.n, self.dev, 2)
        if self.k is None:
            bq.cross_entropy_fp8(*self.head, self.t, self.loss, self.lse, ws, scale=self.scale, stream=stream)
        else:
            self.logp, _ = empty(self.n, self.k, self.dev, self.loss.dtype)
            bq.distill_fp8(*self.head, self.t, self.z, self.loss, self.lse, self.logp, ws, scale=self.scale, stream=stream)
        bq.linear_check(ws, stream)
        return self

    def grad(self, dloss, dx, dw, accumulate=False, ws=None, stream=None):
        ws = workspace(bq.loss_fp8_grad_workspace(self.n, self.rows, self.cols), self.dev) if ws is None else ws
        if self.k is None:
            bq.cross_entropy_fp8_grad(*self.head, self.t, self.loss, self.lse, dloss, dx, dw, ws, scale=self.scale,
                                      accumulate=accumulate, stream=stream)
        else:
            bq.distill_fp8_grad(*self.head, self.t, self.z, self.lse, self.logp, dloss, dx, dw, ws, scale=self.scale,
                                accumulate=accumulate, stream=stream)
        bq.linear_check(ws, stream)

    def check_forward(self):
        loss, lse, logp = O.loss(self.logits, self.pairs)
        top = np.abs(self.logits).max(axis=1)
        sums = self.off + 2.0 ** -22 + (self.rows + 4) * E + 2 * E * top  # of a log-sum, absolutely
        near(f64(self.lse), lse, sums + E * np.abs(lse))
        ids, q, kept = self.pairs
        # a log-probability: its logit and the log-sum; near 0 relative to itself (the others' sum
        d = 2 * self.off + 2.0 ** -21 + 4 * E * top + (self.rows + 4) * E
        # is off by a factor of exp(2 off); each of its terms below 2^-126 counts as 0)
        by = d[:, None] * np.minimum(1.0, 1.5 * np.abs(logp)) + 2 * E * np.abs(logp) + self.rows * 2.0 ** -126
        if self.k is not None:
            got = f64(self.logp)
            assert np.all(got[~kept] == 0)
            near(got[kept], logp[kept], by[kept])
        by = np.where(kept, by, 0)
        # the sum over pairs; log q and q themselves by 2^-20 (the teacher's differences are rounded) and k terms
        terms = np.abs(q * np.log(np.where(q > 0, q, 1))) + np.abs(q * logp)
        extra = 0.0 if self.k is None else ((2.0 ** -20 + self.k * E) * (terms.sum(axis=1) + 1.0))
        near(f64(self.loss), loss, (q * by).sum(axis=1) + extra + E * np.abs(loss))
        return self

    def check_grads(self, dloss, dx, dw, old=None):
        want_x, want_w, size_x, size_w = O.grads(self.x64, self.w64, self.logits, self.pairs, dloss, self.scale)
        some = self.pairs[2].any(axis=1)
        g = np.where(some, np.abs(self.scale * dloss), 0.0)
        p = np.exp(self.logits - O.log_sum(self.logits)[:, None])
        d = 2 * self.off + 2.0 ** -20 + 8 * E * np.abs(self.logits).max(axis=1) + 2 * (self.rows + 4) * E
        u = np.abs(O.dlogits(self.logits, self.pairs))
        # u beside its logits' error (a class's own is 1 - p, precise where p is near 1), q, and fp16's smallest
        # step, 2^-24 at 2^14 u
        if self.k is None:
            du = 1.5 * d[:, None] * u
        else:
            du = d[:, None] * (p + u) + 2.0 ** -19 * O.weights_of(self.pairs, self.rows)
        du = g[:, None] * (du + 2.0 ** -39)
        if dx is not None:
            # few tokens' u as three E4M3 terms, off by 2^-12 of itself and 2^-25 of its 128 words' largest
            few = np.zeros_like(u)
            for j in range(0, self.rows, 128):
                few[:, j:j + 128] = 2.0 ** -25 * u[:, j:j + 128].max(axis=1, keepdims=True)
            by = (du + g[:, None] * few) @ np.abs(self.w64) + (2.2 * H + (self.rows + 8) * 2.0 ** -23) * size_x
            near(f64(dx), want_x, by + U * 1.001 * np.abs(want_x) + U * by)
            assert np.all(f64(dx)[~some] == 0)
        if dw is not None:
            by = du.T @ np.abs(self.x64) + (2.2 * H + (self.n + 8) * 2.0 ** -23) * size_w
            # X * dloss below 2^-24 of its largest by fp16's smallest step
            by = by + 2.0 ** -38 * (u.sum(axis=0)[:, None]
                                    * (g[:, None] * np.abs(self.x64)).max(initial=0.0))
            want = want_w if old is None else want_w + old
            near(f64(dw), want, by + U * 1.001 * np.abs(want) + U * by)


# (words enough to be taken from the tiles of the product: of CTA pairs and of single CTAs, lists of more and fewer words a row)
TEACHERS = [(2000, 900, 1024, 130), (1500, 1300, 2064, 257), (4000, 130, 528, 100), (1000, 2500, 4112, 70), (3000, 400, 512, 1024)]


@pytest.mark.parametrize("n,rows,cols,k", TEACHERS)
@pytest.mark.parametrize("scale", [1.0, -0.5])
def test_distill_of_many_words(cuda, n, rows, cols, k, scale):
    """Several words of a row in one part of the vocabulary, all of them, and none."""
    def edit(c):
        c.ids[::3] = 64 + c.rng.integers(0, 64, c.ids[::3].shape)
        c.ids[1] = -1

    Head(cuda, n, rows, cols, scale=scale, k=k, teacher="fp32", bits=32, spare=2, edit=edit).forward().check_forward()


SIZES = [(1, 1, 16), (42, 1300, 160), (43, 1300, 160), (85, 9000, 144), (1, 130, 128), (2, 300, 144), (7, 256, 272), (33, 1000, 512), (128, 257, 128), (129, 640, 256),
         (200, 2049, 400), (300, 4100, 1040), (520, 1500, 2064)]


@pytest.mark.parametrize("n,rows,cols", SIZES)
@pytest.mark.parametrize("bits", [32, 64])
def test_cross_entropy(cuda, n, rows, cols, bits):
    Head(cuda, n, rows, cols, scale=1.0 if bits == 64 else 0.7, bits=bits).forward().check_forward()


@pytest.mark.parametrize("n,rows,cols", SIZES)
@pytest.mark.parametrize("k,teacher", [(1, "fp32"), (5, "bf16"), (67, "fp32")])
def test_distill(cuda, n, rows, cols, k, teacher):
    Head(cuda, n, rows, cols, scale=0.5, k=k, teacher=teacher, bits=32 if k == 5 else 64).forward().check_forward()


@pytest.mark.parametrize("n,rows,cols", SIZES)
@pytest.mark.parametrize("k", [None, 9])
def test_gradients(cuda, n, rows, cols, k):
    import torch

    c = Head(cuda, n, rows, cols, scale=0.8, k=k, seed=1).forward()
    g = c.rng.standard_normal(n).astype(np.float32) / n
    dx, fx = empty(n, cols, cuda, torch.bfloat16)
    dw, fw = empty(rows, cols, cuda, torch.bfloat16)
    c.grad(torch.as_tensor(g).to(cuda), dx, dw)
    c.check_grads(g, dx, dw)


@pytest.mark.parametrize("n,rows,cols", [(2500, 300, 2000), (3000, 700, 4112), (260, 40000, 528)])
def test_gradients_of_many_tiles(cuda, n, rows, cols):
    """More tiles of dx than pairs of CTAs, and few tiles whose sums are shared out."""
    test_gradients(cuda, n, rows, cols, None)


def test_gradients_in_pieces(cuda):
    """More words than one piece of the vocabulary holds (512 MB of fp16), the last one short, against whole
    sums on the GPU in fp64."""
    import torch

    n, rows, cols = 9000, 3 * 14848 + 129, 128
    c = Head.__new__(Head)
    gen = torch.Generator(device=cuda).manual_seed(3)
    codes = torch.randint(0, 256, (rows, cols), generator=gen, device=cuda, dtype=torch.int32)
    codes = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes).to(torch.uint8)
    w_scale = (0.5 + torch.rand(-(-rows // 128), 1, generator=gen, device=cuda)) * 2e-4
    x = torch.randint(0, 256, (n, cols), generator=gen, device=cuda, dtype=torch.int32)
    x = torch.where((x & 0x7F) == 0x7F, x - 1, x).to(torch.uint8)
    x_scale = (0.5 + torch.rand(1, n, generator=gen, device=cuda)) * 1e-3
    y = torch.randint(0, rows, (n,), generator=gen, device=cuda)
    y[::7] = -1
    w64 = codes.view(torch.float8_e4m3fn).double() * w_scale.double().repeat_interleave(128, 0)[:rows]
    x64 = x.view(torch.float8_e4m3fn).double() * x_scale.double().t()
    c.n, c.rows, c.cols, c.k, c.scale, c.dev = n, rows, cols, None, 1.0, cuda
    c.head, c.t = (x, x_scale, codes, w_scale), y
    c.forward()
    g = torch.randn(n, generator=gen, device=cuda) / n
    dx, _ = empty(n, cols, cuda, torch.bfloat16)
    dw, _ = empty(rows, cols, cuda, torch.bfloat16)
    c.grad(g, dx, dw)
    z = x64 @ w64.t()
    lse = torch.logsumexp(z, 1)
    seen = y >= 0
    at = z.gather(1, y.clamp(min=0)[:, None])[:, 0]
    assert float((c.lse.double() - lse).abs().max()) < 1e-5 and float((c.loss.double() - torch.where(seen, lse - at, 0)).abs().max()) < 1e-5
    u = torch.exp(z.sub_(lse[:, None]))
    u[seen, y[seen]] -= 1
    u *= torch.where(seen, g.double(), 0)[:, None]
    want_x, want_w = u @ w64, u.t() @ x64
    # roundings of u, X (2^-11 each) and the result (2^-8), random in sign: far below in the norm
    assert float((dx.double() - want_x).norm() / want_x.norm()) < 2 ** -8
    assert float((dw.double() - want_w).norm() / want_w.norm()) < 2 ** -8
    size_x, size_w = u.abs() @ w64.abs(), u.abs().t() @ x64.abs()
    assert bool(((dx.double() - want_x).abs() <= U * 1.01 * want_x.abs() + 2.5 * H * size_x).all())
    assert bool(((dw.double() - want_w).abs() <= U * 1.01 * want_w.abs() + 2.5 * H * size_w).all())


# ----------------------------------------------------------------------------- layouts


@pytest.mark.parametrize("k,teacher", [(None, None), (6, "bf16")])
@pytest.mark.parametrize("n,rows,cols", [(5, 300, 144), (150, 1000, 272), (400, 2500, 512)])
def test_pitches_and_alignments(cuda, n, rows, cols, k, teacher):
    """Rows with spare columns (NaN codes, NaN scales), ids and logits inside wider matrices, outputs at odd
    addresses whose surroundings stay as they were."""
    import torch

    for pitch, spare, shift, out_pitch in ((16, 3, 1, 5), (32, 1, 2, 2), (0, 4, 4, 4), (0, 0, 0, 24)):
        c = Head(cuda, n, rows, cols, k=k, teacher=teacher, pitch=pitch, spare=spare, seed=pitch)
        c.forward()
        c.check_forward()
        g = c.rng.standard_normal(n).astype(np.float32)
        dx, fx = empty(n, cols, cuda, torch.bfloat16, out_pitch, shift)
        dw, fw = empty(rows, cols, cuda, torch.bfloat16, out_pitch, shift)
        c.grad(torch.as_tensor(g).to(cuda), dx, dw)
        c.check_grads(g, dx, dw)
        assert outside_kept(dx, fx, shift) and outside_kept(dw, fw, shift)


@pytest.mark.parametrize("n,rows,cols", [(3, 400, 128), (140, 900, 256), (1500, 500, 256)])
def test_one_output_and_accumulation(cuda, n, rows, cols):
    import torch

    c = Head(cuda, n, rows, cols, seed=2).forward()
    g = torch.as_tensor(c.rng.standard_normal(n).astype(np.float32)).to(cuda)
    dx, dw = empty(n, cols, cuda, torch.bfloat16)[0], empty(rows, cols, cuda, torch.bfloat16)[0]
    c.grad(g, dx, dw)
    x, w = torch.empty_like(dx), torch.empty_like(dw)
    c.grad(g, x, None)
    c.grad(g, None, w)
    assert torch.equal(x, dx) and torch.equal(w, dw)
    old = torch.as_tensor(c.rng.standard_normal((rows, cols)).astype(np.float32)).to(cuda).bfloat16()
    w.copy_(old)
    c.grad(g, x, w, accumulate=True)
    assert torch.equal(x, dx)  # never added to
    c.check_grads(f64(g), x, w, old=f64(old))


def test_no_tokens(cuda):
    import torch

    c = Head(cuda, 1, 30, 32)
    none = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=cuda)  # noqa: E731
    head = none(0, 32, t=torch.uint8), none(1, 0), c.w, c.ws_
    dw = torch.full((30, 32), 3.0, dtype=torch.bfloat16, device=cuda)
    ws, wg = workspace(bq.loss_fp8_workspace(0, 30, 32), cuda), workspace(bq.loss_fp8_grad_workspace(0, 30, 32), cuda)
    bq.cross_entropy_fp8(*head, none(0, t=torch.int64), none(0), none(0), ws)
    bq.cross_entropy_fp8_grad(*head, none(0, t=torch.int64), none(0), none(0), none(0), none(0, 32, t=torch.bfloat16), dw, wg,
                              accumulate=True)
    assert bool((dw == 3).all())
    bq.distill_fp8_grad(*head, none(0, 4, t=torch.int32), none(0, 4), none(0), none(0, 4), none(0), None, dw, wg)
    assert not dw.any()


# ----------------------------------------------------------------------------- masks, infinities, sure predictions


@pytest.mark.parametrize("n", [6, 150, 600])
@pytest.mark.parametrize("k", [None, 4])
def test_rows_without_a_target_hold_anything(cuda, n, k):
    """NaN codes, NaN and infinite scales, dloss and logits in rows without a target reach nothing but those
    rows' own log-sums."""
    import torch

    rows, cols = 700, 256

    def none(c):
        if k is None:
            c.targets[1::3] = -1
        else:
            c.ids[1::3] = -1
            c.z[1::3] = float("nan")
            c.z[2, :] = -np.inf  # every weight 0: no target either
            c.z[0, 1] = -np.inf

    c = Head(cuda, n, rows, cols, k=k, seed=5, edit=none)
    some = c.pairs[2].any(axis=1)
    g = c.rng.standard_normal(n).astype(np.float32)
    out = []
    for broken in (False, True):
        if broken:
            c.x[1::3] = 0x7F
            c.xs[:, 1::3] = float("nan")
            c.xs[0, 4::6] = float("inf")
            g[~some] = np.where(np.arange((~some).sum()) % 2, np.nan, np.inf)
        c.forward()
        dx, dw = empty(n, cols, cuda, torch.bfloat16)[0], empty(rows, cols, cuda, torch.bfloat16)[0]
        c.grad(torch.as_tensor(g).to(cuda), dx, dw)
        assert np.all(f64(c.loss)[~some] == 0) and np.all(f64(dx)[~some] == 0)
        out.append([f64(t) for t in (c.loss, c.lse[torch.as_tensor(some).to(cuda)], dx, dw)])
    assert all(np.array_equal(a, b) for a, b in zip(*out))
    c.check_grads(np.where(some, g, 0), dx, dw)


@pytest.mark.parametrize("n", [4, 200])
def test_a_row_of_nan_stays_alone(cuda, n):
    import torch

    rows, cols = 500, 144
    c = Head(cuda, n, rows, cols, seed=6, edit=lambda c: c.targets.__setitem__(slice(None), np.arange(n) % rows))
    c.x[2, 5] = 0x7F
    c.forward()
    bad = np.arange(n) == 2
    for t in (c.loss, c.lse):
        assert np.array_equal(np.isnan(f64(t)), bad)
    dx = empty(n, cols, cuda, torch.bfloat16)[0]
    dw = empty(rows, cols, cuda, torch.bfloat16)[0]
    c.grad(torch.ones(n, device=cuda), dx, dw)
    assert np.array_equal(np.isnan(f64(dx)).any(axis=1), bad) and np.isnan(f64(dx)[2]).all()
    assert np.isnan(f64(dw)).all()  # a sum over tokens, that one among them


def test_a_weight_of_nan_reaches_every_row_with_a_target(cuda):
    import torch

    for n in (3, 300):
        c = Head(cuda, n, 400, 128, seed=7, edit=lambda c: c.targets.__setitem__(0, -1))
        c.w[133, 7] = 0xFF
        c.forward()
        some = c.pairs[2].any(axis=1)
        assert np.array_equal(np.isnan(f64(c.loss)), some)
        dx = empty(n, 128, cuda, torch.bfloat16)[0]
        c.grad(torch.ones(n, device=cuda), dx, None)
        assert np.array_equal(np.isnan(f64(dx)).any(axis=1), some) and np.all(f64(dx)[~some] == 0)


def test_sure_predictions_and_ties(cuda):
    """Losses far below what fp32 holds beside 1, and equal logits (the same words several times)."""
    import torch

    n, rows, cols = 40, 900, 128

    c = Head(cuda, n, rows, cols, scale=6.0, seed=8)
    c.forward().check_forward()
    loss, _, _ = O.loss(c.logits, c.pairs)
    assert np.sum((loss > 0) & (loss < 1e-6)) >= 3
    g = c.rng.standard_normal(n).astype(np.float32)
    dx, dw = empty(n, cols, cuda, torch.bfloat16)[0], empty(rows, cols, cuda, torch.bfloat16)[0]
    c.grad(torch.as_tensor(g).to(cuda), dx, dw)
    c.check_grads(g, dx, dw)
    # every word the same: each has the probability 1 / rows, whichever the target
    c.w[:] = c.w[:1].clone()
    c.ws_[:] = 0.01
    c.forward()
    some = c.pairs[2].any(axis=1)
    # (exact but for the log, the sum of 899 ones and the difference to a logit read apart: 6e-8 of each)
    z = np.abs(f64(c.lse)) + 1
    assert np.all(np.abs(f64(c.loss) - np.log(rows))[some] <= 1e-5 * z[some])


@pytest.mark.parametrize("n", [3, 70])
def test_teachers(cuda, n):
    """One id many times, the most pairs, logits of the type's lowest value and infinities beside others."""
    import torch

    rows, cols, k = 600, 128, 1024

    def edit(c):
        c.ids[0] = 17
        c.ids[1, :] = np.arange(k) % 9
        c.z[1, ::2] = torch.finfo(torch.float32).min
        c.z[2] = torch.finfo(torch.float32).min
        c.ids[2] = np.arange(k) % rows

    c = Head(cuda, n, rows, cols, scale=0.5, k=k, seed=9, edit=edit)
    c.forward().check_forward()
    g = c.rng.standard_normal(n).astype(np.float32)
    dx, dw = empty(n, cols, cuda, torch.bfloat16)[0], empty(rows, cols, cuda, torch.bfloat16)[0]
    c.grad(torch.as_tensor(g).to(cuda), dx, dw)
    c.check_grads(g, dx, dw)


def test_one_pair_of_weight_one_is_a_class(cuda):
    """A teacher that knows one word says what a class says."""
    import torch

    n, rows, cols = 130, 800, 256
    a = Head(cuda, n, rows, cols, seed=10).forward()
    g = torch.as_tensor(a.rng.standard_normal(n).astype(np.float32)).to(cuda)
    dx, dw = empty(n, cols, cuda, torch.bfloat16)[0], empty(rows, cols, cuda, torch.bfloat16)[0]
    a.grad(g, dx, dw)
    want = [f64(t) for t in (a.loss, a.lse, dx, dw)]
    a.k, a.t, a.z = 1, a.t[:, None].contiguous(), torch.zeros(n, 1, device=cuda)
    a.forward()
    a.grad(g, dx, dw)
    for got, w in zip((a.loss, a.lse, dx, dw), want):
        # (the target's logit is read by the same code; q is 1 and log q 0)
        near(f64(got), w, 2 * U * np.abs(w) + 1e-30 if got.dtype == torch.bfloat16 else 4 * E * np.abs(w))


@pytest.mark.parametrize("n", [5, 90, 300])
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60])
def test_sizes_of_gradients(cuda, n, size):
    """Gradients far from 1, and rows whose own differ by 2^16: fp16 operands by common powers of two."""
    import torch

    rows, cols = 700, 256
    c = Head(cuda, n, rows, cols, seed=14).forward()
    g = (c.rng.standard_normal(n) * size * 2.0 ** -c.rng.integers(0, 17, n)).astype(np.float32)
    dx, dw = empty(n, cols, cuda, torch.bfloat16)[0], empty(rows, cols, cuda, torch.bfloat16)[0]
    c.grad(torch.as_tensor(g).to(cuda), dx, dw)
    c.check_grads(g, dx, dw)


def test_gradients_accumulated_over_micro_batches(cuda):
    """The weight's gradient summed over calls on the same buffers, each before the last has been read: the bits of
    calls with a pause between."""
    import torch

    for n, rows, cols, k in ((520, 900, 256, None), (260, 3000, 512, 3)):
        cs = [Head(cuda, n, rows, cols, k=k, seed=30 + i).forward() for i in range(3)]
        ws = workspace(bq.loss_fp8_grad_workspace(n, rows, cols), cuda)
        g = torch.linspace(0.5, 1, n, device=cuda) / n
        x, xs = torch.empty_like(cs[0].x.contiguous()), torch.empty_like(cs[0].xs.contiguous())
        sums = []
        for pause in (True, False):
            dw, dxs = torch.zeros(rows, cols, dtype=torch.bfloat16, device=cuda), []
            for turn in range(6):
                c = cs[turn % 3]
                x.copy_(c.x), xs.copy_(c.xs)  # the same memory for every micro-batch
                head, c.head = c.head, (x, xs, c.w, c.ws_)
                dx = torch.empty(n, cols, dtype=torch.bfloat16, device=cuda)
                if k is None:
                    bq.cross_entropy_fp8_grad(*c.head, c.t, c.loss, c.lse, g, dx, dw, ws, accumulate=True)
                else:
                    bq.distill_fp8_grad(*c.head, c.t, c.z, c.lse, c.logp, g, dx, dw, ws, accumulate=True)
                c.head = head
                dxs.append(dx)
                if pause:
                    torch.cuda.synchronize()
            sums.append([dw, *dxs])
        assert all(torch.equal(a, b) for a, b in zip(*sums))


# ----------------------------------------------------------------------------- derivatives of the kernels' own losses


@pytest.mark.parametrize("k", [None, 8])
def test_gradients_match_differences_of_the_losses(cuda, k):
    """The losses' derivative along the factor of the logits is sum(dx * x) / scale, and sum(dw * w) / scale."""
    import torch

    n, rows, cols, d = 300, 3000, 512, 2.0 ** -6
    c = Head(cuda, n, rows, cols, k=k, seed=11)
    if k:
        c.z.zero_()  # (the teacher's softmax has the factor too: q the same for all)
        c.pairs = O.teacher_pairs(c.ids, np.zeros((n, k)), 1.0, rows)
    g = torch.rand(n, device=cuda) / n
    totals = {}
    for f in (1 - d, 1 + d, 1 - 2 * d, 1 + 2 * d, 1.0):
        c.scale = f
        c.forward()
        totals[f] = float((c.loss.double() * g.double()).sum())
    dx, dw = empty(n, cols, cuda, torch.bfloat16)[0], empty(rows, cols, cuda, torch.bfloat16)[0]
    c.grad(g, dx, dw)
    slope = (8 * (totals[1 + d] - totals[1 - d]) - (totals[1 + 2 * d] - totals[1 - 2 * d])) / (12 * d)
    by_x, by_w = float((f64(dx) * c.x64).sum()), float((f64(dw) * c.w64).sum())
    # the differences are off by their fifth derivative's d^4 / 30 and the losses' 1e-6 / d; the sums by
    # the roundings of dx and dw, 2^-9 of each term at random
    for got, terms in ((by_x, f64(dx) * c.x64), (by_w, f64(dw) * c.w64)):
        assert abs(got - slope) <= 2e-4 * abs(slope) + 1e-4 + 6 * U * np.sqrt(np.sum(terms ** 2))


# ----------------------------------------------------------------------------- streams, graphs, workspaces, offsets


@pytest.mark.parametrize("k", [None, 5])
def test_one_workspace_another_stream_and_graphs(cuda, k):
    """Sizes and inputs in turn on one workspace, on a stream of its own, and in two captured graphs that share
    it, replayed on new inputs: the bits of calls with workspaces of their own."""
    import torch

    sizes = [(2, 900, 144), (50, 2000, 256), (301, 1500, 512), (702, 700, 272), (1101, 3000, 256)]
    cases = [[Head(cuda, *s, k=k, seed=20 + i) for i in range(2)] for s in sizes]
    need = max(max(bq.loss_fp8_workspace(*s), bq.loss_fp8_grad_workspace(*s)) for s in sizes)
    shared = workspace(need, cuda)

    def buffers(c):
        new = lambda *s, t=torch.float32: torch.full(s, 9.0, dtype=t, device=cuda)  # noqa: E731
        b = dict(loss=new(c.n), lse=new(c.n), dx=new(c.n, c.cols, t=torch.bfloat16), dw=new(c.rows, c.cols, t=torch.bfloat16),
                 g=torch.linspace(-1, 1, c.n, device=cuda))
        if k:
            b["logp"] = new(c.n, k)
        return b

    def step(c, b, ws):
        if k is None:
            bq.cross_entropy_fp8(*c.head, c.t, b["loss"], b["lse"], ws)
            bq.cross_entropy_fp8_grad(*c.head, c.t, b["loss"], b["lse"], b["g"], b["dx"], b["dw"], ws)
        else:
            bq.distill_fp8(*c.head, c.t, c.z, b["loss"], b["lse"], b["logp"], ws)
            bq.distill_fp8_grad(*c.head, c.t, c.z, b["lse"], b["logp"], b["g"], b["dx"], b["dw"], ws)

    want = {}
    for i, pair in enumerate(cases):
        for j, c in enumerate(pair):
            b = buffers(c)
            step(c, b, workspace(need, cuda, fill=0x3C))
            want[i, j] = {name: t.clone() for name, t in b.items()}
    same = lambda b, w: all(torch.equal(b[name], w[name]) for name in w)  # noqa: E731
    for _ in range(3):
        for i, pair in enumerate(cases):
            for j, c in enumerate(pair):
                b = buffers(c)
                step(c, b, shared)
                assert same(b, want[i, j]), (i, j)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i, pair in enumerate(cases):
            b = buffers(pair[0])
            step(pair[0], b, shared)
            assert same(b, want[i, 0])
    side.synchronize()

    graphs = []
    for i in (1, 3):  # (their inputs are copied in before each replay)
        c, b = cases[i][0], buffers(cases[i][0])
        held = [t.clone() for t in (*c.head, c.t)] + ([c.z.clone()] if k else [])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(c, b, shared)
        graphs.append((i, graph, b, held))
    for turn in range(3):
        for i, graph, b, held in graphs:
            j = (turn + i) % 2
            c, src = cases[i][0], cases[i][j]
            fresh = held if j == 0 else [*src.head, src.t] + ([src.z] if k else [])
            for to, t in zip([*c.head, c.t] + ([c.z] if k else []), fresh):
                to.copy_(t)
            graph.replay()
            torch.cuda.synchronize()
            assert same(b, want[i, j]), (turn, i)
    bq.linear_check(shared)


def test_offsets_past_32_bits(cuda):
    """A head of more than 2^31 codes, whose gradient has more than 2^32 bytes: targets among its last words."""
    import torch

    rows, cols, n = 263000, 8192, 5
    assert rows * cols > 2 ** 31
    gen = torch.Generator(device=cuda).manual_seed(1)
    w = torch.randint(0, 0x58, (rows, cols), generator=gen, device=cuda, dtype=torch.uint8)
    w[-3000:] |= 0x80
    ws_ = torch.full((-(-rows // 128), cols // 128), 2.0 ** -9, device=cuda)
    x = torch.randint(0, 0x50, (n, cols), generator=gen, device=cuda, dtype=torch.uint8)
    xs = torch.full((cols // 128, n), 2.0 ** -10, device=cuda)
    y = torch.tensor([rows - 1, rows - 2999, 0, -1, rows], device=cuda)
    loss, lse, g = torch.empty(n, device=cuda), torch.empty(n, device=cuda), torch.tensor([1.0, -2.0, 0.5, 3.0, 1.0], device=cuda)
    bq.cross_entropy_fp8(x, xs, w, ws_, y, loss, lse, workspace(bq.loss_fp8_workspace(n, rows, cols), cuda))
    dx = torch.empty(n, cols, dtype=torch.bfloat16, device=cuda)
    dw = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=cuda)
    bq.cross_entropy_fp8_grad(x, xs, w, ws_, y, loss, lse, g, dx, dw, workspace(bq.loss_fp8_grad_workspace(n, rows, cols), cuda))
    x64 = x.view(torch.float8_e4m3fn).double() * 2.0 ** -10
    z = torch.cat([x64 @ (w[i:i + 20000].view(torch.float8_e4m3fn).double() * 2.0 ** -9).t() for i in range(0, rows, 20000)], 1)
    want = torch.logsumexp(z, 1)
    assert float((lse.double() - want).abs().max()) < 1e-5
    seen = [0, 1, 2]
    for t in seen:
        assert abs(float(loss[t]) - float(want[t] - z[t, y[t]])) < 1e-5
    u = torch.exp(z - want[:, None])
    for t in seen:
        u[t, y[t]] -= 1
    u *= torch.where((y >= 0) & (y < rows), g, 0).double()[:, None]
    for part in (slice(0, 300), slice(rows - 3100, rows)):
        ref = u[:, part].t() @ x64
        size = u[:, part].abs().t() @ x64.abs()
        assert bool(((dw[part].double() - ref).abs() <= U * 1.01 * ref.abs() + 2.5 * H * size).all())
    ref = sum(u[:, i:i + 20000] @ (w[i:i + 20000].view(torch.float8_e4m3fn).double() * 2.0 ** -9) for i in range(0, rows, 20000))
    size = sum(u[:, i:i + 20000].abs() @ (w[i:i + 20000].view(torch.float8_e4m3fn).double().abs() * 2.0 ** -9)
               for i in range(0, rows, 20000))
    assert bool(((dx.double() - ref).abs() <= U * 1.01 * ref.abs() + 2.5 * H * size).all())
    assert not dx[3:].any()
    assert bool(torch.isfinite(dw.view(torch.int16)[::1000].view(torch.bfloat16)).all())


# ----------------------------------------------------------------------------- as a model uses them


@pytest.mark.parametrize("k", [None, 6])
def test_the_example_models_head(cuda, k):
    """The last norm's rows, the loss and its gradients as a training step runs them, against fp64 on the same
    FP8 rows and weights."""
    import os
    import sys

    import torch

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from fp8_lm import Model

    vocab, width, n = 900, 256, 300
    m = Model(vocab, width, 256, 1, n, cuda, seed=3)
    ids = torch.randint(0, vocab, (n,), device=cuda)
    rows, _ = m.encode(ids)
    c = Head.__new__(Head)
    codes, scales = m.weight("head")
    c.x64, c.w64 = L.decode_rows(rows[0].cpu().numpy(), rows[1].cpu().numpy()), L.decode_tiles(codes.cpu().numpy(), scales.cpu().numpy())
    c.n, c.rows, c.cols, c.k, c.scale, c.dev = n, vocab, width, k, 1.0, cuda
    c.logits, c.size = O.logits(c.x64, c.w64, 1.0)
    c.off = (width + 4) * 2.0 ** -23 * c.size.max(axis=1)
    rng = np.random.default_rng(0)
    g = rng.random(n).astype(np.float32) / n
    dloss = torch.as_tensor(g).to(cuda)
    if k is None:
        y = rng.integers(-1, vocab, n)
        c.pairs = O.class_pairs(y, vocab)
        loss, dx = m.cross_entropy(rows, torch.as_tensor(y).to(cuda), dloss)
    else:
        y, z = rng.integers(0, vocab, (n, k)), rng.standard_normal((n, k)).astype(np.float32)
        c.pairs = O.teacher_pairs(y, z, 1.0, vocab)
        loss, dx = m.distill(rows, torch.as_tensor(y).to(cuda), torch.as_tensor(z).to(cuda), dloss)
    want, lse, c_logp = O.loss(c.logits, c.pairs)
    near(f64(loss), want, 2e-5 * (1 + np.abs(want)))
    c.check_grads(g, dx, m.grads["head"])
    m.step(ids, torch.as_tensor(y).to(cuda), 1e-3, 1e-4, teacher=None if k is None else torch.as_tensor(z).to(cuda))
    m.check()
