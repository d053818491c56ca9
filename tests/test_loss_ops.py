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
            # at most 42 tokens: u as three E4M3 terms, off by 2^-12 of itself and 2^-25 of its 128 words' largest
            few = np.zeros_like(u)
            if self.n <= 42:
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


SIZES = [(1, 1, 16), (42, 1300, 160), (43, 1300, 160), (1, 130, 128), (2, 300, 144), (7, 256, 272), (33, 1000, 512), (128, 257, 128), (129, 640, 256),
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
    """More words than one piece of the vocabulary holds (256 MB of fp16), the last one short, against whole
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
