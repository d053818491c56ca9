"""The layer operators on the GPU against their formulas in fp64: embedding lookup
and gradient, root-mean-square norm with FP8 rows and its gradients, FP8
projections and theirs.

Tolerances: u = 2^-8 bounds a rounding to bf16 relative to its result, e = 2^-24 one
to fp32.  A sum of k fp32 terms is off by at most k e times the sum of their
magnitudes; a tensor-core sum of k products by k 2^-23 times it (its additions may
truncate)."""

import numpy as np
import pytest

import block_quant_gb300 as bq
from oracle import layer as L
from oracle.codecs import bf16_bits_to_f32, e4m3_decode, e4m3_encode

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_quant_gb300 import build

    build.build()
    return bq.load()


# ----------------------------------------------------------------------------- helpers


def bf16(x, dev, pitch=0, shift=0):
    """A bf16 matrix (or vector) on the GPU with `pitch` spare columns, starting
    `shift` elements past an aligned address, and its values in fp64."""
    import torch

    x = torch.as_tensor(np.asarray(x, np.float32)).bfloat16()
    want = x.double().numpy()
    if x.dim() == 1:
        flat = torch.full((x.shape[0] + shift,), 7.0, dtype=torch.bfloat16, device=dev)
        flat[shift:] = x.to(dev)
        return flat[shift:], want
    n, c = x.shape
    flat = torch.full((n * (c + pitch) + shift,), 7.0, dtype=torch.bfloat16, device=dev)
    m = flat[shift:].view(n, c + pitch)[:, :c]
    m.copy_(x.to(dev))
    return m, want


def empty(n, c, dev, dtype, pitch=0, shift=0, fill=7.0):
    """(matrix, the allocation it lies in) with every value `fill`."""
    import torch

    flat = torch.full((n * (c + pitch) + shift,), fill, dtype=dtype, device=dev)
    return flat[shift:].view(n, c + pitch)[:, :c], flat


def f64(t):
    return t.double().cpu().numpy()


def outside_kept(m, flat, shift, fill=7.0):
    """The spare columns around a strided output still hold what they held."""
    n, c = m.shape
    ld = m.stride(0)
    rest = flat[shift:].double().cpu().numpy().reshape(n, ld)[:, c:]
    return np.all(rest == fill) and np.all(flat[:shift].double().cpu().numpy() == fill)


def fp8_weight(rng, rows, cols, dev):
    """Codes and tile scales of a random weight, and its values in fp64."""
    import torch

    codes = e4m3_encode((rng.standard_normal((rows, cols)) * 60).astype(np.float32))
    scale = (np.exp(rng.standard_normal((-(-rows // 128), -(-cols // 128)))) * 1e-3).astype(np.float32)
    return (torch.as_tensor(codes).to(dev), torch.as_tensor(scale).to(dev), L.decode_tiles(codes, scale))


def fp8_rows(rng, n, cols, dev, pitch=0, spare=0):
    import torch

    codes = e4m3_encode((rng.standard_normal((n, cols)) * 60).astype(np.float32))
    scale = np.exp(rng.standard_normal((-(-cols // 128), n))).astype(np.float32)
    c = torch.full((n, cols + pitch), 0x7F, dtype=torch.uint8, device=dev)  # NaN codes beside the rows
    c[:, :cols] = torch.as_tensor(codes).to(dev)
    s = torch.full((scale.shape[0], n + spare), float("nan"), dtype=torch.float32, device=dev)
    s[:, :n] = torch.as_tensor(scale).to(dev)
    return c[:, :cols], s[:, :n], L.decode_rows(codes, scale)


def check_codes(codes, scale, y, slack):
    """Codes and scales of fp64 rows y whose fp32 value is off by at most slack |y|."""
    got_s, got = f64(scale), e4m3_decode(codes.cpu().view(__import__("torch").uint8).numpy()).astype(np.float64)
    want_s = L.row_scales(y)
    assert np.all(np.abs(got_s - want_s) <= (slack + 4 * E) * want_s)
    s = L.spread_rows(got_s, y.shape[1])
    # E4M3: four significant bits (half a step is 2^-4 of the value), subnormal step 2^-9
    assert np.all(np.abs(got * s - y) <= 2.0 ** -4 * np.abs(got) * s * 1.001 + 2.0 ** -10 * s * 1.001 + slack * np.abs(y))


# ----------------------------------------------------------------------------- embedding


@pytest.mark.parametrize("cols,pitch,shift", [(8, 0, 0), (128, 8, 0), (2880, 0, 0), (1032, 0, 0), (131, 0, 0), (256, 3, 0), (264, 0, 1), (1, 0, 0)])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("bits", [32, 64])
def test_embed(cuda, cols, pitch, shift, kind, bits):
    import torch

    rng = np.random.default_rng(cols + bits)
    rows, n = 300, 41
    ids = rng.integers(-3, rows + 3, n)
    ids[:3] = [-1, rows, rows - 1]
    if bits == 64:
        ids[3] = 2 ** 40
    tid = torch.as_tensor(ids.astype(np.int64 if bits == 64 else np.int32)).to(cuda)
    out, flat = empty(n, cols, cuda, torch.bfloat16, pitch, shift)
    if kind == "fp8":
        t, ts, want = fp8_weight(rng, rows, cols, cuda)
        bq.embed(t, tid, out, scale=0.37, table_scale=ts)
    else:
        t, want = bf16(rng.standard_normal((rows, cols)), cuda, pitch, shift)
        bq.embed(t, tid, out, scale=0.37)
    ref = L.embed(want, ids, np.float64(np.float32(0.37)))
    assert np.all(np.abs(f64(out) - ref) <= U * 1.001 * np.abs(ref))
    assert outside_kept(out, flat, shift)


def test_embed_of_no_tokens_and_one(cuda):
    import torch

    t, want = bf16(np.arange(64, dtype=np.float32).reshape(4, 16), cuda)
    out, _ = empty(0, 16, cuda, torch.bfloat16)
    bq.embed(t, torch.empty(0, dtype=torch.int64, device=cuda), out)
    out, _ = empty(1, 16, cuda, torch.bfloat16)
    bq.embed(t, torch.tensor([3], device=cuda), out)
    assert np.array_equal(f64(out)[0], want[3])


@pytest.mark.parametrize("n,rows,cols,how", [
    (1, 1, 8, "any"), (1, 1000, 264, "any"), (31, 7, 136, "any"), (32, 7, 128, "one"), (33, 7, 128, "one"),
    (64, 65, 8, "one"), (65, 64, 16, "any"), (700, 300, 520, "zipf"), (1000, 513, 131, "zipf"), (777, 90, 1, "one"),
    (5000, 70000, 24, "zipf"), (9000, 300000, 8, "any"), (40000, 1200, 8, "zipf"), (257, 200, 2880, "out"),
    (256, 40000, 16, "any"), (256, 3, 264, "zipf"), (200, 70, 2056, "one"), (1024, 5000, 136, "zipf"), (1025, 5000, 136, "one"),
    (8192, 600, 24, "zipf"), (8193, 600, 24, "any"),
])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad(cuda, n, rows, cols, how, kind, accumulate):
    import torch

    rng = np.random.default_rng(n + rows)
    if how == "one":
        ids = np.full(n, rows - 1)
    elif how == "zipf":
        ids = np.minimum(rng.zipf(1.3, n) - 1, rows)  # `rows`: outside
    elif how == "out":
        ids = np.where(rng.random(n) < 0.5, -1, rows + 5)
    else:
        ids = rng.integers(-1, rows, n)
    pitch = 0 if cols % 8 else 8
    dy, dyv = bf16(rng.standard_normal((n, cols)), cuda, pitch)
    tid = torch.as_tensor(ids.astype(np.int32)).to(cuda)
    dt = torch.bfloat16 if kind == "bf16" else torch.float32
    out, flat = empty(rows, cols, cuda, dt, pitch, 0, 0.5)
    ws = torch.empty(bq.embed_grad_workspace(n, rows, cols), dtype=torch.uint8, device=cuda)
    bq.embed_grad(dy, tid, out, ws, scale=1.5, accumulate=accumulate)
    g, mag = L.embed_grad(dyv, ids, rows, 1.5)
    k = np.bincount(ids[(ids >= 0) & (ids < rows)], minlength=rows)[:, None]
    if accumulate:
        g, mag = g + 0.5, mag + 0.5
    tol = (k + 2) * E * mag + (U * 1.001 * np.abs(g) if kind == "bf16" else 0) + 1e-30
    assert np.all(np.abs(f64(out) - g) <= tol)
    if pitch:
        assert outside_kept(out, flat, 0, 0.5)
    if not accumulate:  # the same bits again, on another stream
        first = out.clone()
        out.fill_(3.0)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            bq.embed_grad(dy, tid, out, ws, scale=1.5)
        s.synchronize()
        assert torch.equal(first, out)


def test_embed_grad_of_no_tokens(cuda):
    import torch

    out = torch.full((5, 12), 3.0, device=cuda)
    ws = torch.empty(bq.embed_grad_workspace(0, 5, 12), dtype=torch.uint8, device=cuda)
    none = torch.empty(0, 12, dtype=torch.bfloat16, device=cuda)
    ids = torch.empty(0, dtype=torch.int64, device=cuda)
    bq.embed_grad(none, ids, out, ws, accumulate=True)
    assert torch.all(out == 3.0)
    bq.embed_grad(none, ids, out, ws)
    assert torch.all(out == 0.0)


# ----------------------------------------------------------------------------- norm

WIDTHS = [1, 7, 8, 100, 127, 128, 129, 136, 256, 264, 1000, 2880, 4096, 8192, 8200, 8193, 16384, 16392, 33000]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(cuda, cols, residual):
    import torch

    rng = np.random.default_rng(cols)
    n, eps = 5, 1e-5
    pitch, shift = (8, 0) if cols % 16 == 0 else (0, 0) if cols % 8 == 0 else (3, 1)
    a = rng.standard_normal((n, cols)) * np.array([1, 1e-4, 1e3, 0, 1])[:, None]
    x, xv = bf16(a, cuda, pitch, shift)
    r, rv = bf16(rng.standard_normal((n, cols)) * (a != 0), cuda, pitch, shift)
    w, wv = bf16(1 + 0.3 * rng.standard_normal(cols), cuda)
    h, hf = empty(n, cols, cuda, torch.bfloat16, pitch, shift)
    y, yf = empty(n, cols, cuda, torch.bfloat16, pitch, shift)
    codes = torch.full((n, cols + pitch), 0x55, dtype=torch.uint8, device=cuda)
    scale = torch.full((-(-cols // 128), n + 2), 7.0, device=cuda)
    rstd = torch.empty(n, device=cuda)
    bq.rmsnorm(x, w, eps, residual=r if residual else None, h=h if residual else None, y=y, codes=codes[:, :cols],
               code_scale=scale[:, :n], rstd=rstd)
    if residual:
        hv = f64(h)
        assert np.all(np.abs(hv - (xv + rv)) <= U * 1.001 * np.abs(xv + rv))
        assert outside_kept(h, hf, shift)
    else:
        hv = xv
    want, rs = L.rmsnorm(hv, wv, np.float64(np.float32(eps)))
    # the sum of squares, its mean and the root: (cols + 4) e, halved by the root, and
    # an approximate reciprocal root of 2^-22
    slack = (cols + 4) * E + 2.0 ** -21
    assert np.all(np.abs(f64(rstd) - rs) <= slack * rs)
    assert np.all(np.abs(f64(y) - want) <= (U * 1.001 + slack) * np.abs(want))
    assert outside_kept(y, yf, shift)
    check_codes(codes[:, :cols], scale[:, :n], want, slack + 2 * E)
    assert torch.all(codes[:, cols:] == 0x55) and torch.all(scale[:, n:] == 7.0)


@pytest.mark.parametrize("n,cols", [(5000, 256), (2600, 520), (1300, 4096), (700, 8192), (640, 8200), (650, 16384)])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_many_rows(cuda, n, cols, residual):
    """Counts of rows that the resident CTAs share: every row as the same row alone, zeros,
    tiny values, infinities and NaN among them."""
    import torch

    rng = np.random.default_rng(cols)
    a = rng.standard_normal((n, cols))
    a[3] = 0
    a[4] *= 2.0 ** -120
    a[5, 17], a[6, 3], a[7, cols - 1] = np.inf, np.nan, -np.inf
    x, _ = bf16(a, cuda, 8)
    r, _ = bf16(rng.standard_normal((n, cols)) * (np.arange(n) > 8)[:, None], cuda)
    w, _ = bf16(1 + 0.3 * rng.standard_normal(cols), cuda)
    got, want = [], []
    for rows in (n, 50):
        outs = []
        for i in range(0, n, rows):
            m = min(rows, n - i)
            h, y = torch.empty(m, cols, dtype=torch.bfloat16, device=cuda), torch.empty(m, cols, dtype=torch.bfloat16, device=cuda)
            codes = torch.empty(m, cols, dtype=torch.uint8, device=cuda)
            scale, rstd = torch.empty(-(-cols // 128), m, device=cuda), torch.empty(m, device=cuda)
            bq.rmsnorm(x[i:i + m], w, 1e-5, residual=r[i:i + m] if residual else None, h=h if residual else None, y=y,
                       codes=codes, code_scale=scale, rstd=rstd)
            outs.append((h if residual else y, y, codes, scale.t(), rstd))
        (got if rows == n else want).extend(torch.cat(t) for t in zip(*outs))
    for a, b in zip(got, want):
        assert torch.equal(a, b) or bool(((a == b) | ((a != a) & (b != b))).all())


def test_rmsnorm_in_place_and_parts(cuda):
    """h over x, h over the residual, and each output on its own give the same bits."""
    import torch

    rng = np.random.default_rng(3)
    x, _ = bf16(rng.standard_normal((9, 520)), cuda)
    r, _ = bf16(rng.standard_normal((9, 520)), cuda)
    w, _ = bf16(1 + 0.1 * rng.standard_normal(520), cuda)
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(9, device=cuda)
    bq.rmsnorm(x, w, 1e-6, residual=r, h=h, y=y, rstd=rstd)
    for k in range(2):
        a, b = x.clone(), r.clone()
        y2 = torch.empty_like(x)
        bq.rmsnorm(a, w, 1e-6, residual=b, h=(a, b)[k], y=y2)
        assert torch.equal((a, b)[k], h) and torch.equal(y2, y)
    rs2 = torch.empty_like(rstd)
    bq.rmsnorm(h, w, 1e-6, rstd=rs2)
    assert torch.equal(rs2, rstd)


@pytest.mark.parametrize("cols", [520, 515])
def test_rmsnorm_rows_of_zeros_infinities_and_nan(cuda, cols):
    import torch

    a = np.ones((4, cols), np.float32)
    a[0] = 0
    a[1, 5] = np.inf
    a[2, 300] = np.nan
    x, _ = bf16(a, cuda)
    w, _ = bf16(np.ones(cols), cuda)
    y = torch.empty(4, cols, dtype=torch.bfloat16, device=cuda)
    codes = torch.empty(4, cols, dtype=torch.uint8, device=cuda)
    scale = torch.empty(-(-cols // 128), 4, device=cuda)
    bq.rmsnorm(x, w, 1e-5, y=y, codes=codes, code_scale=scale)
    y, s, c = f64(y), f64(scale), e4m3_decode(codes.cpu().numpy()).astype(np.float64)
    assert np.all(y[0] == 0) and np.all(s[:, 0] == 0) and np.all(c[0] == 0)
    assert np.isnan(y[1, 5]) and np.all(y[1, :5] == 0)  # 1 / inf, and inf * 0
    assert np.isnan(c[1, 5] * s[0, 1])
    assert np.all(np.isnan(y[2])) and np.all(np.isnan(s[:, 2]))
    assert np.all(np.abs(y[3] - 1) <= 0.01) and np.all(c[3] == 448)  # untouched by its neighbours


@pytest.mark.parametrize("n,cols", [(1, 8), (1, 8192), (2, 7), (3, 129), (37, 264), (301, 2880), (700, 520), (330, 515),
                                    (5, 8200), (4, 8193), (3, 16392), (2, 33000), (5000, 256), (1300, 4096),
                                    (700, 8192), (640, 8200)])
@pytest.mark.parametrize("dh", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_rmsnorm_grad(cuda, n, cols, dh, kind):
    import torch

    rng = np.random.default_rng(n * cols)
    pitch, shift = (8, 0) if cols % 16 == 0 else (0, 0) if cols % 8 == 0 else (3, 1)
    h, hv = bf16(rng.standard_normal((n, cols)), cuda, pitch, shift)
    dy, dyv = bf16(rng.standard_normal((n, cols)), cuda, pitch, shift)
    g, gv = bf16(rng.standard_normal((n, cols)), cuda, pitch, shift)
    w, wv = bf16(1 + 0.3 * rng.standard_normal(cols), cuda)
    rstd = torch.as_tensor(1 / np.sqrt((hv * hv).mean(1) + 1e-5), dtype=torch.float32).to(cuda)
    rv = f64(rstd)
    dx, flat = empty(n, cols, cuda, torch.bfloat16, pitch, shift)
    dt = torch.bfloat16 if kind == "bf16" else torch.float32
    dw = torch.full((cols,), 0.25, dtype=dt, device=cuda)
    ws = torch.empty(bq.rmsnorm_grad_workspace(n, cols), dtype=torch.uint8, device=cuda)
    bq.rmsnorm_grad(dy, h, w, rstd, dx, dw, ws, dh=g if dh else None)
    want, wantw = L.rmsnorm_grad(dyv, hv, wv, rv)
    if dh:
        want = want + gv
    u, t = np.abs(hv * rv[:, None]), np.abs(dyv * wv)
    mag = rv[:, None] * (t + u * np.mean(t * u, axis=1, keepdims=True)) + (np.abs(gv) if dh else 0)
    assert np.all(np.abs(f64(dx) - want) <= U * 1.001 * np.abs(want) + (cols + 8) * E * mag)
    assert outside_kept(dx, flat, shift)
    magw = np.sum(np.abs(dyv) * u, axis=0)
    tolw = (n + 4) * E * magw
    assert np.all(np.abs(f64(dw) - wantw) <= tolw + (U * 1.001 * np.abs(wantw) if kind == "bf16" else 0))
    once = f64(dw)
    bq.rmsnorm_grad(dy, h, w, rstd, dx, dw, ws, dh=g if dh else None, accumulate=True)
    assert np.all(np.abs(f64(dw) - (once + wantw)) <= tolw + 2 * E * np.abs(once) + (U * 1.001 * np.abs(once + wantw) + 2 * U * np.abs(once) if kind == "bf16" else 2 * E * np.abs(wantw)))


def test_rmsnorm_grad_in_place_and_of_no_rows(cuda):
    import torch

    rng = np.random.default_rng(8)
    h, _ = bf16(rng.standard_normal((40, 384)), cuda)
    dy, _ = bf16(rng.standard_normal((40, 384)), cuda)
    g, _ = bf16(rng.standard_normal((40, 384)), cuda)
    w, _ = bf16(rng.standard_normal(384), cuda)
    rstd = torch.rand(40, device=cuda) + 0.5
    ws = torch.empty(bq.rmsnorm_grad_workspace(40, 384), dtype=torch.uint8, device=cuda)
    dx, dw = torch.empty_like(h), torch.empty(384, device=cuda)
    bq.rmsnorm_grad(dy, h, w, rstd, dx, dw, ws, dh=g)
    for k in range(2):
        a, b, dw2 = dy.clone(), g.clone(), torch.empty_like(dw)
        bq.rmsnorm_grad(a, h, w, rstd, (a, b)[k], dw2, ws, dh=b)
        assert torch.equal((a, b)[k], dx) and torch.equal(dw2, dw)
    none = torch.empty(0, 384, dtype=torch.bfloat16, device=cuda)
    bq.rmsnorm_grad(none, none, w, rstd[:0], none, dw, ws, accumulate=True)
    assert torch.equal(dw2, dw)
    bq.rmsnorm_grad(none, none, w, rstd[:0], none, dw, ws)
    assert torch.all(dw == 0)


@pytest.mark.parametrize("cols", [1, 8, 100, 128, 130, 264, 1032, 2881])
def test_quant_rows(cuda, cols):
    import torch

    rng = np.random.default_rng(cols)
    n = 19
    x, xv = bf16(rng.standard_normal((n, cols)) * np.exp(8 * rng.standard_normal((n, 1))), cuda)
    x[3] = 0
    xv[3] = 0
    x[4] = 2.0 ** -130  # 448 / a overflows
    xv[4] = 2.0 ** -130
    codes = torch.empty(n, cols, dtype=torch.float8_e4m3fn, device=cuda)
    scale = torch.empty(-(-cols // 128), n, device=cuda)
    bq.quant_rows_fp8(x, codes, scale)
    keep = np.arange(n) != 4
    check_codes(codes[torch.as_tensor(keep)], scale[:, torch.as_tensor(keep)], xv[keep], 2 * E)
    s4 = f64(scale)[:, 4]
    assert np.all(s4 > 0) and np.all(np.abs(s4 - 2.0 ** -130 / 448) <= 2.0 ** -150)  # a subnormal scale


# ----------------------------------------------------------------------------- projections

SHAPES = [(1, 1, 16), (1, 128, 128), (1, 300, 4096), (2, 130, 144), (8, 256, 1024), (33, 257, 1040), (64, 200, 2064),
          (100, 64, 8192), (128, 128, 128), (129, 300, 272), (256, 256, 256), (300, 520, 2064), (513, 1000, 528),
          (1030, 2881, 272), (2048, 1024, 640), (700, 4000, 1536), (2000, 2050, 2064), (4100, 1000, 1040), (16, 200, 528),
          (17, 72, 272), (90, 1904, 304), (1100, 520, 400), (2000, 3000, 4096), (1950, 4096, 3008)]


def workspace(n, rows, cols, dev):
    import torch

    ws = torch.full((bq.linear_fp8_workspace(n, rows, cols),), 0xFF, dtype=torch.uint8, device=dev)
    ws[:256] = 0
    return ws


def sum_tol(a, b, red):
    """Bound on the fp32 sum over `red` products of scaled codes: k-blocks of 128 on
    the tensor cores, then one fp32 addition and three roundings of scales a block."""
    return (128 * 2.0 ** -23 + (-(-red // 128) + 3) * E) * (np.abs(a) @ np.abs(b))


@pytest.mark.parametrize("n,rows,cols", SHAPES)
def test_linear(cuda, n, rows, cols):
    import torch

    rng = np.random.default_rng(n + rows + cols)
    x, xs, xv = fp8_rows(rng, n, cols, cuda, pitch=16, spare=3)
    w, ws_, wv = fp8_weight(rng, rows, cols, cuda)
    for pitch, shift in [(0, 0), (5, 1)]:
        out, flat = empty(n, rows, cuda, torch.bfloat16, pitch, shift)
        ws = workspace(n, rows, cols, cuda)
        bq.linear_fp8(x, xs, w, ws_, out, ws)
        bq.linear_check(ws)
        ref = xv @ wv.T
        assert np.all(np.abs(f64(out) - ref) <= U * 1.001 * np.abs(ref) + sum_tol(xv, wv.T, cols))
        assert outside_kept(out, flat, shift)


# many rows whose outputs are aligned to 16, 8, 4 and 2 bytes, and end inside a store
@pytest.mark.parametrize("rows,pitch,shift", [(1997, 3, 0), (1996, 0, 0), (1995, 1, 4), (1998, 0, 0), (1997, 1, 2), (1997, 0, 1)])
def test_linear_output_alignment(cuda, rows, pitch, shift):
    import torch

    n, cols = 4001, 272
    rng = np.random.default_rng(rows + pitch)
    x, xs, xv = fp8_rows(rng, n, cols, cuda)
    w, ws_, wv = fp8_weight(rng, rows, cols, cuda)
    out, flat = empty(n, rows, cuda, torch.bfloat16, pitch, shift)
    ws = workspace(n, rows, cols, cuda)
    bq.linear_fp8(x, xs, w, ws_, out, ws)
    bq.linear_check(ws)
    ref = xv @ wv.T
    assert np.all(np.abs(f64(out) - ref) <= U * 1.001 * np.abs(ref) + sum_tol(xv, wv.T, cols))
    assert outside_kept(out, flat, shift)


@pytest.mark.parametrize("n,rows,cols", SHAPES)
def test_linear_dx(cuda, n, rows, cols):
    import torch

    rng = np.random.default_rng(n + rows + cols)
    w, ws_, wv = fp8_weight(rng, rows, cols, cuda)
    dy, _ = bf16(rng.standard_normal((n, rows)), cuda, 3 if rows % 8 else 0)
    # the rows that the call quantises, taken from the row quantiser (tested above)
    q = torch.empty(n, rows, dtype=torch.uint8, device=cuda)
    qs = torch.empty(-(-rows // 128), n, device=cuda)
    bq.quant_rows_fp8(dy, q, qs)
    qv = L.decode_rows(q.cpu().numpy(), qs.cpu().numpy())
    for pitch, shift in [(0, 0), (5, 1)]:
        dx, flat = empty(n, cols, cuda, torch.bfloat16, pitch, shift)
        ws = workspace(n, rows, cols, cuda)
        bq.linear_fp8_dx(dy, w, ws_, dx, ws)
        bq.linear_check(ws)
        ref = qv @ wv
        assert np.all(np.abs(f64(dx) - ref) <= U * 1.001 * np.abs(ref) + sum_tol(qv, wv, rows))
        assert outside_kept(dx, flat, shift)


@pytest.mark.parametrize("n,rows,cols", SHAPES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_linear_dw(cuda, n, rows, cols, accumulate):
    import torch

    rng = np.random.default_rng(n + rows + cols)
    x, xs, xv = fp8_rows(rng, n, cols, cuda, pitch=16, spare=1)
    dy, dv = bf16(rng.standard_normal((n, rows)), cuda, 8 if rows % 64 == 0 else 0)
    dw, flat = empty(rows, cols, cuda, torch.bfloat16, 8, 0, 0.5)
    ws = workspace(n, rows, cols, cuda)
    bq.linear_fp8_dw(dy, x, xs, dw, ws, accumulate=accumulate)
    bq.linear_check(ws)
    mag = np.abs(dv).T @ np.abs(xv)
    ref = dv.T @ xv + (0.5 if accumulate else 0)
    # X is rounded to bf16 once, products summed in fp32
    tol = U * 1.001 * (np.abs(ref) + mag) + n * 2.0 ** -23 * mag
    assert np.all(np.abs(f64(dw) - ref) <= tol)
    assert outside_kept(dw, flat, 0, 0.5)


# outer products in one and in several chunks of tokens, products in one and in several
# shares, with rows that end inside a tile; gradients whose rows are not aligned
@pytest.mark.parametrize("pitch,shift", [(0, 0), (8, 0), (3, 1)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,rows,cols", [(16, 70, 272), (24, 250, 528), (33, 300, 16), (65, 1000, 2064), (130, 700, 528),
                                         (2300, 250, 272), (4100, 520, 272), (5000, 100, 1040)])
def test_linear_dw_rows_and_shares(cuda, n, rows, cols, accumulate, pitch, shift):
    import torch

    rng = np.random.default_rng(n + rows + cols)
    x, xs, xv = fp8_rows(rng, n, cols, cuda)
    dy, dv = bf16(rng.standard_normal((n, rows)), cuda)
    dw, flat = empty(rows, cols, cuda, torch.bfloat16, pitch, shift, -0.25)
    ws = workspace(n, rows, cols, cuda)
    bq.linear_fp8_dw(dy, x, xs, dw, ws, accumulate=accumulate)
    bq.linear_check(ws)
    mag = np.abs(dv).T @ np.abs(xv)
    ref = dv.T @ xv + (-0.25 if accumulate else 0)
    tol = U * 1.001 * (np.abs(ref) + mag) + n * 2.0 ** -23 * mag  # (as above)
    assert np.all(np.abs(f64(dw) - ref) <= tol)
    assert outside_kept(dw, flat, shift, -0.25)


def integer_rows(rng, n, cols, top, dev):
    """FP8 rows of small integers whose scales are powers of two, no two groups of a row
    beside one another the same: (codes, scales, values in fp64)."""
    import torch

    v = rng.integers(-2, 3, (n, cols)).astype(np.float32)
    g = -(-cols // 128)
    power = (np.arange(g)[:, None] * 3 + rng.integers(0, top, (1, n)) + rng.integers(0, 2, (g, n))) % top
    scale = (2.0 ** power).astype(np.float32)
    codes = e4m3_encode(v)
    return torch.as_tensor(codes).to(dev), torch.as_tensor(scale).to(dev), L.decode_rows(codes, scale)


# every sum is a whole number below 2^24, so exact in any order: a k-block that took another
# block's or another tile's scales would show.  Several tiles a CTA pair, k-blocks more
# and fewer than its ring of scales has slots, rows that end inside a lane's four scales, scales
# at a pitch that copies by 16 bytes cannot read
@pytest.mark.parametrize("n,rows,cols,spare", [(4100, 4200, 528, 0), (4098, 3000, 2064, 2), (4099, 2600, 5136, 1)])
def test_linear_scales_exact(cuda, n, rows, cols, spare):
    import torch

    rng = np.random.default_rng(n)
    x, s, xv = integer_rows(rng, n, cols, 8, cuda)
    xs = torch.full((s.shape[0], n + spare), float("nan"), device=cuda)[:, :n]
    xs.copy_(s)
    wv = rng.integers(-2, 3, (rows, cols)).astype(np.float32)
    tiles = (2.0 ** rng.integers(0, 4, (-(-rows // 128), -(-cols // 128)))).astype(np.float32)
    codes = e4m3_encode(wv)
    wv = L.decode_tiles(codes, tiles)
    w, ws_ = torch.as_tensor(codes).to(cuda), torch.as_tensor(tiles).to(cuda)
    # |sum| <= 2 * 2 * 2^7 * 2^3 * cols < 2^12 * 5136 = 1.25 * 2^24 at worst; as drawn:
    ref = torch.as_tensor(xv).to(cuda) @ torch.as_tensor(wv).to(cuda).t()
    assert float((torch.as_tensor(np.abs(xv)).to(cuda) @ torch.as_tensor(np.abs(wv)).to(cuda).t()).max()) < 2 ** 24
    ws = workspace(n, rows, cols, cuda)
    for _ in range(3):
        out = torch.zeros(n, rows, dtype=torch.bfloat16, device=cuda)
        bq.linear_fp8(x, xs, w, ws_, out, ws)
        bq.linear_check(ws)
        assert torch.equal(out, ref.float().bfloat16())


def test_linear_of_no_tokens(cuda):
    import torch

    rng = np.random.default_rng(1)
    w, ws_, _ = fp8_weight(rng, 48, 32, cuda)
    x = torch.empty(0, 32, dtype=torch.uint8, device=cuda)
    xs = torch.empty(1, 0, device=cuda)
    y = torch.empty(0, 48, dtype=torch.bfloat16, device=cuda)
    ws = workspace(0, 48, 32, cuda)
    bq.linear_fp8(x, xs, w, ws_, y, ws)
    bq.linear_fp8_dx(y, w, ws_, torch.empty(0, 32, dtype=torch.bfloat16, device=cuda), ws)
    dw = torch.full((48, 32), 2.0, dtype=torch.bfloat16, device=cuda)
    bq.linear_fp8_dw(y, x, xs, dw, ws, accumulate=True)
    assert torch.all(dw == 2.0)
    bq.linear_fp8_dw(y, x, xs, dw, ws)
    assert torch.all(dw == 0.0)


def test_linear_same_bits_again_and_rows_apart(cuda):
    """The same call gives the same bits, a row's result does not depend on the rows
    beside it, and a NaN stays in its row."""
    import torch

    rng = np.random.default_rng(5)
    n, rows, cols = 40, 384, 1024
    x, xs, _ = fp8_rows(rng, n, cols, cuda)
    w, ws_, _ = fp8_weight(rng, rows, cols, cuda)
    ws = workspace(n, rows, cols, cuda)
    a, b = (torch.empty(n, rows, dtype=torch.bfloat16, device=cuda) for _ in range(2))
    bq.linear_fp8(x, xs, w, ws_, a, ws)
    bq.linear_fp8(x, xs, w, ws_, b, ws)
    assert torch.equal(a, b)
    x2 = x.clone()
    x2[7, 100] = 0x7F
    bq.linear_fp8(x2, xs, w, ws_, b, ws)
    bad = torch.isnan(b).any(dim=1).cpu().numpy()
    assert bad[7] and bad.sum() == 1
    keep = np.arange(n) != 7
    assert torch.equal(a[torch.as_tensor(keep)], b[torch.as_tensor(keep)])


# ----------------------------------------------------------------------------- streams, graphs, large offsets


def test_another_stream_and_a_graph(cuda):
    """One step's chain on a stream of its own, then captured and replayed on new inputs:
    the same bits as on the current stream."""
    import torch

    n, rows, cols, vocab = 300, 520, 272, 700
    rng = np.random.default_rng(7)
    table, ts, _ = fp8_weight(rng, vocab, cols, cuda)
    w, ws_, _ = fp8_weight(rng, rows, cols, cuda)
    gain = bf16(rng.standard_normal(cols), cuda)[0]
    new = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=cuda)  # noqa: E731
    ids = new(n, t=torch.int64)
    ws = workspace(n, rows, cols, cuda)
    ws_e = new(bq.embed_grad_workspace(n, vocab, cols), t=torch.uint8)
    ws_n = new(bq.rmsnorm_grad_workspace(n, cols), t=torch.uint8)
    x, h, dh, dx, dy = new(n, cols), new(n, cols), new(n, cols), new(n, cols), new(n, rows)
    q, qs, rstd = new(n, cols, t=torch.uint8), new(3, n, t=torch.float32), new(n, t=torch.float32)
    y, dw, dg, dt = new(n, rows), new(rows, cols), new(cols), new(vocab, cols)

    def chain():
        bq.embed(table, ids, x, table_scale=ts)
        bq.rmsnorm(x, gain, 1e-5, residual=x, h=h, codes=q, code_scale=qs, rstd=rstd)
        bq.linear_fp8(q, qs, w, ws_, y, ws)
        bq.linear_fp8_dw(dy, q, qs, dw, ws)
        bq.linear_fp8_dx(dy, w, ws_, dh, ws)
        bq.rmsnorm_grad(dh, h, gain, rstd, dx, dg, ws_n)
        bq.embed_grad(dx, ids, dt, ws_e)
        return [t.clone() for t in (x, h, q, qs, rstd, y, dw, dh, dx, dg, dt)]

    def inputs(seed):
        r = np.random.default_rng(seed)
        ids.copy_(torch.as_tensor(r.integers(0, vocab, n)))
        dy.copy_(torch.as_tensor(r.standard_normal((n, rows)).astype(np.float32)))

    want = []
    for seed in (1, 2, 3):
        inputs(seed)
        want.append(chain())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        inputs(1)
        got = chain()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = chain()
    for seed in (2, 3):
        inputs(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[seed - 1]))
    bq.linear_check(ws)


def test_offsets_past_32_bits(cuda):
    """Tables, batches and outputs of more than 2^31 elements: their last rows."""
    import torch

    rng = np.random.default_rng(3)
    rows, cols = 525000, 4096  # 2.15 G elements, 4.3 GB
    assert rows * cols > 2 ** 31
    big = torch.zeros(rows, cols, dtype=torch.bfloat16, device=cuda)
    last, lv = bf16(rng.standard_normal((3, cols)), cuda)
    big[-3:] = last
    ids = torch.tensor([rows - 1, 0, rows - 3, rows - 1], device=cuda)
    out = torch.empty(4, cols, dtype=torch.bfloat16, device=cuda)
    bq.embed(big, ids, out)
    assert torch.equal(out[0], last[2]) and torch.equal(out[2], last[0]) and not out[1].any()
    ws = torch.empty(bq.embed_grad_workspace(4, rows, cols), dtype=torch.uint8, device=cuda)
    dy, dv = bf16(rng.standard_normal((4, cols)), cuda)
    bq.embed_grad(dy, ids, big, ws)
    want = dv[0] + dv[3]
    assert np.all(np.abs(f64(big[-1]) - want) <= U * np.abs(want) + 2 * E * (np.abs(dv[0]) + np.abs(dv[3])))
    assert torch.equal(big[-3], dy[2]) and torch.equal(big[0], dy[1]) and not big[-2].any() and not big[1:-3].any()

    # as many rows through the norm: the last ones as by themselves
    big[-3:] = last
    gain = bf16(rng.standard_normal(cols), cuda)[0]
    q = torch.empty(rows, cols, dtype=torch.uint8, device=cuda)
    qs = torch.empty(cols // 128, rows, device=cuda)
    bq.rmsnorm(big, gain, 1e-5, codes=q, code_scale=qs)
    q1, qs1 = torch.empty(3, cols, dtype=torch.uint8, device=cuda), torch.empty(cols // 128, 3, device=cuda)
    bq.rmsnorm(last, gain, 1e-5, codes=q1, code_scale=qs1)
    assert torch.equal(q[-3:], q1) and torch.equal(qs[:, -3:], qs1)

    # and a product that writes as many
    k = 32
    w, ws_, wv = fp8_weight(rng, cols, k, cuda)
    x, xs, xv = fp8_rows(rng, 256, k, cuda)
    many = x.repeat(rows // 256 + 1, 1)[:rows].contiguous()
    scales = xs.repeat(1, rows // 256 + 1)[:, :rows].contiguous()
    ws = workspace(rows, cols, k, cuda)
    bq.linear_fp8(many, scales, w, ws_, big, ws)
    bq.linear_check(ws)
    at = (rows - 200 + np.arange(200)) % 256
    ref = xv[at] @ wv.T
    assert np.all(np.abs(f64(big[-200:]) - ref) <= U * 1.001 * np.abs(ref) + sum_tol(xv[at], wv.T, k))


# ----------------------------------------------------------------------------- row quantiser, group by group


def quantise(y):
    """(codes, scales [groups, n]) of fp32 rows by the rule of the codes, each operation
    rounded to fp32 once: s = a / 448, code = e4m3(y * (448 / a)).  Ordinary groups only."""
    n, cols = y.shape
    g = -(-cols // 128)
    p = np.zeros((n, g * 128), np.float32)
    p[:, :cols] = y
    a = np.abs(p.reshape(n, g, 128)).max(axis=2)
    r = np.repeat(np.float32(448) / a, 128, axis=1)[:, :cols]
    return e4m3_encode(y * r), (a / np.float32(448)).T


@pytest.mark.parametrize("cols", [1, 8, 100, 128, 130, 264, 1032, 2881])
def test_quant_rows_zero_and_tiny(cuda, cols):
    """Rows of zeros have scales and codes of 0; rows whose 448 / a overflows get their codes by
    dividing by the scale: 2^-130 / s is within 2^-10 of 448, every code the largest."""
    import torch

    n = 19
    x, _ = bf16(np.random.default_rng(cols).standard_normal((n, cols)), cuda)
    x[3], x[4], x[5] = 0, 2.0 ** -130, -(2.0 ** -130)
    codes = torch.full((n, cols), 0x55, dtype=torch.uint8, device=cuda)
    scale = torch.empty(-(-cols // 128), n, device=cuda)
    bq.quant_rows_fp8(x, codes, scale)
    assert not codes[3].any() and not scale[:, 3].any()
    assert torch.all(codes[4] == 0x7E) and torch.all(codes[5] == 0xFE)


# many rows (four spans a warp) and few (one); rows of whole words, rows that are not, codes that
# are not.  A warp's groups are of every kind beside one another
@pytest.mark.parametrize("n,cols,pitch,shift", [(1300, 4096, 0, 0), (700, 1032, 8, 0), (1300, 264, 3, 1), (650, 2872, 5, 3),
                                                (1300, 2881, 0, 0), (1300, 131, 2, 1), (40, 1032, 0, 0), (40, 1032, 3, 1),
                                                (40, 1031, 0, 0)])
def test_quant_rows_groups(cuda, n, cols, pitch, shift):
    import torch

    rng = np.random.default_rng(n + cols)
    g = -(-cols // 128)
    kind = rng.choice(["plain", "zero", "tiny", "nan", "inf"], (n, g), p=[0.6, 0.1, 0.1, 0.1, 0.1])
    kind[::3] = "plain"  # (rows whose warps see nothing else)
    spread = lambda v: np.repeat(v, 128, axis=1)[:, :cols]  # noqa: E731
    of = spread(kind)
    factor = np.exp(4 * rng.standard_normal((n, g)))
    a = rng.standard_normal((n, cols)) * spread(factor)
    a[of == "zero"] = 0
    a[of == "tiny"] *= (2.0 ** -125 / spread(factor))[of == "tiny"]
    first = np.arange(g) * 128
    at = np.minimum(first[None, :] + rng.integers(0, 128, (n, g)), cols - 1)
    rows = np.broadcast_to(np.arange(n)[:, None], (n, g))
    a[rows[kind == "nan"], at[kind == "nan"]] = np.nan
    a[rows[kind == "inf"], at[kind == "inf"]] = -np.inf
    x, xv = bf16(a, cuda, pitch, shift)
    codes = torch.full((n, cols), 0x55, dtype=torch.uint8, device=cuda)
    scale = torch.empty(g, n, device=cuda)
    bq.quant_rows_fp8(x, codes, scale)
    got, s = codes.cpu().numpy(), scale.cpu().numpy()
    plain, zero, tiny = of == "plain", of == "zero", of == "tiny"
    # ordinary groups bit for bit
    ordinary = np.where(plain, xv, 1.0).astype(np.float32)
    want, want_s = quantise(ordinary)
    assert np.array_equal(got[plain], want[plain])
    assert np.array_equal(s.T[kind == "plain"], want_s.T[kind == "plain"])
    assert not (got[zero] & 0x7F).any() and not s.T[kind == "zero"].any()
    # tiny groups: a scale within half a step of the subnormals, codes within half a step of y / s
    top = np.where(tiny, np.abs(xv), 0)
    top = np.pad(top, ((0, 0), (0, g * 128 - cols))).reshape(n, g, 128).max(axis=2)
    st = s.T.astype(np.float64)
    assert np.all(np.abs(st - top / 448)[kind == "tiny"] <= 2.0 ** -150)
    v, sv = e4m3_decode(got).astype(np.float64), spread(st)
    with np.errstate(invalid="ignore"):
        y = xv / sv
        off = np.abs(v - np.clip(y, -448, 448)) <= 2.0 ** -4 * np.abs(v) * 1.001 + 2.0 ** -10 * 1.001
    assert np.all(off[tiny])
    # a NaN makes its group's scale NaN; an infinity makes its scale infinite and its own code NaN
    assert np.all(np.isnan(s.T[kind == "nan"]))
    assert np.all(np.isposinf(s.T[kind == "inf"]))
    assert np.all(np.isnan(e4m3_decode(got[rows[kind == "inf"], at[kind == "inf"]])))


# the input gradient against rows quantised here, bit for bit the quantiser's
@pytest.mark.parametrize("n,rows,cols", [(33, 257, 1040), (300, 520, 2064), (2048, 1024, 640), (700, 4000, 1536),
                                         (4100, 1000, 1040), (1100, 520, 400), (1950, 4096, 3008), (1300, 1001, 272)])
def test_linear_dx_of_rows_quantised_apart(cuda, n, rows, cols):
    import torch

    rng = np.random.default_rng(n + rows + cols)
    w, ws_, wv = fp8_weight(rng, rows, cols, cuda)
    dy, dv = bf16(rng.standard_normal((n, rows)), cuda)
    q, qs = quantise(dv.astype(np.float32))
    codes, scale = torch.empty(n, rows, dtype=torch.uint8, device=cuda), torch.empty(-(-rows // 128), n, device=cuda)
    bq.quant_rows_fp8(dy, codes, scale)
    assert np.array_equal(codes.cpu().numpy(), q) and np.array_equal(scale.cpu().numpy(), qs)
    qv = L.decode_rows(q, qs)
    dx = torch.empty(n, cols, dtype=torch.bfloat16, device=cuda)
    ws = workspace(n, rows, cols, cuda)
    bq.linear_fp8_dx(dy, w, ws_, dx, ws)
    bq.linear_check(ws)
    ref = qv @ wv
    assert np.all(np.abs(f64(dx) - ref) <= U * 1.001 * np.abs(ref) + sum_tol(qv, wv, rows))


# ----------------------------------------------------------------------------- products of whole numbers: exact


def small_integers(rng, shape, dev):
    import torch

    v = rng.integers(-3, 4, shape).astype(np.float32)
    return torch.as_tensor(v).bfloat16().to(dev), v.astype(np.float64)


# Every product is a whole number of at most 3 * 2 * 2^3 and every sum below 2^24, so exact
# however it is split: a token, a share or a tail left out or counted twice shows
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,rows,cols", SHAPES + [(16, 70, 272), (24, 250, 528), (33, 300, 16), (65, 1000, 2064), (130, 700, 528),
                                                  (2300, 250, 272), (4100, 520, 272), (5000, 100, 1040), (8191, 1024, 1024),
                                                  (63, 520, 528), (64, 520, 528)])
def test_linear_dw_exact(cuda, n, rows, cols, accumulate):
    import torch

    rng = np.random.default_rng(n + rows + cols)
    x, xs, xv = integer_rows(rng, n, cols, 4, cuda)
    dy, dv = small_integers(rng, (n, rows), cuda)
    dw, old = small_integers(rng, (rows, cols), cuda)
    assert n * 48 < 2 ** 24
    ref = torch.as_tensor(dv).to(cuda).t() @ torch.as_tensor(xv).to(cuda)
    if accumulate:
        ref += torch.as_tensor(old).to(cuda)
    ws = workspace(n, rows, cols, cuda)
    bq.linear_fp8_dw(dy, x, xs, dw, ws, accumulate=accumulate)
    bq.linear_check(ws)
    assert torch.equal(dw, ref.float().bfloat16())


@pytest.mark.parametrize("n,rows,cols", SHAPES)
def test_linear_exact(cuda, n, rows, cols):
    import torch

    rng = np.random.default_rng(n + rows + cols)
    x, xs, xv = integer_rows(rng, n, cols, 8, cuda)
    codes = e4m3_encode(rng.integers(-2, 3, (rows, cols)).astype(np.float32))
    tiles = (2.0 ** rng.integers(0, 3, (-(-rows // 128), -(-cols // 128)))).astype(np.float32)
    wv = L.decode_tiles(codes, tiles)
    assert 4 * 2 ** 9 * cols <= 2 ** 24
    ref = torch.as_tensor(xv).to(cuda) @ torch.as_tensor(wv).to(cuda).t()
    out, ws = torch.empty(n, rows, dtype=torch.bfloat16, device=cuda), workspace(n, rows, cols, cuda)
    bq.linear_fp8(x, xs, torch.as_tensor(codes).to(cuda), torch.as_tensor(tiles).to(cuda), out, ws)
    bq.linear_check(ws)
    assert torch.equal(out, ref.float().bfloat16())


# ----------------------------------------------------------------------------- parameters gathered from several devices


def test_weights_gathered_from_several_devices(cuda):
    """The staging buffers of a layout over several devices, all of whose shards are held here
    (what an AllGather leaves): a weight cut by device boundaries is read from its start and
    its first scale slot."""
    import torch

    shapes = [(300, 272), (1, 777), (900, 528), (129, 2064)]
    descs = [(r, c, int(np.lcm(128 * c, 256)) if r > 1 else 256, bq.ADAM_FLAT256, int(r > 1)) for r, c in shapes]
    layout = bq.plan(descs, 4)
    t = layout.export()
    S, n, ni, nf = int(t[3]), int(t[4]), int(t[5]), int(t[7])
    places = t[8 + 7 * n:8 + 7 * n + 7 * ni].reshape(ni, 7)
    tables = torch.empty(layout.upload_bytes(0, 4), dtype=torch.uint8, device=cuda)
    shard = layout.upload(0, 4, tables)
    rng = np.random.default_rng(4)
    master = torch.as_tensor(rng.standard_normal(4 * S).astype(np.float32)).to(cuda)
    codes, scales = torch.zeros(4 * S, dtype=torch.uint8, device=cuda), torch.zeros(nf, device=cuda)
    bq.quant_fp8(shard, master, codes, scales)
    spanning = 0
    for i, (r, c) in enumerate(shapes):
        if r == 1:
            continue
        mine = places[places[:, 1] == i]
        spanning += len(mine) > 1
        at, slot = int(mine[0, 0] * S + mine[0, 4]), int(mine[0, 6])
        w, ws_ = codes[at:at + r * c].view(r, c), scales[slot:slot + -(-r // 128) * -(-c // 128)]
        wv, m = L.decode_tiles(w.cpu().numpy(), ws_.cpu().numpy()), f64(master[at:at + r * c].view(r, c))
        s = L.spread_tiles(ws_.cpu().numpy(), r, c)
        assert np.all(np.abs(wv - m) <= 2.0 ** -4 * np.abs(wv) * 1.001 + 2.0 ** -10 * s * 1.001)
        x, xs, xv = fp8_rows(rng, 40, c, cuda)
        out, ws = torch.empty(40, r, dtype=torch.bfloat16, device=cuda), workspace(40, r, c, cuda)
        bq.linear_fp8(x, xs, w, ws_, out, ws)
        bq.linear_check(ws)
        ref = xv @ wv.T
        assert np.all(np.abs(f64(out) - ref) <= U * 1.001 * np.abs(ref) + sum_tol(xv, wv.T, c))
        ids = torch.as_tensor(rng.integers(0, r, 50)).to(cuda)
        rows = torch.empty(50, c, dtype=torch.bfloat16, device=cuda)
        bq.embed(w, ids, rows, table_scale=ws_)
        want = wv[ids.cpu().numpy()]
        assert np.all(np.abs(f64(rows) - want) <= U * 1.001 * np.abs(want))
    assert spanning
