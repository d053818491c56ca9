"""The layer operators without a GPU: what the C ABI and the binding refuse, and the
oracle's gradients against differences of its forward passes."""

import ctypes as C

import numpy as np
import pytest

import block_quant_gb300 as bq
from oracle import layer as L

P = 4096  # an aligned address that no refused call reads


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_quant_gb300 import build

    build.build()
    return bq.load()


def test_norm_gradient_matches_differences():
    rng = np.random.default_rng(0)
    h, w, dy = rng.standard_normal((3, 17)), rng.standard_normal(17), rng.standard_normal((3, 17))
    eps, d = 1e-3, 1e-5
    _, rstd = L.rmsnorm(h, w, eps)
    dh, dw = L.rmsnorm_grad(dy, h, w, rstd)
    loss = lambda h, w: np.sum(dy * L.rmsnorm(h, w, eps)[0])  # noqa: E731
    # central differences: off by the third derivative times d^2 / 6 and rounding of 1e-16 / d
    for i in range(3):
        for c in range(17):
            e = np.zeros_like(h)
            e[i, c] = d
            assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * d) - dh[i, c]) < 1e-7
    for c in range(17):
        e = np.zeros_like(w)
        e[c] = d
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * d) - dw[c]) < 1e-7


def test_embedding_gradient_matches_differences():
    rng = np.random.default_rng(1)
    table, dy = rng.standard_normal((6, 5)), rng.standard_normal((9, 5))
    ids = np.array([0, 5, 5, -1, 2, 6, 5, 2, 0])
    g, _ = L.embed_grad(dy, ids, 6, 1.5)
    for v in range(6):
        for c in range(5):
            e = np.zeros_like(table)
            e[v, c] = 1.0  # linear: any step
            diff = np.sum(dy * (L.embed(table + e, ids, 1.5) - L.embed(table, ids, 1.5)))
            assert abs(diff - g[v, c]) < 1e-12


def test_projection_gradients_match_differences():
    rng = np.random.default_rng(2)
    x, w, dy = rng.standard_normal((4, 6)), rng.standard_normal((5, 6)), rng.standard_normal((4, 5))
    dx, dw = dy @ w, dy.T @ x
    loss = lambda x, w: np.sum(dy * (x @ w.T))  # noqa: E731
    for a, g in ((x, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + 1
            up = loss(x, w)
            a[i] = old
            assert abs(up - loss(x, w) - g[i]) < 1e-12


def _embed(lib, **k):
    a = dict(table=P, kind=0, ts=None, rows=10, cols=8, ldt=8, ids=P, bits=32, n=4, scale=1.0, out=P, ldo=8)
    a.update(k)
    return lib.bq_embed(*a.values(), None)


def _embed_grad(lib, **k):
    a = dict(dy=P, ldd=8, ids=P, bits=64, n=4, scale=1.0, rows=10, cols=8, out=P, kind=0, ldo=8, acc=0, ws=P, wb=1 << 20)
    a.update(k)
    return lib.bq_embed_grad(*a.values(), None)


def _norm(lib, **k):
    a = dict(x=P, ldx=8, res=None, ldr=0, w=P, eps=1e-5, n=4, cols=8, h=None, ldh=0, y=P, ldy=8, codes=None, ldc=0,
             scale=None, lds=0, rstd=None)
    a.update(k)
    return lib.bq_rmsnorm(*a.values(), None)


def _norm_grad(lib, **k):
    a = dict(dy=P, ldy=8, h=P, ldh=8, w=P, rstd=P, dh=None, ldg=0, n=4, cols=8, dx=P, ldx=8, dw=P, kind=0, acc=0, ws=P,
             wb=1 << 20)
    a.update(k)
    return lib.bq_rmsnorm_grad(*a.values(), None)


def _quant(lib, **k):
    a = dict(x=P, ldx=8, n=4, cols=8, codes=P, ldc=8, scale=P, lds=4)
    a.update(k)
    return lib.bq_quant_rows_fp8(*a.values(), None)


def _lin(lib, **k):
    a = dict(x=P, ldx=32, xs=P, lds=4, w=P, ldw=32, ws_=P, n=4, rows=16, cols=32, out=P, ldo=16, ws=P, wb=1 << 20)
    a.update(k)
    return lib.bq_linear_fp8(*a.values(), None)


def _lin_dx(lib, **k):
    a = dict(dy=P, ldy=16, w=P, ldw=32, ws_=P, n=4, rows=16, cols=32, dx=P, ldx=32, ws=P, wb=1 << 20)
    a.update(k)
    return lib.bq_linear_fp8_dx(*a.values(), None)


def _lin_dw(lib, **k):
    a = dict(dy=P, ldy=16, x=P, ldx=32, xs=P, lds=4, n=4, rows=16, cols=32, dw=P, ldw=32, acc=0, ws=P, wb=1 << 20)
    a.update(k)
    return lib.bq_linear_fp8_dw(*a.values(), None)


INV, ALIGN, SPACE = bq.BQ_EINVAL, bq.BQ_EALIGN, bq.BQ_ENOSPC
REFUSED = [
    (_embed, dict(table=None), INV), (_embed, dict(ids=None), INV), (_embed, dict(out=None), INV),
    (_embed, dict(kind=1), INV), (_embed, dict(kind=2), INV), (_embed, dict(bits=16), INV), (_embed, dict(n=-1), INV),
    (_embed, dict(rows=0), INV), (_embed, dict(cols=0), INV), (_embed, dict(cols=65537, ldt=70000, ldo=70000), INV),
    (_embed, dict(ldt=7), INV), (_embed, dict(ldo=7), INV), (_embed, dict(out=P + 1), ALIGN),
    (_embed, dict(table=P + 1), ALIGN), (_embed, dict(ids=P + 2), ALIGN), (_embed, dict(kind=2, ts=P + 2), ALIGN),
    (_embed_grad, dict(dy=None), INV), (_embed_grad, dict(out=None), INV), (_embed_grad, dict(ids=None), INV),
    (_embed_grad, dict(kind=2), INV), (_embed_grad, dict(ldd=4), INV), (_embed_grad, dict(ldo=4), INV),
    (_embed_grad, dict(ws=None), INV), (_embed_grad, dict(ws=P + 16), ALIGN), (_embed_grad, dict(wb=64), SPACE),
    (_embed_grad, dict(ids=P + 4), ALIGN), (_embed_grad, dict(kind=1, out=P + 2), ALIGN),
    (_embed_grad, dict(n=(1 << 27) + 1), INV), (_embed_grad, dict(rows=(1 << 30) + 1), INV),
    (_norm, dict(x=None), INV), (_norm, dict(w=None), INV), (_norm, dict(y=None), INV), (_norm, dict(res=P, ldr=8), INV),
    (_norm, dict(codes=P, ldc=8), INV), (_norm, dict(codes=P, ldc=4, scale=P, lds=4), INV),
    (_norm, dict(cols=136, ldx=136, ldy=136, codes=P, ldc=136, scale=P, lds=3), INV), (_norm, dict(eps=-1.0), INV),
    (_norm, dict(eps=float("nan")), INV), (_norm, dict(ldx=7), INV), (_norm, dict(x=P + 1), ALIGN),
    (_norm, dict(rstd=P + 2), ALIGN), (_norm, dict(n=-1), INV),
    (_norm_grad, dict(dy=None), INV), (_norm_grad, dict(rstd=None), INV), (_norm_grad, dict(dw=None), INV),
    (_norm_grad, dict(kind=2), INV), (_norm_grad, dict(ldh=4), INV), (_norm_grad, dict(dh=P, ldg=4), INV),
    (_norm_grad, dict(wb=16), SPACE), (_norm_grad, dict(ws=P + 8), ALIGN), (_norm_grad, dict(kind=1, dw=P + 2), ALIGN),
    (_quant, dict(x=None), INV), (_quant, dict(codes=None), INV), (_quant, dict(scale=None), INV),
    (_quant, dict(ldc=4), INV), (_quant, dict(scale=P + 1), ALIGN),
    (_lin, dict(x=None), INV), (_lin, dict(w=None), INV), (_lin, dict(ws_=None), INV), (_lin, dict(out=None), INV),
    (_lin, dict(ws=None), INV), (_lin, dict(wb=128), SPACE), (_lin, dict(wb=256), SPACE), (_lin, dict(ws=P + 128), ALIGN), (_lin, dict(x=P + 8), ALIGN),
    (_lin, dict(w=P + 8), ALIGN), (_lin, dict(ldx=40), ALIGN), (_lin, dict(ldw=40), ALIGN),
    (_lin, dict(cols=24), ALIGN), (_lin, dict(ldx=16), INV), (_lin, dict(ldo=8), INV),
    (_lin, dict(cols=144, ldx=144, ldw=144, lds=3), INV), (_lin, dict(rows=(1 << 24) + 1, ldo=1 << 25), INV),
    (_lin_dx, dict(dy=None), INV), (_lin_dx, dict(dx=None), INV), (_lin_dx, dict(wb=300), SPACE),
    (_lin_dx, dict(ldy=8), INV), (_lin_dx, dict(ldx=16), INV), (_lin_dx, dict(dx=P + 1), ALIGN),
    (_lin_dw, dict(dy=None), INV), (_lin_dw, dict(x=None), INV), (_lin_dw, dict(dw=None), INV),
    (_lin_dw, dict(wb=300), SPACE), (_lin_dw, dict(ldw=16), INV), (_lin_dw, dict(x=P + 4), ALIGN),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refused(built, i):
    call, change, code = REFUSED[i]
    assert call(built, **change) == code, (call.__name__, change, built.bq_last_error())
    assert built.bq_last_error()


def test_no_tokens_is_no_work(built):
    """Counts of zero return before anything is launched (there may be no GPU here)."""
    assert _embed(built, n=0, table=None, ids=None, out=None) == bq.BQ_OK
    assert _norm(built, n=0) == bq.BQ_OK
    assert _quant(built, n=0) == bq.BQ_OK
    assert _embed_grad(built, n=0, acc=1) == bq.BQ_OK
    assert _norm_grad(built, n=0, acc=1) == bq.BQ_OK
    assert _lin(built, n=0) == bq.BQ_OK
    assert _lin_dx(built, n=0) == bq.BQ_OK
    assert _lin_dw(built, n=0, acc=1) == bq.BQ_OK


def test_workspace_sizes(built):
    b = C.c_size_t()
    assert built.bq_linear_fp8_workspace(8, 16, 24, C.byref(b)) == ALIGN
    assert built.bq_linear_fp8_workspace(8, 16, 32, None) == INV
    assert bq.linear_fp8_workspace(0, 1, 16) >= 256
    assert bq.embed_grad_workspace(0, 1, 1) > 0
    # room for the larger of: codes and scales of dy; bf16 rows of X and of dy
    assert bq.linear_fp8_workspace(1000, 4096, 2048) >= 1000 * 2 * (4096 + 2048)


def test_binding_refuses_shapes_and_types():
    import torch

    t = torch.zeros(10, 16, dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int64)
    out = torch.zeros(4, 16, dtype=torch.bfloat16)
    bad = [
        lambda: bq.embed(t.half(), ids, out, stream=0),
        lambda: bq.embed(t, ids.float(), out, stream=0),
        lambda: bq.embed(t, ids, out[:3], stream=0),
        lambda: bq.embed(t.t(), ids, out, stream=0),
        lambda: bq.embed(t.to(torch.uint8), ids, out, stream=0),  # FP8 without scales
        lambda: bq.rmsnorm(out, torch.zeros(8, dtype=torch.bfloat16), 1e-5, y=out, stream=0),
        lambda: bq.rmsnorm(out.float(), t[0], 1e-5, y=out, stream=0),
        lambda: bq.rmsnorm(out, t[0], 1e-5, codes=torch.zeros(4, 16, dtype=torch.uint8),
                           code_scale=torch.zeros(4, 1), stream=0),
        lambda: bq.linear_fp8(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(1, 4), torch.zeros(8, 16, dtype=torch.uint8),
                              torch.zeros(2), torch.zeros(4, 8, dtype=torch.bfloat16), None, stream=0),
    ]
    for call in bad:
        with pytest.raises(bq.BQError) as e:
            call()
        assert e.value.code == bq.BQ_EINVAL
    with pytest.raises(bq.BQError, match="not on a GPU"):  # right shapes and types
        bq.embed(t, ids, out, stream=0)


def test_packed_call_refuses_what_it_does_not_know(built):
    words = bytes(8 * 24)
    assert built.bq_call(99, words) == INV
    assert built.bq_call(-1, words) == INV
    assert built.bq_call(0, None) == INV


@pytest.mark.parametrize("seed", range(12))
def test_gathered_weights_are_one_run(built, seed):
    """A matrix whose shards lie on several devices: in the gathered buffers (the devices' shards
    one after another) its codes are one row-major run from its start and its tile scales one
    run from its first slot, as the projections and the lookup read them."""
    rng = np.random.default_rng(seed)
    descs = []
    for _ in range(int(rng.integers(3, 12))):
        if rng.random() < 0.3:
            descs.append((1, int(rng.integers(1, 3000)), 256, bq.ADAM_FLAT256, 0))
            continue
        rows, cols = int(rng.integers(2, 2000)), 16 * int(rng.integers(1, 60))
        descs.append((rows, cols, int(np.lcm(128 * cols, 256)), bq.ADAM_FLAT256, 1))
    spanning = 0
    for V in (1, 2, 3, 8):
        t = bq.plan(descs, V, start_align=16).export()
        S, n, ni = int(t[3]), int(t[4]), int(t[5])
        starts = t[8:8 + 7 * n].reshape(n, 7)[:, 0]
        rows = t[8 + 7 * n:8 + 7 * n + 7 * ni].reshape(ni, 7)  # dev, tensor, t_off, len, local_off, mslot, fslot
        for i, (r, c, _, _, fp8) in enumerate(descs):
            if not fp8:
                continue
            mine = rows[rows[:, 1] == i]
            spanning += len(mine) > 1
            at, slot, first = 0, int(mine[0, 6]), int(mine[0, 0] * S + mine[0, 4])
            assert first == starts[i] and first % 16 == 0
            for dev, _, off, size, local, _, fslot in mine:
                assert off == at and dev * S + local == first + at  # no gap in the codes
                assert off % (128 * c) == 0 and fslot == slot + off // (128 * c) * -(-c // 128)  # nor in the scales
                at += int(size)
            assert at == r * c
    assert spanning
