"""The losses over an FP8 head without a GPU: what the C ABI and the binding refuse, the
oracle's gradients against differences of its losses, and the bit patterns that the
kernels rely on."""

import ctypes as C

import numpy as np
import pytest

import block_quant_gb300 as bq
from oracle import loss as O
from test_layer_binding import Tensor, library  # noqa: F401  (the library's stand-in)

P = 4096  # an aligned address that no refused call reads
INV, ALIGN, NOSPC = bq.BQ_EINVAL, bq.BQ_EALIGN, bq.BQ_ENOSPC
WS = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_quant_gb300 import build

    build.build()
    return bq.load()


# ----------------------------------------------------------------------------- the oracle


@pytest.mark.parametrize("kind", ["class", "teacher"])
def test_gradients_match_differences(kind):
    rng = np.random.default_rng(4)
    n, rows, cols, k, scale, d = 5, 7, 6, 4, 0.7, 1e-5
    x, w, g = rng.standard_normal((n, cols)), rng.standard_normal((rows, cols)), rng.standard_normal(n)
    if kind == "class":
        pairs = O.class_pairs(np.array([2, -1, 6, 7, 0]), rows)
    else:
        ids = np.array([[0, 3, 3, -1], [-1, -1, 9, -1], [6, 5, 4, 1], [2, 2, 2, 2], [1, 0, 6, 3]])
        z = rng.standard_normal((n, k))
        z[2, 1] = z[4, 0] = -np.inf
        pairs = O.teacher_pairs(ids, z, scale, rows)
        assert not pairs[2][1].any()

    def total(x, w):
        return np.sum(g * O.loss(O.logits(x, w, scale)[0], pairs)[0])

    dx, dw, _, _ = O.grads(x, w, O.logits(x, w, scale)[0], pairs, g, scale)
    # central differences: off by the third derivative times d^2 / 6 and rounding of 1e-15 / d
    for a, grad, f in ((x, dx, lambda e: total(x + e, w)), (w, dw, lambda e: total(x, w + e))):
        for i in np.ndindex(a.shape):
            e = np.zeros_like(a)
            e[i] = d
            assert abs((f(e) - f(-e)) / (2 * d) - grad[i]) < 1e-8


def test_log_probabilities_near_zero():
    """-log(1 + s) for others of sum s, far below what 1 - p could hold."""
    z = np.array([[0.0, -50.0, -60.0]])
    want = -np.exp(-50.0) - np.exp(-60.0)  # (s^2 is 1e-43 of it)
    assert abs(O.log_probs(z, np.array([[0]]))[0, 0] - want) < 1e-12 * -want


# ----------------------------------------------------------------------------- refusals


HEAD = dict(x=P, ldx=32, xs=P, lds=4, w=P, ldw=32, ws_=P, n=4, rows=16, cols=32)
TEACHER = dict(ids=P, bits=64, ldi=3, z=P, kind=0, ldz=3, k=3, scale=1.0)
CALLS = {
    "bq_cross_entropy_fp8": {**HEAD, **dict(y=P, bits=64, scale=1.0, loss=P, lse=P, ws=P, wb=WS)},
    "bq_cross_entropy_fp8_grad": {**HEAD, **dict(y=P, bits=64, scale=1.0, loss=P, lse=P, dloss=P, dx=P, ldd=32, dw=P, ldg=32,
                                                 acc=0, ws=P, wb=WS)},
    "bq_distill_fp8": {**HEAD, **TEACHER, **dict(loss=P, lse=P, logp=P, ldp=3, ws=P, wb=WS)},
    "bq_distill_fp8_grad": {**HEAD, **TEACHER, **dict(lse=P, logp=P, ldp=3, dloss=P, dx=P, ldd=32, dw=P, ldg=32, acc=0, ws=P,
                                                      wb=WS)},
}
SHARED = [(dict(n=-1), INV), (dict(n=2 ** 27 + 1), INV), (dict(rows=0), INV), (dict(rows=2 ** 24 + 1), INV), (dict(cols=0), INV),
          (dict(cols=65552), INV), (dict(cols=24, ldx=32, ldw=32), ALIGN), (dict(x=None), INV), (dict(xs=None), INV),
          (dict(w=None), INV), (dict(ws_=None), INV), (dict(lse=None), INV), (dict(ldx=16), INV), (dict(ldw=16), INV),
          (dict(ldx=40), ALIGN), (dict(ldw=40), ALIGN), (dict(x=P + 8), ALIGN), (dict(w=P + 4), ALIGN), (dict(xs=P + 2), ALIGN),
          (dict(ws_=P + 1), ALIGN), (dict(lse=P + 2), ALIGN), (dict(bits=16), INV), (dict(scale=float("nan")), INV),
          (dict(scale=float("inf")), INV), (dict(n=2 ** 21, rows=2 ** 21), INV), (dict(ws=None), INV), (dict(ws=P + 128), ALIGN), (dict(wb=512), NOSPC),
          (dict(lds=3, cols=144, ldx=144, ldw=144, ldd=144, ldg=144), INV)]
GRAD = [(dict(dloss=None), INV), (dict(dx=None, dw=None), INV), (dict(ldd=31), INV), (dict(ldg=31), INV), (dict(dx=P + 1), ALIGN),
        (dict(dw=P + 1), ALIGN), (dict(dloss=P + 2), ALIGN)]
PAIRS = [(dict(ids=None), INV), (dict(z=None), INV), (dict(logp=None), INV), (dict(k=0), INV), (dict(k=1025, ldi=1025, ldz=1025, ldp=1025), INV),
         (dict(ldi=2), INV), (dict(ldz=2), INV), (dict(ldp=2), INV), (dict(kind=2), INV), (dict(ids=P + 4), ALIGN),
         (dict(z=P + 1), ALIGN), (dict(kind=1, z=P + 2), ALIGN), (dict(logp=P + 2), ALIGN)]
CLASS = [(dict(y=None), INV), (dict(loss=None), INV), (dict(y=P + 4), ALIGN), (dict(loss=P + 1), ALIGN)]


@pytest.mark.parametrize("name", CALLS)
def test_refused(built, name):
    args, f = CALLS[name], getattr(built, name)
    bad = SHARED + (GRAD if name.endswith("grad") else []) + (PAIRS if "distill" in name else CLASS)
    for change, code in bad:
        change = {k: v for k, v in change.items() if k in args}
        assert change
        assert f(*{**args, **change}.values(), None) == code, change
    if name == "bq_distill_fp8":
        assert f(*{**args, "loss": None}.values(), None) == INV


@pytest.mark.parametrize("name", CALLS)
def test_no_tokens(built, name):
    """Nothing is read, and nothing launched where nothing is to be written."""
    args = {**CALLS[name], "n": 0}
    for key in ("x", "xs", "w", "ws_", "y", "ids", "z", "loss", "lse", "logp", "dloss", "dx", "dw"):
        if key in args:
            args[key] = None
    assert getattr(built, name)(*args.values(), None) == bq.BQ_OK


def test_workspaces_are_sized(built):
    for f in (bq.loss_fp8_workspace, bq.loss_fp8_grad_workspace):
        for bad, code in (((-1, 8, 16), INV), ((1, 0, 16), INV), ((1, 8, 24), ALIGN), ((1, 2 ** 24 + 1, 16), INV), ((2 ** 27 + 1, 8, 16), INV)):
            with pytest.raises(bq.BQError) as e:
                f(*bad)
            assert e.value.code == code
        assert f(0, 8, 16) > 0 and f(1, 1, 16) > 0
    assert built.bq_loss_fp8_workspace(1, 8, 16, None) == INV
    # a piece of the vocabulary, not the logits: 8192 tokens of 128256 words
    logits = 8192 * 128256 * 2
    assert bq.loss_fp8_workspace(8192, 128256, 4096) < logits / 8
    assert bq.loss_fp8_grad_workspace(8192, 128256, 4096) < logits / 2


def test_packed_calls_are_those_of_their_names(built):
    """Each packed call with the workspace left out is refused as the call itself is."""
    import struct

    for op, name in ((8, "bq_cross_entropy_fp8"), (9, "bq_cross_entropy_fp8_grad"), (10, "bq_distill_fp8"), (11, "bq_distill_fp8_grad")):
        def packed(args):
            return b"".join(struct.pack("<d", v) if isinstance(v, float) else struct.pack("<q", v or 0) for v in args.values()) + bytes(8)

        assert built.bq_call(op, packed({**CALLS[name], "ws": None})) == INV
        assert name in built.bq_last_error().decode()
        assert built.bq_call(op, packed({**CALLS[name], "wb": 512})) == NOSPC
        assert built.bq_call(op, packed({**CALLS[name], "scale": float("nan")})) == INV
        for key, code in (("lse", ALIGN), ("x", ALIGN), ("w", ALIGN)):
            assert built.bq_call(op, packed({**CALLS[name], key: P + 1})) == code
        if name.endswith("grad"):
            assert built.bq_call(op, packed({**CALLS[name], "dw": P + 1})) == ALIGN
            assert built.bq_call(op, packed({**CALLS[name], "ldd": 1})) == INV
        if "distill" in name:
            assert built.bq_call(op, packed({**CALLS[name], "ldp": 1})) == INV


# ----------------------------------------------------------------------------- the binding


def tensors(grad, distill, **change):
    n, rows, cols, k = 4, 8, 32, 3
    a = dict(codes=Tensor("u8", n, cols), code_scale=Tensor("f32", 1, n), w=Tensor("u8", rows, cols), w_scale=Tensor("f32", 1))
    if distill:
        a.update(ids=Tensor("i32", n, k), teacher=Tensor("f32", n, k), lse=Tensor("f32", n), logp=Tensor("f32", n, k))
    else:
        a.update(targets=Tensor("i64", n), loss=Tensor("f32", n), lse=Tensor("f32", n))
    if grad:
        a.update(dloss=Tensor("f32", n), dx=Tensor("bf16", n, cols), dw=Tensor("bf16", rows, cols))
    elif distill:
        a["loss"] = Tensor("f32", n)
    a["ws"] = Tensor("u8", 1 << 20)
    a.update(change)
    return a


def call(grad, distill, **change):
    f = {(0, 0): bq.cross_entropy_fp8, (1, 0): bq.cross_entropy_fp8_grad, (0, 1): bq.distill_fp8, (1, 1): bq.distill_fp8_grad}
    f[int(grad), int(distill)](**tensors(grad, distill, **change), stream=0)


@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("distill", [0, 1])
def test_the_binding_refuses(library, grad, distill):  # noqa: F811
    call(grad, distill)
    assert len(library.calls) == 1 and library.calls[0][0] == 8 + grad + 2 * distill
    bad = [dict(codes=Tensor("bf16", 4, 32)), dict(codes=Tensor("u8", 4, 16)), dict(code_scale=Tensor("f32", 1, 5)),
           dict(code_scale=Tensor("f32", 2, 4)), dict(w=Tensor("bf16", 8, 32)), dict(w_scale=Tensor("f32", 2)),
           dict(w_scale=Tensor("bf16", 1)), dict(lse=Tensor("f32", 5)), dict(lse=Tensor("bf16", 4)), dict(lse=None),
           dict(ws=None), dict(ws=Tensor("u8", 1 << 20, gpu=-1)), dict(ws=Tensor("u8", 1 << 20, contiguous=False)),
           dict(lse=Tensor("f32", 4, gpu=1)), dict(lse=Tensor("f32", 4, gpu=-1)), dict(lse=Tensor("f32", 4, contiguous=False))]
    if distill:
        bad += [dict(ids=Tensor("i32", 4)), dict(ids=Tensor("f32", 4, 3)), dict(ids=Tensor("i32", 5, 3)), dict(ids=None),
                dict(teacher=Tensor("f32", 4, 2)), dict(teacher=Tensor("u8", 4, 3)), dict(teacher=None),
                dict(logp=Tensor("f32", 4, 2)), dict(logp=Tensor("bf16", 4, 3)), dict(ids=Tensor("i32", 4, 3, gpu=1))]
    else:
        bad += [dict(targets=Tensor("f32", 4)), dict(targets=Tensor("i64", 5)), dict(targets=Tensor("i64", 4, 1)),
                dict(loss=Tensor("f32", 3)), dict(loss=None)]
    if grad:
        bad += [dict(dloss=Tensor("f32", 3)), dict(dloss=Tensor("bf16", 4)), dict(dx=Tensor("f32", 4, 32)),
                dict(dx=Tensor("bf16", 4, 16)), dict(dw=Tensor("bf16", 4, 32)), dict(dw=Tensor("f32", 8, 32))]
    for change in bad:
        with pytest.raises(bq.BQError) as e:
            call(grad, distill, **change)
        assert e.value.code == INV, change
    library.current = 1
    with pytest.raises(bq.BQError, match="current device"):
        call(grad, distill)
    library.current = 0
    if grad:
        call(grad, distill, dx=None)
        call(grad, distill, dw=None)
    assert len(library.calls) == 1 + 2 * grad
